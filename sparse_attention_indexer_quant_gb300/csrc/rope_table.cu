// Rotary cosine/sine tables.
//
// The angle of row p, column i is p * w_i.  As a fraction of a turn it is
// p * (w_i / 2 pi) mod 1, and with the frequency as a 64-bit fraction the
// product and the reduction are one integer addition per row that wraps: no
// fp64 arithmetic (which this chip runs at a small fraction of its fp32 rate)
// and no loss at far positions.  The fraction is split into a quarter turn q and
// 32 bits of remainder u in [-1, 1] eighths of a turn, whose sine and cosine are
// polynomials in u^2: Chebyshev interpolation of sin(pi u / 4) / u and
// cos(pi u / 4) over u^2 in [0, 1], degrees 3 and 4, off by 2.4e-9 and 5e-11
// before fp32 rounding.  With u's rounding to fp32 and their own they are off by
// at most 1.35 * 2^-24 (every fp32 u tried); the factor mscale adds its rounding
// and the product's, 2^-24 each.  With sincospif in their place the kernel was
// bound by its instructions: 35 us for 262144 x 64 pairs (134 MB) against 20.5 us now.
//
// Bound by its stores (8 bytes per pair): a thread owns four columns, walks
// down the rows by adding its frequencies times the row step, and stores
// 16 bytes of cosines and of sines per row.
#include "common.cuh"
#include "launch.h"
#include "serving.h"

namespace idx {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void cos_sin_turn(unsigned long long phase, float* c, float* s) {
  const unsigned turn = (unsigned)(phase >> 32);
  const unsigned q = (turn + (1u << 29)) >> 30;  // nearest quarter, mod 4
  // 32 bits of the rest: [-1, 1] eighths of a turn
  const float u = (float)(int)__funnelshift_l((unsigned)phase, turn - (q << 30), 2) * 0x1p-31f;
  const float z = u * u;
  // the sine's first term on its own, so that its sum is rounded once
  const float sx = fmaf(u, 0.7853981609766182f,
                        u * z * fmaf(fmaf(-3.595429072400257e-05f, z, 0.002490006801490165f), z,
                                     -0.08074543470810033f));
  const float cx = fmaf(fmaf(fmaf(fmaf(3.5297971415016813e-06f, z, -0.00032593858595389604f), z,
                                  0.01585432522845092f), z, -0.3084251351582918f), z, 1.f);
  const float a = (q & 1) ? sx : cx, b = (q & 1) ? cx : sx;
  // cosine negative in quarters 1 and 2, sine in 2 and 3
  *c = __uint_as_float(__float_as_uint(a) ^ (((q + 1) & 2) << 30));
  *s = __uint_as_float(__float_as_uint(b) ^ ((q & 2) << 30));
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  const int groups = (a.half + 3) / 4;  // of four columns
  const int per_block = kThreads / groups;
  const int row_in_block = threadIdx.x / groups, col = 4 * (threadIdx.x % groups);
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel may still read the buffers written here
  if (row_in_block >= per_block) return;
  unsigned long long turn[4], step[4];
  const int64_t row0 = (int64_t)blockIdx.x * per_block + row_in_block;
  const int64_t stride = (int64_t)gridDim.x * per_block;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long f = col + i < a.half ? a.turns[col + i] : 0;
    turn[i] = f * (unsigned long long)(a.pos0 + row0);
    step[i] = f * (unsigned long long)stride;
  }
  for (int64_t r = row0; r < a.num_pos; r += stride) {
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cos_sin_turn(turn[i], &c[i], &s[i]);
      c[i] *= a.mscale;
      s[i] *= a.mscale;
      turn[i] += step[i];
    }
    const int64_t at = r * a.half + col;
    if (VEC) {
      *reinterpret_cast<float4*>(a.cos_out + at) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(a.sin_out + at) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < a.half) {
          a.cos_out[at + i] = c[i];
          a.sin_out[at + i] = s[i];
        }
    }
  }
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs& a, int sms, cudaStream_t stream) {
  const int per_block = kThreads / ((a.half + 3) / 4);
  const int64_t want = (a.num_pos + per_block - 1) / per_block;
  const int64_t most = (int64_t)sms * 8;
  const int grid = (int)(want > most ? most : want);
  // four columns as one 16-byte store where every row starts on 16 bytes
  const bool vec = a.half % 4 == 0 &&
                   ((reinterpret_cast<uintptr_t>(a.cos_out) | reinterpret_cast<uintptr_t>(a.sin_out)) & 15) == 0;
  return vec ? launch_dependent(rope_table_kernel<true>, dim3(grid), dim3(kThreads), 0, stream, a)
             : launch_dependent(rope_table_kernel<false>, dim3(grid), dim3(kThreads), 0, stream, a);
}

}  // namespace idx
