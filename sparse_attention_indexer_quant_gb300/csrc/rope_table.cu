// Rotary cosine/sine tables.
//
// The angle of row p, column i is p * w_i.  As a fraction of a turn it is
// p * (w_i / 2 pi) mod 1, and with the frequency as a 64-bit fraction the
// product and the reduction are one integer multiplication that wraps: no
// fp64 arithmetic (which this chip runs at a small fraction of its fp32 rate)
// and no loss at far positions.  The fraction is split into a quarter turn q
// and a remainder in [-1/8, 1/8) turn, which fp32 holds to 24 bits.
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

__device__ __forceinline__ void cos_sin_turn(unsigned long long turn, float* c, float* s) {
  const unsigned q = (unsigned)((turn + (1ull << 61)) >> 62);         // nearest quarter, mod 4
  const long long r = (long long)(turn - ((unsigned long long)q << 62));  // [-2^61, 2^61)
  // half turns: r * 2^-63; the top 32 bits of r << 2 keep 30 bits below the sign
  const float x = (float)(int)((unsigned long long)(r << 2) >> 32) * 0x1p-33f;
  float sx, cx;
  sincospif(x, &sx, &cx);
  const float a = (q & 1) ? sx : cx, b = (q & 1) ? cx : sx;
  *c = (q == 1 || q == 2) ? -a : a;
  *s = (q & 2) ? -b : b;
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
