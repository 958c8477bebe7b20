"""What stands beside a sequence does not change a bit of its rows: other sequences' queries,
keys and values, with and without a cap."""
import pytest
import torch

from test_gpu_prompt_attention import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_quant_gb300 import binding
    binding.check_device(torch.cuda.current_device())
    return binding


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap", [0.0, 6.0])
@pytest.mark.parametrize("lens,keys,window", [([20, 50, 90], [20, 50, 90], 0), ([20, 50, 90], [300, 450, 600], 0),
                                              ([20, 50, 90], [300, 450, 600], 100), ([6, 40], [3000, 5000], 0)])
def test_other_sequences_do_not_reach_a_row(idx, D, dtype, softcap, lens, keys, window):
    """Scores of one sequence stay below half of the cap, its neighbours' pass it by far or not."""
    q, k, v = make(lens, keys, 4, 2, D, dtype, peak=0.5)
    base = run(idx, q, k, v, lens, keys, softcap=softcap, window=window)
    for b in range(len(lens)):
        t0, s0 = sum(lens[:b]), sum(keys[:b])
        mine = slice(t0, t0 + lens[b])
        for size in (30.0, float("inf")):
            x, y, z = (torch.full_like(t, size) if size > 100 else t * size for t in (q, k, v))
            x[mine], y[s0:s0 + keys[b]], z[s0:s0 + keys[b]] = q[mine], k[s0:s0 + keys[b]], v[s0:s0 + keys[b]]
            out, lse = run(idx, x, y, z, lens, keys, softcap=softcap, window=window)
            assert torch.equal(lse[mine], base[1][mine]), (b, size)
            assert torch.equal(out[mine], base[0][mine]), (b, size)
