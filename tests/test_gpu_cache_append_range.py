"""Appends whose values come near the ends of bf16's range, to blocks that become complete: the pooled
key is a mean, so it is finite where the keys are."""
import numpy as np
import pytest

from test_gpu_cache import Pool, _append_case, _bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("exponent", [124, -85])
@pytest.mark.parametrize("what", ["step", "prompt", "both"])
@pytest.mark.parametrize("ps,D,H,bs", [(16, 64, 2, 256), (128, 128, 1, 8192), (64, 64, 1, 1024)])
def test_pooled_keys_of_any_magnitude(ps, D, H, bs, what, exponent, fmt, cuda_device):
    import torch
    import block_sparse_attention_gate_b200 as mb
    rng = np.random.default_rng(ps + len(what))
    B, max_len = 2, 2 * bs + 5
    P = B * -(-max_len // ps)
    p = mb.MobaCacheParams(B, max_len, P, ps, H, H, D, bs, 1, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    scale = 2.0 ** (exponent - (9 if fmt == "e4m3" else 7))
    pool.Ks = torch.full_like(pool.Ks, scale)
    pool.Vs = torch.full_like(pool.Vs, scale)
    # one token that completes a block, a prompt of two blocks, or a prompt that goes on in a begun block
    add, old = {"step": ([1, 0], [bs - 1, 3]), "prompt": ([2 * bs, 1], [0, bs - 1]),
                "both": ([bs + 7, 1], [bs // 2 + 3, 0])}[what]
    add, old = np.array(add), np.array(old)
    N = int(add.sum()) + 1
    # all of one sign, so that sums are as large as they can be
    kv = _bf16(rng.uniform(0.5, 1, (N, 2, H, D)) * 2.0 ** exponent)
    kbar = torch.full((B, p.max_blocks, H, D), 7.0, device="cuda")
    done = _append_case(rng, p, pool, old, add, N, (kv[:, 0], kv[:, 1]), fmt, ps, bs, D, H, kbar)
    assert done == {"step": 1, "prompt": 3, "both": 1}[what] and kbar.isfinite().all()
