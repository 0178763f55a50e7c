"""Append where one request of many slots holds most of a small budget of tokens."""
import numpy as np
import pytest

from test_gpu_cache import Pool, _append_case, _bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,ps,D,H,bs,long,spare", [
    (256, 16, 64, 2, 128, 700, 0), (256, 64, 128, 1, 256, 1024, 0), (300, 32, 64, 1, 512, 900, 1)])
def test_one_long_run_among_many_slots(B, ps, D, H, bs, long, spare, fmt, cuda_device):
    """At most four tokens a slot in all (spare 0), or one more than that."""
    import torch
    import block_sparse_attention_gate_b200 as mb
    rng = np.random.default_rng(B + ps)
    max_len = long + 130
    add = np.zeros(B, np.int64)
    add[::3] = 1 if long < 4 * B - B // 3 - 1 else 0
    add[B // 2] = long
    old = rng.integers(0, 130, B)
    N = 4 * B + spare
    assert add.sum() <= N
    P = B * -(-max_len // ps)
    p = mb.MobaCacheParams(B, max_len, P, ps, H, H, D, bs, 1, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    kv = _bf16(rng.standard_normal((N, 2, H, D)))
    kbar = torch.full((B, p.max_blocks, H, D), 7.0, device="cuda")
    assert _append_case(rng, p, pool, old, add, N, (kv[:, 0], kv[:, 1]), fmt, ps, bs, D, H, kbar) > 0
