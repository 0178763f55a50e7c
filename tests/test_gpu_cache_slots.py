"""Which of an append's slots count: the first of each run, that is of a request's new tokens in one page."""
import numpy as np
import pytest

import _cache_ref as ref
from test_gpu_cache import Pool, _bf16, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [100, 260])  # one page after the other, and as a prompt
@pytest.mark.parametrize("bad", [-1, 5 * 32 + 1, 16 * 32, 24 * 32, 2 ** 31 - 32])
@pytest.mark.parametrize("at", ["middle", "first"])
def test_the_first_slot_of_a_run_decides(at, bad, n, cuda_device):
    import torch
    import block_sparse_attention_gate_b200 as mb
    rng = np.random.default_rng(n)
    B, max_len, ps, H, D, bs = 2, 256 + 128, 32, 2, 64, 128
    P = B * max_len // ps
    p = mb.MobaCacheParams(B, max_len, P, ps, H, H, D, bs, 1)
    pool = Pool(rng, B, max_len, P, ps, H, D, "e4m3")
    x = rng.standard_normal((n, H, D))
    K = _bf16(x)
    old = 8  # the first run is 24 tokens in a begun page, the second a page of its own
    pos = old + np.arange(n)
    good = (pool.tab[0, pos // ps] * ps + pos % ps).astype(np.int32)
    slots = good.copy()
    slots[24 if at == "first" else 30] = min(bad, 2 ** 31 - 1)
    cu, lens = np.array([0, n, n], np.int32), np.array([old + n, 0], np.int32)
    kc, vc, ks, vs = pool.values()
    seen = good.copy()
    fits = bad == 16 * 32  # an offset of 0 in one of the 24 pages, one that this call writes nothing else to
    assert 16 not in pool.tab[0, :(old + n + ps - 1) // ps]
    if at == "first":  # the run goes there, or is left out
        seen[24:56] = bad + np.arange(32) if fits else -1
    want = ref.append("e4m3", ps, bs, K.double().cpu().numpy(), cu, lens, seen, kc, ks)
    mb.moba_cache_append(p, K, K, _dev(cu), _dev(lens), _dev(slots), _dev(pool.tab), pool.Kc, pool.Vc, pool.Ks, pool.Vs,
                         torch.zeros(B, 3, H, D, device="cuda"))
    torch.cuda.synchronize()
    # a negative slot is no error, nor is one that is not looked at
    assert mb.moba_read_device_error(clear=True) == (2 if at == "first" and bad >= 0 and not fits else 0)
    got = pool.values()
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[2], want[1])
