"""Gated decode where the pages' value scales lie as far apart as appends can write them (zeros get a
scale of 2^-104, the largest bf16 values one of 2^119 or, as int8, 2^121): the sum of the softmax does
not depend on the values, however their scales are spread.  The bounds are those of test_gpu_cache.py."""
import numpy as np
import pytest

import _cache_ref as ref
from test_gpu_cache import Pool, _bf16, _check_decode, _decode, _dev, _kbar_of, _no_error

pytestmark = pytest.mark.gpu

LOWEST, HIGHEST = -104.8, {"e4m3": 119.0, "int8": 120.5}


def _scales(e):
    """2^e to 8 significant bits."""
    s = np.exp2(e).astype(np.float32)
    return _dev((s.view(np.uint32) & 0xffff0000).view(np.float32))


def _zero_pages(pool, pages):
    import torch
    pool.Vc.view(torch.uint8)[pages] = 0
    pool.Vs[pages] = float(ref.scale_of(np.zeros(1), pool.fmt)[0])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("what", ["zeros_first", "zeros_last", "largest", "smallest", "spread"])
@pytest.mark.parametrize("ps,Hq,H,D,bs,k", [(16, 4, 2, 64, 128, 4), (64, 3, 1, 128, 256, 3), (128, 16, 1, 64, 512, 2)])
def test_value_scales(ps, Hq, H, D, bs, k, what, fmt, cuda_device):
    import block_sparse_attention_gate_b200 as mb
    rng = np.random.default_rng(len(what) * ps)
    B, max_len = 4, 2000
    MP = -(-max_len // ps)
    P = B * MP
    p = mb.MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    shape = tuple(pool.Vs.shape)
    if what == "largest":
        pool.Vs = _scales(HIGHEST[fmt] - rng.uniform(0, 2, shape))
    elif what == "smallest":
        pool.Vs = _scales(LOWEST + rng.uniform(0.1, 8, shape))
    elif what == "spread":
        pool.Vs = _scales(rng.uniform(LOWEST + 0.1, HIGHEST[fmt], shape))
    else:
        # pages in turns, the zeros first or last, beside values of about 2^40
        pool.Vs = _scales(rng.uniform(30, 40, shape))
        first = 0 if what == "zeros_first" else 1
        _zero_pages(pool, pool.tab[:, first::2].ravel())
    kbar = _kbar_of(pool, B, max_len, ps, bs, H, D)
    lens = np.array([2000, 1, 2 * ps, 1111])
    q = _bf16(rng.standard_normal((B, Hq, D)) * 2)
    _check_decode(p, pool, q, kbar, lens, pool.tab, _decode(p, pool, q, kbar, lens, pool.tab))
    _no_error()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("ps,D,low", [(16, 64, 32), (128, 64, 32), (64, 128, 4096)])
def test_many_keys_without_values(ps, D, low, fmt, cuda_device):
    """131072 keys whose values are all zero; in turns, `low` keys and then as many that weigh 2^7.8 times
    as much."""
    import torch
    import block_sparse_attention_gate_b200 as mb
    rng = np.random.default_rng(3)
    n, bs, k = 131072, 8192, 16
    P = n // ps
    p = mb.MobaCacheParams(1, n, P, ps, 1, 1, D, bs, k, fmt)
    pool = Pool(rng, 1, n, P, ps, 1, D, fmt)
    _zero_pages(pool, np.arange(P))
    high = (np.arange(n) // low % 2).reshape(P, 1, ps, 1)
    one = {"e4m3": 0x38, "int8": 1}[fmt]
    codes = torch.zeros_like(pool.Kc.view(torch.uint8))
    codes[pool.tab[0]] = _dev((high * one).astype(np.uint8)).expand(-1, -1, -1, D)
    pool.Kc = codes.view(pool.Kc.dtype)
    pool.Ks = _scales(np.full((P, 1), np.log2(7.8 * np.log(2) / np.sqrt(D))))
    q = torch.ones(1, 1, D, dtype=torch.bfloat16, device="cuda")
    kbar = _kbar_of(pool, 1, n, ps, bs, 1, D)
    lens = np.array([n])
    got = _decode(p, pool, q, kbar, lens, pool.tab)
    _check_decode(p, pool, q, kbar, lens, pool.tab, got)
    assert (got[0] == 0).all()
    _no_error()
