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


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("exponent", [6, 12, 16, 24, 50])
@pytest.mark.parametrize("ps,Hq,H,D,bs,k", [(16, 4, 2, 64, 128, 4), (64, 3, 1, 128, 256, 3), (128, 16, 1, 64, 512, 2)])
def test_logits_of_any_magnitude(ps, Hq, H, D, bs, k, exponent, fmt, cuda_device):
    """Queries and keys times 2^exponent each, logits from about 2^12 to 2^100.  Where the best logit leads by
    more than 64 times what fp32 rounds (half a step, for D products and a few factors), every other weight is below
    e^-20 of it (the lead is at least 60): O is the best key's value and LSE its logit, to their roundings."""
    import block_sparse_attention_gate_b200 as mb
    rng = np.random.default_rng(exponent * ps)
    B, max_len = 4, 2000
    P = B * -(-max_len // ps)
    p = mb.MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    pool.Ks *= 2.0 ** exponent
    kbar = _kbar_of(pool, B, max_len, ps, bs, H, D)
    lens = np.array([2000, 1, 2 * ps, 1111])
    q = _bf16(rng.standard_normal((B, Hq, D)) * 2.0 ** exponent)
    O, LSE, sel = (t.double().cpu().numpy() for t in _decode(p, pool, q, kbar, lens, pool.tab))
    _no_error()
    assert np.isfinite(O).all() and np.isfinite(LSE).all()
    kc, vc, ks, vs = pool.values()
    qf, led = q.double().cpu().numpy(), 0
    want_sel = ref.decode(qf, kc, vc, ks, vs, kbar.double().cpu().numpy(), lens, pool.tab, ps, bs, k, D ** -0.5)[2]
    np.testing.assert_array_equal(sel, want_sel)
    for s in range(B):
        for h in range(Hq):
            blocks = [int(b) for b in want_sel[s, h] if b >= 0]
            pos = np.concatenate([np.arange(b * bs, min((b + 1) * bs, lens[s])) for b in blocks])
            page, g = pool.tab[s, pos // ps], h // (Hq // H)
            key = kc[page, g, pos % ps] * ks[page, g, None]
            z, zabs = key @ qf[s, h] * D ** -0.5, (np.abs(key) @ np.abs(qf[s, h])).max() * D ** -0.5
            order, dz = np.argsort(-z), (D + 8) * 2.0 ** -24 * zabs
            lead = z[order[0]] - z[order[1]] if len(z) > 1 else np.inf
            assert abs(LSE[s, h] - z[order[0]]) <= dz + 4 * 2.0 ** -24 * zabs + np.log(len(z))
            if lead < 60 or lead < 64 * dz:
                continue
            led += 1
            top = order[0]
            v, rest = vc[page[top], g, pos[top] % ps] * vs[page[top], g], np.abs(vc).max() * vs.max() * 2e-9 * len(z)
            assert np.all(np.abs(O[s, h] - v) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(v) + rest)
    assert led >= B  # the request of one token leads by itself
