"""Prefill attention over bf16 prompts, their keys and values into the paged cache, then decode of each
prompt's last token: both results against 64-bit attention, one over the bf16 inputs and one over the
stored codes, and against each other.

Bounds (half a rounding step is 2^-8 of the value in bf16):
  * a stored value is off by half a step of its code: scale / 2 in int8, max(2^-4 |x|, 2^-10 scale) in
    e4m3 (both and 2^-16 of it, for scale * code taken in 64 bits);
  * decode: the bounds of test_gpu_cache.py;
  * prefill: its output's rounding 2^-8 |O|, the probabilities' 2^-8 sum_j p_j |v_j|, and a quarter of
    that for fp16 partial rows (2^-11) and fp32 sums; LSE 1e-3 as in the prefill's own parity rule;
  * prefill and decode against each other: both bounds, about the difference that the stored codes make
    in 64 bits.
  * selection: that of the pooled stored keys, exactly; that of the prefill wherever the last chosen and
    the first unchosen score lie further apart than the pooled keys' errors can move them.
"""
import numpy as np
import pytest

import _cache_ref as ref
from test_gpu_cache import _bf16, _dev, _no_error, _values

pytestmark = pytest.mark.gpu


def _attend(q, k, v, scale):
    z = k @ q * scale
    p = np.exp(z - z.max())
    lse = z.max() + np.log(p.sum())
    p /= p.sum()
    return p @ v, lse, p @ np.abs(v), (np.abs(k) @ np.abs(q)).max() * scale


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,ps", [(128, 64), (64, 16)])
def test_prefill_and_decode_agree(D, ps, fmt, cuda_device):
    import torch
    import block_sparse_attention_gate_b200 as mb
    rng = np.random.default_rng(D)
    lens, Hq, H, bs, k = [900, 1, 513, 2000], 8, 2, 128, 4
    G, B, cu = Hq // H, len(lens), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    Q, K, V = (_bf16(rng.standard_normal((T, h, D))) for h in (Hq, H, H))
    p = mb.MobaParams(cu, Hq, H, D, bs, k)
    O, LSE = torch.empty_like(Q), torch.empty(T, Hq, device="cuda")
    sel = torch.empty(T, Hq, k, dtype=torch.int32, device="cuda")
    mb.moba_fwd(p, Q, K, V, mb.alloc_workspace(p), O, LSE, sel=sel)
    c = mb.MobaCache(mb.MobaCacheParams(B, 2048, B * 2048 // ps, ps, Hq, H, D, bs, k, fmt))
    c.append(K, V, c.extend(_dev(np.array(lens, np.int32)), T))
    last = torch.from_numpy(cu[1:].astype(np.int64) - 1).cuda()
    dsel = torch.empty(B, Hq, k, dtype=torch.int32, device="cuda")
    dO, dL = c.decode(Q[last].contiguous(), sel=dsel)
    _no_error()

    q, kx, vx = (t.double().cpu().numpy() for t in (Q[last], K, V))
    O, LSE, sel = (t[last].double().cpu().numpy() for t in (O, LSE, sel))
    dO, dL, dsel = (t.double().cpu().numpy() for t in (dO, dL, dsel))
    tab, compared, strong = c.tables.cpu().numpy(), 0, 0
    codes = [_values(x, fmt) * s.cpu().numpy().astype(np.float64)[:, :, None, None]
             for x, s in ((c.Kc, c.Ks), (c.Vc, c.Vs))]
    scales = [s.cpu().numpy().astype(np.float64) for s in (c.Ks, c.Vs)]
    kbar = c.Kbar.double().cpu().numpy()
    for s, n in enumerate(lens):
        pos = np.arange(n)
        page = tab[s, pos // ps]
        stored = []
        for x, val, sc in zip((kx, vx), codes, scales):
            got, want, step = val[page, :, pos % ps], x[cu[s]:cu[s + 1]], sc[page][:, :, None]
            half = step / 2 if fmt == "int8" else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * step)
            assert np.all(np.abs(got - want) <= half * (1 + 2.0 ** -16))
            stored.append(got)
        i = (n - 1) // bs
        exact = kx[cu[s]:cu[s] + i * bs].reshape(i, bs, H, D).mean(1)
        for h in range(Hq):
            g, chosen = h // G, {int(b) for b in dsel[s, h] if b >= 0}
            score, truth = kbar[s, :i, g] @ q[s, h], exact[:, g] @ q[s, h]
            assert chosen == {i} | set(np.argsort(-score, kind="stable")[:k - 1].tolist())
            same = chosen == {int(b) for b in sel[s, h] if b >= 0}
            if i > k - 1:
                order = np.sort(truth)[::-1]
                # the prefill sums its pooled keys and scores in fp32
                moved = np.abs(score - truth).max() + 2.0 ** -12 * (np.abs(exact[:, g]) @ np.abs(q[s, h])).max()
                strong += order[k - 2] - order[k - 1] > 2 * moved
                assert same or order[k - 2] - order[k - 1] <= 2 * moved
            else:
                assert same
            if not same:
                continue
            compared += 1
            rows = np.concatenate([np.arange(b * bs, min((b + 1) * bs, n)) for b in sorted(chosen)])
            o, lse, wide, _ = _attend(q[s, h], kx[cu[s] + rows, g], vx[cu[s] + rows, g], D ** -0.5)
            so, slse, swide, zabs = _attend(q[s, h], stored[0][rows, g], stored[1][rows, g], D ** -0.5)
            dz = (D + 8) * 2.0 ** -24 * zabs + 2.0 ** -21
            tol_d = 2.0 ** -8 * np.abs(so) + (2.0 ** -10 + 2 * dz) * swide
            tol_p = 2.0 ** -8 * np.abs(o) + 1.25 * 2.0 ** -8 * wide
            assert np.all(np.abs(dO[s, h] - so) <= tol_d)
            assert np.all(np.abs(O[s, h] - o) <= tol_p)
            assert np.all(np.abs(dO[s, h] - O[s, h] - (so - o)) <= tol_d + tol_p)
            assert np.abs(dL[s, h] - LSE[s, h] - (slse - lse)) <= 1e-3 + dz + 2.0 ** -22 * (np.abs(lse) + 24 + zabs)
            # the bounds tell an output from zeros and from the next head's
            assert np.mean(np.abs(o) > tol_d + tol_p) > 0.5
    assert compared >= 0.75 * B * Hq and strong > 0
