"""GPU parity of the paged 8-bit KV cache (tables, append, gated decode) against the 64-bit reference.

Whole numbers, codes and scales are compared exactly.  Bounds of the rest:
  * Kbar: an fp32 sum of bs terms in chains of at most bs / 32 + 16 additions and one division, each
    off by at most 2^-24 of what it adds up: (bs / 32 + 17) * 2^-24 * mean |v|.
  * logits: fp32 dots of D terms (any order), times the scale of the page and the softmax scale:
    dz = (D + 8) * 2^-24 * zabs, zabs = max_j scale * sum_d |q_d k_jd|; the exponential's own error,
    2^-21, is added.
  * LSE: dz, and 4 * 2^-24 of its magnitude in bits (running maximum plus logarithm, fp32).
  * O: bf16's half step 2^-8 |O|; the weights may be rounded to fp16 (half step 2^-11, and 2^-25 of the
    largest weight where fp16 has no more bits, over at most 16 * 8192 keys: 2^-11 of it covers
    2^14 such keys), and each is off by 2 dz: (2^-10 + 2 dz) * sum_j p_j |v_j|.
"""
import numpy as np
import pytest

import _cache_ref as ref

pytestmark = pytest.mark.gpu


def _mb():
    import block_sparse_attention_gate_b200 as mb
    return mb


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf16(a):
    return _dev(a.astype(np.float32)).bfloat16()


def _code_dtype(fmt):
    import torch
    return torch.float8_e4m3fn if fmt == "e4m3" else torch.int8


def _values(codes, fmt):
    import torch
    return ref.code_values(fmt)[codes.view(torch.uint8).cpu().numpy()]


def _no_error():
    import torch
    torch.cuda.synchronize()
    assert _mb().moba_read_device_error(clear=True) == 0


# ---------------------------------------------------------------------------------- tables

def _tables_state(rng, B, max_len, ps, P, add, lens):
    MP = -(-max_len // ps)
    perm = rng.permutation(P).astype(np.int32)
    tab, at = np.full((B, MP), -1, np.int32), 0
    for s in range(B):
        h = -(-int(lens[s]) // ps) if 0 <= lens[s] <= max_len else 0
        tab[s, :h] = perm[at:at + h]
        at += h
    head = int(rng.integers(P))
    ring = np.full(P, -1, np.int32)
    ring[(head + np.arange(P - at)) % P] = perm[at:]
    return tab, ring, np.array([head, P - at], np.int32)


def _run_tables(p, add, lens, tab, ring, state, max_tokens, in_place=False):
    import torch
    mb = _mb()
    i32 = dict(dtype=torch.int32, device="cuda")
    d = {k: _dev(v.astype(np.int32)) for k, v in dict(add=add, lens=lens, tab=tab, ring=ring, state=state).items()}
    lo, so = (d["lens"], d["state"]) if in_place else (torch.full_like(d["lens"], -9), torch.full_like(d["state"], -9))
    cu, slots, status = torch.full((len(add) + 1,), -9, **i32), torch.full((max_tokens,), -9, **i32), torch.full((1,), -9, **i32)
    mb.moba_cache_tables(p, d["add"], d["lens"], d["tab"], d["ring"], d["state"], lo, so, cu, slots, status)
    _no_error()
    return dict(lens=lo, tables=d["tab"], ring=d["ring"], state=so, cu=cu, slots=slots, status=status)


def _check_tables(got, want):
    for k in ("lens", "tables", "ring", "state", "cu", "slots"):
        np.testing.assert_array_equal(got[k].cpu().numpy(), want[k], err_msg=k)
    assert int(got["status"]) == want["status"]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,max_len,ps,new", [
    (1, 1, 16, 1), (1, 100000, 16, 70001), (3, 50, 32, 20), (65, 4097, 64, 1), (64, 300, 128, 300), (1024, 100, 16, 7),
    (1025, 100, 16, 33), (3000, 257, 32, 257), (7, 40000, 64, 30000), (200, 3000, 16, 2000)])
def test_tables(B, max_len, ps, new, in_place, cuda_device):
    rng = np.random.default_rng(B + new)
    MP = -(-max_len // ps)
    P = B * MP + 5
    p = _mb().MobaCacheParams(B, max_len, P, ps, 1, 1, 64, 128, 1)
    add = rng.integers(0, new + 1, B).astype(np.int64)
    add[rng.random(B) < 0.2] = 0
    add[rng.random(B) < 0.15] = -1 - rng.integers(3)
    lens = np.array([rng.integers(0, max_len - max(a, 0) + 1) for a in add])
    tab, ring, state = _tables_state(rng, B, max_len, ps, P, add, lens)
    N = int(np.maximum(add, 0).sum()) + int(rng.integers(0, 3)) * 17
    want = ref.tables(ps, P, max_len, add, lens.astype(np.int32), tab, ring, state, N)
    assert want["status"] == 0
    _check_tables(_run_tables(p, add, lens, tab, ring, state, N, in_place), want)


@pytest.mark.parametrize("what", ["pages", "long", "slots", "len", "head", "count", "all_idle", "all_end", "exact_pages",
                                  "huge_add", "two"])
def test_tables_status(what, cuda_device):
    rng = np.random.default_rng(3)
    B, max_len, ps = 5, 200, 16
    P = 40
    p = _mb().MobaCacheParams(B, max_len, P, ps, 1, 1, 64, 128, 1)
    add, lens, N = np.array([3, 17, 0, -1, 40]), np.array([16, 30, 5, 100, 0]), 64
    if what == "long":
        add[1] = 171
    if what == "slots":
        N = 59
    if what == "huge_add":
        add[1] = 2 ** 31 - 1
    if what == "all_idle":
        add[:] = 0
    if what == "all_end":
        add[:] = -1
    tab, ring, state = _tables_state(rng, B, max_len, ps, P, add, lens)
    if what in ("pages", "two"):
        state[1] = 4
    if what == "exact_pages":
        state[1] = 5  # 3 -> 2 pages: 1, 30 -> 47: 1, 0 -> 40: 3
    if what == "two":
        N = 3
    if what == "len":
        lens[2] = 201
    if what == "head":
        state[0] = P
    if what == "count":
        state[1] = P + 1
    want = ref.tables(ps, P, max_len, add, lens.astype(np.int32), tab, ring, state, N)
    expect = {"pages": 1, "long": 2, "slots": 4, "len": 8, "head": 8, "count": 8, "huge_add": 2, "two": 5}
    assert want["status"] == expect.get(what, 0)
    _check_tables(_run_tables(p, add, lens, tab, ring, state, N), want)
    _check_tables(_run_tables(p, add, lens, tab, ring, state, N, in_place=True), want)


def test_tables_with_a_bad_page_in_the_ring(cuda_device):
    p = _mb().MobaCacheParams(2, 100, 10, 16, 1, 1, 64, 128, 1)
    add, lens = np.array([20, 5]), np.array([0, 0])
    tab, ring, state = np.full((2, 7), -1, np.int32), np.array([3, 99, 4, 5, 6, 7, 8, 9, 0, 1], np.int32), np.array([0, 10])
    want = ref.tables(16, 10, 100, add, lens, tab, ring, state, 25)
    assert (want["slots"][16:20] == -1).all() and want["slots"][20] == 64
    _check_tables(_run_tables(p, add, lens, tab, ring, state, 25), want)


def test_tables_without_tokens(cuda_device):
    p = _mb().MobaCacheParams(2, 100, 10, 16, 1, 1, 64, 128, 1)
    add, lens = np.array([0, -1]), np.array([5, 33])
    rng = np.random.default_rng(1)
    tab, ring, state = _tables_state(rng, 2, 100, 16, 10, add, lens)
    want = ref.tables(16, 10, 100, add, lens, tab, ring, state, 0)
    _check_tables(_run_tables(p, add, lens, tab, ring, state, 0), want)


# ---------------------------------------------------------------------------------- append

class Pool:
    """A pool with random codes and scales, rows of distinct pages in any order."""

    def __init__(self, rng, B, max_len, P, ps, H, D, fmt, garbage=True):
        import torch
        self.fmt, self.ps, self.P = fmt, ps, P
        MP = -(-max_len // ps)
        assert P >= B * MP
        self.tab = rng.permutation(P)[:B * MP].reshape(B, MP).astype(np.int32)
        raw = rng.integers(0, 256, (2, P, H, ps, D)).astype(np.uint8)
        if fmt == "int8":
            raw[raw == 128] = 127
        else:
            raw[(raw & 127) == 127] = 0x30
            raw &= 0xBF  # magnitudes below 2, so that a page is not ruled by its few largest codes
        self.Kc, self.Vc = (torch.from_numpy(raw[i]).cuda().view(_code_dtype(fmt)) for i in range(2))
        sc = np.exp2(rng.uniform(-6, -5, (2, P, H)) - (0 if fmt == "e4m3" else 5)).astype(np.float32)
        sc = (sc.view(np.uint32) & 0xffff0000).view(np.float32)
        if fmt == "e4m3":
            sc *= 32
        self.Ks, self.Vs = _dev(sc[0]), _dev(sc[1])

    def values(self):
        return (_values(self.Kc, self.fmt), _values(self.Vc, self.fmt), self.Ks.cpu().numpy().astype(np.float64),
                self.Vs.cpu().numpy().astype(np.float64))


def _append_case(rng, p, pool, old, add, N, kv, fmt, ps, bs, D, H, kbar):
    """Runs the append once and compares everything that it may touch with the reference."""
    import torch
    mb = _mb()
    B = len(old)
    cu = np.zeros(B + 1, np.int32)
    cu[1:] = np.cumsum(add)
    lens = (old + add).astype(np.int32)
    slots = np.full(N, -1, np.int32)
    for s in range(B):
        for j in range(add[s]):
            pos = old[s] + j
            slots[cu[s] + j] = pool.tab[s, pos // ps] * ps + pos % ps
    kc, vc, ks, vs = pool.values()
    K, V = kv
    kf, vf = K.double().cpu().numpy(), V.double().cpu().numpy()
    want_k, want_ks = ref.append(fmt, ps, bs, kf, cu, lens, slots, kc, ks)
    want_v, want_vs = ref.append(fmt, ps, bs, vf, cu, lens, slots, vc, vs)
    pooled = ref.pooled(ps, bs, cu, lens, pool.tab, want_k, want_ks)
    before = kbar.clone()
    args = (_dev(cu), _dev(lens), _dev(slots), _dev(pool.tab), pool.Kc, pool.Vc, pool.Ks, pool.Vs, kbar)
    for _ in range(2):  # the second time changes nothing more
        mb.moba_cache_append(p, K, V, *args)
        _no_error()
        np.testing.assert_array_equal(_values(pool.Kc, fmt), want_k)
        np.testing.assert_array_equal(_values(pool.Vc, fmt), want_v)
        np.testing.assert_array_equal(pool.Ks.cpu().numpy(), want_ks)
        np.testing.assert_array_equal(pool.Vs.cpu().numpy(), want_vs)
        got = kbar.cpu().numpy().astype(np.float64)
        rest = before.cpu().numpy().astype(np.float64)
        for (s, b), (mean, mag) in pooled.items():
            np.testing.assert_array_less(np.abs(got[s, b] - mean), (bs / 32 + 17) * 2.0 ** -24 * mag + 1e-40)
            rest[s, b] = got[s, b]
        np.testing.assert_array_equal(got, rest)
    return len(pooled)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,max_len,ps,H,D,bs,new", [
    (1, 1, 16, 1, 64, 128, 1), (5, 300, 32, 2, 64, 128, 1), (4, 700, 128, 3, 128, 256, 9), (3, 1500, 64, 2, 128, 384, 700),
    (2, 1030, 16, 1, 128, 128, 900), (9, 400, 16, 8, 64, 128, 60), (1, 2300, 128, 2, 128, 1024, 2300),
    (40, 130, 32, 1, 64, 128, 2), (300, 220, 16, 1, 64, 128, 200), (140, 600, 32, 2, 128, 256, 400)])
def test_append(B, max_len, ps, H, D, bs, new, fmt, cuda_device):
    import torch
    rng = np.random.default_rng(B * 7 + new)
    P = B * -(-max_len // ps) + 3
    p = _mb().MobaCacheParams(B, max_len, P, ps, H, H, D, bs, 1, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    add = np.minimum(rng.integers(0, new + 1, B), max_len)
    add[rng.integers(B)] = new
    old = np.array([rng.integers(0, max_len - a + 1) for a in add])
    if max_len % bs == 0 or B > 3:  # one that ends with its block, one that begins on a page
        s = int(np.argmax(add))
        old[s] = max(0, (old[s] + add[s]) // bs * bs - add[s])
    N = int(add.sum()) + 5
    # K and V side by side in one projection; some rows far larger than the pages' scales
    kv = rng.standard_normal((N, 2, H, D)) * np.exp(rng.standard_normal((N, 1, 1, 1)))
    kv[N - 5:] = np.nan  # rows behind the last token are not read
    kv = _bf16(kv)
    kbar = torch.full((B, p.max_blocks, H, D), 7.0, device="cuda")
    _append_case(rng, p, pool, old, add, N, (kv[:, 0], kv[:, 1]), fmt, ps, bs, D, H, kbar)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("ps,D,H,bs", [(32, 64, 2, 128), (16, 128, 5, 256), (64, 128, 1, 512), (128, 64, 3, 384)])
def test_append_long_runs_beside_short_ones(ps, D, H, bs, fmt, cuda_device):
    """Requests with a long prompt, at and around four pages, with single tokens and with none, in one call."""
    import torch
    rng = np.random.default_rng(ps)
    B, max_len = 150, 1500
    add = rng.integers(0, 3, B)
    for s, n in zip((3, 40, 41, 129, 149), (1100, 4 * ps, 4 * ps - 1, 4 * ps + 1, 2 * ps)):
        add[s] = n
    old = np.array([rng.integers(0, min(max_len - a, 400) + 1) for a in add])
    N = int(add.sum()) + 3
    assert 4 * ps <= N < 2 * ps * B and N > 4 * B  # two launches
    P = B * -(-max_len // ps)
    p = _mb().MobaCacheParams(B, max_len, P, ps, H, H, D, bs, 1, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    kv = _bf16(rng.standard_normal((N, 2, H, D)) * np.exp(rng.standard_normal((N, 1, 1, 1))))
    kbar = torch.full((B, p.max_blocks, H, D), 7.0, device="cuda")
    assert _append_case(rng, p, pool, old, add, N, (kv[:, 0], kv[:, 1]), fmt, ps, bs, D, H, kbar) > 2


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_values_at_the_edges(fmt, cuda_device):
    """Zero pages, the smallest and largest magnitudes, infinities and NaN, exact ties."""
    import torch
    rng = np.random.default_rng(9)
    B, max_len, ps, H, D, bs = 6, 64, 16, 1, 64, 128
    P = B * 4
    p = _mb().MobaCacheParams(B, max_len, P, ps, H, H, D, bs, 1, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    add, old = np.array([16, 16, 16, 16, 16, 3]), np.array([0, 0, 16, 0, 16, 5])
    N = int(add.sum())
    x = rng.standard_normal((N, 2, H, D))
    x[0:16] = 0
    x[16:32] *= 2.0 ** -120
    x[32:48] *= 2.0 ** 120
    x[50, :, :, 3], x[51, :, :, 4], x[52, :, :, 5] = np.inf, -np.inf, np.nan
    # multiples of half a step under a power of two: exact ties
    x[64:80] = rng.integers(-255, 256, (16, 2, H, D)) / 2.0
    x[64, :, :, 0] = ref.QMAX[fmt]
    kv = _bf16(x)
    kbar = torch.zeros(B, 1, H, D, device="cuda")
    _append_case(rng, p, pool, old, add, N, (kv[:, 0].contiguous(), kv[:, 1].contiguous()), fmt, ps, bs, D, H, kbar)


def test_append_grows_a_page_token_by_token(cuda_device):
    """Each token larger than the last: every step moves the page's older codes to the new scale."""
    import torch
    mb = _mb()
    for fmt in ("e4m3", "int8"):
        p = mb.MobaCacheParams(1, 64, 8, 32, 1, 1, 64, 128, 1, fmt)
        c = mb.MobaCache(p)
        rng = np.random.default_rng(4)
        codes, scales = np.zeros((8, 1, 32, 64)), np.zeros((8, 1))
        for t in range(40):
            x = rng.standard_normal((1, 1, 64)) * 1.2 ** t
            K = _bf16(x)
            slots = c.extend(torch.ones(1, dtype=torch.int32, device="cuda"), 1)
            c.append(K, K, slots)
            cu, lens = np.array([0, 1]), np.array([t + 1])
            codes, scales = ref.append(fmt, 32, 128, K.double().cpu().numpy(), cu, lens, slots.cpu().numpy(), codes, scales)
        _no_error()
        np.testing.assert_array_equal(_values(c.Kc, fmt), codes)
        np.testing.assert_array_equal(c.Vs.cpu().numpy(), scales)


def test_append_refuses_bad_slots_and_pages(cuda_device):
    """Slots outside the pool or not at the token's offset, and bad table entries, are left out and
    reported; a negative slot is only left out."""
    import torch
    mb = _mb()
    B, max_len, ps, H, D, bs = 2, 256, 32, 2, 64, 128
    p = mb.MobaCacheParams(B, max_len, 16, ps, H, H, D, bs, 1)
    for bad, err in ((-1, 0), (16 * ps, 2), (2 ** 31 - 32, 2), (5 * ps + 1, 2)):
        rng = np.random.default_rng(2)
        pool = Pool(rng, B, max_len, 16, ps, H, D, "e4m3")
        before = pool.values()
        K = _bf16(rng.standard_normal((40, H, D)))
        slots = np.full(40, -1, np.int32)
        slots[:32], slots[32:] = pool.tab[0, 0] * ps + np.arange(32), bad
        kbar = torch.zeros(B, 2, H, D, device="cuda")
        mb.moba_cache_append(p, K, K, _dev(np.array([0, 40, 40], np.int32)), _dev(np.array([40, 0], np.int32)),
                             _dev(slots), _dev(pool.tab), pool.Kc, pool.Vc, pool.Ks, pool.Vs, kbar)
        torch.cuda.synchronize()
        assert mb.moba_read_device_error(clear=True) == err
        after = pool.values()
        rest = np.ones(16, bool)
        rest[pool.tab[0, 0]] = False
        for a, b in zip(before, after):
            np.testing.assert_array_equal(a[rest], b[rest])
        assert (after[2][pool.tab[0, 0]] != before[2][pool.tab[0, 0]]).any()
    # a table that names no page where a block is pooled
    rng = np.random.default_rng(2)
    pool = Pool(rng, B, max_len, 16, ps, H, D, "e4m3")
    tab = pool.tab.copy()
    tab[0, 1] = 16
    K = _bf16(rng.standard_normal((128, H, D)))
    slots = (pool.tab[0, np.arange(128) // ps] * ps + np.arange(128) % ps).astype(np.int32)
    mb.moba_cache_append(p, K, K, _dev(np.array([0, 128, 128], np.int32)), _dev(np.array([128, 0], np.int32)),
                         _dev(slots), _dev(tab), pool.Kc, pool.Vc, pool.Ks, pool.Vs,
                         torch.zeros(B, 2, H, D, device="cuda"))
    torch.cuda.synchronize()
    assert mb.moba_read_device_error(clear=True) == 2


# ---------------------------------------------------------------------------------- decode

def _decode(p, pool, q, kbar, lens, tab, sel=True):
    import torch
    mb = _mb()
    B, Hq, D = q.shape
    ws = torch.full((p.workspace_bytes,), 0xff, dtype=torch.uint8, device="cuda")
    O = torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((B, Hq), float("nan"), device="cuda")
    s = torch.full((B, Hq, p.c.top_k), -7, dtype=torch.int32, device="cuda") if sel else None
    mb.moba_cache_decode_fwd(p, q, pool.Kc, pool.Vc, pool.Ks, pool.Vs, kbar, _dev(lens.astype(np.int32)), _dev(tab),
                             ws, O, LSE, sel=s)
    torch.cuda.synchronize()
    return O, LSE, s


def _check_decode(p, pool, q, kbar, lens, tab, got):
    O, LSE, sel = got
    c = p.c
    kc, vc, ks, vs = pool.values()
    scale = c.softmax_scale if c.softmax_scale > 0 else c.head_dim ** -0.5
    o, lse, want_sel, wide, zabs = ref.decode(q.double().cpu().numpy(), kc, vc, ks, vs,
                                              kbar.double().cpu().numpy(), lens, tab, c.page_size, c.block_size,
                                              c.top_k, scale)
    if sel is not None:
        np.testing.assert_array_equal(sel.cpu().numpy(), want_sel)
    dz = (c.head_dim + 8) * 2.0 ** -24 * zabs + 2.0 ** -21
    got_l, got_o = LSE.double().cpu().numpy(), O.double().cpu().numpy()
    np.testing.assert_array_equal(np.isneginf(got_l), np.isneginf(lse))
    fin = np.isfinite(lse)
    bits = np.abs(lse[fin]) + 24 + zabs[fin]
    assert np.all(np.abs(got_l[fin] - lse[fin]) <= dz[fin] + 4 * 2.0 ** -24 * bits)
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * dz[..., None]) * wide
    assert np.all(np.abs(got_o - o) <= tol), np.max(np.abs(got_o - o) - tol)


def _kbar_of(pool, B, max_len, ps, bs, H, D):
    kc, _, ks, _ = pool.values()
    out = np.full((B, -(-max_len // bs), H, D), np.nan, np.float32)  # incomplete blocks are not read
    for s in range(B):
        for b in range(max_len // bs):
            pages = pool.tab[s, b * bs // ps:(b + 1) * bs // ps]
            out[s, b] = (kc[pages] * ks[pages][:, :, None, None]).sum((0, 2)) / bs
    return _dev(out)


DECODE = [
    # B, max_len, ps, Hq, Hkv, D, bs, k
    (1, 1, 16, 1, 1, 64, 128, 1),
    (4, 700, 16, 4, 2, 128, 128, 3),
    (3, 2000, 32, 8, 1, 64, 256, 5),          # eight heads on one KV head
    (2, 1500, 128, 16, 1, 128, 128, 2),       # more heads than one matrix tile holds
    (2, 1111, 64, 36, 2, 64, 384, 4),         # 18 heads to a group
    (5, 999, 64, 6, 2, 128, 128, 16),         # top_k 16 with at most 8 blocks
    (1, 9000, 128, 3, 1, 128, 128, 8),        # 70 candidate blocks, an odd group
    (1, 20000, 32, 2, 2, 64, 128, 16),        # 156 candidate blocks
    (2, 17000, 64, 4, 2, 128, 8192, 3),       # the largest block
    (70, 300, 16, 4, 4, 64, 128, 3),          # many short requests
    (2, 5000, 64, 4, 1, 128, 2048, 3),
    (1, 70000, 16, 2, 1, 64, 128, 4),         # 546 candidate blocks, small pages
    (1, 140000, 128, 1, 1, 64, 128, 3),       # 1093 candidate blocks
    (5, 127, 16, 6, 2, 64, 128, 4),           # requests of one block at most: nothing to choose from
    (7, 2000, 64, 36, 2, 128, 2048, 3),       # the same, 18 heads to a group
    (3, 1000, 32, 10, 2, 128, 256, 1),        # top_k 1: the own block alone
    (900, 130, 32, 4, 2, 128, 256, 3),        # the same with a long work list
    (800, 20, 16, 2, 2, 128, 128, 2),         # more entries of the work list than are counted one by one
    (1200, 140, 16, 2, 2, 64, 128, 2),
    (40, 2100, 64, 8, 8, 64, 1024, 2),        # units of two pieces
    (30, 1500, 128, 16, 8, 128, 512, 6),      # three units and more for each warp
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,max_len,ps,Hq,H,D,bs,k", DECODE)
def test_decode(B, max_len, ps, Hq, H, D, bs, k, fmt, cuda_device):
    rng = np.random.default_rng(max_len + k)
    P = B * -(-max_len // ps) + 2
    p = _mb().MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    kbar = _kbar_of(pool, B, max_len, ps, bs, H, D)
    edges = [max_len, 1, 0, bs, bs + 1, 2 * bs - 1, ps, ps + 1, max_len - 1, 3 * ps - 1]
    lens = np.array([max(0, min(edges[s % len(edges)], max_len)) for s in range(B)])
    q = _bf16(rng.standard_normal((B, Hq, D)))
    got = _decode(p, pool, q, kbar, lens, pool.tab)
    _check_decode(p, pool, q, kbar, lens, pool.tab, got)
    _no_error()
    # again, without a selection and at other lengths: the same rows of the work space, nothing left over
    lens2 = rng.integers(0, max_len + 1, B)
    _check_decode(p, pool, q, kbar, lens2, pool.tab, _decode(p, pool, q, kbar, lens2, pool.tab, sel=False))
    # deterministic
    again = _decode(p, pool, q, kbar, lens, pool.tab)
    assert all((a.view(dtype=t) == b.view(dtype=t)).all() for a, b, t in zip(got, again, _int_types()))


def _int_types():
    import torch
    return torch.int16, torch.int32, torch.int32


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_is_blind_to_what_lies_behind(fmt, cuda_device):
    """NaN codes behind the newest token, NaN scales of pages that no request holds, table entries behind a
    request's last page: without effect."""
    import torch
    rng = np.random.default_rng(8)
    B, max_len, ps, Hq, H, D, bs, k = 4, 600, 64, 4, 2, 128, 256, 2
    P = B * 10 + 4
    p = _mb().MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    kbar = _kbar_of(pool, B, max_len, ps, bs, H, D)
    lens = np.array([600, 65, 193, 1])
    q = _bf16(rng.standard_normal((B, Hq, D)))
    clean = _decode(p, pool, q, kbar, lens, pool.tab)
    _check_decode(p, pool, q, kbar, lens, pool.tab, clean)
    tab = pool.tab.copy()
    kc, vc = pool.Kc.view(torch.uint8), pool.Vc.view(torch.uint8)
    used = set()
    for s in range(B):
        n = int(lens[s])
        last = (n - 1) // ps
        kc[pool.tab[s, last], :, (n - 1) % ps + 1:] = 0x7f
        vc[pool.tab[s, last], :, (n - 1) % ps + 1:] = 0xff
        tab[s, last + 1:] = [(-1, P, 2 ** 31 - 1, -2 ** 31)[i % 4] for i in range(tab.shape[1] - last - 1)]
        used |= set(pool.tab[s, :last + 1].tolist())
    free = torch.tensor([i for i in range(P) if i not in used], device="cuda")
    pool.Ks[free], pool.Vs[free] = float("nan"), float("inf")
    dirty = _decode(p, pool, q, kbar, lens, tab)
    _no_error()
    assert all((a.view(dtype=t) == b.view(dtype=t)).all() for a, b, t in zip(clean, dirty, _int_types()))


def test_decode_with_bad_pages_and_lengths(cuda_device):
    """Keys of a page outside the pool are masked and reported; with none left the row is empty.  A
    length outside the range counts as 0."""
    rng = np.random.default_rng(8)
    B, max_len, ps, Hq, H, D, bs, k = 4, 600, 32, 4, 2, 64, 128, 3
    P = B * 19
    mb = _mb()
    p = mb.MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k)
    pool = Pool(rng, B, max_len, P, ps, H, D, "e4m3")
    kbar = _kbar_of(pool, B, max_len, ps, bs, H, D)
    q = _bf16(rng.standard_normal((B, Hq, D)))
    tab = pool.tab.copy()
    tab[0, ::2], tab[1, :] = P, -1
    lens = np.array([600, 100, 77, 300])
    got = _decode(p, pool, q, kbar, lens, tab)
    assert mb.moba_read_device_error(clear=True) == 2
    _check_decode(p, pool, q, kbar, lens, tab, got)
    assert (got[0][1] == 0).all() and (got[1][1] == -np.inf).all()
    got = _decode(p, pool, q, kbar, np.array([601, -5, 77, 2 ** 31 - 1]), pool.tab)
    _no_error()
    _check_decode(p, pool, q, kbar, np.array([0, 0, 77, 0]), pool.tab, got)


def test_decode_ties_and_non_finite(cuda_device):
    """Equal scores go to the lower block; a NaN query gives NaN and a valid selection; a NaN pooled key
    ranks last; other rows are untouched by either."""
    import torch
    rng = np.random.default_rng(8)
    B, max_len, ps, Hq, H, D, bs, k = 3, 40 * 128, 128, 8, 2, 64, 128, 6
    P = B * 40
    p = _mb().MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k)
    pool = Pool(rng, B, max_len, P, ps, H, D, "e4m3")
    kbar = _kbar_of(pool, B, max_len, ps, bs, H, D)
    kbar[0, 5:30] = kbar[0, 4]       # ties among 26 blocks
    kbar[1, :, 1] = 0                # all tie
    kbar[1, 3, 1] = -0.0
    kbar[2, 7, 0] = float("nan")
    q = rng.standard_normal((B, Hq, D))
    q[2, 6] = np.nan
    q[2, 7, 5] = np.inf
    q = _bf16(q)
    lens = np.array([max_len, max_len - 3, max_len])
    O, LSE, sel = _decode(p, pool, q, kbar, lens, pool.tab)
    _no_error()
    assert O[2, 6].isnan().all() and LSE[2, 6].isnan()
    s = sel.cpu().numpy()
    assert (s[2, 6:] >= 0).all() and (s[2, 6:] < 40).all() and all(len(set(r)) == k for r in s[2, 6:])
    assert (s[1, 4:] == [39, 0, 1, 2, 3, 4]).all()
    live = np.array([h for h in range(Hq) if h < 6])
    sub = _mb().MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k)
    qq = q.clone()
    qq[2, 6:] = 0
    want = _decode(sub, pool, qq, kbar, lens, pool.tab)
    _check_decode(sub, pool, qq, kbar, lens, pool.tab, want)
    assert (want[0][:, live].view(torch.int16) == O[:, live].view(torch.int16)).all()
    assert (want[2][:, live] == sel[:, live]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_wide_range_of_scales(fmt, cuda_device):
    """Pages whose scales lie far apart, queries far from 1, a softmax scale of the caller's: the weights of
    pages with small values keep their precision."""
    import torch
    rng = np.random.default_rng(12)
    B, max_len, ps, Hq, H, D, bs, k = 3, 400, 16, 4, 2, 64, 128, 3
    P = B * 25
    for vexp, qexp, zs in ((30, 0, 0.0), (8, -60, 2.0 ** 58), (0, 40, 2.0 ** -43)):
        p = _mb().MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k, fmt, zs)
        pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
        pool.Vs *= torch.exp2(torch.from_numpy(rng.integers(-vexp, vexp + 1, tuple(pool.Vs.shape))).cuda()).float()
        pool.Vc.view(torch.uint8)[pool.tab[0, 3]] = 0
        pool.Vs[pool.tab[0, 3]] = 2.0 ** -104  # what a page of zeros gets
        kbar = _kbar_of(pool, B, max_len, ps, bs, H, D)
        q = _bf16(rng.standard_normal((B, Hq, D)) * 2.0 ** qexp)
        lens = np.array([400, 129, 64])
        _check_decode(p, pool, q, kbar, lens, pool.tab, _decode(p, pool, q, kbar, lens, pool.tab))
        _no_error()


def test_decode_refuses_other_tensors(cuda_device):
    import torch
    mb = _mb()
    rng = np.random.default_rng(1)
    p = mb.MobaCacheParams(2, 100, 10, 32, 2, 1, 64, 128, 1)
    pool = Pool(rng, 2, 100, 10, 32, 1, 64, "e4m3")
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    kbar, lens = torch.zeros(2, 1, 1, 64, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    O, LSE, ws = torch.zeros_like(q), torch.zeros(2, 2, device="cuda"), mb.alloc_cache_workspace(p)
    tab = _dev(pool.tab)

    def call(**kw):
        a = dict(Q=q, Kc=pool.Kc, Vc=pool.Vc, Ks=pool.Ks, Vs=pool.Vs, Kbar=kbar, lens=lens, tables=tab, workspace=ws,
                 O=O, LSE=LSE)
        a.update(kw)
        mb.moba_cache_decode_fwd(p, **a)

    call()
    for bad in (dict(Q=q.float()), dict(Q=q.transpose(0, 1)), dict(Kc=pool.Kc.view(torch.uint8)), dict(lens=lens.cpu()),
                dict(tables=tab[:, :3]), dict(O=O.expand(2, 2, 64)[:1]), dict(workspace=ws[:-1]), dict(LSE=LSE.double())):
        with pytest.raises(mb.MobaError):
            call(**bad)
    _no_error()


def test_decode_far_into_a_large_pool(cuda_device):
    """Pages whose codes lie behind 4 GB, appended to and read."""
    import torch
    mb = _mb()
    H, ps, D, fmt = 2, 128, 128, "int8"
    P = 140000  # 4.6 GB of codes each for keys and values
    p = mb.MobaCacheParams(2, 600, P, ps, 4, H, D, 256, 3, fmt)
    rng = np.random.default_rng(6)
    tab = (P - 1 - rng.permutation(10)).reshape(2, 5).astype(np.int32)
    add, cu = np.array([600, 333], np.int32), np.array([0, 600, 933], np.int32)
    slots = np.concatenate([tab[s, np.arange(n) // ps] * ps + np.arange(n) % ps for s, n in enumerate(add)]).astype(np.int32)
    kv, q = _bf16(rng.standard_normal((933, 2, H, D))), _bf16(rng.standard_normal((2, 4, D)))
    Kc, Vc = (torch.empty(P, H, ps, D, dtype=torch.int8, device="cuda") for _ in range(2))
    Ks, Vs = (torch.empty(P, H, device="cuda") for _ in range(2))
    kbar = torch.zeros(2, 3, H, D, device="cuda")
    mb.moba_cache_append(p, kv[:, 0], kv[:, 1], _dev(cu), _dev(add), _dev(slots), _dev(tab), Kc, Vc, Ks, Vs, kbar)
    small = type("P", (), {})()  # the ten pages by themselves
    order = tab.flatten().astype(np.int64)
    at = torch.from_numpy(order).cuda()
    kc, vc = (ref.code_values(fmt)[x[at].view(torch.uint8).cpu().numpy()] for x in (Kc, Vc))
    ks, vs = (x[at].cpu().numpy().astype(np.float64) for x in (Ks, Vs))
    zero = np.zeros((10, H, ps, D)), np.zeros((10, H))
    place = np.full(P, -1)
    place[order] = np.arange(10)
    near = place[slots // ps] * ps + slots % ps
    for got, scales, x in ((kc, ks, kv[:, 0]), (vc, vs, kv[:, 1])):
        want, want_s = ref.append(fmt, ps, 256, x.double().cpu().numpy(), cu, add, near, *zero)
        used = [place[tab[s, j]] for s, n in enumerate(add) for j in range(-(-n // ps))]
        np.testing.assert_array_equal(scales[used], want_s[used])
        for s, n in enumerate(add):
            for pos in (0, 127, 128, n - 1):
                np.testing.assert_array_equal(got[place[tab[s, pos // ps]], :, pos % ps], want[place[tab[s, pos // ps]], :, pos % ps])
    O, LSE, sel = torch.empty_like(q), torch.empty(2, 4, device="cuda"), torch.empty(2, 4, 3, dtype=torch.int32, device="cuda")
    mb.moba_cache_decode_fwd(p, q, Kc, Vc, Ks, Vs, kbar, _dev(add), _dev(tab), mb.alloc_cache_workspace(p), O, LSE, sel=sel)
    _no_error()
    small.values = lambda: (kc, vc, ks, vs)
    _check_decode(p, small, q, kbar, add, place[tab], (O, LSE, sel))


@pytest.mark.parametrize("B,max_len,Hq,H,D,bs,k", [(2, 3000, 8, 2, 128, 256, 4), (40, 900, 8, 4, 64, 128, 3)])
def test_decode_calls_back_to_back_share_a_workspace(B, max_len, Hq, H, D, bs, k, cuda_device):
    """Calls on different inputs, one behind the other without a wait, on one work space."""
    import torch
    mb = _mb()
    rng = np.random.default_rng(B)
    ps = 32
    P = B * -(-max_len // ps)
    p = mb.MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k)
    pool = Pool(rng, B, max_len, P, ps, H, D, "e4m3")
    kbar, tab = _kbar_of(pool, B, max_len, ps, bs, H, D), _dev(pool.tab)
    sets = []
    for _ in range(5):
        lens = rng.integers(0, max_len + 1, B)
        q = _bf16(rng.standard_normal((B, Hq, D)))
        sets.append((q, _dev(lens.astype(np.int32)), _decode(p, pool, q, kbar, lens, pool.tab)))
    ws, got = mb.alloc_cache_workspace(p), []
    for i in range(60):
        q, lens, _ = sets[i % 5]
        O, LSE = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
        sel = torch.empty(B, Hq, k, dtype=torch.int32, device="cuda")
        mb.moba_cache_decode_fwd(p, q, pool.Kc, pool.Vc, pool.Ks, pool.Vs, kbar, lens, tab, ws, O, LSE, sel=sel)
        got.append((O, LSE, sel))
    _no_error()
    for i, g in enumerate(got):
        assert all((a.view(dtype=t) == b.view(dtype=t)).all() for a, b, t in zip(g, sets[i % 5][2], _int_types()))


# ---------------------------------------------------------------------------------- together

class Model:
    """The reference's copy of one cache, step by step."""

    def __init__(self, p, fmt):
        c = p.c
        self.c, self.fmt = c, fmt
        pool = (c.num_pages, c.num_kv_heads)
        self.kc, self.vc = np.zeros(pool + (c.page_size, c.head_dim)), np.zeros(pool + (c.page_size, c.head_dim))
        self.ks, self.vs = np.zeros(pool), np.zeros(pool)
        self.lens, self.tab = np.zeros(c.max_seqs, np.int32), np.zeros((c.max_seqs, p.pages_per_seq), np.int32)
        self.ring, self.state = np.arange(c.num_pages, dtype=np.int32), np.array([0, c.num_pages])

    def step(self, add, K, V, N):
        c = self.c
        t = ref.tables(c.page_size, c.num_pages, c.max_seqlen, add, self.lens, self.tab, self.ring, self.state, N)
        self.lens, self.tab, self.ring, self.state = t["lens"], t["tables"], t["ring"], t["state"]
        args = (self.fmt, c.page_size, c.block_size)
        self.kc, self.ks = ref.append(*args, K.double().cpu().numpy(), t["cu"], self.lens, t["slots"], self.kc, self.ks)
        self.vc, self.vs = ref.append(*args, V.double().cpu().numpy(), t["cu"], self.lens, t["slots"], self.vc, self.vs)
        return t


def _serve(p, fmt, steps, seed, graph):
    """A small server: prompts, single tokens, requests that end and slots that are taken again."""
    import torch
    mb = _mb()
    c, rng = p.c, np.random.default_rng(seed)
    B, N = c.max_seqs, 300
    cache, model = mb.MobaCache(p), Model(p, fmt)
    add_d = torch.zeros(B, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(N, c.num_q_heads + 2 * c.num_kv_heads, c.head_dim, dtype=torch.bfloat16, device="cuda")
    Q = torch.zeros(B, c.num_q_heads, c.head_dim, dtype=torch.bfloat16, device="cuda")
    sel = torch.zeros(B, c.num_q_heads, c.top_k, dtype=torch.int32, device="cuda")
    K, V = qkv[:, c.num_q_heads:c.num_q_heads + c.num_kv_heads], qkv[:, c.num_q_heads + c.num_kv_heads:]

    def step():
        slots = cache.extend(add_d, N)
        cache.append(K, V, slots)
        return cache.decode(Q, sel=sel)

    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # add is all 0: nothing changes
        torch.cuda.current_stream().wait_stream(side)
        G = torch.cuda.CUDAGraph()
        with torch.cuda.graph(G):
            O, LSE = step()
    for i in range(steps):
        add = np.where(model.lens > 0, 1, 0)
        for s in range(B):
            if model.lens[s] == 0 and rng.random() < 0.5:
                add[s] = rng.integers(1, 1 + min(N // B, c.max_seqlen - 8))
            elif model.lens[s] > 0 and (rng.random() < 0.1 or model.lens[s] >= c.max_seqlen):
                add[s] = -1
            elif model.lens[s] > 0 and rng.random() < 0.2:
                add[s] = min(int(rng.integers(2, N // B)), c.max_seqlen - int(model.lens[s]))
        add_d.copy_(_dev(add.astype(np.int32)))
        qkv.copy_(_bf16(rng.standard_normal(tuple(qkv.shape)) * 2.0 ** rng.integers(-2, 3)))
        Q.copy_(_bf16(rng.standard_normal(tuple(Q.shape))))
        if graph:
            G.replay()
        else:
            O, LSE = step()
        torch.cuda.synchronize()
        model.step(add, K, V, N)
        assert int(cache.status) == 0
        np.testing.assert_array_equal(cache.lens.cpu().numpy(), model.lens)
        for got, want in ((cache.tables, model.tab), (cache.free_pages, model.ring), (cache.free_state, model.state),
                          (cache.Ks, model.ks), (cache.Vs, model.vs)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        np.testing.assert_array_equal(_values(cache.Kc, fmt), model.kc)
        np.testing.assert_array_equal(_values(cache.Vc, fmt), model.vc)
        pool = type("P", (), dict(values=lambda self: (model.kc, model.vc, model.ks, model.vs)))()
        _check_decode(p, pool, Q, cache.Kbar, model.lens, model.tab, (O, LSE, sel))
        for s in range(B):  # the pooled keys in use are those of the stored keys
            for b in range(max(0, (int(model.lens[s]) - 1) // c.block_size)):
                pages = model.tab[s, b * c.block_size // c.page_size:(b + 1) * c.block_size // c.page_size]
                v = model.kc[pages] * model.ks[pages][:, :, None, None]
                d = np.abs(cache.Kbar[s, b].double().cpu().numpy() - v.sum((0, 2)) / c.block_size)
                assert np.all(d <= (c.block_size / 32 + 17) * 2.0 ** -24 * np.abs(v).sum((0, 2)) / c.block_size)
    _no_error()


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("fmt,ps,D,Hq,H,bs", [("e4m3", 16, 64, 4, 2, 128), ("int8", 64, 128, 3, 1, 256)])
def test_serving_steps(fmt, ps, D, Hq, H, bs, graph, cuda_device):
    B, max_len = 6, 700
    p = _mb().MobaCacheParams(B, max_len, B * -(-max_len // ps), ps, Hq, H, D, bs, 3, fmt)
    _serve(p, fmt, 30, seed=ps, graph=graph)


def test_graph_replays_without_a_wait_between_them(cuda_device):
    """A captured step that advances the lengths itself, replayed at once many times: the same as the steps
    one by one."""
    import torch
    mb = _mb()
    rng = np.random.default_rng(5)
    p = mb.MobaCacheParams(3, 500, 60, 32, 4, 2, 64, 128, 3, "int8")
    kv, q = _bf16(rng.standard_normal((200, 2, 2, 64))), _bf16(rng.standard_normal((3, 4, 64)))
    first, one = _dev(np.array([100, 33, 60], np.int32)), torch.ones(3, dtype=torch.int32, device="cuda")
    out = []
    for graph in (False, True):
        c = mb.MobaCache(p)
        c.append(kv[:193, 0], kv[:193, 1], c.extend(first, 193))

        def step():
            slots = c.extend(one, 3)
            c.append(kv[:3, 0], kv[:3, 1], slots)
            return c.decode(q)

        O, LSE = step()
        if graph:
            G = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(G):
                O, LSE = step()
            for _ in range(300):
                G.replay()
        else:
            for _ in range(300):
                O, LSE = step()
        _no_error()
        out.append((O, LSE, c.lens, c.tables, c.free_pages, c.free_state, c.Kc, c.Vc, c.Ks, c.Vs, c.Kbar))
    assert out[0][2].tolist() == [401, 334, 361]
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_streams_given_by_object_and_by_address(cuda_device):
    import torch
    mb = _mb()
    rng = np.random.default_rng(78)
    p = mb.MobaCacheParams(2, 900, 30, 64, 4, 2, 64, 128, 3)
    kv, q = _bf16(rng.standard_normal((1000, 2, 2, 64))), _bf16(rng.standard_normal((2, 4, 64)))
    add = _dev(np.array([700, 300], np.int32))
    want = None
    for how in (None, "object", "address"):
        c = mb.MobaCache(p)
        side = torch.cuda.Stream()
        st = None if how is None else side if how == "object" else side.cuda_stream
        slots, O, LSE = torch.empty(1000, dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty(2, 4, device="cuda")
        torch.cuda.synchronize()
        mb.moba_cache_tables(p, add, c.lens, c.tables, c.free_pages, c.free_state, c.lens, c.free_state, c.cu_new, slots,
                             c.status, stream=st)
        mb.moba_cache_append(p, kv[:, 0], kv[:, 1], c.cu_new, c.lens, slots, c.tables, c.Kc, c.Vc, c.Ks, c.Vs, c.Kbar,
                             stream=st)
        mb.moba_cache_decode_fwd(p, q, c.Kc, c.Vc, c.Ks, c.Vs, c.Kbar, c.lens, c.tables, c.workspace, O, LSE, stream=st)
        _no_error()
        assert int(c.status) == 0 and LSE.isfinite().all()
        want = want or (O, LSE)
        assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])


def test_two_caches_on_two_streams(cuda_device):
    """Independent caches on streams of their own, at the same time."""
    import torch
    mb = _mb()
    out = []
    for run in range(2):
        streams = [torch.cuda.Stream() for _ in range(2)] if run else [torch.cuda.current_stream()] * 2
        rng = np.random.default_rng(77)
        work = []
        for i in range(2):
            p = mb.MobaCacheParams(4, 4000, 4 * 63, 64, 8, 2, 128, 256, 4, ("e4m3", "int8")[i])
            kv, q = _bf16(rng.standard_normal((8000, 2, 2, 128))), _bf16(rng.standard_normal((4, 8, 128)))
            work.append((mb.MobaCache(p), kv, q, _dev(np.array([3000, 1, 2500, 2000], np.int32))))
        torch.cuda.synchronize()
        res = []
        for _ in range(3):
            for (c, kv, q, add), st in zip(work, streams):
                with torch.cuda.stream(st):
                    slots = c.extend(add if not res else (add > 0).int(), 8000)
                    c.append(kv[:, 0], kv[:, 1], slots)
                    res.append(c.decode(q))
        torch.cuda.synchronize()
        out.append(res)
    _no_error()
    for (a, b), (x, y) in zip(*out):
        assert torch.equal(a, x) and torch.equal(b, y)


def test_prompts_through_prefill_then_decode(cuda_device):
    """The pieces as a server uses them: prefill attention over the bf16 prompt, its keys and values into the
    cache, then decode; the row of the prompt's last token agrees with the prefill's up to the 8-bit rounding."""
    import torch
    mb = _mb()
    rng = np.random.default_rng(31)
    lens, Hq, H, D, bs, k, ps = [900, 1, 513], 8, 2, 128, 128, 4, 64
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    Q, K, V = (_bf16(rng.standard_normal((T, h, D))) for h in (Hq, H, H))
    p = mb.MobaParams(cu, Hq, H, D, bs, k)
    O, LSE = torch.empty_like(Q), torch.empty(T, Hq, device="cuda")
    sel = torch.empty(T, Hq, k, dtype=torch.int32, device="cuda")
    mb.moba_fwd(p, Q, K, V, mb.alloc_workspace(p), O, LSE, sel=sel)
    c = mb.MobaCache(mb.MobaCacheParams(3, 1024, 48, ps, Hq, H, D, bs, k, "int8"))
    slots = c.extend(_dev(np.array(lens, np.int32)), T)
    c.append(K, V, slots)
    last = torch.from_numpy(cu[1:].astype(np.int64) - 1).cuda()
    dsel = torch.empty(3, Hq, k, dtype=torch.int32, device="cuda")
    dO, dL = c.decode(Q[last].contiguous(), sel=dsel)
    _no_error()
    same = (dsel.sort(-1).values == sel[last].sort(-1).values).all(-1)
    assert same.float().mean() > 0.5  # the gate sees the stored keys: close scores may change places
    # int8 with a scale for 64 tokens: each key and value is off by half a step of at most max/127
    # (max about 4.5): 0.018; logits by at most 0.018 * sum |q| / sqrt(D), about 0.018 * 0.8 * sqrt(D) = 0.17
    # in the worst case of all signs alike, and by a tenth of that in the mean over independent errors
    assert (dL - LSE[last])[same].abs().max() < 0.17
    assert (dO.float() - O[last].float())[same].abs().max() < 0.17 * 4.5
