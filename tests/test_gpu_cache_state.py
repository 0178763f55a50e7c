"""Block tables of a paged cache whose state does not add up: refused, nothing changed.

A call takes ring positions [head, head + need) and writes [head + count, head + count + back), both
modulo the pool, without an order between the two: they are apart exactly if count + back is at most
the pool.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _run(B, max_len, P, ps, add, lens, tab, ring, state, N, in_place):
    """Status, and whether everything that a refused call leaves alone is as it was."""
    import torch
    import block_sparse_attention_gate_b200 as mb
    p = mb.MobaCacheParams(B, max_len, P, ps, 1, 1, 64, 128, 1)
    d = [torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda() for a in (add, lens, tab, ring, state)]
    was = [t.clone() for t in d]
    lens_out, state_out = (d[1], d[4]) if in_place else (torch.full_like(d[1], -9), torch.full_like(d[4], -9))
    cu, slots, status = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (B + 1, N, 1))
    mb.moba_cache_tables(p, *d, lens_out, state_out, cu, slots, status)
    torch.cuda.synchronize()
    assert mb.moba_read_device_error(clear=True) == 0
    same = torch.equal(d[2], was[2]) and torch.equal(d[3], was[3])
    same &= torch.equal(lens_out, was[1]) and torch.equal(state_out, was[4])
    same &= bool((cu == 0).all()) and bool((slots == -1).all())
    return int(status), same, (lens_out, d[2], d[3], state_out, cu, slots)


def _state(B, ends, ps, take, P, count, head):
    """`ends` requests of two pages each end, the last request takes `take` pages; `count` are free."""
    MP = max(take, 2)
    lens, add = np.zeros(B, np.int64), np.zeros(B, np.int64)
    lens[:ends], add[:ends] = 2 * ps, -1
    add[B - 1] = take * ps
    tab = np.full((B, MP), -1)
    tab[:ends, :2] = np.arange(2 * ends).reshape(ends, 2) % P
    ring = (np.arange(P) * 7 + 3) % P if P % 7 else np.arange(P)[::-1]
    return add, lens, tab, ring, np.array([head, count]), MP * ps


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [5, 1500])  # one pass over the requests, and two
@pytest.mark.parametrize("over", [0, 1, 4])
def test_pages_given_back_never_reach_those_taken(B, over, in_place, cuda_device):
    """count + back = pool + over, while count - need + back fits."""
    ps, P, ends, take = 16, 40, 4, 6
    count = P - 2 * ends + over
    add, lens, tab, ring, state, max_len = _state(B, ends, ps, take, P, count, head=37)
    assert count - take + 2 * ends <= P
    N = take * ps
    status, same, got = _run(B, max_len, P, ps, add, lens, tab, ring, state, N, in_place)
    if over:
        assert status == 8 and same
        return
    # the largest state that adds up: everything is taken and given back
    assert status == 0
    lens_out, tables, free, st, cu, slots = (t.cpu().numpy() for t in got)
    taken = ring[(37 + np.arange(take)) % P]
    np.testing.assert_array_equal(tables[B - 1, :take], taken)
    np.testing.assert_array_equal(slots, (taken[:, None] * ps + np.arange(ps)).ravel())
    want = ring.copy()
    want[(37 + count + np.arange(2 * ends)) % P] = tab[:ends, :2].ravel()
    np.testing.assert_array_equal(free, want)
    assert st.tolist() == [(37 + take) % P, count - take + 2 * ends]
    assert lens_out[:ends].tolist() == [0] * ends and lens_out[B - 1] == N and cu[B] == N


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [3, 1500])
@pytest.mark.parametrize("what", ["one_ends", "both_end", "none_ends"])
def test_shared_pages_are_refused(what, B, in_place, cuda_device):
    """Ten pages, four of which two requests hold, six free; a third request takes five: whoever ends,
    no page that is still read may be handed out."""
    ps, P = 16, 10
    lens, add = np.zeros(B, np.int64), np.zeros(B, np.int64)
    tab = np.full((B, 5), -1)
    lens[0] = lens[B - 2] = 4 * ps
    tab[0, :4] = tab[B - 2, :4] = np.arange(4)
    ring = np.array([4, 5, 6, 7, 8, 9, -1, -1, -1, -1])
    add[0] = 0 if what == "none_ends" else -1
    add[B - 2] = -1 if what == "both_end" else 0
    add[B - 1] = 5 * ps
    status, same, _ = _run(B, 5 * ps, P, ps, add, lens, tab, ring, np.array([0, 6]), 5 * ps, in_place)
    assert status == 8 and same
    # the same with pages of its own for each: served
    tab[B - 2, :4] = np.arange(4, 8)
    ring = np.array([8, 9] + [-1] * 8)
    add[B - 1] = 2 * ps
    status, _, got = _run(B, 5 * ps, P, ps, add, lens, tab, ring, np.array([0, 2]), 5 * ps, in_place)
    assert status == 0 and got[1][B - 1, :2].tolist() == [8, 9]


def test_one_sharer_ends_and_another_request_grows(cuda_device):
    """Rows made to share pages behind the cache's back: the sharer that stays keeps its stored values."""
    import torch
    import block_sparse_attention_gate_b200 as mb
    p = mb.MobaCacheParams(3, 80, 10, 16, 2, 1, 64, 128, 1)
    c = mb.MobaCache(p)
    i32 = dict(dtype=torch.int32, device="cuda")
    kv = torch.randn(80, 1, 64, device="cuda").bfloat16()
    c.append(kv[:64], kv[:64], c.extend(torch.tensor([64, 0, 0], **i32), 64))
    c.tables[1], c.lens[1] = c.tables[0], 64  # a second request over the same pages
    q = torch.randn(3, 2, 64, device="cuda").bfloat16()
    before = [t[1].clone() for t in c.decode(q)]
    for add in ([-1, 0, 0], [0, 0, 80], [-1, 0, 80], [0, 0, 80]):
        slots = c.extend(torch.tensor(add, **i32), 80)
        assert int(c.status) == 8 and bool((slots == -1).all())
        c.append(kv, kv, slots)
        after = [t[1] for t in c.decode(q)]
        assert all(torch.equal(a, b) for a, b in zip(before, after))
    torch.cuda.synchronize()
    assert mb.moba_read_device_error(clear=True) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_over_rows_that_share_pages(fmt, cuda_device):
    """Tables of the caller's own: requests over one prefix, each with a last page of its own."""
    from test_gpu_cache import Pool, _bf16, _check_decode, _decode, _kbar_of, _no_error
    import block_sparse_attention_gate_b200 as mb
    rng = np.random.default_rng(21)
    B, max_len, ps, Hq, H, D, bs, k = 5, 700, 32, 4, 2, 64, 128, 3
    P = B * -(-max_len // ps)
    p = mb.MobaCacheParams(B, max_len, P, ps, Hq, H, D, bs, k, fmt)
    pool = Pool(rng, B, max_len, P, ps, H, D, fmt)
    pool.tab[1:, :20] = pool.tab[0, :20]
    kbar = _kbar_of(pool, B, max_len, ps, bs, H, D)
    lens = np.array([700, 650, 641, 700, 333])
    q = _bf16(rng.standard_normal((B, Hq, D)))
    _check_decode(p, pool, q, kbar, lens, pool.tab, _decode(p, pool, q, kbar, lens, pool.tab))
    _no_error()
