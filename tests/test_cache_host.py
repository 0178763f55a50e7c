"""Paged 8-bit cache, without a GPU: sizes, refusals of bad arguments before any CUDA call, and the
reference of the parity tests against independent statements of the same formulas."""
import ctypes

import numpy as np
import pytest

import _cache_ref as ref
import block_sparse_attention_gate_b200 as mb

GOOD = dict(max_seqs=3, max_seqlen=1000, num_pages=50, page_size=32, num_q_heads=4, num_kv_heads=2, head_dim=64,
            block_size=128, top_k=3)


@pytest.mark.parametrize("change,status", [
    (dict(max_seqs=0), 1), (dict(max_seqs=65536), 2), (dict(max_seqlen=0), 1), (dict(max_seqlen=(1 << 30) + 1), 2),
    (dict(num_pages=0), 1), (dict(num_pages=1 << 27), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
    (dict(page_size=256), 2), (dict(num_kv_heads=3), 1), (dict(num_q_heads=0), 1), (dict(head_dim=96), 2),
    (dict(num_q_heads=512, num_kv_heads=512), 2), (dict(block_size=100), 2), (dict(block_size=16384), 2),
    (dict(top_k=0), 2), (dict(top_k=17), 2), (dict(max_seqlen=1 << 22, block_size=128), 2),
    (dict(max_seqs=65535, max_seqlen=1 << 20, page_size=16), 2)])
def test_bad_params_are_refused(change, status):
    with pytest.raises(mb.MobaError) as e:
        mb.MobaCacheParams(**{**GOOD, **change})
    assert e.value.status == status
    p = mb.MobaCacheParams(**GOOD)
    for name, value in change.items():
        setattr(p.c, name, value)
    lib = mb.load()
    assert lib.moba_cache_decode_workspace_size(p.ref()) == 0
    rc = lib.moba_cache_tables(p.ref(), 16, 16, 16, 16, 16, 16, 16, 16, 16, 8, 16, None)
    assert rc == status and lib.moba_last_error()


def test_bad_format_is_refused():
    with pytest.raises(mb.MobaError, match="format"):
        mb.MobaCacheParams(**GOOD, format="int4")
    p = mb.MobaCacheParams(**GOOD)
    p.c.format = 2
    assert mb.load().moba_cache_decode_workspace_size(p.ref()) == 0


def test_pointers_are_checked_before_any_cuda_call():
    lib, p = mb.load(), mb.MobaCacheParams(**GOOD)
    n = 9
    good = [16] * n
    for i in range(n):
        args = list(good)
        args[i] = None
        assert lib.moba_cache_tables(p.ref(), *args, 8, 16, None) == 1
        args[i] = 18
        assert lib.moba_cache_tables(p.ref(), *args, 8, 16, None) == 3
    assert lib.moba_cache_tables(p.ref(), *good, -1, 16, None) == 1
    assert lib.moba_cache_tables(p.ref(), *good, 8, None, None) == 1
    row = GOOD["num_kv_heads"] * GOOD["head_dim"]
    rest = [16] * 9
    assert lib.moba_cache_append(p.ref(), None, row, 16, row, 8, *rest, None) == 1
    assert lib.moba_cache_append(p.ref(), 24, row, 16, row, 8, *rest, None) == 3
    assert lib.moba_cache_append(p.ref(), 16, row - 8, 16, row, 8, *rest, None) == 1
    assert lib.moba_cache_append(p.ref(), 16, row, 16, row + 4, 8, *rest, None) == 3
    assert lib.moba_cache_append(p.ref(), 16, row, 16, row, -1, *rest, None) == 1
    assert lib.moba_cache_append(p.ref(), None, row, None, row, 0, *[None] * 9, None) == 0  # nothing to write
    for i in range(9):
        args = list(rest)
        args[i] = None
        assert lib.moba_cache_append(p.ref(), 16, row, 16, row, 8, *args, None) == 1
    ws = p.workspace_bytes
    for i in range(8):
        args = [16] * 8
        args[i] = None
        assert lib.moba_cache_decode_fwd(p.ref(), *args, None, 256, ws, 16, 16, None) == 1
    assert lib.moba_cache_decode_fwd(p.ref(), *[16] * 8, 18, 256, ws, 16, 16, None) == 3
    assert lib.moba_cache_decode_fwd(p.ref(), *[16] * 8, None, None, ws, 16, 16, None) == 4
    assert lib.moba_cache_decode_fwd(p.ref(), *[16] * 8, None, 272, ws, 16, 16, None) == 4
    assert lib.moba_cache_decode_fwd(p.ref(), *[16] * 8, None, 256, ws - 1, 16, 16, None) == 4
    assert lib.moba_cache_decode_fwd(p.ref(), *[16] * 8, None, 256, ws, None, 16, None) == 1


def test_tensor_checks():
    import torch
    p = mb.MobaCacheParams(**GOOD)
    cpu = torch.device("cpu")
    p.check(cpu, add=torch.zeros(3, dtype=torch.int32), Kc=torch.zeros(50, 2, 32, 64).to(torch.float8_e4m3fn))
    for bad in (torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=torch.int32),
                torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(mb.MobaError):
            p.check(cpu, add=bad)
    with pytest.raises(mb.MobaError):
        p.check(cpu, Kc=torch.zeros(50, 2, 32, 64, dtype=torch.int8))
    with pytest.raises(mb.MobaError):
        p.check(torch.device("cuda:0"), add=torch.zeros(3, dtype=torch.int32))
    kv = torch.zeros(5, 2, 2, 64, dtype=torch.bfloat16)
    p.check(cpu, K=kv[:, 0], V=kv[:, 1])  # rows apart
    with pytest.raises(mb.MobaError):
        p.check(cpu, K=kv.transpose(0, 1)[0].transpose(0, 1).contiguous().transpose(0, 1))
    i32 = dict(dtype=torch.int32)
    add = torch.zeros(3, **i32)
    with pytest.raises(mb.MobaError, match="CUDA"):
        mb.moba_cache_tables(p, add, add, torch.zeros(3, 32, **i32), torch.zeros(50, **i32), torch.zeros(2, **i32),
                             add, torch.zeros(2, **i32), torch.zeros(4, **i32), torch.zeros(7, **i32),
                             torch.zeros(1, **i32))
    q = mb.MobaCacheParams(**GOOD, format="int8")
    q.check(cpu, Kc=torch.zeros(50, 2, 32, 64, dtype=torch.int8))


def test_buffers_match_the_header():
    p = mb.MobaCacheParams(**GOOD)
    assert p.pages_per_seq == 32 and p.max_blocks == 8
    assert ctypes.sizeof(mb._CCacheParams) == 44
    # a partial O row and its statistics for each (request, head, slot), at the least
    assert p.workspace_bytes >= 3 * 4 * 3 * (64 + 1) * 4
    assert mb.moba_cache_decode_workspace_size(p) == p.workspace_bytes


def test_reference_codes():
    import torch
    b = torch.arange(256).to(torch.uint8)
    np.testing.assert_array_equal(ref.code_values("e4m3"), b.view(torch.float8_e4m3fn).double().numpy())
    np.testing.assert_array_equal(ref.code_values("int8"), b.view(torch.int8).double().numpy())
    x = torch.cat([torch.linspace(-460, 460, 20011), torch.randn(5000) * 1e-2]).double()
    got = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.to_codes(x.float().double().numpy(), "e4m3"), got)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_bf16_over_a_scale_is_never_near_a_tie(fmt):
    """Every quotient of two numbers of 8 significant bits is a midpoint of codes or at least 2^-17 away
    from there, so that fp32 quotients round as the exact ones do."""
    a, b = np.arange(128, 256.0)[:, None], np.arange(128, 256.0)[None]
    for e in range(-3, 9):
        q = a / b * 2.0 ** e
        if fmt == "int8":
            mid = np.floor(q) + 0.5
        else:
            step = np.exp2(np.floor(np.log2(np.maximum(q, 2.0 ** -6))) - 3)
            mid = (np.floor(q / step) + 0.5) * step
        if fmt == "int8" and e > 7:
            continue  # beyond the largest code
        d = np.abs(q - mid) / mid
        assert d[d > 0].min() >= 2.0 ** -17
        np.testing.assert_array_equal(ref.to_codes(q, fmt), ref.to_codes(q.astype(np.float32).astype(np.float64), fmt))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_reference_scale(fmt):
    rng = np.random.default_rng(5)
    big = np.concatenate([[0.0, 2.0 ** -97, 448.0, 127.0, 3.0e38], np.exp2(rng.uniform(-90, 100, 1000))])
    s = ref.scale_of(big, fmt)
    m, _ = np.frexp(s)
    assert np.all(m * 256 == np.rint(m * 256))                       # 8 significant bits
    assert np.all(s * ref.QMAX[fmt] >= np.maximum(big, ref.TINY))    # takes big to the largest code
    assert np.all(s * (1 - 2.0 ** -7) * ref.QMAX[fmt] < np.maximum(big, ref.TINY))  # and is the least such
