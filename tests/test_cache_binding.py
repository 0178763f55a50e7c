"""Python surface of the paged 8-bit cache, without a GPU: numbers that the C structure cannot hold, and
layouts that torch calls contiguous."""
import pytest

import block_sparse_attention_gate_b200 as mb

GOOD = dict(max_seqs=3, max_seqlen=1000, num_pages=50, page_size=32, num_q_heads=4, num_kv_heads=2, head_dim=64,
            block_size=128, top_k=3)


@pytest.mark.parametrize("name", GOOD)
@pytest.mark.parametrize("turn", [1 << 32, -(1 << 32), 1 << 40])
def test_numbers_beyond_32_bits_are_refused(name, turn):
    """A value that is good modulo 2^32 is not taken for that one."""
    with pytest.raises(mb.MobaError) as e:
        mb.MobaCacheParams(**{**GOOD, name: GOOD[name] + turn})
    assert e.value.status == 2 and name in str(e.value)


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 5])
def test_slot_maps_beyond_32_bits_are_refused(n):
    import torch
    p = mb.MobaCacheParams(**GOOD)
    with pytest.raises(mb.MobaError, match="slots"):
        p._slots(-1, torch.empty(n, dtype=torch.int32, device="meta"))


def test_keys_of_one_head_may_come_transposed():
    """[1, n, D] seen as [n, 1, D]: contiguous, whatever the stride of the one head."""
    import torch
    cpu = torch.device("cpu")
    p = mb.MobaCacheParams(**{**GOOD, "num_kv_heads": 1})
    kv = torch.zeros(2, 1, 7, 64, dtype=torch.bfloat16)
    K, V = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    assert K.is_contiguous() and K.stride(1) != 64
    p.check(cpu, K=K, V=V)
    p.check(cpu, K=torch.zeros(1, 7, 128, dtype=torch.bfloat16)[:, :, :64].transpose(0, 1))  # rows apart
    with pytest.raises(mb.MobaError):
        p.check(cpu, K=torch.zeros(7, 1, 64, 2, dtype=torch.bfloat16)[..., 0])
    with pytest.raises(mb.MobaError):  # more heads: their stride counts
        mb.MobaCacheParams(**GOOD).check(cpu, K=torch.zeros(2, 7, 64, dtype=torch.bfloat16).transpose(0, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 40])
def test_append_of_keys_of_one_head_transposed(n, cuda_device):
    import torch
    p = mb.MobaCacheParams(**{**GOOD, "num_kv_heads": 1})
    kv = torch.randn(2, 1, n, 64, device="cuda").bfloat16()
    caches = []
    for plain in (True, False):
        c = mb.MobaCache(p)
        K, V = (x.transpose(0, 1).reshape(n, 1, 64).clone() if plain else x.transpose(0, 1) for x in kv)
        c.append(K, V, c.extend(torch.tensor([n, 0, 0], dtype=torch.int32, device="cuda"), n))
        caches.append((c.Kc.view(torch.uint8), c.Vc.view(torch.uint8), c.Ks, c.Vs))
    assert all(torch.equal(a, b) for a, b in zip(*caches)) and bool((caches[0][0] != 0).any())
