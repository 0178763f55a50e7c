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
