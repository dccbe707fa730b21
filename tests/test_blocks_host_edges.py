"""Refusals of the calls of a decode step over selected pages that need no GPU: objects whose tensors were exchanged."""

import pytest
import torch


@pytest.fixture(scope="module")
def pk():
    from paged_kv_attention_slot_gb300 import build as B

    B.build()
    import paged_kv_attention_slot_gb300 as pk

    pk._lib.lib()
    return pk


def _cache(pk, P=11, ps=16, H=2, D=128):
    k = torch.zeros((P, ps, H, D), dtype=torch.bfloat16)
    return pk.KVCache(k, k.clone())


@pytest.mark.parametrize("other", [torch.zeros(32, dtype=torch.int64), torch.zeros(64, dtype=torch.int32),
                                   torch.zeros(128, dtype=torch.int64)[::2], torch.zeros((64, 1), dtype=torch.int64)])
def test_rope_store_refuses_another_phase_step(pk, other):
    rot = pk.Rotary(128, device="cpu")
    q, k, i = torch.zeros((3, 8, 128), dtype=torch.bfloat16), torch.zeros((3, 2, 128), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    rot.phase_step = other
    with pytest.raises(ValueError, match="phase_step"):
        pk.rope_store(q, k, k, i, i, _cache(pk), rot)
