"""Refusals of the calls of a decode step over selected pages that need no GPU: objects whose tensors were exchanged."""

import numpy as np
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


@pytest.mark.parametrize("name, other", [
    ("codes", torch.zeros((11, 2, 2, 128), dtype=torch.int16)), ("codes", torch.zeros((11, 2, 2, 128), dtype=torch.uint8)),
    ("codes", torch.zeros((1, 2, 2, 128), dtype=torch.int8).expand(11, 2, 2, 128)), ("codes", torch.zeros((11, 2, 1, 128), dtype=torch.int8)),
    ("codes", torch.zeros((11, 2, 2, 256), dtype=torch.int8)[..., ::2]), ("codes", torch.zeros((11, 2, 256), dtype=torch.int8)),
    ("scale", torch.ones((2, 128), dtype=torch.bfloat16)), ("scale", torch.ones(())), ("scale", torch.ones(128)),
    ("scale", torch.ones((1, 128)).expand(2, 128)), ("scale", torch.ones((2, 64)))])
def test_bounds_whose_tensors_were_exchanged_are_refused(pk, name, other):
    b, cache = pk.KeyBounds.of(_cache(pk), 0.03), _cache(pk)
    setattr(b, name, other)
    plan = pk.Plan().plan([0, 1, 2], [0, 7, 11], list(range(11)), [4, 2], num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                          mode="decode", num_sms=152, host_only=True, num_blocks=4)
    with pytest.raises(ValueError, match="contiguous"):
        plan.bound_keys(cache, b)
    with pytest.raises(ValueError, match="contiguous"):
        plan.select(torch.zeros((2, 8, 128), dtype=torch.bfloat16), b)


@pytest.mark.parametrize("yes", [np.True_, [1], "yes", torch.tensor(True)])
def test_flags_are_truth_values(pk, yes):
    # (as in the calls over every page; on host tensors everything but the device is accepted)
    cache, rot = _cache(pk), pk.Rotary(128, device="cpu")
    b, q = pk.KeyBounds.of(cache, 0.03), torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    k, i = torch.zeros((2, 2, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    plan = pk.Plan().plan([0, 1, 2], [0, 7, 11], list(range(11)), [4, 2], num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                          mode="decode", num_sms=152, host_only=True, num_blocks=4)
    for f in (lambda: plan.bound_keys(cache, b, all_pages=yes), lambda: pk.rope_store(q, k, k, i, i, cache, rot, return_k=yes),
              lambda: plan.run(q, cache, blocks=torch.zeros((2, 2, 4), dtype=torch.int32), return_lse=yes)):
        with pytest.raises(ValueError, match="CUDA device"):
            f()
