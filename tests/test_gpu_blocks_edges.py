"""A decode step over selected pages on the GPU where its parts meet the rest of a program: objects dropped while their
calls are in flight, forms of the selection by number of units and pages, bounds of quantised pools step by step."""

import re
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import blocks as OB
from tests.test_gpu_blocks import Selection, Server, _cache, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import paged_kv_attention_slot_gb300 as pk

    pk._lib.lib()
    assert pk.device_error() == 0
    yield
    assert pk.device_error() == 0


def _pk():
    import paged_kv_attention_slot_gb300 as pk

    return pk


@pytest.mark.parametrize("given", [False, True])
def test_a_rotary_dropped_while_its_call_waits_on_another_stream(given):
    pk = _pk()
    cache, _ = _cache("bf16", 4, 16, 2, 128, "nhd")
    q = torch.randn((9, 4, 128), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    k = torch.randn((9, 2, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    pos, slots = torch.arange(5, 14, device="cuda"), torch.arange(9, device="cuda")
    want = pk.rope_store(q, k, k, pos, slots, cache, pk.Rotary(128))
    assert not torch.equal(want, q)
    side = torch.cuda.Stream()
    warm = [torch.zeros(64, dtype=torch.int64, device="cuda") for _ in range(200)]
    del warm
    torch.cuda.synchronize()
    rot, out = pk.Rotary(128), torch.empty_like(q)
    address = rot.phase_step.data_ptr()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(800_000_000)  # about 0.4 s
    if given:
        pk.rope_store(q, k, k, pos, slots, cache, rot, q_out=out, stream=side)
    else:
        with torch.cuda.stream(side):
            pk.rope_store(q, k, k, pos, slots, cache, rot, q_out=out)
    del rot
    taken = [torch.zeros(64, dtype=torch.int64, device="cuda") for _ in range(100)]  # (angles of zero, were they read)
    assert not side.query() and address not in [t.data_ptr() for t in taken]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
