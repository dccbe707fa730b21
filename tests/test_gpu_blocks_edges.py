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


# ---- forms of the selection ----
_SOURCE = (Path(__file__).parent.parent / "paged_kv_attention_slot_gb300" / "csrc" / "block_select.cu").read_text()
FEW = int(re.search(r"kFewPages = (\d+);", _SOURCE).group(1))  # competing pages that one small CTA takes in any case


def _form(units, competing):
    """What the launcher chooses: a small CTA per unit, or wide ones, in clusters as far as they run at once."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return "wide" if competing > FEW and units <= sms else "narrow"


FORMS = [
    # what, requests, pages beyond FEW of the longest and how far below the others may lie, heads, kv_heads, D, form
    ("one wide CTA per unit", 76, 90, 30, 4, 2, 128, "wide"),
    ("one wide CTA per unit", 95, 60, 20, 1, 1, 64, "wide"),
    ("clusters of a middle size", 16, 1400, 600, 4, 2, 128, "wide"),
    ("clusters of a middle size", 22, 3000, 2500, 2, 1, 128, "wide"),
    ("clusters of a middle size", 17, 2300, 900, 2, 1, 64, "wide"),
    ("clusters of two", 36, 2500, 100, 4, 2, 128, "wide"),
    ("clusters, 64 dims", 2, 1500, 700, 6, 2, 64, "wide"),
    ("query heads beyond those a thread keeps", 2, 900, 200, 40, 1, 128, "wide"),
    ("query heads beyond those a thread keeps", 1, 2000, 0, 256, 2, 64, "wide"),
    ("query heads beyond those a thread keeps", 76, 200, 50, 46, 2, 128, "wide"),
    ("units beyond the SMs", 100, 150, 60, 4, 2, 128, "narrow"),
    ("units beyond the SMs", 160, 40, 30, 3, 1, 64, "narrow"),
    ("the last count that is few", 4, 0, 5, 4, 2, 128, "narrow"),
    ("the first that is many", 4, 1, 5, 4, 2, 128, "wide"),
]


@pytest.mark.parametrize("kind", ["random", "few", "equal", "outlier"])
@pytest.mark.parametrize("what, requests, more, spread, heads, kv_heads, D, form", FORMS)
def test_selection_in_every_form(what, requests, more, spread, heads, kv_heads, D, form, kind):
    ps, K, sink, recent = 8, 37, 1, 2
    r = np.random.RandomState(requests)
    longest = FEW + more + sink + recent
    pages = [longest] + [longest - int(r.randint(0, spread + 1)) for _ in range(requests - 1)]
    assert _form(requests * kv_heads, longest - sink - recent) == form
    Selection([n * ps - int(r.randint(0, ps)) for n in pages], heads, kv_heads, ps, D, K, kind=kind, seed=1).check(sink, recent)


# ---- bounds of quantised pools, step by step ----
def _values(s):
    """What attention reads of the K pool, float32 [pages, page_size, kv_heads, head_dim]."""
    k = s.cache.k
    if s.dtype == "e4m3":
        return k.view(torch.float8_e4m3fn).float() * torch.tensor(s.cache.k_scale, dtype=torch.float32, device="cuda")
    codes = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    x = torch.stack((codes[(k & 15).long()], codes[(k >> 4).long()]), -1).flatten(-2)
    sf = s.cache.k_sf.view(torch.float8_e4m3fn) if s.cache.k_sf.dtype == torch.uint8 else s.cache.k_sf
    return x * sf.float().repeat_interleave(16, -1) * torch.tensor(s.cache.k_scale, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("dtype, heads, kv_heads, ps", [("e4m3", 4, 4, 32), ("e4m3", 4, 2, 16), ("nvfp4", 16, 2, 16), ("nvfp4", 4, 2, 64)])
def test_bounds_of_quantised_pools_after_every_step(dtype, heads, kv_heads, ps):
    prompts = [5, 333, 1000, 64]
    s = Server(prompts, heads, kv_heads, ps, dtype, 6, seed=4)
    pk = s.pk
    s.lens = list(prompts)
    q, k, v = s.tokens(sum(prompts))
    pk.rope_store(q, k, v, *s.plan(prompts, "prefill", kv_dtype="bf16").token_map(), s.cache, s.rot)
    s.plan([1] * 4, "decode").bound_keys(s.cache, s.bounds, all_pages=True)
    for step in range(6):
        if step:
            s.lens = [n + 1 for n in s.lens]
            q, k, v = s.tokens(4)
            p = s.plan([1] * 4, "decode", num_blocks=s.K)
            pk.rope_store(q, k, v, *p.token_map(), s.cache, s.rot)
            p.bound_keys(s.cache, s.bounds)
        K, codes, idx = _np(_values(s)), _np(s.bounds.codes), s.index([1] * 4)
        for i, n in enumerate(s.lens):
            for b, page in enumerate(idx[2][idx[1][i]:idx[1][i + 1]]):
                assert np.array_equal(codes[page], OB.page_bounds(K[page, :min(ps, n - b * ps)], _np(s.bounds.scale))), (step, i, b)
