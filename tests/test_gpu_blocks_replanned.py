"""Captured calls of a decode step over selected pages whose plan is made anew in place: for the same lengths over other
pages, as documented, and for anything else that leaves the workspace's layout alone, which must end in a recorded error
or in rows that say so, never in an access out of range."""

import numpy as np
import pytest
import torch

from oracle import blocks as OB
from tests.test_gpu_blocks import Chosen, Selection, _batch, _np

pytestmark = pytest.mark.gpu

SLOT_RANGE, PAGE_RANGE, CAPACITY = 1, 2, 4


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


def _capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fn()
    return graph


def _front(plan):
    """What stands in front of the request table and the page list in a plan's workspace: where it differs, a captured call
    would read something else in their place, and is not replayed."""
    i = plan.info()
    return i["num_work"], i["num_merge"], i["batch_size"]


# ---- selection ----
@pytest.mark.parametrize("heads, kv_heads, D, short, long", [
    (8, 8, 128, 60, 63),       # within the same 32 pages of scores: served
    (8, 8, 128, 60, 200),      # one CTA per unit
    (4, 2, 64, 700, 769),
    (4, 2, 128, 2000, 2600),   # clusters
    (2, 1, 64, 2000, 9000),
    (2, 1, 128, 40000, 49152)])
def test_a_captured_selection_refuses_longer_requests(heads, kv_heads, D, short, long):
    # request 1 grows from `short` to `long` pages; the other, as long as it was, is served beside it
    ps, K, keep = 8, 8, 30
    s = Selection([keep * ps - 3, short * ps - 5], heads, kv_heads, ps, D, K, seed=1)
    t = Selection([keep * ps - 3, long * ps - 5], heads, kv_heads, ps, D, K, seed=2)
    pk = _pk()
    P = len(t.codes)
    codes = torch.zeros((P, kv_heads, 2, D), dtype=torch.int8, device="cuda")
    codes[:len(s.codes)] = s.b.codes
    b, q = pk.KeyBounds(codes, s.b.scale.clone()), s.q.cuda()
    blocks = torch.empty((2, kv_heads, K), dtype=torch.int32, device="cuda")
    kw = dict(num_qo_heads=heads, num_kv_heads=kv_heads, head_dim=D, page_size=ps, mode="decode", num_blocks=K)
    at, front = s.plan.workspace.data_ptr(), _front(s.plan)
    graph = _capture(lambda: s.plan.select(q, b, num_sink=1, num_recent=2, blocks=blocks))
    want = s.want(1, 2)
    for _ in range(2):
        s.plan.plan(*s.idx, **kw)
        codes[:len(s.codes)] = s.b.codes
        b.scale.copy_(s.b.scale)
        q.copy_(s.q)
        blocks.fill_(99)
        graph.replay()
        assert pk.device_error() == 0 and np.array_equal(_np(blocks), want)
        s.plan.plan(*t.idx, **kw)
        assert s.plan.workspace.data_ptr() == at and _front(s.plan) == front
        codes.copy_(t.b.codes)
        b.scale.copy_(t.b.scale)
        q.copy_(t.q)
        blocks.fill_(99)
        graph.replay()
        other = t.want(1, 2)
        if long - 3 > -(-(short - 3) // 32) * 32:
            assert pk.device_error() == CAPACITY
            other[1] = -1
        else:
            assert pk.device_error() == 0
        assert np.array_equal(_np(blocks), other)


# ---- pages ----
def _batch_kw(heads, kv_heads, D, ps, **kw):
    return dict(num_qo_heads=heads, num_kv_heads=kv_heads, head_dim=D, page_size=ps, **kw)


@pytest.mark.parametrize("lens, D", [([300, 45], 128), ([9000, 500], 64), ([9000, 500], 128)])
def test_a_captured_selection_serves_other_pages_and_records_those_it_has_no_bounds_of(lens, D):
    pk, ps, H, K = _pk(), 8, 2, 9
    s = Selection(lens, 4, H, ps, D, K, seed=3)
    q, blocks = s.q.cuda(), torch.empty((2, H, K), dtype=torch.int32, device="cuda")
    graph = _capture(lambda: s.plan.select(q, s.b, num_sink=1, num_recent=1, blocks=blocks))
    P, first = len(s.codes), s.idx
    for seed in (4, 5):
        idx = np.random.RandomState(seed).permutation(P)[:len(first[2])].astype(np.int32)
        s.idx = (first[0], first[1], idx, first[3])
        s.plan.plan(*s.idx, **_batch_kw(4, H, D, ps, mode="decode", num_blocks=K))
        blocks.fill_(99)
        graph.replay()
        assert pk.device_error() == 0 and np.array_equal(_np(blocks), s.want(1, 1))
    # pages of request 0 that the bounds do not have, competing ones and the last one, which is selected in any case
    for page in (P, 2 ** 31 - 1):
        for at in (1, len(first[2]) // 2, first[1][1] - 1):
            bad = idx.copy()
            bad[at] = page
            s.plan.plan(first[0], first[1], bad, first[3], **_batch_kw(4, H, D, ps, mode="decode", num_blocks=K))
            blocks.fill_(99)
            graph.replay()
            assert pk.device_error() == PAGE_RANGE
            got = _np(blocks)
            assert np.array_equal(got[1], s.want(1, 1)[1])
            assert np.all((got[0] >= 0) & (got[0] < first[1][1])) and np.all(np.diff(got[0]) > 0)


@pytest.mark.parametrize("dtype, mode, every, ps", [
    *((d, "decode", e, ps) for d in ("bf16", "e4m3", "nvfp4") for e, ps in ((False, 16), (True, 16), (True, 64))),
    ("bf16", "prefill", False, 16), ("bf16", "prefill", True, 64)])
def test_captured_bounds_serve_other_pages_and_record_those_outside_the_pool(dtype, mode, every, ps):
    pk, H, P = _pk(), 2, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    if dtype == "bf16":
        k = torch.randn((P, ps, H, 128), generator=g, device="cuda").to(torch.bfloat16)
        cache = pk.KVCache(k, k.clone())
    elif dtype == "e4m3":
        k = torch.randn((P, ps, H, 128), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        cache = pk.KVCache(k, k.clone(), 0.7, 0.7)
    else:
        cache = pk.KVCache.nvfp4(P, ps, H, 128, 0.01, 0.01)
        cache.k.random_(0, 256, generator=g)
        cache.k_sf.random_(0x30, 0x50, generator=g)
    lens, q_lens = ([5 * ps - 3, 9 * ps, 17], [1, 1, 0]) if mode == "decode" else ([5 * ps - 3, 9 * ps, 17], [ps + 2, 3, 17])
    idx, _ = _batch(lens, q_lens, ps)
    kw = _batch_kw(2, H, 128, ps, mode=mode, kv_dtype=dtype, max_splits=1)
    room = torch.full((P + 2, H, 2, 128), 99, dtype=torch.int8, device="cuda")  # (a page before and one behind the bounds)
    b = pk.KeyBounds(room[1:P + 1], torch.full((H, 128), 0.03, device="cuda"))
    plan, other = pk.Plan().plan(*idx, **kw), pk.Plan()
    graph = _capture(lambda: plan.bound_keys(cache, b, all_pages=every))

    def replayed():
        room.fill_(99)
        graph.replay()
        return pk.device_error(), room.clone()

    def eager(*batch):
        want = torch.full_like(room, 99)
        other.plan(*batch, **kw).bound_keys(cache, pk.KeyBounds(want[1:P + 1], b.scale), all_pages=every)
        assert pk.device_error() == 0
        return want

    for seed in (2, 3):
        pages = np.random.RandomState(seed).permutation(P)[:len(idx[2])].astype(np.int32)
        plan.plan(idx[0], idx[1], pages, idx[3], **kw)
        code, got = replayed()
        assert code == 0 and torch.equal(got, eager(idx[0], idx[1], pages, idx[3]))
    want = eager(idx[0], idx[1], pages, idx[3])
    for page in (P, 2 ** 31 - 1):
        at = int(idx[1][1]) - 1  # request 0's last page
        bad = pages.copy()
        bad[at] = page
        plan.plan(idx[0], idx[1], bad, idx[3], **kw)
        code, got = replayed()
        assert code == PAGE_RANGE
        rest = want.clone()
        rest[1 + pages[at]] = 99
        assert torch.equal(got, rest)
    # a shorter request 1: the entries of the captured call behind the list's end are nobody's pages
    lens[1] = 6 * ps
    short, _ = _batch(lens, q_lens, ps)
    front = _front(plan)
    plan.plan(*short, **kw)
    assert _front(plan) == front
    code, got = replayed()
    assert code == 0 and torch.equal(got, eager(*short))


# ---- attention ----
@pytest.mark.parametrize("dtype, keys, ps, K, more", [("bf16", 200, 16, 4, 8), ("nvfp4", 200, 16, 4, 8), ("e4m3", 12000, 8, 1100, 1300),
                                                      ("bf16", 12000, 8, 1000, 1300)])
def test_a_captured_run_records_a_plan_made_anew_for_more_blocks(dtype, keys, ps, K, more):
    pk = _pk()
    c = Chosen([keys], 4, 2, ps, dtype, layout="hnd", seed=2)
    p, chosen = c.plan(num_blocks=K, max_splits=1), c.choose(K)
    # blocks that the rows behind the selection would give, were they read
    room = torch.zeros((1, 4, K), dtype=torch.int32, device="cuda")
    blocks, out = room[:, :2], torch.empty_like(c.q)
    blocks.copy_(chosen)
    want = p.run(c.q, c.cache, blocks=blocks)
    graph = _capture(lambda: p.run(c.q, c.cache, blocks=blocks, out=out))
    graph.replay()
    assert pk.device_error() == 0 and torch.equal(out, want)
    b = c.b
    kw = _batch_kw(4, 2, 128, ps, mode="decode", kv_dtype=dtype, max_splits=1)
    front = _front(p)
    p.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, num_blocks=more, **kw)
    assert _front(p) == front
    graph.replay()
    assert pk.device_error() == PAGE_RANGE
    p.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, num_blocks=K, **kw)
    out.zero_()
    graph.replay()
    assert pk.device_error() == 0 and torch.equal(out, want)


# ---- token map ----
@pytest.mark.parametrize("mode, lens, first, then", [
    ("decode", [40, 9, 700, 33], [1, 1, 1, 1], [1, 1, 0, 0]), ("decode", [40, 9, 700, 33], [1, 1, 1, 1], [0, 1, 0, 0]),
    ("prefill", [300, 41], [100, 41], [90, 3])])
def test_rows_of_a_captured_token_map_behind_the_last_token_are_padding(mode, lens, first, then):
    pk = _pk()
    kw = _batch_kw(4, 1, 128, 16, mode=mode, max_splits=1, num_sms=152)
    # (the lists in front of the request table take as many 256-byte lines: it stays where the captured call reads it)
    size = [pk.Plan.workspace_size(*_batch(lens, n, 16)[0], **kw) for n in (first, then)]
    assert size[0] == size[1]
    p = pk.Plan().plan(*_batch(lens, first, 16)[0], **kw)
    off = torch.arange(len(lens), device="cuda") * 1000
    at = p.workspace.data_ptr()
    kept = []
    graph = _capture(lambda: kept.extend(p.token_map(off)))
    for q_lens in (first, then, first):
        idx, _ = _batch(lens, q_lens, 16)
        p.plan(*idx, **kw)
        assert p.workspace.data_ptr() == at
        for x in kept:
            x.fill_(77)
        graph.replay()
        n = sum(q_lens)
        pos, slots = OB.token_map(*idx, 16, _np(off))
        assert np.array_equal(_np(kept[0]), np.concatenate([pos, np.zeros(sum(first) - n, np.int64)]))
        assert np.array_equal(_np(kept[1]), np.concatenate([slots, np.full(sum(first) - n, -1)]))
