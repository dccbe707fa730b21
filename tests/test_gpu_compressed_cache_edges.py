"""The compressed cache at the edges of what its entry points accept.

Tolerances are those of tests/test_gpu_compressed_cache.py (derived in its docstring)."""

import ctypes as C

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import eviction as OE
from oracle import nvfp4 as O4
from tests.test_gpu_compressed_cache import Case, _check_evict, _check_scores, _np, _pk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import paged_kv_attention_slot_gb300 as pk

    pk._lib.lib()
    assert pk.device_error() == 0
    yield
    assert pk.device_error() == 0


# ------------------------------------------------------------------------------------------------
# strides
# ------------------------------------------------------------------------------------------------
def test_nvfp4_pool_whose_rows_lie_a_gigabyte_apart():
    # [page_size, pages, heads, ...] pools: 2^29 bytes from a token's codes to the next one's, so eight tokens
    # are 2^32 bytes apart
    pk = _pk()
    P, ps, H, Hq = 1 << 20, 16, 8, 32
    pools = [torch.empty((ps, P, H, w), dtype=torch.uint8, device="cuda").permute(1, 0, 2, 3) for w in (64, 64, 8, 8)]
    cache = pk.KVCache(pools[0], pools[1], 0.002, 0.002, k_sf=pools[2], v_sf=pools[3])
    assert cache.k.stride(1) == 2 ** 29
    pages = np.array([P - 1, 3, P - 30, P - 7, 11, P - 2], np.int32)
    L = 6 * ps - 5
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((L, H, 128), generator=g).to(torch.bfloat16) for _ in range(2))
    slots = torch.from_numpy(pages.astype(np.int64)[np.arange(L) // ps] * ps + np.arange(L) % ps).cuda()
    pk.kv_store(k.cuda(), v.cuda(), slots, cache)
    lk, lv = pk.kv_load(slots, cache)
    K, V = (O4.dequantize(*O4.quantize(x.float().numpy(), 0.002), 0.002) for x in (k, v))
    for got, ref in ((lk, K), (lv, V)):
        assert np.all(np.abs(_np(got.float()) - ref) <= 2.0 ** -8 * (1 + 2.0 ** -12) * np.abs(ref))
    q = torch.randn((1, Hq, 128), generator=g).to(torch.bfloat16)
    plan = pk.Plan().plan([0, 1], [0, 6], pages, [L - 5 * ps], num_qo_heads=Hq, num_kv_heads=H, head_dim=128, page_size=ps,
                          kv_dtype="nvfp4")
    out, lse = plan.run(q.cuda(), cache, return_lse=True)
    qn = q[0].double().numpy()
    scale = 1 / np.sqrt(128)
    for h in range(Hq):
        Kh, Vh = K[:, h // 4], V[:, h // 4]
        o, l = OA.attend(qn[h], Kh, Vh, 0, L - 1, scale)
        absv, _ = OA.attend(qn[h], Kh, np.abs(Vh), 0, L - 1, scale)
        dx = 2.0 ** -16 * scale * float(np.max(np.abs(Kh) @ np.abs(qn[h])))
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * dx + 2.0 ** -18) * absv * (1 + 2.0 ** -8) + L * 2.0 ** -25 * np.abs(Vh).max()
        assert np.all(np.abs(_np(out[0, h].float()) - o) <= tol), h
        assert abs(float(lse[0, h]) - l) <= dx + 2.0 ** -22 * (1 + abs(l)) + 2.0 ** -20, h
    scores = torch.zeros((P, H, ps), device="cuda")
    scores[torch.from_numpy(pages).cuda().long()] = torch.rand((6, H, ps), generator=g).cuda()
    kept = _np(plan.evict(cache, scores, 40, num_sink=2, num_recent=8))
    ek, ev = pk.kv_load(slots[:40], cache)
    for h in range(H):
        old = torch.from_numpy(kept[0, h]).cuda().long()
        assert torch.equal(ek[:, h], lk[old, h]) and torch.equal(ev[:, h], lv[old, h])


# ------------------------------------------------------------------------------------------------
# signed zeros
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("scale", [1.0, 0.0017, 2.0 ** 20])
def test_store_keeps_the_sign_of_zeros_beside_other_values(scale):
    # zeros of both signs, and values whose quotient or scaled value is too small for any code but a zero
    pk = _pk()
    T, H = 48, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, H, 128), generator=g) * scale
    r = torch.rand((T, H, 128), generator=g)
    for lo, val in ((0.0, 0.0), (0.2, -0.0), (0.4, -1e-4 * scale), (0.5, 1e-4 * scale), (0.6, -1e-40), (0.7, 1e-40)):
        x[(r >= lo) & (r < lo + 0.1)] = val
    k = x.to(torch.bfloat16)
    cache = pk.KVCache.nvfp4(T // 16, 16, H, 128, scale, scale)
    pk.kv_store(k.cuda(), (-k).cuda(), torch.arange(T, device="cuda"), cache)
    for pool, sf, y in ((cache.k, cache.k_sf, k), (cache.v, cache.v_sf, -k)):
        codes, f = O4.quantize(y.float().numpy(), scale)
        assert np.array_equal(_np(sf).reshape(T, H, 8), f)
        assert np.array_equal(_np(pool).reshape(T, H, 64), codes)
        assert (O4.unpack(codes) == 8).any() and (O4.unpack(codes) == 0).any()
    back, _ = pk.kv_load(torch.arange(T, device="cuda"), cache)
    minus = (k == 0) & torch.signbit(k)
    assert minus.any() and torch.signbit(back.cpu()[minus]).all() and not back.cpu()[minus].any()


# ------------------------------------------------------------------------------------------------
# query heads of one group
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("what", [float("nan"), float("inf"), 2.0 ** 16])
@pytest.mark.parametrize("heads, kv_heads", [(8, 2), (16, 2), (32, 2), (40, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_a_head_does_not_depend_on_its_neighbours(dtype, heads, kv_heads, what):
    # every other head holds a NaN, an infinity or large values; the heads between them are what they are without
    c = Case([200, 90, 700], heads, kv_heads, 16, dtype, seed=6)
    bad = np.arange(heads) % 2 == 1
    out, lse = c.plan(num_sms=8).run(c.q, c.cache, return_lse=True)
    q = c.q.clone()
    if what == 2.0 ** 16:
        q[:, bad] = (q[:, bad].float() * what).to(torch.bfloat16)
    else:
        q[:, bad, 5] = what
    o2, l2 = c.plan(num_sms=8).run(q, c.cache, return_lse=True)
    out[:, ~bad], lse[:, ~bad] = o2[:, ~bad], l2[:, ~bad]
    c.check(out, lse)
    if what == 2.0 ** 16:
        assert torch.isfinite(o2.float()).all() and torch.isfinite(l2).all()
    else:
        assert not torch.isfinite(l2[:, bad]).any()


# ------------------------------------------------------------------------------------------------
# streams
# ------------------------------------------------------------------------------------------------
def test_memory_for_work_on_another_stream_is_not_taken_from_the_current_one():
    # a block that the current stream has just freed may still be in use there: the plan's workspace and
    # scratch and a run's outputs, all written on `side`, must not be given it
    pk = _pk()
    c = Case([700, 45], 32, 8, 16, "nvfp4", seed=32)
    side = torch.cuda.Stream()
    c.plan(scored=True).run(c.q, c.cache, return_lse=True, scores=torch.zeros((c.cache.num_pages, 8, 16), device="cuda"))
    scores = torch.zeros((c.cache.num_pages, 8, 16), device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = [1 << 20, 800 * 32 * 4 * 5 // 4, c.q.numel() * 2, c.q.shape[0] * 32 * 4]
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in held]
    del held  # the current stream's free blocks
    side.wait_stream(torch.cuda.current_stream())
    b = c.b
    p = pk.Plan().plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, num_qo_heads=32, num_kv_heads=8, head_dim=128,
                       page_size=16, kv_dtype="nvfp4", scored=True, stream=side)
    out, lse = p.run(c.q, c.cache, return_lse=True, scores=scores, stream=side)
    kept = p.evict(c.cache, scores, 100, stream=side)
    k, v = pk.kv_load(torch.arange(8, device="cuda"), c.cache, stream=side)
    for name, t in dict(workspace=p.workspace, scratch=p.scratch, out=out, lse=lse, kept=kept, k=k, v=v).items():
        assert not any(lo <= t.data_ptr() < hi for lo, hi in spans), name
    torch.cuda.current_stream().wait_stream(side)
    c.check(out, lse)


def test_a_stream_from_elsewhere_may_be_gone_before_the_plan():
    c = Case([700, 45], 32, 8, 16, "nvfp4", seed=32)
    scores = torch.zeros((c.cache.num_pages, 8, 16), device="cuda")
    rt = torch.cuda.cudart()
    handle = C.c_uint64(0)
    assert int(rt.cudaStreamCreate(C.addressof(handle))) == 0
    ext = torch.cuda.ExternalStream(handle.value)
    ext.wait_stream(torch.cuda.current_stream())
    p = c.plan(scored=True, stream=ext)
    out, lse = p.run(c.q, c.cache, return_lse=True, scores=scores, stream=ext)
    with torch.cuda.stream(ext):
        out2 = p.run(c.q, c.cache)
    ext.synchronize()
    c.check(out, lse)
    c.check(out2, lse)
    assert int(rt.cudaStreamDestroy(handle.value)) == 0
    del p, out, lse, out2  # their memory goes back without a look at the stream
    again = torch.empty(8 << 20, dtype=torch.uint8, device="cuda").zero_()
    torch.cuda.synchronize()
    assert not again.any()


def test_runs_on_a_side_stream_inside_a_capture():
    c = Case([700, 45, 2000], 32, 8, 16, "nvfp4", seed=33)
    p = c.plan(num_sms=40, scored=True)
    scores = torch.zeros((c.cache.num_pages, 8, 16), device="cuda")
    p.run(c.q, c.cache, scores=scores)
    scores.zero_()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out, lse = p.run(c.q, c.cache, return_lse=True, scores=scores, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        total = out.float().sum()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    c.check(out, lse)
    _check_scores(c, scores, torch.zeros_like(scores), times=2)
    assert torch.isfinite(total)


# ------------------------------------------------------------------------------------------------
# eviction with more units than run at once
# ------------------------------------------------------------------------------------------------
def _many(units_per_sm):
    """Requests (of 8 KV heads) so that there are more than this many units for each SM."""
    n = torch.cuda.get_device_properties(0).multi_processor_count
    return int(units_per_sm * n) // 8 + 1


@pytest.mark.parametrize("dtype, D, layout", [("bf16", 64, "nhd"), ("bf16", 128, "hnd"), ("e4m3", 128, "nhd"), ("nvfp4", 128, "hnd"),
                                              ("nvfp4", 128, "padded")])
@pytest.mark.parametrize("kind, budget, sink, recent", [("heavy", 96, 4, 16), ("ties", 100, 0, 90), ("wild", 33, 1, 0)])
def test_evict_by_one_cta_per_unit(dtype, D, layout, kind, budget, sink, recent):
    # more than 2.5 units per SM: a unit has one CTA, which moves K, V, both block scales and the scores
    n = _many(2.5)
    lens = [101 + 13 * (i % 9) for i in range(n)]
    assert min(lens) > budget and 2 * n * 8 > 5 * torch.cuda.get_device_properties(0).multi_processor_count
    _check_evict(lens, 8, 16, dtype, budget, sink, recent, kind=kind, D=D, layout=layout, seed=n)


def test_evict_by_one_cta_per_unit_in_several_rounds_of_the_list():
    # more moves per unit than one list (512) holds
    n = _many(2.5)
    _check_evict([1400 + i for i in range(n)], 8, 16, "bf16", 700, 0, 64, kind="wild", D=64, seed=3)


# ------------------------------------------------------------------------------------------------
# very many query heads
# ------------------------------------------------------------------------------------------------
def test_scored_decode_of_the_largest_group():
    c = Case([20, 33], 12288, 1, 16, "bf16", D=64, seed=60)
    start = torch.rand((c.cache.num_pages, 1, 16), generator=torch.Generator().manual_seed(1)).cuda()
    scores = start.clone()
    c.check(*c.plan(scored=True).run(c.q, c.cache, return_lse=True, scores=scores))
    b = c.b
    w = np.zeros((c.cache.num_pages, 1, 16))
    OE.add_weights(w, b.q.double().numpy(), c.K, b.kv_indptr, b.kv_indices, b.last_page_len, b.qo_indptr, 16)
    # 12288 weights of relative error 2 dx + 2^-19 are added in sequence: their sum is off by at most 12288 * 2^-24
    # of itself on top
    ref = _np(start).astype(np.float64) + w
    tol = w * (2 * c.dx() + 2.0 ** -19 + 12288 * 2.0 ** -24) + 2.0 ** -23 * ref
    assert np.all(np.abs(_np(scores) - ref) <= tol)
    assert np.array_equal(_np(scores)[w == 0], _np(start)[w == 0])


# ------------------------------------------------------------------------------------------------
# scores at any 4-byte address
# ------------------------------------------------------------------------------------------------
def _unaligned(t):
    """A contiguous copy that starts 4 bytes past a 16-byte boundary."""
    u = torch.empty(t.numel() + 4, dtype=t.dtype, device=t.device)[1:t.numel() + 1].view(t.shape)
    assert u.data_ptr() % 16 == 4 and u.is_contiguous()
    return u.copy_(t)


@pytest.mark.parametrize("sms", [0, 4])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_scores_need_not_be_aligned_to_vectors(dtype, sms):
    # the single-key forms of the score update and of eviction's reads, on pages that vectors would fit
    pk = _pk()
    c = Case([700, 45, 130], 16, 2, 16, dtype, seed=61)
    start = torch.rand((c.cache.num_pages, 2, 16), generator=torch.Generator().manual_seed(1)).cuda()
    scores = _unaligned(start)
    p = c.plan(num_sms=sms, scored=True)
    c.check(*p.run(c.q, c.cache, return_lse=True, scores=scores))
    _check_scores(c, scores, start)
    pools = [x.clone() for x in c.pools]
    aligned = scores.clone()
    want = p.evict(c.cache, aligned, 100, num_sink=2, num_recent=10)
    moved = [x.clone() for x in c.pools]
    for x, y in zip(c.pools, pools):
        x.copy_(y)
    assert torch.equal(p.evict(c.cache, scores, 100, num_sink=2, num_recent=10), want)
    assert torch.equal(scores, aligned) and all(torch.equal(x, y) for x, y in zip(c.pools, moved))
    x = torch.ones((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    pk.kv_store(x, x, torch.tensor([int(c.b.kv_indices[0]) * 16 + 3], device="cuda"), c.cache, scores=scores)
    aligned[int(c.b.kv_indices[0]), :, 3] = 0
    assert torch.equal(scores, aligned)


def test_evict_of_a_long_request_with_unaligned_scores():
    pk = _pk()
    L, ps, b = 14000, 16, 3000
    n = -(-L // ps)
    fresh = torch.rand((n, 1, ps), generator=torch.Generator().manual_seed(2)).cuda()
    k = torch.randn((n, ps, 1, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    plan = pk.Plan().plan([0, 1], [0, n], np.arange(n), [L - (n - 1) * ps], num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=ps)
    got = []
    for s in (fresh.clone(), _unaligned(fresh)):
        cache = pk.KVCache(k.clone(), -k)
        kept = plan.evict(cache, s, b, num_sink=4, num_recent=100)
        got.append((kept, s.clone(), cache.k, cache.v))
    assert all(torch.equal(x, y) for x, y in zip(*got))


# ------------------------------------------------------------------------------------------------
# two calls at once
# ------------------------------------------------------------------------------------------------
def test_layers_evicted_at_once_on_one_plan():
    # eviction only reads the plan: the layers of a step may be evicted side by side
    pk = _pk()
    c = Case([3000, 900, 2000], 8, 8, 16, "bf16", seed=62)
    p = c.plan()
    layers = []
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        scores = torch.rand((c.cache.num_pages, 8, 16), generator=g).cuda()
        pools = [x.clone().mul_(i + 1) for x in c.pools]
        layers.append((pk.KVCache(*pools), scores, [x.clone() for x in pools], scores.clone()))
    want = []
    for cache, scores, pools, fresh in layers:
        kept = p.evict(cache, scores, 800, num_sink=4, num_recent=64)
        want.append((kept, scores.clone(), cache.k.clone(), cache.v.clone()))
        cache.k.copy_(pools[0])
        cache.v.copy_(pools[1])
        scores.copy_(fresh)
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    kept = [p.evict(cache, scores, 800, num_sink=4, num_recent=64, stream=s) for (cache, scores, _, _), s in zip(layers, streams)]
    torch.cuda.synchronize()
    for (cache, scores, _, _), k, w in zip(layers, kept, want):
        assert all(torch.equal(x, y) for x, y in zip((k, scores, cache.k, cache.v), w))


# ------------------------------------------------------------------------------------------------
# more rows than one launch indexes
# ------------------------------------------------------------------------------------------------
def test_store_and_load_of_more_rows_than_one_launch_covers():
    # 2^26 (token, head) rows per launch; the token behind them goes with a second one
    pk = _pk()
    H, T = 65536, 1026
    x = torch.empty((T, H, 128), dtype=torch.bfloat16, device="cuda")
    row = torch.randn((H, 128), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    for t in range(T):
        x[t] = row.roll(t, 0)
    cache = pk.KVCache.nvfp4(T, 1, H, 128, 0.002, 0.002)
    slots = torch.arange(T, device="cuda").flip(0).contiguous()
    pk.kv_store(x, x, slots, cache)
    k, v = pk.kv_load(slots, cache)
    one = pk.KVCache.nvfp4(1, 1, H, 128, 0.002, 0.002)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    for t in (0, 1, 500, 1022, 1023, 1024, 1025):
        pk.kv_store(x[t:t + 1], x[t:t + 1], zero, one)
        a = pk.kv_load(zero, one)[0][0]
        assert torch.equal(cache.k[T - 1 - t, 0], one.k[0, 0]) and torch.equal(cache.v_sf[T - 1 - t, 0], one.v_sf[0, 0])
        assert torch.equal(k[t], a) and torch.equal(v[t], a)
    del x, k, v, cache
    torch.cuda.empty_cache()
