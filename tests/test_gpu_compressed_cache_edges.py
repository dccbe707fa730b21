"""The compressed cache at the edges of what its entry points accept.

Tolerances are those of tests/test_gpu_compressed_cache.py (derived in its docstring)."""

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import nvfp4 as O4
from tests.test_gpu_compressed_cache import Case, _np, _pk

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
