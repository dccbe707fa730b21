"""The compressed cache on the GPU: NVFP4 write, read back and decode, decode that accumulates attention
weights, eviction by them, and a run of all of them, against the float64 oracle.

Tolerances are worst-case bounds of the arithmetic, computed per element:
* stored codes, block scales, moved rows, kept positions: equal;
* values read back: one rounding to bf16 (2^-8 relative) after float32 products (2^-22);
* decode outputs: a rounding to bf16 of the output (2^-8 |o|) and of each probability to the 16-bit type of
  the second product (bf16 2^-8 or f16 2^-11, relative, times sum_j p_j |v_j|; an f16 probability below
  2^-14 of the reference maximum is off by at most 2^-25 of it), and the scores' own error;
* scores x = scale q.k in float32: at most 128 additions, each off by 2^-23 of the largest partial sum,
  which sum_d |q_d k_d| bounds: dx = 2^-16 scale max_j sum_d |q_d k_jd|; a weight exp(x - lse) is off by 2 dx
  relative (x and lse), and 2^-20 for the exponentials; the log-sum-exp by dx + 2^-22 (1 + |lse|)."""

import ctypes as C

import numpy as np
import pytest
import torch

import workloads as W
from oracle import attention as OA
from oracle import eviction as OE
from oracle import nvfp4 as O4
from tests import gpu_common as G

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


def _np(t):
    return t.detach().cpu().numpy()


# ------------------------------------------------------------------------------------------------
# NVFP4 pools
# ------------------------------------------------------------------------------------------------
def _fp4_pools(P, ps, H, layout, fill=0xA5):
    """Code and scale pools of the given memory layout, filled with a byte pattern."""
    def one(w):
        if layout == "nhd":
            return torch.full((P, ps, H, w), fill, dtype=torch.uint8, device="cuda")
        if layout == "hnd":
            return torch.full((P, H, ps, w), fill, dtype=torch.uint8, device="cuda").transpose(1, 2)
        if layout == "head pools":  # one contiguous pool per head
            return torch.full((H, P, ps, w), fill, dtype=torch.uint8, device="cuda").permute(1, 2, 0, 3)
        # padded rows: more than the row between tokens, heads and pages
        pad = 64 if w >= 64 else 8
        return torch.full((P, ps + 1, H + 1, w + pad), fill, dtype=torch.uint8, device="cuda")[:, :ps, :H, :w]
    return one(64), one(64), one(8), one(8)


def _special_rows(T, H, seed):
    """bf16 rows with zeros, ties, subnormal and huge blocks, infinities and NaN among N(0, 1) ones."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, 128), generator=g)
    flat = x.view(-1, 16)
    n = flat.shape[0]
    for k, f in enumerate((0.0, 1e-3, 2.0 ** -12, 1e-38, 1e30, 300.0)):
        flat[k::23] *= f
    flat[7::29] = torch.randint(-12, 13, flat[7::29].shape, generator=g) * 0.25   # ties once the scale is 1 / 2 / 4
    flat[11 % n, 3] = float("inf")
    flat[13 % n, 5] = float("-inf")
    flat[17 % n, 0] = float("nan")
    flat[19 % n, :] = -0.0
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "padded", "head pools"])
@pytest.mark.parametrize("T, H, ps, scale", [(1, 1, 1, 1.0), (7, 3, 5, 0.125), (64, 8, 16, 0.0017), (301, 2, 128, 0.37)])
def test_store_writes_the_oracles_codes_and_load_reads_them_back(T, H, ps, scale, layout):
    pk = _pk()
    P = (T + ps - 1) // ps + 2
    pools = _fp4_pools(P, ps, H, layout)
    cache = pk.KVCache(pools[0], pools[1], scale, 1.0, k_sf=pools[2], v_sf=pools[3])
    k, v = _special_rows(T, H, 1), _special_rows(T, H, 2)
    slots = torch.randperm(P * ps, generator=torch.Generator().manual_seed(3))[:T]
    if T > 4:
        slots[2] = -1  # padding
    want = [_np(p).copy() for p in pools]
    for n, (x, s) in enumerate(((k, scale), (v, 1.0))):
        codes, sf = O4.quantize(x.float().numpy(), s)
        for t, slot in enumerate(slots.tolist()):
            if slot >= 0:
                want[n][slot // ps, slot % ps] = codes[t]
                want[2 + n][slot // ps, slot % ps] = sf[t]
    pk.kv_store(k.cuda(), v.cuda(), slots.cuda(), cache)
    for got, w in zip(pools, want):
        assert np.array_equal(_np(got), w)  # the other slots keep their bytes
    # read back: repeats, padding, any order
    take = torch.cat([slots, slots.flip(0), torch.tensor([-5])])
    lk, lv = pk.kv_load(take.cuda(), cache)
    for n, (got, s) in enumerate(((lk, scale), (lv, 1.0))):
        got = _np(got.float()).astype(np.float64)
        t = take.numpy()
        p = np.maximum(t, 0)
        ref = O4.dequantize(want[n][p // ps, p % ps], want[2 + n][p // ps, p % ps], s)
        ref[t < 0] = 0.0
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        ok = ~np.isnan(ref)
        assert np.all(np.abs(got - ref)[ok] <= np.abs(ref[ok]) * 2.0 ** -8 * (1 + 2.0 ** -12))


@pytest.mark.parametrize("scale", [1.0, 0.00186, 5.0 / 2688.0, 77.7])
def test_store_rounds_every_bf16_magnitude_like_the_oracle(scale):
    # all positive finite bf16 values up to 2^20 of the scale, in blocks of one binade each and of
    # mixed binades: every halfway case of both formats occurs
    pk = _pk()
    bits = np.arange(0x3000, 0x4A00, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    g = torch.Generator().manual_seed(5)
    rows = torch.cat([x, x[torch.randperm(len(x), generator=g)], -x])
    rows = torch.cat([rows, rows[: (-len(rows)) % 128]]).view(-1, 1, 128)
    T = rows.shape[0]
    cache = pk.KVCache.nvfp4(1, T, 1, 128, scale, scale)
    pk.kv_store(rows.cuda(), (-rows).cuda(), torch.arange(T, device="cuda"), cache)
    codes, sf = O4.quantize(rows.float().numpy(), scale)
    assert np.array_equal(_np(cache.k[0]), codes) and np.array_equal(_np(cache.k_sf[0]), sf)
    codes, sf = O4.quantize(-rows.float().numpy(), scale)
    assert np.array_equal(_np(cache.v[0]), codes) and np.array_equal(_np(cache.v_sf[0]), sf)


@pytest.mark.parametrize("dtype, D", [("bf16", 64), ("bf16", 128), ("e4m3", 128), ("e4m3", 64)])
def test_load_reads_bf16_and_fp8_pools(dtype, D):
    pk = _pk()
    P, ps, H = 5, 3, 3
    x = torch.randn((P, ps, H, D), generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    take = torch.tensor([0, 14, 3, 3, -1, 7])
    i = take.clamp(min=0)
    if dtype == "bf16":
        cache = pk.KVCache(x.cuda(), -x.cuda())
        ref = x.float().numpy()[i // ps, i % ps]
        tol = 0.0
    else:
        codes = torch.randint(0, 256, (P, ps, H, D), generator=torch.Generator().manual_seed(8), dtype=torch.uint8)
        codes[(codes & 127) == 127] = 5
        cache = pk.KVCache(codes.cuda(), (codes ^ 128).cuda(), 0.3, 0.3)
        ref = OA.to_f64(codes.numpy()[i // ps, i % ps], "e4m3", 0.3)
        tol = 2.0 ** -8 * (1 + 2.0 ** -12)
    ref = np.where(take.numpy()[:, None, None] < 0, 0.0, ref)
    k, v = pk.kv_load(take.cuda(), cache)
    for got, r in ((k, ref), (v, -ref)):
        assert np.all(np.abs(_np(got.float()) - r) <= tol * np.abs(r))


def test_store_and_load_of_no_tokens_and_of_a_slot_out_of_range():
    pk = _pk()
    cache = pk.KVCache.nvfp4(2, 4, 2, 128)
    none = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    pk.kv_store(none, none, slots, cache)
    assert pk.kv_load(slots, cache)[0].shape == (0, 2, 128)
    x = torch.ones((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([3, 8], device="cuda")
    pk.kv_store(x, x, far, cache)
    assert pk.device_error() == 1  # PKV_DEVERR_SLOT_RANGE
    k, _ = pk.kv_load(far, cache)
    assert pk.device_error() == 1
    # a block of ones: the scale is E4M3(1 / 6) = 1.375 * 2^-3, the code 6: 6 * 0.171875 = 1.03125
    assert torch.all(k[0] == 1.03125) and not k[1].any()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_store_starts_the_scores_of_written_slots_only(dtype):
    pk = _pk()
    P, ps, H = 3, 4, 5
    if dtype == "nvfp4":
        cache = pk.KVCache.nvfp4(P, ps, H, 128)
    else:
        t = torch.bfloat16 if dtype == "bf16" else torch.uint8
        cache = pk.KVCache(torch.zeros((P, ps, H, 128), dtype=t, device="cuda"), torch.zeros((P, ps, H, 128), dtype=t, device="cuda"))
    scores = torch.full((P, H, ps), 7.0, device="cuda")
    x = torch.randn((4, H, 128), device="cuda").to(torch.bfloat16)
    pk.kv_store(x, x, torch.tensor([0, 6, -1, 11], device="cuda"), cache, scores=scores)
    want = torch.full((P, H, ps), 7.0)
    want[0, :, 0] = want[1, :, 2] = want[2, :, 3] = 0
    assert torch.equal(scores.cpu(), want)


# ------------------------------------------------------------------------------------------------
# decode
# ------------------------------------------------------------------------------------------------
class Case:
    """A batch with a pool of any type on the GPU and its float64 values for the oracle."""

    def __init__(self, lens, heads, kv_heads, ps, dtype, D=128, layout="hnd", window=-1, seed=0, q_scale=1.0, q_lens=None,
                 k_scale=0.002, v_scale=0.0021):
        pk = _pk()
        self.b = b = W.make_batch(lens, q_lens or [1] * len(lens), ps, heads, kv_heads, D, seed, window_left=window)
        self.dtype, self.window = dtype, window
        P = b.k_pool.shape[0]
        if q_scale != 1.0:
            b.q = (b.q.float() * q_scale).to(torch.bfloat16)
        if dtype == "bf16":
            self.pools = [b.k_pool.cuda(), b.v_pool.cuda()]
            if layout == "hnd":
                self.pools = [p.transpose(1, 2).contiguous().transpose(1, 2) for p in self.pools]
            self.cache = pk.KVCache(*self.pools)
            self.K, self.V = b.k_pool.double().numpy(), b.v_pool.double().numpy()
        elif dtype == "e4m3":
            ks = vs = 0.01
            codes = [G.quantize_chunked(x, s) for x, s in ((b.k_pool, ks), (b.v_pool, vs))]
            self.pools = [torch.from_numpy(c).cuda() for c in codes]
            self.cache = pk.KVCache(*self.pools, ks, vs)
            self.K, self.V = (OA.to_f64(c, "e4m3", s) for c, s in zip(codes, (ks, vs)))
        else:
            ks, vs = k_scale, v_scale
            self.pools = list(_fp4_pools(P, ps, kv_heads, layout, fill=0x7F))
            qs = [O4.quantize(x.float().numpy(), s) for x, s in ((b.k_pool, ks), (b.v_pool, vs))]
            for n in range(2):
                self.pools[n].copy_(torch.from_numpy(qs[n][0]))
                self.pools[2 + n].copy_(torch.from_numpy(qs[n][1]))
            self.cache = pk.KVCache(self.pools[0], self.pools[1], ks, vs, k_sf=self.pools[2], v_sf=self.pools[3])
            self.K, self.V = (O4.dequantize(c, f, s) for (c, f), s in zip(qs, (ks, vs)))
        self.q = b.q.cuda()
        self.scale = 1.0 / np.sqrt(D)

    def plan(self, **kw):
        b = self.b
        a = dict(num_qo_heads=b.num_qo_heads, num_kv_heads=b.num_kv_heads, head_dim=b.head_dim, page_size=b.page_size,
                 mode="decode", window_left=self.window, kv_dtype=self.dtype)
        a.update(kw)
        return _pk().Plan().plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, **a)

    def oracle(self):
        b = self.b
        a = (b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, b.page_size)
        q = b.q.double().numpy()
        o, lse = OA.paged_attention(q, self.K, self.V, *a, window_left=self.window)
        absv, _ = OA.paged_attention(q, self.K, np.abs(self.V), *a, window_left=self.window)
        return o, lse, absv

    def dx(self):
        """Bound of a float32 score's error (see the module's docstring)."""
        q = np.abs(self.b.q.double().numpy())
        k = np.abs(self.K).reshape(-1, *self.K.shape[2:])
        rep = q.shape[1] // k.shape[1]
        top = max(float(np.max(q[:, h] @ k[:, h // rep].T)) if q.shape[0] else 0.0 for h in range(q.shape[1]))
        return 2.0 ** -16 * self.scale * top

    def check(self, out, lse, rows=None):
        o, l, absv = self.oracle()
        dx = self.dx()
        got, gl = _np(out.float()).astype(np.float64), _np(lse).astype(np.float64)
        rows = np.arange(len(o)) if rows is None else rows
        p_round = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -11
        n = int(self.b.kv_len.max())
        small = 0.0 if self.dtype == "bf16" else n * 2.0 ** -25 * float(np.abs(self.V).max())
        tol = 2.0 ** -8 * np.abs(o) + (p_round + 2 * dx + 2.0 ** -18) * absv * (1 + 2.0 ** -8) + small
        bad = np.abs(got - o)[rows] > tol[rows]
        assert not bad.any(), (np.abs(got - o)[rows].max(), tol[rows].min(), int(bad.sum()))
        assert np.all(np.abs(gl - l)[rows] <= dx + 2.0 ** -22 * (1 + np.abs(l[rows])) + 2.0 ** -20)


DECODE = [
    # lens, heads, kv_heads, page, window, num_sms
    ([1], 4, 1, 16, -1, 0),
    ([7, 16, 33, 64, 1, 15], 8, 2, 16, -1, 0),
    ([300, 5, 4097], 28, 4, 16, -1, 8),
    ([1000, 31], 32, 2, 1, -1, 0),        # token-granular pages, 16 query heads per KV head
    ([517, 2000, 1], 32, 1, 5, -1, 4),     # odd pages, two head groups
    ([2500, 900], 8, 8, 64, 700, 16),      # window, one query head per KV head
    ([129, 128, 127], 18, 2, 128, 0, 0),   # window of the last key alone, 9 query heads
]


@pytest.mark.parametrize("layout", ["nhd", "hnd", "padded", "head pools"])
@pytest.mark.parametrize("lens, heads, kv_heads, ps, window, sms", DECODE)
def test_nvfp4_decode(lens, heads, kv_heads, ps, window, sms, layout):
    c = Case(lens, heads, kv_heads, ps, "nvfp4", layout=layout, window=window, seed=len(lens))
    c.check(*c.plan(num_sms=sms).run(c.q, c.cache, return_lse=True))


def test_nvfp4_decode_unsplit_and_repeated_on_one_plan():
    c = Case([3000, 1500], 32, 8, 16, "nvfp4", seed=5)
    for kw in (dict(max_splits=1), dict(num_sms=152), dict(num_sms=3)):
        p = c.plan(**kw)
        for _ in range(2):
            c.check(*p.run(c.q, c.cache, return_lse=True))


def test_nvfp4_decode_of_large_queries():
    # |q| far beyond f16: the kernel scales its rows; scores stay moderate through a small pool scale
    c = Case([200, 90], 8, 2, 16, "nvfp4", seed=6, q_scale=2.0 ** 14, k_scale=0.002)
    c.cache.struct.k_scale = 0.002 * 2.0 ** -14
    c.K = c.K * 2.0 ** -14
    c.check(*c.plan().run(c.q, c.cache, return_lse=True))


@pytest.mark.parametrize("power", [-24, -60, -100])
def test_nvfp4_decode_of_small_queries(power):
    # |q| far below f16's normal range against a pool of large scale: the scores stay moderate
    c = Case([200, 90], 8, 2, 16, "nvfp4", seed=6, q_scale=2.0 ** power, k_scale=0.002)
    c.cache.struct.k_scale = 0.002 * 2.0 ** -power
    c.K = c.K * 2.0 ** -power
    c.check(*c.plan().run(c.q, c.cache, return_lse=True))


def test_nvfp4_decode_of_zero_queries_is_the_mean_of_v():
    c = Case([40, 7], 8, 2, 16, "nvfp4", seed=6, q_scale=0.0)
    out, lse = c.plan().run(c.q, c.cache, return_lse=True)
    c.check(out, lse)
    assert np.allclose(_np(lse), np.log([[40.0], [7.0]]), atol=1e-5)


def test_nvfp4_decode_with_requests_without_new_tokens_and_empty_ones():
    c = Case([40, 0, 17, 64], 8, 2, 16, "nvfp4", q_lens=[1, 0, 0, 1], seed=8)
    out, lse = c.plan().run(c.q, c.cache, return_lse=True)
    c.check(out, lse)
    p = c.plan(mode="mixed")
    c.check(*p.run(c.q, c.cache, return_lse=True))


def test_nvfp4_noalloc_decode_equals_the_workspace_one():
    pk = _pk()
    c = Case([900, 3, 2048], 32, 8, 16, "nvfp4", seed=9)
    host = c.plan(num_sms=64, host_only=True)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    for _ in range(2):
        pk._lib.check(pk._lib.lib().pkv_attn_decode_run_noalloc(host._h, c.q.data_ptr(), C.byref(c.cache.struct), out.data_ptr(),
                                                                lse.data_ptr(), torch.cuda.current_stream().cuda_stream))
        c.check(out, lse)


def test_nvfp4_masked_rows_never_read_their_scales():
    # codes and scales behind a request's end are NaN scales: nothing of them may reach the output
    c = Case([1, 5, 17, 30], 8, 2, 16, "nvfp4", seed=10)
    b = c.b
    for i, L in enumerate(b.kv_len):
        for j in range(int(L), len(b.block_rows[i]) * 16):
            page = int(b.block_rows[i][j // 16])
            for t in (2, 3):
                c.pools[t][page, j % 16] = 0x7F
            for t in (0, 1):
                c.pools[t][page, j % 16] = 0x77
    c.check(*c.plan().run(c.q, c.cache, return_lse=True))


def test_nvfp4_run_refuses_a_pool_of_another_type():
    pk = _pk()
    c = Case([40], 8, 2, 16, "nvfp4", seed=11)
    other = Case([40], 8, 2, 16, "e4m3", seed=11)
    with pytest.raises(pk.PkvError, match="dtype"):
        c.plan().run(c.q, other.cache)
    with pytest.raises(pk.PkvError, match="dtype"):
        other.plan().run(c.q, c.cache)


def test_extend_over_an_nvfp4_prefix_through_kv_load():
    # the documented way: load the cached prefix as bf16, attend to it with a ragged plan
    pk = _pk()
    c = Case([150, 70], 8, 2, 16, "nvfp4", seed=12)
    b = c.b
    pos = [np.arange(int(L)) for L in b.kv_len]
    slots = np.concatenate([np.asarray(b.block_rows[i])[p // 16] * 16 + p % 16 for i, p in enumerate(pos)])
    k, v = pk.kv_load(torch.from_numpy(slots).cuda(), c.cache)
    kv_indptr = np.concatenate([[0], np.cumsum(b.kv_len)]).astype(np.int32)
    q = torch.randn((9, 8, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    qo = np.array([0, 5, 9], np.int32)
    p = pk.Plan().plan(qo, kv_indptr, None, None, num_qo_heads=8, num_kv_heads=2, head_dim=128, mode="ragged")
    out, lse = p.run_ragged(q.cuda(), k, v, return_lse=True)
    ro, rl = OA.ragged_attention(q.double().numpy(), _np(k.float()).astype(np.float64), _np(v.float()).astype(np.float64), qo,
                                 kv_indptr)
    G.compare(out, lse, ro, rl)


# ------------------------------------------------------------------------------------------------
# scores
# ------------------------------------------------------------------------------------------------
def _check_scores(c, got, start, times=1):
    """start + times * the oracle's weights."""
    b = c.b
    P, ps, H = c.K.shape[:3]
    w = np.zeros((P, H, ps))
    OE.add_weights(w, b.q.double().numpy(), c.K, b.kv_indptr, b.kv_indices, b.last_page_len, b.qo_indptr, ps, c.window)
    got, start = _np(got).astype(np.float64), _np(start).astype(np.float64)
    ref = start + times * w
    tol = times * w * (2 * c.dx() + 2.0 ** -19) + (times + 1) * 2.0 ** -24 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))
    assert np.array_equal(got[w == 0], start[w == 0])  # slots of no visible key


SCORED = [(*d, "nvfp4", 128) for d in DECODE] + [(*d, "bf16", 128) for d in DECODE] + [(*d, "bf16", 64) for d in DECODE[:5]] + [
    (*d, "e4m3", 128) for d in DECODE]


@pytest.mark.parametrize("lens, heads, kv_heads, ps, window, sms, dtype, D", SCORED)
def test_scored_decode(lens, heads, kv_heads, ps, window, sms, dtype, D):
    c = Case(lens, heads, kv_heads, ps, dtype, D=D, window=window, seed=20 + len(lens))
    P = c.cache.num_pages
    start = torch.rand((P, kv_heads, ps), generator=torch.Generator().manual_seed(1)).cuda()
    scores = start.clone()
    p = c.plan(num_sms=sms, scored=True)
    c.check(*p.run(c.q, c.cache, return_lse=True, scores=scores))
    _check_scores(c, scores, start)
    out = p.run(c.q, c.cache, scores=scores)  # without an lse of the caller's, and once more on the same plan
    assert torch.isfinite(out.float()).all()
    _check_scores(c, scores, start, times=2)


def test_scored_decode_unsplit_long_range():
    c = Case([5000, 12], 8, 2, 16, "bf16", seed=30)
    scores = torch.zeros((c.cache.num_pages, 2, 16), device="cuda")
    c.check(*c.plan(max_splits=1, scored=True).run(c.q, c.cache, return_lse=True, scores=scores))
    _check_scores(c, scores, torch.zeros_like(scores))


def test_scored_mixed_plan_scores_the_one_token_rows():
    c = Case([300, 200, 90], 8, 2, 16, "bf16", layout="nhd", q_lens=[1, 20, 1], seed=31)
    scores = torch.zeros((c.cache.num_pages, 2, 16), device="cuda")
    out, lse = c.plan(mode="mixed", scored=True).run(c.q, c.cache, return_lse=True, scores=scores)
    o, l, _ = c.oracle()
    G.compare(out, lse, o, l)
    _check_scores(c, scores, torch.zeros_like(scores))


def test_scored_run_on_a_side_stream_and_in_a_captured_graph():
    c = Case([700, 45, 2000], 32, 8, 16, "nvfp4", seed=32)
    p = c.plan(num_sms=40, scored=True)
    scores = torch.zeros((c.cache.num_pages, 8, 16), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = p.run(c.q, c.cache, return_lse=True, scores=scores, stream=side)
    with torch.cuda.stream(side):
        out2 = torch.empty_like(out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            p.run(c.q, c.cache, out=out2, lse=lse, scores=scores)
        for _ in range(3):
            graph.replay()
    torch.cuda.current_stream().wait_stream(side)
    c.check(out, lse)
    c.check(out2, lse)
    _check_scores(c, scores, torch.zeros_like(scores), times=4)


def test_scored_run_refuses_a_small_scratch_and_a_prefill_plan():
    pk = _pk()
    c = Case([40, 20], 8, 2, 16, "bf16", layout="nhd", seed=33)
    p = c.plan(scored=True)
    L = pk._lib.lib()
    scores = torch.zeros((c.cache.num_pages, 2, 16), device="cuda")
    out = torch.empty_like(c.q)
    args = (c.q.data_ptr(), C.byref(c.cache.struct), out.data_ptr(), None, scores.data_ptr())
    n = C.c_size_t(0)
    assert L.pkv_attn_scored_scratch_size(p._h, C.byref(n)) == 0
    buf = torch.empty(n.value + 256, dtype=torch.uint8, device="cuda")
    assert L.pkv_attn_decode_run_scored(p._h, *args, buf.data_ptr(), n.value - 1, None) == pk._lib.PKV_EWORKSPACE
    assert L.pkv_attn_decode_run_scored(p._h, *args, None, n.value, None) == pk._lib.PKV_EWORKSPACE
    assert L.pkv_attn_decode_run_scored(p._h, *args, buf.data_ptr() + 64, n.value, None) == pk._lib.PKV_EINVAL
    assert L.pkv_attn_decode_run_scored(p._h, *args[:4], None, buf.data_ptr(), n.value, None) == pk._lib.PKV_EINVAL
    pre = c.plan(mode="prefill")
    assert L.pkv_attn_decode_run_scored(pre._h, *args, buf.data_ptr(), n.value, None) == pk._lib.PKV_EINVAL
    assert not scores.any()


# ------------------------------------------------------------------------------------------------
# eviction
# ------------------------------------------------------------------------------------------------
def _score_values(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "heavy":
        return torch.exp(2 * torch.randn(shape, generator=g)) * (torch.rand(shape, generator=g) > 0.2)
    if kind == "ties":
        return torch.randint(0, 4, shape, generator=g).float()
    if kind == "zero":
        return torch.zeros(shape)
    x = torch.randn(shape, generator=g)  # "wild": signs, infinities, NaN, signed zeros, the type's extremes
    r = torch.rand(shape, generator=g)
    for lo, val in ((0.0, float("nan")), (0.1, float("inf")), (0.15, float("-inf")), (0.2, 0.0), (0.3, -0.0),
                    (0.4, torch.finfo(torch.float32).min), (0.45, torch.finfo(torch.float32).max), (0.5, 1e-45)):
        x[(r >= lo) & (r < lo + 0.05)] = val
    return x


def _bits(t):
    t = t.detach().cpu().contiguous()
    return t.view({2: torch.int16, 4: torch.int32, 1: torch.uint8}[t.element_size()]).numpy().copy()


def _check_evict(lens, H, ps, dtype, budget, sink, recent, kind="heavy", D=128, layout="hnd", mode="decode", seed=0, q_lens=None):
    pk = _pk()
    b = W.make_batch(lens, q_lens or [min(1, int(L)) for L in lens], ps, H, H, D, seed)
    P = b.k_pool.shape[0]
    if dtype == "nvfp4":
        pools = list(_fp4_pools(P, ps, H, layout))
        for n, p in enumerate(pools):
            p.copy_(torch.randint(0, 256, p.shape, generator=torch.Generator().manual_seed(n + 1), dtype=torch.uint8))
        cache = pk.KVCache(pools[0], pools[1], k_sf=pools[2], v_sf=pools[3])
    else:
        pools = [b.k_pool.cuda(), b.v_pool.cuda()]
        if dtype == "e4m3":
            pools = [torch.randint(0, 256, p.shape, device="cuda", dtype=torch.uint8) for p in pools]
        if layout == "hnd" and mode == "decode":
            pools = [p.transpose(1, 2).contiguous().transpose(1, 2) for p in pools]
        cache = pk.KVCache(*pools)
    scores = _score_values(kind, (P, H, ps), seed + 1).cuda()
    plan = pk.Plan().plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, num_qo_heads=H, num_kv_heads=H, head_dim=D,
                          page_size=ps, mode=mode, kv_dtype=dtype)
    want = [_bits(p) for p in pools]
    ws = _bits(scores)
    values = _np(scores)
    # the oracle ranks float values and moves bit patterns
    idx = np.zeros((P, H, ps), dtype=np.int64) + np.arange(P * H * ps).reshape(P, H, ps)
    B = len(lens)
    kept = np.full((B, H, budget), -1, dtype=np.int32)
    for i in range(B):
        pages = np.asarray(b.block_rows[i], dtype=np.int64)
        L = int(lens[i])
        j = np.arange(L)
        for h in range(H):
            old = np.array(OE.kept_positions(values[pages[j // ps], h, j % ps], budget, sink, recent) if L else [], dtype=np.int64)
            kept[i, h, :len(old)] = old
            dst = np.arange(len(old))
            for p in want:
                p[pages[dst // ps], dst % ps, h] = p[pages[old // ps], old % ps, h].copy()
            ws[pages[dst // ps], h, dst % ps] = ws[pages[old // ps], h, old % ps].copy()
    got = plan.evict(cache, scores, budget, num_sink=sink, num_recent=recent)
    assert np.array_equal(_np(got), kept)
    for g, w in zip(pools, want):
        assert np.array_equal(_bits(g), w)
    assert np.array_equal(_bits(scores), ws)


EVICT = [
    # lens, kv heads, page, budget, sink, recent
    ([1, 2, 3], 2, 16, 1, 0, 0),
    ([5, 0, 9, 4], 1, 4, 4, 1, 1),
    ([40, 33, 32, 31, 64], 2, 16, 32, 4, 8),
    ([100, 70], 3, 1, 30, 0, 30),           # nothing but the recent keys
    ([100, 70], 2, 5, 30, 30, 0),           # nothing but the first keys
    ([100, 70], 2, 5, 30, 10, 20),          # first and recent fill the budget
    ([65, 66, 300], 2, 16, 64, 0, 32),      # the recent keys overlap themselves
    ([700, 1025, 64], 2, 16, 640, 4, 600),  # and in several tiles
    ([1000, 999], 2, 128, 100, 0, 0),
    ([4000, 2100, 2048], 1, 16, 2000, 4, 64),
]


@pytest.mark.parametrize("kind", ["heavy", "ties", "zero", "wild"])
@pytest.mark.parametrize("lens, H, ps, budget, sink, recent", EVICT)
def test_evict(lens, H, ps, budget, sink, recent, kind):
    _check_evict(lens, H, ps, "bf16", budget, sink, recent, kind=kind, D=64, seed=len(lens))


@pytest.mark.parametrize("dtype, D, layout", [("bf16", 128, "nhd"), ("bf16", 128, "hnd"), ("e4m3", 128, "nhd"), ("nvfp4", 128, "nhd"),
                                              ("nvfp4", 128, "hnd"), ("nvfp4", 128, "padded")])
def test_evict_moves_whole_rows_of_every_pool_type(dtype, D, layout):
    _check_evict([300, 130, 90, 260], 4, 16, dtype, 128, 3, 20, D=D, layout=layout, seed=3)
    _check_evict([300, 257], 2, 3, dtype, 256, 0, 250, D=D, layout=layout, seed=4)


def test_evict_with_many_units_and_more_moves_than_one_list_holds():
    # 160 units: one CTA each; 2,500 survivors of 5,000 keys with ascending scores all move
    _check_evict([5000] * 20, 8, 16, "bf16", 2500, 0, 0, kind="heavy", D=64, seed=5)
    pk = _pk()
    L, ps, b = 5000, 8, 2500
    pool = torch.zeros((L // ps, ps, 1, 64), dtype=torch.bfloat16, device="cuda")
    pool[..., 0] = torch.arange(L, device="cuda").view(-1, ps, 1) // 32
    cache = pk.KVCache(pool, pool.clone())
    pages = np.arange(L // ps, dtype=np.int32)
    plan = pk.Plan().plan([0, 1], [0, len(pages)], pages, [ps], num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=ps)
    scores = torch.arange(L, device="cuda", dtype=torch.float32).view(-1, 1, ps).contiguous()
    kept = plan.evict(cache, scores, b)
    assert torch.equal(kept[0, 0].cpu(), torch.arange(b, L, dtype=torch.int32))
    assert torch.equal(scores.view(-1)[:b].cpu(), torch.arange(b, L, dtype=torch.float32))
    assert torch.equal(cache.k[:, :, 0, 0].reshape(-1)[:b].cpu().float(), (torch.arange(b, L) // 32).to(torch.bfloat16).float())


SLICED = [
    # lens, kv heads, page, budget, sink, recent: requests beyond the whole form's 12288 keys
    ([20000, 13000, 100, 12289], 2, 16, 5000, 4, 300),
    ([20000, 12500], 1, 16, 12400, 0, 12000),  # recent keys that overlap themselves, in tiles of the cluster
    ([15001], 3, 5, 7000, 0, 0),               # odd pages
    ([13000], 2, 1, 600, 300, 300),            # nothing of the body
    ([33000], 1, 128, 30000, 16, 1000),        # more holes than one round of the lists holds
]


@pytest.mark.parametrize("kind", ["heavy", "ties", "zero", "wild"])
@pytest.mark.parametrize("lens, H, ps, budget, sink, recent", SLICED)
def test_evict_of_long_requests(lens, H, ps, budget, sink, recent, kind):
    _check_evict(lens, H, ps, "bf16", budget, sink, recent, kind=kind, D=64, seed=len(lens))


@pytest.mark.parametrize("dtype, layout", [("e4m3", "nhd"), ("nvfp4", "padded"), ("nvfp4", "hnd"), ("bf16", "hnd")])
def test_evict_of_long_requests_moves_every_pool_type(dtype, layout):
    _check_evict([14000, 12800], 2, 16, dtype, 12000, 4, 2000, layout=layout, seed=9)


def test_evict_of_more_long_units_than_clusters_run_at_once():
    _check_evict([12300] * 40, 4, 16, "bf16", 12200, 0, 40, kind="ties", D=64, seed=10)


def test_evict_with_survivors_all_behind_the_budget():
    # ascending scores: every survivor is a mover, in many rounds of the lists, in both forms
    pk = _pk()
    for L, b in ((12000, 5000), (100000, 45000)):
        ps = 8
        pool = torch.zeros((L // ps, ps, 1, 64), dtype=torch.bfloat16, device="cuda")
        pool[..., 0] = (torch.arange(L, device="cuda") // 512).view(-1, ps, 1)
        cache = pk.KVCache(pool, pool.clone())
        pages = np.random.RandomState(0).permutation(L // ps).astype(np.int32)
        at = torch.from_numpy(pages).cuda().long()
        plan = pk.Plan().plan([0, 1], [0, len(pages)], pages, [ps], num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=ps)
        scores = torch.empty((L // ps, 1, ps), device="cuda")
        scores[at, 0] = torch.arange(L, device="cuda", dtype=torch.float32).view(-1, ps)
        before = cache.k[at, :, 0, 0].reshape(-1).clone()
        kept = plan.evict(cache, scores, b)
        got = kept[0, 0].long()
        assert torch.equal(got.sort().values, torch.arange(L - b, L, device="cuda"))
        assert torch.equal(scores[at, 0].reshape(-1)[:b], got.float())
        for x in (cache.k, cache.v):
            assert torch.equal(x[at, :, 0, 0].reshape(-1)[:b], before[got])


@pytest.mark.parametrize("layout", ["pages outermost", "heads outermost"])
def test_pools_beyond_four_gigabytes(layout):
    # rows at byte offsets past 2^32 of an NVFP4 pool (by their page, or by their head alone): write, read
    # back, scored decode, eviction
    pk = _pk()
    P, ps, H = 640000, 16, 8
    if layout == "pages outermost":
        cache = pk.KVCache.nvfp4(P, ps, H, 128, 0.002, 0.002)
        assert cache.k.stride(0) * (P - 30) > 2 ** 32
    else:
        pools = [torch.empty((H, P, ps, w), dtype=torch.uint8, device="cuda").permute(1, 2, 0, 3) for w in (64, 64, 8, 8)]
        cache = pk.KVCache(pools[0], pools[1], 0.002, 0.002, k_sf=pools[2], v_sf=pools[3])
        assert cache.k.stride(0) * P < 2 ** 32 < cache.k.stride(2) * (H - 1)
    scores = torch.zeros((P, H, ps), device="cuda")
    pages = np.array([P - 1, 3, P - 30, P - 7, 11, P - 2], np.int32)
    L = 6 * ps - 5
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((L, H, 128), generator=g).to(torch.bfloat16) for _ in range(2))
    slots = torch.from_numpy(pages.astype(np.int64)[np.arange(L) // ps] * ps + np.arange(L) % ps).cuda()
    pk.kv_store(k.cuda(), v.cuda(), slots, cache, scores=scores)
    lk, lv = pk.kv_load(slots, cache)
    K, V = (O4.dequantize(*O4.quantize(x.float().numpy(), 0.002), 0.002) for x in (k, v))
    for got, ref in ((lk, K), (lv, V)):
        assert np.all(np.abs(_np(got.float()) - ref) <= 2.0 ** -8 * (1 + 2.0 ** -12) * np.abs(ref))
    q = torch.randn((1, 32, 128), generator=g).to(torch.bfloat16)
    plan = pk.Plan().plan([0, 1], [0, 6], pages, [L - 5 * ps], num_qo_heads=32, num_kv_heads=8, head_dim=128, page_size=ps,
                          kv_dtype="nvfp4", scored=True)
    out, lse = plan.run(q.cuda(), cache, return_lse=True, scores=scores)
    qn = q[0].double().numpy()
    for h in range(32):
        o, l = OA.attend(qn[h], K[:, h // 4], V[:, h // 4], 0, L - 1, 1 / np.sqrt(128))
        assert np.abs(_np(out[0, h].float()) - o).max() <= 2e-2 and abs(float(lse[0, h]) - l) <= 2e-3
    w = OE.key_weights(qn, K, 0, L - 1, 1 / np.sqrt(128), 4)
    got = _np(scores[torch.from_numpy(pages).cuda().long()]).transpose(0, 2, 1).reshape(-1, H)[:L]
    assert np.abs(got - w).max() <= 1e-4
    kept = _np(plan.evict(cache, scores, 40, num_sink=2, num_recent=8))
    ek, _ = pk.kv_load(slots[:40], cache)
    for h in range(H):
        assert torch.equal(ek[:, h], lk[torch.from_numpy(kept[0, h]).cuda().long(), h])


def test_evict_of_a_request_longer_than_the_score_cache():
    _check_evict([300000, 20], 1, 64, "bf16", 20000, 4, 100, D=64, seed=6)


@pytest.mark.parametrize("mode", ["prefill", "mixed"])
def test_evict_on_prefill_and_mixed_plans(mode):
    _check_evict([200, 140, 60], 2, 16, "bf16", 100, 4, 16, layout="nhd", mode=mode, q_lens=[30, 1, 5], seed=7)


def test_evict_refusals():
    pk = _pk()
    c = Case([100, 70], 8, 2, 16, "bf16", layout="nhd", seed=40)
    scores = torch.zeros((c.cache.num_pages, 2, 16), device="cuda")
    p = c.plan()
    for b, s, r in ((0, 0, 0), (-1, 0, 0), (10, -1, 0), (10, 0, -1), (10, 6, 5), (2 ** 21 + 1, 0, 0)):
        with pytest.raises(ValueError):
            p.evict(c.cache, scores, b, num_sink=s, num_recent=r)
        kept = torch.empty(16, dtype=torch.int32, device="cuda")
        assert pk._lib.lib().pkv_kv_evict(p._h, C.byref(c.cache.struct), scores.data_ptr(), b, s, r, kept.data_ptr(), None) in (
            pk._lib.PKV_EINVAL, pk._lib.PKV_EUNSUPPORTED)
    with pytest.raises(ValueError):
        p.evict(c.cache, scores, 10, kept=torch.empty((2, 2, 11), dtype=torch.int32, device="cuda"))
    with pytest.raises(pk.PkvError, match="window"):
        Case([100, 70], 8, 2, 16, "bf16", layout="nhd", window=10, seed=40).plan().evict(c.cache, scores, 10)
    b = c.b
    ix = b.kv_indices.copy()
    ix[1] = ix[0]
    shared = pk.Plan().plan(b.qo_indptr, b.kv_indptr, ix, b.last_page_len, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16)
    with pytest.raises(pk.PkvError, match="listed twice"):
        shared.evict(c.cache, scores, 10)
    rag = pk.Plan().plan([0, 1], [0, 5], None, None, num_qo_heads=8, num_kv_heads=2, head_dim=128, mode="ragged")
    with pytest.raises(ValueError):
        rag.evict(c.cache, scores, 10)
    with pytest.raises(pk.PkvError, match="dtype"):
        q4 = Case([100, 70], 8, 2, 16, "nvfp4", seed=40)
        p.evict(q4.cache, scores[:q4.cache.num_pages], 10)
    assert not scores.any()


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "nvfp4"])
def test_serving_steps_with_eviction(dtype):
    """Prompt write, scored decode steps, eviction, re-plan with the kept lengths, further steps: every step's
    output is the attention over the keys a host copy says are cached."""
    pk = _pk()
    H, Hq, ps, P, S, R, budget, D = 2, 8, 16, 24, 4, 16, 64, 128
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    if dtype == "nvfp4":
        cache = pk.KVCache.nvfp4(P, ps, H, D, 0.002, 0.002)
    else:
        cache = pk.KVCache(torch.zeros((P, ps, H, D), dtype=torch.bfloat16, device="cuda"),
                           torch.zeros((P, ps, H, D), dtype=torch.bfloat16, device="cuda"))
    scores = torch.full((P, H, ps), 1e9, device="cuda")  # stale values of the slots' last owners
    perm = torch.randperm(P, generator=g).tolist()
    rows = [perm[:10], perm[10:20]]
    lens = [150, 40]
    host = [[], []]  # per request: list over positions of (k, v) [H, D] as stored

    def stored(x):
        if dtype == "bf16":
            return x.double().numpy()
        q, f = O4.quantize(x.float().numpy(), 0.002)
        return O4.dequantize(q, f, 0.002)

    def write(i, pos, k, v):
        slots = torch.tensor([rows[i][p // ps] * ps + p % ps for p in pos])
        pk.kv_store(k.cuda(), v.cuda(), slots.cuda(), cache, scores=scores)
        host[i].extend(zip(stored(k), stored(v)))

    for i in range(2):
        write(i, range(lens[i]), rnd(lens[i], H, D), rnd(lens[i], H, D))
    plan = pk.Plan()

    def make_plan(scored):
        need = [-(-n // ps) for n in lens]
        plan.plan([0, 1, 2], np.concatenate([[0], np.cumsum(need)]), np.concatenate([rows[i][:need[i]] for i in range(2)]),
                  [n - (c - 1) * ps for n, c in zip(lens, need)], num_qo_heads=Hq, num_kv_heads=H, head_dim=D, page_size=ps,
                  kv_dtype=dtype, scored=scored)

    weights = [np.zeros((n, H)) for n in lens]

    def step():
        for i in range(2):
            write(i, [lens[i]], rnd(1, H, D), rnd(1, H, D))
            lens[i] += 1
            weights[i] = np.vstack([weights[i], np.zeros((1, H))])
        make_plan(True)
        q = rnd(2, Hq, D)
        out, lse = plan.run(q.cuda(), cache, return_lse=True, scores=scores)
        for i in range(2):
            K, V = (np.stack([kv[n] for kv in host[i]]) for n in (0, 1))
            qn = q[i].double().numpy()
            for hq in range(Hq):
                o, l = OA.attend(qn[hq], K[:, hq // 4], V[:, hq // 4], 0, lens[i] - 1, 1 / np.sqrt(D))
                assert np.abs(_np(out[i, hq].float()) - o).max() <= 2e-2
                assert abs(float(lse[i, hq]) - l) <= 2e-3
            weights[i] += OE.key_weights(qn, K, 0, lens[i] - 1, 1 / np.sqrt(D), Hq // H)
            j = np.arange(lens[i])
            got = _np(scores)[np.asarray(rows[i])[j // ps], :, j % ps]
            assert np.abs(got - weights[i]).max() <= 1e-4

    for phase in range(2):
        for _ in range(5):
            step()
        kept = _np(plan.evict(cache, scores, budget, num_sink=S, num_recent=R))
        for i in range(2):
            n = min(lens[i], budget)
            old = kept[i, :, :n]
            assert np.all(kept[i, :, n:] == -1)
            for h in range(H):
                assert sorted(set(old[h])) == sorted(old[h])
                if lens[i] > budget:  # the survivors outweigh the evicted, up to the scores' rounding
                    body = np.setdiff1d(old[h], np.r_[0:S, lens[i] - R:lens[i]])
                    out = np.setdiff1d(np.arange(S, lens[i] - R), body)
                    assert weights[i][body, h].min() >= weights[i][out, h].max() - 1e-4
            host[i] = [tuple(np.stack([host[i][old[h, p]][n][h] for h in range(H)]) for n in (0, 1)) for p in range(n)]
            weights[i] = np.stack([weights[i][old[h], h] for h in range(H)], axis=1)
            lens[i] = n
    step()


def test_eviction_step_in_a_captured_graph():
    pk = _pk()
    c = Case([300, 200], 8, 2, 16, "bf16", layout="nhd", seed=50)
    fresh = _score_values("heavy", (c.cache.num_pages, 2, 16), 3).cuda()
    scores = fresh.clone()
    p = c.plan(scored=True)
    kept = torch.empty((2, 2, 128), dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    pools = [x.clone() for x in c.pools]

    def fn():
        for x, y in zip(c.pools, pools):
            x.copy_(y)
        scores.copy_(fresh)
        p.run(c.q, c.cache, out=out, lse=lse, scores=scores)
        p.evict(c.cache, scores, 128, num_sink=4, num_recent=32, kept=kept)

    fn()
    torch.cuda.synchronize()
    want = [x.clone() for x in (*c.pools, scores, kept, lse)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fn()
    for t in (*c.pools, scores, kept):
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*c.pools, scores, kept, lse), want):
        if a.dtype == torch.float32:
            assert torch.allclose(a, b, rtol=1e-5, atol=1e-6)
        else:
            assert torch.equal(a, b)
