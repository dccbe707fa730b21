"""A decode step over selected pages on the GPU -- token map, rotary KV write, key bounds, selection, attention over the
selection, and a run of all of them -- against the oracle.

Tolerances:
* positions, slots, bounds, selected pages, pool contents against a KV write of the same keys: equal;
* turned elements: one rounding to bf16 (2^-8 relative) of a float32 value, whose error is bounded by (|x1| + |x2|) amplitude
  times: the phase's top 32 bits (2^-32 of a turn: 2^-29 rad) as a float (2^-24 of at most pi: 2^-22), sine and cosine (2 units
  in the last place, 2^-23 each), the amplitude's product and two products and a sum (2^-24 each): 2^-20 in all;
* attention: the bounds of test_gpu_compressed_cache, which this file's cases use.
"""

import ctypes as C
import math
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import blocks as OB
from tests.test_gpu_compressed_cache import Case, _fp4_pools, _np

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


def _batch(lens, q_lens, ps, seed=0):
    """Index arrays of a batch over shuffled pages, and the number of pages of its pool."""
    need = [-(-n // ps) for n in lens]
    P = sum(need) + 3
    idx = np.random.RandomState(seed).permutation(P)[:sum(need)].astype(np.int32)
    last = np.array([n - (k - 1) * ps if k else 0 for n, k in zip(lens, need)], np.int32)
    return (np.cumsum([0] + q_lens).astype(np.int32), np.cumsum([0] + need).astype(np.int32), idx, last), P


# ------------------------------------------------------------------------------------------------
# token map
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("mode, lens, q_lens, ps", [
    ("decode", [1], [1], 16), ("decode", [5, 0, 16, 17, 300], [1, 0, 1, 0, 1], 16), ("decode", list(range(1, 400)), [1] * 399, 5),
    ("mixed", [40, 7, 0, 900, 33], [40, 0, 0, 1, 30], 16), ("mixed", [0, 9, 9, 0], [0, 0, 9, 0], 1),
    ("prefill", [2000, 1, 128, 129], [2000, 1, 100, 129], 128), ("prefill", [3, 4], [0, 0], 16)])
@pytest.mark.parametrize("shifted", [False, True])
def test_token_map(mode, lens, q_lens, ps, shifted):
    pk = _pk()
    idx, P = _batch(lens, q_lens, ps)
    off = np.random.RandomState(1).randint(-5, 1 << 40, len(lens)) if shifted else None
    p = pk.Plan().plan(*idx, num_qo_heads=4, num_kv_heads=2, head_dim=128, page_size=ps, mode=mode)
    pos, slots = p.token_map(None if off is None else torch.from_numpy(off).cuda())
    want = OB.token_map(*idx, ps, off)
    assert pos.dtype == slots.dtype == torch.int64 and pos.is_contiguous() and slots.is_contiguous()
    assert np.array_equal(_np(pos), want[0]) and np.array_equal(_np(slots), want[1])


def test_token_map_refusals():
    pk = _pk()
    idx, P = _batch([40, 20], [1, 1], 16)
    kw = dict(num_qo_heads=4, num_kv_heads=2, head_dim=128, page_size=16)
    p = pk.Plan().plan(*idx, mode="decode", **kw)
    for off in (torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64)):
        with pytest.raises(ValueError, match="offsets"):
            p.token_map(off)
    with pytest.raises(pk.PkvError, match="positions"):
        pk.Plan().plan(*idx, mode="prefill", causal=False, **kw).token_map()
    for mode in ("ragged", "paged_ragged"):
        with pytest.raises(pk.PkvError, match="needs a PKV_MODE_DECODE"):
            pk.Plan().plan(idx[0], idx[0] if mode == "ragged" else idx[1], idx[2], idx[3], mode=mode, **kw).token_map()


# ------------------------------------------------------------------------------------------------
# rotary KV write
# ------------------------------------------------------------------------------------------------
def _cache(dtype, P, ps, H, D, layout):
    """A cache of any type filled with a byte pattern, and its tensors."""
    pk = _pk()
    if dtype == "nvfp4":
        t = list(_fp4_pools(P, ps, H, layout))
        return pk.KVCache(t[0], t[1], 0.002, 0.0017, k_sf=t[2], v_sf=t[3]), t
    kind, fill = (torch.bfloat16, 7.0) if dtype == "bf16" else (torch.uint8, 0xA5)
    shape = (P, H, ps, D) if layout == "hnd" else (P, ps, H, D)
    t = [torch.full(shape, fill, dtype=kind, device="cuda") for _ in range(2)]
    if layout == "hnd":
        t = [x.transpose(1, 2) for x in t]
    return (pk.KVCache(*t) if dtype == "bf16" else pk.KVCache(*t, 0.013, 0.017)), t


def _turned(rot, x, pos):
    """Oracle rows, and the tolerance of each element."""
    x = x.double().cpu().numpy()
    angle = 2 * math.pi * OB.turns(pos, rot.phase_step.cpu().numpy().view(np.uint64).tolist())
    want = OB.rotate(x, angle, rot.interleaved, rot.amplitude)
    R = rot.rotary_dim
    a = np.abs(x[..., :R])
    if rot.interleaved:
        both = np.repeat(a[..., 0::2] + a[..., 1::2], 2, -1)
    else:
        both = np.tile(a[..., :R // 2] + a[..., R // 2:], 2)
    tol = 2.0 ** -8 * np.abs(want)
    tol[..., :R] += 2.0 ** -20 * abs(rot.amplitude) * both
    tol[..., R:] = 0.0  # (passes through)
    return want, tol


def _near(got, want, tol):
    d = np.abs(got.double().cpu().numpy() - want)
    assert np.all(d <= tol), (float(d.max()), int((d > tol).sum()))


ROPE = [
    # dtype, D, rotary, interleaved, heads, kv_heads, tokens, page, layout
    ("bf16", 128, 128, False, 32, 8, 64, 16, "nhd"),
    ("bf16", 128, 128, True, 8, 2, 7, 1, "hnd"),
    ("bf16", 128, 32, False, 28, 4, 33, 5, "nhd"),
    ("bf16", 128, 48, True, 1, 1, 1, 128, "nhd"),
    ("bf16", 64, 64, False, 5, 5, 301, 64, "hnd"),
    ("bf16", 64, 16, True, 3, 1, 2, 16, "nhd"),
    ("bf16", 64, 48, False, 128, 8, 9, 16, "nhd"),  # more rows than threads
    ("e4m3", 128, 128, False, 32, 8, 65, 16, "nhd"),
    ("e4m3", 128, 64, True, 64, 8, 17, 1, "hnd"),
    ("e4m3", 64, 32, False, 4, 2, 5, 3, "nhd"),
    ("nvfp4", 128, 128, False, 32, 8, 65, 16, "hnd"),
    ("nvfp4", 128, 128, True, 8, 2, 7, 16, "nhd"),
    ("nvfp4", 128, 16, False, 8, 2, 3, 16, "padded"),
    ("nvfp4", 128, 48, False, 40, 8, 11, 128, "head pools"),
    ("nvfp4", 128, 80, False, 4, 4, 6, 16, "hnd"),
    ("nvfp4", 128, 112, True, 128, 8, 4, 1, "hnd"),
    # more tokens than SMs: several rounds of fewer threads
    ("bf16", 128, 128, False, 32, 8, 200, 16, "nhd"),
    ("bf16", 64, 32, True, 40, 8, 153, 16, "hnd"),
    ("e4m3", 128, 96, False, 32, 8, 160, 64, "nhd"),
    ("nvfp4", 128, 96, False, 28, 4, 170, 16, "hnd"),
]


@pytest.mark.parametrize("dtype, D, R, interleaved, heads, kv_heads, T, ps, layout", ROPE)
def test_rope_store(dtype, D, R, interleaved, heads, kv_heads, T, ps, layout):
    pk = _pk()
    g = torch.Generator().manual_seed(T + R)
    qkv = torch.randn((T, heads + 2 * kv_heads, D), generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
    P = -(-T // ps) + 2
    slots = torch.randperm(P * ps, generator=g)[:T].cuda()
    if T > 4:
        slots[3] = -1
    pos = torch.randint(0, 131072, (T,), generator=g)
    pos[0] = 0
    rot = pk.Rotary(D, rotary_dim=R, base=500000.0, interleaved=interleaved, amplitude=1.2 if R == 48 else None)
    cache, pools = _cache(dtype, P, ps, kv_heads, D, layout)
    other, want_pools = _cache(dtype, P, ps, kv_heads, D, layout)
    before = qkv.clone()
    qo, ko = pk.rope_store(q, k, v, pos.cuda(), slots, cache, rot, return_k=True)
    assert torch.equal(qkv, before) and qo.is_contiguous() and ko.is_contiguous()
    _near(qo, *_turned(rot, q, pos.tolist()))
    _near(ko, *_turned(rot, k, pos.tolist()))
    pk.kv_store(ko, v.contiguous(), slots, other)
    for a, b in zip(pools, want_pools):
        assert torch.equal(a, b)
    # without the turned keys, over given outputs
    cache2, pools2 = _cache(dtype, P, ps, kv_heads, D, layout)
    out = torch.empty_like(qo)
    assert pk.rope_store(q, k, v, pos.cuda(), slots, cache2, rot, q_out=out) is out and torch.equal(out, qo)
    for a, b in zip(pools2, want_pools):
        assert torch.equal(a, b)


def test_rope_store_in_place_and_broadcast_inputs():
    pk = _pk()
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((6, h, 128), generator=g).to(torch.bfloat16).cuda() for h in (8, 2, 2))
    pos, slots = torch.arange(6).cuda() * 1000, torch.arange(6).cuda()
    rot = pk.Rotary(128)
    a, pa = _cache("bf16", 1, 16, 2, 128, "nhd")
    qo, ko = pk.rope_store(q, k, v, pos, slots, a, rot, return_k=True)
    b, pb = _cache("bf16", 1, 16, 2, 128, "nhd")
    q2, k2 = q.clone(), k.clone()
    ret = pk.rope_store(q2, k2, v, pos, slots, b, rot, q_out=q2, k_out=k2)
    assert ret[0] is q2 and ret[1] is k2 and torch.equal(q2, qo) and torch.equal(k2, ko) and torch.equal(pa[0], pb[0])
    # one row for all tokens and heads
    one = q[:1, :1].expand(6, 8, 128)
    assert torch.equal(pk.rope_store(one, k, v, pos, slots, b, rot), pk.rope_store(one.contiguous(), k, v, pos, slots, b, rot))


def test_rope_store_of_single_rows_of_any_stride():
    # the stride of a dimension of one is not used
    pk = _pk()
    base = torch.randn(4096, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    one = base[:512].view(4, 128)
    rot = pk.Rotary(128)
    pos, slot = torch.tensor([77], device="cuda"), torch.tensor([3], device="cuda")
    a, pa = _cache("bf16", 1, 16, 1, 128, "nhd")
    b, pb = _cache("bf16", 1, 16, 1, 128, "nhd")
    want = pk.rope_store(one[None], one[None, :1], one[None, 1:2], pos, slot, a, rot)
    got = pk.rope_store(torch.as_strided(base, (1, 4, 128), (13, 128, 1)), torch.as_strided(base, (1, 1, 128), (1, 3, 1)),
                        torch.as_strided(base, (1, 1, 128), (5, 7, 1), 128), pos, slot, b, rot)
    assert torch.equal(got, want) and torch.equal(pa[0], pb[0]) and torch.equal(pa[1], pb[1])
    with pytest.raises(pk.PkvError, match="strides"):
        pk.rope_store(torch.as_strided(base, (2, 4, 128), (516, 128, 1)), torch.zeros((2, 1, 128), dtype=torch.bfloat16, device="cuda"),
                      torch.zeros((2, 1, 128), dtype=torch.bfloat16, device="cuda"), pos.expand(2).contiguous(), slot.expand(2).contiguous(), b, rot)


def test_rope_store_of_far_and_negative_positions():
    pk = _pk()
    pos = [-1, -131072, 2 ** 31 - 1, 2 ** 31, 2 ** 40 + 12345, -2 ** 63, 2 ** 63 - 1, 2 ** 20]
    T = len(pos)
    q = torch.randn((T, 4, 128), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    k = q[:, :1].contiguous()
    rot = pk.Rotary(128, inv_freq=np.linspace(0.0, 6.3, 64))
    cache, pools = _cache("bf16", 1, 16, 1, 128, "nhd")
    qo, ko = pk.rope_store(q, k, k, torch.tensor(pos).cuda(), torch.arange(T).cuda(), cache, rot, return_k=True)
    _near(qo, *_turned(rot, q, pos))
    assert torch.equal(pools[0][0, :T], ko) and torch.equal(pools[1][0, :T], k)


def test_rope_store_passes_infinities_and_nan_to_their_pair_only():
    pk = _pk()
    q = torch.randn((2, 4, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    clean = q.clone()
    q[0, 1, 5], q[1, 2, 70] = float("inf"), float("nan")
    k = clean[:, :1].contiguous()
    rot = pk.Rotary(128)
    args = (torch.tensor([3, 4]).cuda(), torch.arange(2).cuda(), _cache("bf16", 1, 16, 1, 128, "nhd")[0], rot)
    a, b = pk.rope_store(q, k, k, *args), pk.rope_store(clean, k, k, *args)
    bad = torch.zeros_like(a, dtype=torch.bool)
    bad[0, 1, [5, 69]] = bad[1, 2, [6, 70]] = True
    assert torch.equal(a[~bad], b[~bad]) and not a[bad].isfinite().any()


def test_rope_store_slots_out_of_range_and_scores():
    pk = _pk()
    q, k = torch.randn((5, 4, 128), device="cuda").to(torch.bfloat16), torch.randn((5, 2, 128), device="cuda").to(torch.bfloat16)
    cache, pools = _cache("bf16", 3, 4, 2, 128, "nhd")
    scores = torch.full((3, 2, 4), 7.0, device="cuda")
    slots = torch.tensor([0, 12, 6, -3, 2 ** 40], device="cuda")
    rot, pos = pk.Rotary(128), torch.arange(5, device="cuda")
    qo, ko = pk.rope_store(q, k, k, pos, slots, cache, rot, scores=scores, return_k=True)
    assert pk.device_error() == 1 and pk.device_error() == 0
    _near(qo, *_turned(rot, q, range(5)))
    want = torch.full((3, 2, 4), 7.0)
    want[0, :, 0] = want[1, :, 2] = 0
    assert torch.equal(scores.cpu(), want)
    wk = torch.full((3, 4, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    wk[0, 0], wk[1, 2] = ko[0], ko[2]
    assert torch.equal(pools[0], wk)
    # nothing to write
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert pk.rope_store(e, e[:, :2], e[:, :2], none, none, cache, rot).shape == (0, 4, 128)
    with pytest.raises(ValueError, match="rotary must be on"):
        pk.rope_store(q, k, k, pos, slots, cache, pk.Rotary(128, device="cpu"))


# ------------------------------------------------------------------------------------------------
# key bounds
# ------------------------------------------------------------------------------------------------
def _want_codes(c, codes, scale, q_lens, every):
    b = c.b
    for i, n in enumerate(b.kv_len):
        for blk in range(int(b.kv_indptr[i + 1] - b.kv_indptr[i])):
            lo, hi = blk * b.page_size, min(int(n), (blk + 1) * b.page_size)
            if not every and (q_lens[i] == 0 or hi <= n - q_lens[i]):
                continue
            page = int(b.kv_indices[b.kv_indptr[i] + blk])
            codes[page] = OB.page_bounds(c.K[page, :hi - lo], scale)
    return codes


BOUNDS = [
    # dtype, lens, heads, kv_heads, page, D, layout, q_lens, mode
    ("bf16", [1, 15, 16, 17, 33], 4, 2, 16, 128, "hnd", None, "decode"),
    ("bf16", [200, 7, 129], 4, 4, 64, 64, "nhd", None, "decode"),
    ("bf16", [300, 8, 9], 2, 1, 8, 128, "nhd", None, "decode"),
    ("bf16", [250, 1000, 31], 4, 2, 24, 128, "hnd", [1, 0, 1], "decode"),
    ("bf16", [100, 70, 40, 33], 4, 2, 16, 128, "nhd", [50, 0, 1, 33], "mixed"),
    ("bf16", [100, 70, 256], 4, 2, 128, 128, "nhd", [100, 3, 128], "prefill"),
    ("e4m3", [1, 15, 16, 17, 500], 4, 2, 16, 128, "nhd", None, "decode"),
    ("e4m3", [260, 128], 8, 8, 128, 128, "nhd", None, "decode"),
    ("nvfp4", [1, 15, 16, 17, 500], 4, 2, 16, 128, "hnd", None, "decode"),
    ("nvfp4", [260, 128, 3], 2, 1, 128, 128, "padded", [1, 1, 0], "decode"),
    ("nvfp4", [31, 64], 4, 4, 32, 128, "head pools", None, "decode"),
    # more pages than one CTA each takes, their rows in several rounds
    ("bf16", [7000, 5001], 4, 4, 40, 64, "nhd", None, "decode"),
    ("bf16", [9000, 1], 2, 2, 33, 128, "hnd", [3000, 1], "mixed"),
    ("e4m3", [8000, 39], 4, 4, 40, 128, "nhd", None, "decode"),
    ("nvfp4", [8000, 121], 4, 4, 40, 128, "hnd", None, "decode"),
]


@pytest.mark.parametrize("every", [False, True])
@pytest.mark.parametrize("dtype, lens, heads, kv_heads, ps, D, layout, q_lens, mode", BOUNDS)
def test_bound_keys(dtype, lens, heads, kv_heads, ps, D, layout, q_lens, mode, every):
    pk = _pk()
    c = Case(lens, heads, kv_heads, ps, dtype, D=D, layout=layout, seed=5, q_lens=q_lens)
    r = np.random.RandomState(0)
    scale = (r.rand(kv_heads, D) * 0.03 + 0.02).astype(np.float32)
    scale[0, 3] = 0.001  # most keys lie beyond 127 steps
    start = r.randint(-127, 128, (c.cache.num_pages, kv_heads, 2, D)).astype(np.int8)
    b = pk.KeyBounds(torch.from_numpy(start).cuda(), torch.from_numpy(scale).cuda())
    c.plan(mode=mode).bound_keys(c.cache, b, all_pages=every)
    want = _want_codes(c, start.copy(), scale, q_lens or [1] * len(lens), every)
    assert np.array_equal(_np(b.codes), want)


def test_bound_keys_of_special_values():
    pk = _pk()
    k = torch.randn((4, 16, 2, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    for j, x in enumerate((float("nan"), float("inf"), float("-inf"), -0.0, 3e38, 1e-40)):
        k[0, j, 0, 10 + j], k[1, 9, 1, 10 + j] = x, x
    k[2, :, :, 7] = 0.0
    k[3, 5:] = float("nan")  # behind the request's end
    scale = np.full((2, 128), 0.25, np.float32)
    scale[1, 12], scale[0, 7], scale[1, 7] = 3e38, 0.0, np.inf  # (0 / 0 and 0 / inf)
    cache = pk.KVCache(k.cuda(), k.cuda().clone())
    b = pk.KeyBounds(torch.zeros((4, 2, 2, 128), dtype=torch.int8, device="cuda"), torch.from_numpy(scale).cuda())
    p = pk.Plan().plan([0, 1], [0, 4], [0, 1, 2, 3], [5], num_qo_heads=2, num_kv_heads=2, head_dim=128, page_size=16, mode="decode")
    p.bound_keys(cache, b, all_pages=True)
    K = k.double().numpy()
    want = np.stack([OB.page_bounds(K[i, :5 if i == 3 else 16], scale) for i in range(4)])
    assert np.array_equal(_np(b.codes), want)


def test_bound_keys_of_many_requests_some_without_pages():
    pk = _pk()
    lens = [(37 * i) % 90 for i in range(700)]
    idx, P = _batch(lens, [1 if n and i % 3 else 0 for i, n in enumerate(lens)], 16, seed=4)
    k = torch.randn((P, 16, 1, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    cache = pk.KVCache(k, k.clone())
    p = pk.Plan().plan(*idx, num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=16, mode="decode")
    for every in (False, True):
        b = pk.KeyBounds.of(cache, 0.03)
        p.bound_keys(cache, b, all_pages=every)
        valid = np.zeros(P, np.int64)  # keys of the pages that are looked at
        for i, n in enumerate(lens):
            pages = idx[2][idx[1][i]:idx[1][i + 1]]
            if every:
                valid[pages] = 16
            if len(pages) and (every or idx[0][i + 1] > idx[0][i]):
                valid[pages[-1]] = idx[3][i]
        x = k.float()
        there = torch.from_numpy(valid).cuda()[:, None] > torch.arange(16, device="cuda")
        s = torch.tensor(0.03, device="cuda")
        lo = torch.floor(x.masked_fill(~there[..., None, None], math.inf).amin(1) / s)
        hi = torch.ceil(x.masked_fill(~there[..., None, None], -math.inf).amax(1) / s)
        want = torch.stack((lo, hi), 2).clamp(-127, 127)
        want[torch.from_numpy(valid).cuda() == 0] = 0
        assert torch.equal(b.codes.float(), want)


def test_bound_keys_refusals():
    pk = _pk()
    c = Case([40, 20], 4, 2, 4, "bf16", layout="nhd")
    with pytest.raises(pk.PkvError, match="page_size"):
        c.plan().bound_keys(c.cache, pk.KeyBounds.of(c.cache, 1.0))
    c = Case([40, 20], 4, 2, 16, "bf16", layout="nhd")
    b, p = pk.KeyBounds.of(c.cache, 1.0), c.plan()
    other = pk.KVCache(torch.zeros_like(c.cache.k).view(torch.uint8)[..., :128].contiguous(), torch.zeros_like(c.cache.k).view(torch.uint8)[..., :128].contiguous())
    with pytest.raises(pk.PkvError, match="geometry"):
        p.bound_keys(other, b)
    L = pk._lib.lib()
    args = (p._h, C.byref(c.cache.struct))
    assert L.pkv_key_bounds_update(*args, None, b.scale.data_ptr(), 0, None) == -1
    assert L.pkv_key_bounds_update(*args, b.codes.data_ptr() + 8, b.scale.data_ptr(), 0, None) == -1
    assert L.pkv_key_bounds_update(*args, b.codes.data_ptr(), None, 0, None) == -1
    assert not b.codes.any()
    none = pk.Plan().plan([0], [0], [], [], num_qo_heads=4, num_kv_heads=2, head_dim=128, page_size=16, mode="decode")
    none.bound_keys(c.cache, b)
    assert not b.codes.any()


# ------------------------------------------------------------------------------------------------
# selection
# ------------------------------------------------------------------------------------------------
class Selection:
    def __init__(self, lens, heads, kv_heads, ps, D, num_blocks, q_lens=None, kind="random", seed=0):
        pk = _pk()
        r = np.random.RandomState(seed)
        self.q_lens = q_lens or [1] * len(lens)
        self.lens, self.ps, self.K = lens, ps, num_blocks
        self.idx, P = _batch(lens, self.q_lens, ps, seed)
        mid, half = r.randn(P, kv_heads, 1, D) * 20, r.rand(P, kv_heads, 1, D) * 40
        codes = np.concatenate([mid - half, mid + half], 2)
        if kind == "few":    # a handful of different pages: many equal scores
            codes = codes[r.randint(0, 3, P)]
        if kind == "equal":
            codes[:] = codes[:1]
        if kind == "outlier":  # one page far above the others: most scores share a digit
            codes = np.where(np.arange(P)[:, None, None, None] == self.idx[2][-1], 127, codes * 0.05)
        if kind == "extreme":
            codes = np.where(r.rand(*codes.shape) < 0.5, -127, 127)
        self.codes = np.clip(np.rint(codes), -127, 127).astype(np.int8)
        self.scale = (r.rand(kv_heads, D) * 0.05 + 0.01).astype(np.float32)
        q = torch.from_numpy(r.randn(sum(self.q_lens), heads, D)).to(torch.bfloat16)
        if kind == "extreme":
            q = torch.sign(q)
            self.scale[:] = 1.0
        if kind == "wild":
            q[0] = 0
            q[1, 0, 3], q[1, 1, 4], q[1, 2, 5] = float("nan"), float("inf"), float("-inf")
            q[2] *= 1e38
            q[3] *= 1e-40
        self.q = q
        self.b = pk.KeyBounds(torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scale).cuda())
        self.plan = pk.Plan().plan(*self.idx, num_qo_heads=heads, num_kv_heads=kv_heads, head_dim=D, page_size=ps, mode="decode",
                                   num_blocks=num_blocks)

    def want(self, sink, recent):
        qo, kv, pages, _ = self.idx
        H = self.codes.shape[1]
        G = self.q.shape[1] // H
        q = self.q.float().numpy()
        out = np.full((len(q), H, self.K), -1, np.int32)
        for i in range(len(self.lens)):
            if qo[i + 1] > qo[i]:
                mine = pages[kv[i]:kv[i + 1]]
                for h in range(H):
                    out[qo[i], h] = OB.select(q[qo[i], h * G:(h + 1) * G], self.codes[mine, h], self.scale[h], len(mine), self.K, sink, recent)
        return out

    def check(self, sink, recent, **kw):
        got = self.plan.select(self.q.cuda(), self.b, num_sink=sink, num_recent=recent, **kw)
        want = self.want(sink, recent)
        assert np.array_equal(_np(got), want), np.argwhere(_np(got) != want)[:5]
        return got


SELECT = [
    # lens, heads, kv_heads, page, D, blocks, sink, recent
    ([1, 16, 17, 63, 64, 65, 81, 1000], 8, 2, 16, 128, 4, 1, 1),
    ([500, 513], 8, 8, 16, 128, 1, 0, 1),             # the last page alone
    ([500, 513, 30], 5, 1, 16, 64, 3, 1, 2),          # no page competes
    ([800, 13, 4096], 28, 4, 8, 128, 100, 2, 4),
    ([4000, 3999, 2, 700], 16, 1, 32, 64, 33, 0, 2),
    ([4096] * 3, 40, 2, 64, 128, 63, 1, 1),           # all but one
    ([4096] * 3, 40, 2, 64, 128, 64, 1, 1),           # every page
    ([9000], 128, 1, 64, 128, 20, 1, 1),              # 128 query heads
    ([33000, 60000, 5], 8, 2, 16, 128, 200, 1, 4),    # several CTAs per unit
    ([131071], 4, 1, 8, 128, 700, 3, 5),
    ([300 + i for i in range(300)], 4, 2, 16, 64, 9, 1, 1),
    ([5000] * 30 + [6001], 4, 2, 16, 128, 60, 1, 1),   # a CTA per unit, an SM each
    ([4700 + 9 * i for i in range(80)], 4, 2, 16, 128, 40, 1, 2),  # more units than SMs
    ([9000, 8000], 6, 2, 16, 64, 50, 0, 3),            # several CTAs per unit, head_dim 64
]


@pytest.mark.parametrize("kind", ["random", "few", "equal", "extreme", "outlier"])
@pytest.mark.parametrize("lens, heads, kv_heads, ps, D, K, sink, recent", SELECT)
def test_select(lens, heads, kv_heads, ps, D, K, sink, recent, kind):
    Selection(lens, heads, kv_heads, ps, D, K, kind=kind, seed=len(lens)).check(sink, recent)


def test_select_of_special_queries():
    Selection([700, 600, 500, 400, 300], 6, 2, 16, 128, 8, kind="wild").check(1, 1)


def test_select_with_requests_without_new_tokens():
    s = Selection([0, 500, 40, 700, 0], 4, 2, 16, 128, 6, q_lens=[0, 1, 0, 1, 0])
    out = torch.full((2, 2, 6), 99, dtype=torch.int32, device="cuda")
    assert s.check(1, 2, blocks=out) is out
    none = Selection([500, 40], 4, 2, 16, 128, 6, q_lens=[0, 0])
    assert none.check(1, 2).shape == (0, 2, 6)


def test_select_of_the_longest_requests():
    # as many pages as one CTA's shared memory holds scores of, and codes beyond 2^31 bytes
    pk = _pk()
    P, H, D = 49152 + 37, 192, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    codes = torch.randint(-127, 128, (P, H, 2, D), generator=g, device="cuda", dtype=torch.int8)
    q = torch.randn((1, H, D), generator=g, device="cuda").to(torch.bfloat16)
    scale = torch.rand((H, D), generator=g, device="cuda") + 0.5
    pages = torch.randperm(P, generator=g, device="cuda")[:49152]
    p = pk.Plan().plan([0, 1], [0, 49152], pages.cpu().numpy(), [3], num_qo_heads=H, num_kv_heads=H, head_dim=D, page_size=8,
                       mode="decode", num_blocks=1000)
    got = _np(p.select(q, pk.KeyBounds(codes, scale), num_sink=2, num_recent=2))
    for h in (0, 100, 191):
        want = OB.select(q[0, h:h + 1].float().cpu().numpy(), codes[pages, h].cpu().numpy(), scale[h].cpu().numpy(), 49152, 1000, 2, 2)
        assert got[0, h].tolist() == want


def test_select_refusals():
    pk = _pk()
    s = Selection([500, 300], 4, 2, 16, 128, 6)
    q = s.q.cuda()
    for sink, recent in ((-1, 1), (0, 0), (5, 2), (2 ** 31 - 1, 2 ** 31 - 1)):
        with pytest.raises(pk.PkvError, match="num_sink"):
            s.plan.select(q, s.b, num_sink=sink, num_recent=recent)
    for kw in (dict(num_sink=2 ** 32), dict(num_recent=2 ** 32 + 1), dict(num_sink=-2 ** 31 - 1)):
        with pytest.raises(ValueError, match="32 bits"):
            s.plan.select(q, s.b, **kw)
    with pytest.raises(pk.PkvError, match="bounds have"):
        s.plan.select(q, pk.KeyBounds(s.b.codes[:20].clone(), s.b.scale))
    with pytest.raises(ValueError, match="blocks"):
        s.plan.select(q, s.b, blocks=torch.zeros((2, 2, 5), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="q must"):
        s.plan.select(s.q, s.b)


# ------------------------------------------------------------------------------------------------
# attention over selected pages
# ------------------------------------------------------------------------------------------------
def _choose(c, K, seed, q_lens=None):
    """Random selections: ascending pages, the last one among them."""
    b, r = c.b, np.random.RandomState(seed)
    rows = []
    for i in range(len(b.kv_len)):
        if b.qo_indptr[i + 1] == b.qo_indptr[i]:
            continue
        N = int(b.kv_indptr[i + 1] - b.kv_indptr[i])
        for _ in range(b.num_kv_heads):
            n = min(N, K)
            pick = sorted(r.permutation(N - 1)[:n - 1]) + [N - 1]
            rows.append(pick + [-1] * (K - n))
    return np.array(rows, np.int32).reshape(-1, b.num_kv_heads, K)


class Chosen(Case):
    """A case whose oracle sees the selected pages only."""

    def choose(self, K, seed=0):
        self.blocks = _choose(self, K, seed)
        return torch.from_numpy(self.blocks).cuda()

    def oracle(self):
        b = self.b
        a = (b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, b.page_size)
        q = b.q.double().numpy()
        o, lse = OB.attend_blocks(q, self.K, self.V, self.blocks, *a)
        return o, lse, OB.attend_blocks(q, self.K, np.abs(self.V), self.blocks, *a)[0]


ATTEND = [
    # dtype, lens, heads, kv_heads, page, D, layout, blocks, num_sms
    ("bf16", [1, 16, 17, 300, 1000], 8, 2, 16, 128, "hnd", 5, 0),
    ("bf16", [2500, 33], 28, 4, 8, 64, "nhd", 31, 0),
    ("bf16", [900, 901, 77], 32, 2, 24, 128, "nhd", 7, 0),     # pages that end inside a tile, 16 query heads per KV head
    ("bf16", [5000, 4000], 40, 1, 64, 128, "hnd", 50, 8),      # head groups, shared units
    ("bf16", [700, 65], 4, 4, 128, 128, "nhd", 1, 0),          # the last page alone
    ("e4m3", [3000, 17, 450], 32, 8, 16, 128, "nhd", 40, 4),
    ("e4m3", [700, 1, 640], 18, 2, 40, 128, "nhd", 6, 0),
    ("nvfp4", [3000, 17, 450], 32, 8, 16, 128, "hnd", 40, 4),
    ("nvfp4", [700, 1, 640], 16, 2, 24, 128, "padded", 6, 0),
    ("nvfp4", [6000, 8000], 20, 1, 128, 128, "hnd", 30, 16),
    ("bf16", [12000, 8191], 4, 2, 8, 128, "nhd", 1025, 0),     # more pages than are looked up ahead
    ("e4m3", [9000], 4, 1, 8, 128, "nhd", 1100, 4),
    ("nvfp4", [33000], 8, 1, 16, 128, "hnd", 1500, 20),
]


@pytest.mark.parametrize("dtype, lens, heads, kv_heads, ps, D, layout, K, sms", ATTEND)
def test_attention_over_selected_pages(dtype, lens, heads, kv_heads, ps, D, layout, K, sms):
    c = Chosen(lens, heads, kv_heads, ps, dtype, D=D, layout=layout, seed=7)
    p = c.plan(num_blocks=K, num_sms=sms)
    blocks = c.choose(K)
    for _ in range(2):  # the shared units' counters are ready again
        out, lse = p.run(c.q, c.cache, return_lse=True, blocks=blocks)
        c.check(out, lse)
    assert torch.equal(p.run(c.q, c.cache, blocks=blocks).isfinite(), torch.ones_like(out, dtype=torch.bool))


def test_attention_with_requests_without_new_tokens():
    c = Chosen([300, 200, 0, 90], 8, 2, 16, "bf16", layout="nhd", q_lens=[1, 0, 0, 1], seed=8)
    out, lse = c.plan(num_blocks=4).run(c.q, c.cache, return_lse=True, blocks=c.choose(4))
    c.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_every_page_selected_is_the_dense_run(dtype):
    c = Case([300, 17, 2000], 8, 2, 16, dtype, layout="hnd", seed=9)
    blocks = torch.full((3, 2, 200), -1, dtype=torch.int32)
    for i, n in enumerate((300, 17, 2000)):
        blocks[i, :, :-(-n // 16)] = torch.arange(-(-n // 16))
    a = c.plan(num_blocks=200, max_splits=1).run(c.q, c.cache, return_lse=True, blocks=blocks.cuda())
    b = c.plan(max_splits=1).run(c.q, c.cache, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_one_kv_head_is_the_dense_run_over_the_selected_pages(dtype):
    pk = _pk()
    c = Chosen([3000, 700, 15], 4, 1, 16, dtype, layout="hnd", seed=10)
    blocks = c.choose(12)
    a = c.plan(num_blocks=12, max_splits=1).run(c.q, c.cache, return_lse=True, blocks=blocks)
    b, lists = c.b, []
    for i in range(3):
        mine = b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i + 1]]
        lists.append(mine[[x for x in c.blocks[i, 0] if x >= 0]])
    p = pk.Plan().plan(b.qo_indptr, np.cumsum([0] + [len(x) for x in lists]), np.concatenate(lists), b.last_page_len, num_qo_heads=4,
                       num_kv_heads=1, head_dim=128, page_size=16, mode="decode", kv_dtype=dtype, max_splits=1)
    d = p.run(c.q, c.cache, return_lse=True)
    assert torch.equal(a[0], d[0]) and torch.equal(a[1], d[1])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_a_block_outside_its_request_is_recorded(dtype):
    pk = _pk()
    c = Chosen([300, 200], 8, 2, 16, dtype, layout="hnd", seed=11)
    p, blocks = c.plan(num_blocks=4), c.choose(4)
    good = p.run(c.q, c.cache, blocks=blocks)
    assert pk.device_error() == 0
    for x in (-1, 13, 2 ** 31 - 1, -2 ** 31):  # (200 keys are 13 pages: 0 .. 12)
        bad = blocks.clone()
        bad[1, 1, 2] = x
        out = p.run(c.q, c.cache, blocks=bad)
        assert pk.device_error() == 2
        assert torch.equal(out[0], good[0]) and torch.equal(out[1, :4], good[1, :4])


def test_runs_over_every_page_refuse_a_plan_over_selected_pages():
    pk = _pk()
    c = Chosen([300, 200], 8, 2, 16, "bf16", layout="nhd", seed=12)
    p, blocks = c.plan(num_blocks=4), c.choose(4)
    with pytest.raises(pk.PkvError, match="decode_run_blocks"):
        p.run(c.q, c.cache)
    L = pk._lib.lib()
    out, n = torch.empty_like(c.q), C.c_size_t(0)
    assert L.pkv_attn_decode_run_noalloc(p._h, c.q.data_ptr(), C.byref(c.cache.struct), out.data_ptr(), None, None) == -1
    assert L.pkv_attn_scored_scratch_size(p._h, C.byref(n)) == -1
    d = c.plan()
    assert L.pkv_attn_decode_run_blocks(d._h, c.q.data_ptr(), C.byref(c.cache.struct), blocks.data_ptr(), out.data_ptr(), None, None) == -1
    assert L.pkv_attn_decode_run_blocks(p._h, c.q.data_ptr(), C.byref(c.cache.struct), None, out.data_ptr(), None, None) == -1
    assert L.pkv_block_select(d._h, c.q.data_ptr(), out.data_ptr(), out.data_ptr(), 100, 1, 1, blocks.data_ptr(), None) == -1
    with pytest.raises(ValueError, match="blocks need"):
        p.run(c.q, c.cache, blocks=blocks, scores=torch.zeros((c.cache.num_pages, 2, 16), device="cuda"))
    with pytest.raises(ValueError, match="out must"):
        p.run(c.q, c.cache, blocks=blocks, out=out[:1])


# ------------------------------------------------------------------------------------------------
# all of them
# ------------------------------------------------------------------------------------------------
class Server:
    """Requests that grow by a token per step over one layer's cache, with a copy of every turned key and value."""

    def __init__(self, prompts, heads, kv_heads, ps, dtype, num_blocks, D=128, room=8, seed=0):
        pk = _pk()
        self.pk, self.heads, self.H, self.ps, self.dtype, self.K, self.D = pk, heads, kv_heads, ps, dtype, num_blocks, D
        self.r = torch.Generator().manual_seed(seed)
        need = [-(-(n + room) // ps) for n in prompts]
        self.P = sum(need) + 2
        perm = np.random.RandomState(seed).permutation(self.P).astype(np.int32)
        self.tables = np.split(perm[:sum(need)], np.cumsum(need)[:-1])
        self.cache, self.pools = _cache(dtype, self.P, ps, kv_heads, D, "hnd")
        self.rot = pk.Rotary(D, base=500000.0)
        self.bounds = pk.KeyBounds.of(self.cache, 0.04)
        self.lens, self.dropped = [0] * len(prompts), [0] * len(prompts)

    def index(self, q_lens):
        need = [-(-n // self.ps) for n in self.lens]
        idx = np.concatenate([t[:k] for t, k in zip(self.tables, need)])
        last = [n - (k - 1) * self.ps for n, k in zip(self.lens, need)]
        return (np.cumsum([0] + q_lens).astype(np.int32), np.cumsum([0] + need).astype(np.int32), idx, np.array(last, np.int32))

    def tokens(self, T):
        return tuple(torch.randn((T, h, self.D), generator=self.r).to(torch.bfloat16).cuda() for h in (self.heads, self.H, self.H))

    def plan(self, q_lens, mode, num_blocks=0, kv_dtype=None):
        kw = dict(num_qo_heads=self.heads, num_kv_heads=self.H, head_dim=self.D, page_size=self.ps, kv_dtype=kv_dtype or self.dtype)
        return self.pk.Plan().plan(*self.index(q_lens), mode=mode, num_blocks=num_blocks, **kw)

    def values(self):
        slots = torch.arange(self.P * self.ps).cuda()
        k, v = self.pk.kv_load(slots, self.cache)
        return [x.double().cpu().numpy().reshape(self.P, self.ps, self.H, self.D) for x in (k, v)]


@pytest.mark.parametrize("dtype, heads, kv_heads, ps", [("bf16", 8, 2, 16), ("e4m3", 4, 4, 32), ("nvfp4", 16, 2, 16)])
def test_serving_steps_over_selected_pages(dtype, heads, kv_heads, ps):
    prompts = [5, 333, 1000, 64]
    s = Server(prompts, heads, kv_heads, ps, dtype, 6)
    pk = s.pk
    # the prompts: positions and slots from a prefill plan (of a bf16 view: the map does not read the pool)
    s.lens = list(prompts)
    q, k, v = s.tokens(sum(prompts))
    first = s.plan(prompts, "prefill", kv_dtype="bf16")
    pk.rope_store(q, k, v, *first.token_map(), s.cache, s.rot)
    if dtype == "bf16":
        first.bound_keys(s.cache, s.bounds)
    else:
        s.plan([1] * 4, "decode").bound_keys(s.cache, s.bounds, all_pages=True)
    for step in range(5):
        s.lens = [n + 1 for n in s.lens]
        q, k, v = s.tokens(4)
        p = s.plan([1] * 4, "decode", num_blocks=s.K)
        pos, slots = p.token_map()
        assert pos.tolist() == [n - 1 for n in s.lens]
        q = pk.rope_store(q, k, v, pos, slots, s.cache, s.rot)
        p.bound_keys(s.cache, s.bounds)
        blocks = p.select(q, s.bounds, num_sink=1, num_recent=2)
        out, lse = p.run(q, s.cache, return_lse=True, blocks=blocks)
        # the bounds are those of the pool, the selection that of the bounds, the outputs those of the selection
        K, V = s.values()
        idx = s.index([1] * 4)
        codes, scale = _np(s.bounds.codes), _np(s.bounds.scale)
        G = heads // kv_heads
        for i, n in enumerate(s.lens):
            pages = idx[2][idx[1][i]:idx[1][i + 1]]
            for b, page in enumerate(pages):
                valid = K[page, :min(ps, n - b * ps)]
                if dtype != "nvfp4":  # (kv_load rounds a 4-bit value to bf16)
                    if dtype == "bf16":
                        assert np.array_equal(codes[page], OB.page_bounds(valid, scale))
                assert np.all(codes[page, :, 0] * 0.04 <= valid.min(0) + 0.04) and np.all(codes[page, :, 1] * 0.04 >= valid.max(0) - 0.04)
            for h in range(kv_heads):
                want = OB.select(q[i, h * G:(h + 1) * G].float().cpu().numpy(), codes[pages, h], scale[h], len(pages), s.K, 1, 2)
                assert blocks[i, h].tolist() == want
        o, l = OB.attend_blocks(q.double().cpu().numpy(), K, V, _np(blocks), *idx, ps)
        # (values read back are rounded to bf16, 2^-8: as far off as the probabilities; N(0, 1) rows)
        assert np.abs(out.double().cpu().numpy() - o).max() <= 0.04 and np.abs(_np(lse) - l).max() <= 0.04


def test_steps_after_eviction_have_fresh_bounds_and_true_positions():
    s = Server([400, 90], 8, 2, 16, "bf16", 4, seed=3)
    pk = s.pk
    s.lens = [400, 90]
    q, k, v = s.tokens(490)
    first = s.plan([400, 90], "prefill")
    pos, slots = first.token_map()
    pk.rope_store(q, k, v, pos, slots, s.cache, s.rot)
    first.bound_keys(s.cache, s.bounds)
    scores = torch.rand((s.P, 2, 16), device="cuda")
    s.plan([1, 1], "decode", num_blocks=4).evict(s.cache, scores, 128, num_sink=4, num_recent=16)
    s.lens, s.dropped = [128 + 1, 90 + 1], [400 - 128, 0]
    p = s.plan([1, 1], "decode", num_blocks=4)
    pos, slots = p.token_map(torch.tensor(s.dropped).cuda())
    assert pos.tolist() == [400, 90]
    q, k, v = s.tokens(2)
    q = pk.rope_store(q, k, v, pos, slots, s.cache, s.rot)
    p.bound_keys(s.cache, s.bounds, all_pages=True)
    K, _ = s.values()
    idx, codes = s.index([1, 1]), _np(s.bounds.codes)
    for i, n in enumerate(s.lens):
        for b, page in enumerate(idx[2][idx[1][i]:idx[1][i + 1]]):
            assert np.array_equal(codes[page], OB.page_bounds(K[page, :min(16, n - 16 * b)], _np(s.bounds.scale)))


@pytest.mark.parametrize("lens", [[700, 45, 3000], [70000, 9]])
def test_a_step_on_a_side_stream_and_in_a_captured_graph(lens):
    s = Server(lens, 8, 2, 16, "bf16", 8, seed=5)
    pk = s.pk
    s.lens = list(lens)
    for x in s.pools:
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"))
    p = s.plan([1] * len(lens), "decode", num_blocks=8)
    q, k, v = s.tokens(len(lens))
    p.bound_keys(s.cache, s.bounds, all_pages=True)
    blocks = torch.empty((len(lens), 2, 8), dtype=torch.int32, device="cuda")
    out, qo = torch.empty_like(q), torch.empty_like(q)

    def step(stream=None):
        pos, slots = p.token_map(stream=stream)
        pk.rope_store(q, k, v, pos, slots, s.cache, s.rot, q_out=qo, stream=stream)
        p.bound_keys(s.cache, s.bounds, stream=stream)
        p.select(qo, s.bounds, blocks=blocks, stream=stream)
        p.run(qo, s.cache, out=out, blocks=blocks, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (*s.pools, s.bounds.codes, blocks, qo)]
    o = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def again(run):
        for x in (s.pools[0][:, 0], s.bounds.codes[p_last], blocks, qo, out):
            x.zero_()
        s.pools[0].copy_(start[0])
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        for a, b in zip((*s.pools, s.bounds.codes, blocks, qo), want):
            assert torch.equal(a, b)
        # (shared units claim their keys at run time: float32 sums in another order, one rounding)
        assert torch.allclose(out.float(), o.float(), rtol=2.0 ** -6, atol=2.0 ** -10)

    start = [x.clone() for x in s.pools]
    p_last = torch.tensor([t[-(-n // 16) - 1] for t, n in zip(s.tables, lens)]).long().cuda()
    again(lambda: step(side))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    again(graph.replay)
    again(graph.replay)


def test_memory_of_results_on_another_stream():
    # results for a given stream come from its memory: blocks freed on the current one may be in use there
    s = Server([700, 45], 8, 2, 16, "bf16", 8, seed=6)
    s.lens = [700, 45]
    p = s.plan([1, 1], "decode", num_blocks=8)
    q, k, v = s.tokens(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pos, slots = p.token_map(stream=side)
    qo = s.pk.rope_store(q, k, v, pos, slots, s.cache, s.rot, stream=side)
    p.bound_keys(s.cache, s.bounds, all_pages=True, stream=side)
    blocks = p.select(qo, s.bounds, stream=side)
    a = p.run(qo, s.cache, blocks=blocks, stream=side)
    side.synchronize()
    pos2, slots2 = p.token_map()
    qo2 = s.pk.rope_store(q, k, v, pos2, slots2, s.cache, s.rot)
    b2 = p.select(qo2, s.bounds)
    assert torch.equal(pos, pos2) and torch.equal(slots, slots2) and torch.equal(qo, qo2) and torch.equal(blocks, b2)
    assert torch.equal(a, p.run(qo2, s.cache, blocks=b2))


def test_calls_return_the_given_outputs_and_keep_nothing():
    s = Server([700, 45], 8, 2, 16, "bf16", 8, seed=7)
    s.lens = [700, 45]
    p = s.plan([1, 1], "decode", num_blocks=8)
    q, k, v = s.tokens(2)
    p.bound_keys(s.cache, s.bounds, all_pages=True)
    given = [torch.empty_like(q), torch.empty_like(k), torch.empty((2, 2, 8), dtype=torch.int32, device="cuda"), torch.empty_like(q),
             torch.empty((2, 8), device="cuda")]
    qo, ko, blocks, out, lse = given

    def step(give):
        pos, slots = p.token_map()
        r = s.pk.rope_store(q, k, v, pos, slots, s.cache, s.rot, *((qo, ko) if give else ()), return_k=True)
        p.bound_keys(s.cache, s.bounds)
        b = p.select(r[0], s.bounds, blocks=blocks if give else None)
        return (*r, b, *p.run(r[0], s.cache, *((out, lse) if give else ()), return_lse=True, blocks=b))

    assert all(a is b for a, b in zip(step(True), given))
    assert all(torch.equal(a, b) for a, b in zip(step(False)[:3], given))
    everything = [*given, q, k, v, p, p.workspace, p._streams, s.cache, s.cache.struct, s.bounds.codes, s.rot.phase_step]
    before, memory = [sys.getrefcount(x) for x in everything], torch.cuda.memory_allocated()
    for i in range(60):
        step(i % 2 == 0)
    assert [sys.getrefcount(x) for x in everything] == before and torch.cuda.memory_allocated() == memory


def test_steps_from_several_threads_and_streams():
    servers = [Server([700 + 16 * i, 45], 8, 2, 16, "bf16", 8, seed=8 + i) for i in range(4)]
    work = []
    for i, s in enumerate(servers):
        for x in s.pools:
            x.copy_(torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda"))
        s.lens = [700 + 16 * i, 45]
        p, stream = s.plan([1, 1], "decode", num_blocks=8), torch.cuda.Stream()
        p.bound_keys(s.cache, s.bounds, all_pages=True)
        work.append((s, p, stream, s.tokens(2)))

    def step(s, p, t):
        pos, slots = p.token_map()
        qo = s.pk.rope_store(*t, pos, slots, s.cache, s.rot)
        p.bound_keys(s.cache, s.bounds)
        blocks = p.select(qo, s.bounds)
        return pos, slots, qo, blocks, p.run(qo, s.cache, blocks=blocks)

    want = [[x.clone() for x in step(s, p, t)] for s, p, _, t in work]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def run(i):
        try:
            s, p, stream, t = work[i]
            with torch.cuda.stream(stream):
                for _ in range(100):
                    got[i] = step(s, p, t)
                stream.synchronize()
                assert stream.cuda_stream in p._streams  # the plan's workspace is recorded on it
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))
        # (shared units claim their keys at run time: float32 sums in another order, one rounding)
        assert torch.allclose(a[4].float(), b[4].float(), rtol=2.0 ** -6, atol=2.0 ** -10)


def test_host_tensors_with_a_stream_are_refused():
    pk = _pk()
    k = torch.zeros((11, 16, 2, 128), dtype=torch.bfloat16)
    cache, side = pk.KVCache(k, k.clone()), torch.cuda.Stream()
    p = pk.Plan().plan(*_batch([100, 50], [1, 1], 16)[0], num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, mode="decode",
                       num_blocks=4)
    q, kv, i = torch.zeros((2, 8, 128), dtype=torch.bfloat16), torch.zeros((2, 2, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    b, blocks = pk.KeyBounds.of(cache, 1.0), torch.zeros((2, 2, 4), dtype=torch.int32)
    for f in (lambda: pk.rope_store(q, kv, kv, i, i, cache, pk.Rotary(128, device="cpu"), stream=side), lambda: p.bound_keys(cache, b, stream=side),
              lambda: p.select(q, b, stream=side), lambda: p.run(q, cache, blocks=blocks, stream=side, return_lse=True)):
        with pytest.raises(ValueError, match="current CUDA device"):
            f()
    with pytest.raises(ValueError, match="offsets"):
        p.token_map(i, stream=side)
