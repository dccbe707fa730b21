"""Decode over selected pages on the host (no GPU): the oracle pinned to closed forms and brute force, the frequencies and
phase steps of Rotary, the plans over selected pages, and every refusal of the entry points."""

import ctypes as C
import math
import sys

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import blocks as OB


@pytest.fixture(scope="module")
def pk():
    from paged_kv_attention_slot_gb300 import build as B

    B.build()
    import paged_kv_attention_slot_gb300 as pk

    pk._lib.lib()
    return pk


# ---- oracle ----
def test_token_map_worked_example():
    # request 0: 5 keys on pages 7, 2 (page size 4), 2 of them new; request 1: nothing new; request 2: 1 key on page 0
    pos, slots = OB.token_map([0, 2, 2, 3], [0, 2, 3, 4], [7, 2, 5, 0], [1, 4, 1], 4, offsets=[10, 0, -1])
    assert pos.tolist() == [13, 14, -1] and slots.tolist() == [7 * 4 + 3, 2 * 4, 0]


def test_rotate_is_a_turn_of_the_complex_plane():
    r = np.random.RandomState(0)
    x, angle = r.randn(3, 2, 64), r.randn(3, 16)
    half, near = OB.rotate(x, angle, False, 1.5), OB.rotate(x, angle, True, 1.5)
    z = 1.5 * np.exp(1j * angle)[:, None]
    w = (x[..., :16] + 1j * x[..., 16:32]) * z
    assert np.allclose(half, np.concatenate([w.real, w.imag, x[..., 32:]], -1), atol=1e-14)
    w = (x[..., 0:32:2] + 1j * x[..., 1:32:2]) * z
    assert np.allclose(near[..., 0:32:2], w.real, atol=1e-14) and np.allclose(near[..., 1:32:2], w.imag, atol=1e-14)
    assert np.array_equal(near[..., 32:], x[..., 32:])


def test_turns_depend_on_position_differences_only():
    r = np.random.RandomState(1)
    steps = r.randint(0, 2 ** 62, 8).astype(np.uint64)
    q, k = r.randn(1, 1, 16), r.randn(1, 1, 16)
    dots = []
    for shift in (0, 5, 2 ** 40, -17):
        a, b = (OB.rotate(x, 2 * math.pi * OB.turns([p + shift], steps), True) for x, p in ((q, 11), (k, 4)))
        dots.append(float((a * b).sum()))
    assert np.allclose(dots, dots[0], atol=1e-12)


def test_page_bounds_bound_the_keys():
    r = np.random.RandomState(2)
    K = r.randn(9, 2, 8).astype(np.float32)
    scale = (r.rand(2, 8) * 0.02 + 0.04).astype(np.float32)
    c = OB.page_bounds(K, scale).astype(np.float64)
    assert np.all(c[:, 0] * scale <= K.min(0) + 1e-6) and np.all(c[:, 1] * scale >= K.max(0) - 1e-6)
    assert np.all(c[:, 0] * scale > K.min(0) - scale - 1e-6) and np.all(c[:, 1] * scale < K.max(0) + scale + 1e-6)


def test_page_bounds_special_values():
    K = np.zeros((2, 1, 6), np.float32)
    K[:, 0] = [[np.nan, np.inf, -1e30, 2.0, -0.0, np.nan], [1, 1, 1, 2.0, 0.0, np.inf]]
    c = OB.page_bounds(K, np.ones((1, 6), np.float32))[0]
    assert c[0].tolist() == [-127, 1, -127, 2, 0, -127] and c[1].tolist() == [127, 127, 1, 2, 0, 127]


def test_selection_keeps_the_pages_of_the_largest_bounds():
    r = np.random.RandomState(3)
    for _ in range(50):
        G, D, N = int(r.randint(1, 6)), 8, int(r.randint(1, 30))
        S, R = int(r.randint(0, 3)), int(r.randint(1, 3))
        n = int(r.randint(S + R, S + R + 12))
        lo = r.randint(-127, 128, (N, D))
        codes = np.stack([lo, np.minimum(127, lo + r.randint(0, 60, (N, D)))], 1).astype(np.int8)
        q, scale = r.randn(G, D).astype(np.float32), np.ones(D, np.float32)
        got = OB.select(q, codes, scale, N, n, S, R)
        live = [b for b in got if b >= 0]
        assert live == sorted(set(live)) and len(got) == n and len(live) == min(N, n)
        if N > n:
            assert live[:S] == list(range(S)) and live[len(live) - R:] == list(range(N - R, N))
            # the real bound, to the rounding of the codes (half a unit each, times 127, per head and channel)
            real = (np.maximum(q[:, None] * codes[None, :, 0], q[:, None] * codes[None, :, 1])).sum((0, 2))
            slack = 127 * G * D * 0.5 * np.abs(q).max() / (32767 // G)
            out = sorted(set(range(S, N - R)) - set(live))
            if out and n > S + R:
                assert real[sorted(set(live) - set(range(S)) - set(range(N - R, N)))].min() >= real[out].max() - 2 * slack


def test_selection_ties_go_to_the_lower_page_and_nothing_counts_without_a_query():
    codes = np.full((9, 2, 4), 3, np.int8)
    assert OB.select(np.ones((2, 4)), codes, np.ones(4), 9, 5, 1, 2) == [0, 1, 2, 7, 8]
    wild = np.random.RandomState(0).randint(-127, 128, (9, 2, 4)).astype(np.int8)
    for q in (np.zeros((2, 4)), np.full((2, 4), np.nan), np.full((2, 4), np.inf)):
        assert OB.select(q, wild, np.ones(4), 9, 5, 0, 1) == [0, 1, 2, 3, 8]


def test_attention_over_every_page_is_attention():
    r = np.random.RandomState(4)
    k, v, q = r.randn(6, 4, 2, 8), r.randn(6, 4, 2, 8), r.randn(2, 4, 8)
    a = ([0, 1, 1, 2], [0, 2, 4, 6], [3, 0, 5, 2, 1, 4], [3, 4, 1], 4)
    blocks = np.tile(np.array([0, 1, -1], np.int32), (2, 2, 1))
    o, lse = OB.attend_blocks(q, k, v, blocks, *a)
    wo, wl = OA.paged_attention(q, k, v, *a)
    assert np.allclose(o, wo, atol=1e-13) and np.allclose(lse, wl, atol=1e-13)


# ---- Rotary ----
def test_rotary_frequencies(pk):
    f = 500000.0 ** (-np.arange(0, 128, 2) / 128)
    assert np.array_equal(pk.Rotary(128, base=500000.0, device="cpu").inv_freq, f)
    assert np.allclose(pk.Rotary(128, base=500000.0, scaling="linear", factor=4, device="cpu").inv_freq, f / 4, rtol=1e-15)
    g = pk.Rotary(128, base=500000.0, scaling="base", factor=4, device="cpu").inv_freq
    assert g[0] == 1 and np.isclose(g[-1], f[-1] / 4, rtol=1e-12) and np.all(np.diff(g / f) < 0)
    w = pk.Rotary(128, base=500000.0, scaling="wavelength", factor=8, device="cpu")
    t = 8192 * f / (2 * np.pi)
    assert np.array_equal(w.inv_freq[t >= 4], f[t >= 4]) and np.allclose(w.inv_freq[t <= 1], f[t <= 1] / 8, rtol=1e-15)
    mid = (t > 1) & (t < 4)
    assert mid.any() and np.allclose(w.inv_freq[mid], f[mid] * ((t[mid] - 1) / 3 + (4 - t[mid]) / 3 / 8), rtol=1e-12)
    assert w.amplitude == 1.0
    y = pk.Rotary(64, scaling="ramp", factor=4, original_positions=4096, low_turns=1, high_turns=32, device="cpu")
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    # pairs that turn 32 times and once: indices 10.46 and 22.5
    assert np.array_equal(y.inv_freq[:11], f[:11]) and np.allclose(y.inv_freq[23:], f[23:] / 4, rtol=1e-15)
    assert np.isclose(y.inv_freq[16], f[16] * (7 / 13 + 6 / 13 / 4), rtol=1e-12)
    assert np.isclose(y.amplitude, 0.1 * math.log(4) + 1)
    assert pk.Rotary(64, scaling="ramp", factor=4, amplitude=1.25, device="cpu").amplitude == 1.25
    own = pk.Rotary(64, rotary_dim=32, inv_freq=f[:16] * 3, interleaved=True, device="cpu")
    assert np.array_equal(own.inv_freq, f[:16] * 3) and own.phase_step.shape == (16,) and own.interleaved


def test_rotary_phase_steps_are_turns_per_position(pk):
    r = pk.Rotary(64, inv_freq=np.linspace(-7.0, 40.0, 32), device="cpu")
    steps = r.phase_step.numpy().view(np.uint64)
    for f, s in zip(r.inv_freq, steps.tolist()):
        # 2 pi in float64 and the quotient: two roundings of 2^-53, relative to the turns
        off = (s / 2.0 ** 64 - f / (2 * math.pi)) % 1.0
        assert min(off, 1 - off) <= 2.0 ** -51 * (1 + abs(f))


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=144), dict(base=0.0), dict(base=float("inf")), dict(scaling="other"),
    dict(scaling="linear", factor=0.0), dict(scaling="wavelength", factor=2.0, low_turns=4.0, high_turns=4.0),
    dict(scaling="ramp", factor=2.0, base=1.0), dict(inv_freq=[1.0] * 63), dict(inv_freq=[1.0] * 64, scaling="linear"),
    dict(inv_freq=[float("nan")] * 64), dict(amplitude=float("nan")), dict(scaling="wavelength", original_positions=0)])
def test_rotary_refusals(pk, kw):
    with pytest.raises(ValueError):
        pk.Rotary(128, device="cpu", **kw)


# ---- plans over selected pages ----
def _plan(pk, lens, num_blocks, q_lens=None, ps=16, heads=8, kv_heads=2, **kw):
    need = [-(-n // ps) for n in lens]
    q = [1] * len(lens) if q_lens is None else q_lens
    a = dict(num_qo_heads=heads, num_kv_heads=kv_heads, head_dim=128, page_size=ps, mode="decode", num_sms=152, host_only=True,
             num_blocks=num_blocks)
    a.update(kw)
    return pk.Plan().plan(np.cumsum([0] + q), np.cumsum([0] + need), np.arange(sum(need)),
                          [n - (k - 1) * ps if k else 0 for n, k in zip(lens, need)], **a)


def test_plan_reads_the_selected_keys_only(pk):
    lens = [1, 16, 17, 160, 161, 1000, 100000]
    p = _plan(pk, lens, 10)
    items = p.work_items()
    for i, n in enumerate(lens):
        pages = -(-n // 16)
        want = n if pages <= 10 else 9 * 16 + n - (pages - 1) * 16
        mine = items[items[:, 0] == i]
        assert set(mine[:, 1]) == {0, 1} and np.all(mine[:, 3] == 0) and np.all(mine[:, 4] == want)
    assert p.info()["kv_tokens"] == sum(int(items[items[:, 0] == i][0, 4]) for i in range(len(lens)))
    assert p.info()["max_page_id"] == sum(-(-n // 16) for n in lens) - 1


def test_plan_over_more_pages_than_there_are_is_the_dense_plan(pk):
    lens = [5, 700, 3000]
    a, b = _plan(pk, lens, 1000), _plan(pk, lens, 0)
    assert np.array_equal(a.work_items(), b.work_items())
    assert a.info() == b.info()


def test_workspace_size_of_selected_pages(pk):
    ps, lens = 16, [40000, 70000]
    need = [-(-n // ps) for n in lens]
    args = (np.arange(3), np.cumsum([0] + need), np.arange(sum(need)), [n - (k - 1) * ps for n, k in zip(lens, need)])
    kw = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=ps, mode="decode", num_sms=152)
    n = pk.Plan.workspace_size(*args, num_blocks=64, **kw)
    assert n == _plan(pk, lens, 64).info()["workspace_bytes"] < pk.Plan.workspace_size(*args, **kw)


@pytest.mark.parametrize("kw, status", [
    (dict(mode="prefill", num_blocks=4), "PKV_EINVAL"), (dict(mode="mixed", num_blocks=4), "PKV_EINVAL"),
    (dict(window_left=100, num_blocks=4), "PKV_EINVAL"), (dict(num_blocks=-1), "PKV_EINVAL"),
    (dict(num_blocks=49153), "PKV_EUNSUPPORTED"), (dict(num_blocks=4, ps=7), "PKV_EUNSUPPORTED"),
    (dict(num_blocks=4, heads=258), "PKV_EUNSUPPORTED")])
def test_plan_refusals(pk, kw, status):
    kw = dict(kw)
    with pytest.raises(pk.PkvError, match=status):
        _plan(pk, [100, 50], kw.pop("num_blocks"), **kw)


def test_plan_refuses_scores_and_too_long_requests(pk):
    with pytest.raises(ValueError, match="exclude"):
        _plan(pk, [100], 4, scored=True)
    with pytest.raises(pk.PkvError, match="49152 pages"):
        _plan(pk, [8 * 49152 + 1], 4, ps=8)
    assert _plan(pk, [8 * 49152], 4, ps=8).info()["kv_tokens"] == 32
    # (a request without a new token is not selected from)
    assert _plan(pk, [8 * 49152 + 1, 9], 4, ps=8, q_lens=[0, 1]).info()["kv_tokens"] == 9


@pytest.mark.parametrize("n", [2 ** 32 + 5, -2 ** 33])
def test_plan_refuses_counts_beyond_32_bits(pk, n):
    with pytest.raises(ValueError, match="32 bits"):
        _plan(pk, [100], n)


def test_replanning_forgets_the_selection(pk):
    p = _plan(pk, [100], 4)
    assert p.num_blocks == 4
    p.plan([0, 1], [0, 7], np.arange(7), [4], num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, mode="decode", num_sms=152,
           host_only=True)
    assert p.num_blocks == 0 and p.info()["kv_tokens"] == 100


# ---- refusals before anything runs (host tensors: nothing may be launched) ----
def _cache(pk, P=8, ps=16, H=2, D=128):
    k = torch.zeros((P, ps, H, D), dtype=torch.bfloat16)
    return pk.KVCache(k, k.clone())


def test_rope_store_refusals(pk):
    cache, rot = _cache(pk), pk.Rotary(128, device="cpu")
    q, k = torch.zeros((3, 8, 128), dtype=torch.bfloat16), torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int64)
    good = dict(q=q, k=k, v=k, positions=i, slot_mapping=i, cache=cache, rotary=rot)
    bad = [dict(q=q[:2]), dict(q=q.float()), dict(q=q[..., :64]), dict(q=q[0]), dict(k=k[:, :1]), dict(v=k[:2]), dict(v=k.float()),
           dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(positions=i.int()), dict(positions=i[:2]),
           dict(slot_mapping=torch.zeros((3, 1), dtype=torch.int64)), dict(slot_mapping=torch.zeros(6, dtype=torch.int64)[::2]),
           dict(rotary=pk.Rotary(64, device="cpu")), dict(q_out=q.float()), dict(q_out=q[:2]), dict(k_out=q),
           dict(k_out=torch.zeros((3, 2, 256), dtype=torch.bfloat16)[..., :128])]
    for kw in bad:
        with pytest.raises(ValueError):
            pk.rope_store(**{**good, **kw})
    with pytest.raises(ValueError, match="current CUDA device|CUDA"):
        pk.rope_store(**good)


def _rope_args(pk, **kw):
    x = torch.zeros(4096, dtype=torch.int64)
    p = (x.data_ptr() + 15) // 16 * 16
    a = dict(q=p, k=p, v=p, q_out=p, k_out=None, positions=p, slot_mapping=p, phase_step=p, scores=None, num_tokens=2,
             q_stride_token=1024, q_stride_head=128, k_stride_token=256, k_stride_head=128, v_stride_token=256, v_stride_head=128,
             num_qo_heads=8, rotary_dim=128, interleaved=0, amplitude=1.0)
    a.update(kw)
    return x, pk._lib.pkv_rope_args(**a)


@pytest.mark.parametrize("kw, status", [
    (dict(num_tokens=-1), -1), (dict(num_tokens=2 ** 31), -2), (dict(num_qo_heads=0), -1), (dict(num_qo_heads=65537), -1),
    (dict(rotary_dim=0), -2), (dict(rotary_dim=24), -2), (dict(rotary_dim=144), -2), (dict(interleaved=2), -1),
    (dict(amplitude=float("inf")), -1), (dict(q_stride_token=1028), -1), (dict(k_stride_head=-128), -1), (dict(v_stride_head=4), -1),
    (dict(q=None), -1), (dict(q_out=None), -1), (dict(positions=None), -1), (dict(phase_step=None), -1), (dict(q=8), -1),
    (dict(k_out=24), -1), (dict(positions=4), -1), (dict(scores=2), -1)])
def test_rope_store_abi_refusals(pk, kw, status):
    keep, a = _rope_args(pk, **kw)
    assert pk._lib.lib().pkv_rope_kv_store(C.byref(a), C.byref(_cache(pk).struct), None) == status


def test_rope_store_abi_accepts_no_tokens_and_refuses_null(pk):
    L = pk._lib.lib()
    keep, a = _rope_args(pk, num_tokens=0, q=None)
    assert L.pkv_rope_kv_store(C.byref(a), C.byref(_cache(pk).struct), None) == 0
    assert L.pkv_rope_kv_store(C.byref(a), None, None) == -1
    assert L.pkv_rope_kv_store(None, C.byref(_cache(pk).struct), None) == -1


def test_key_bounds_refusals(pk):
    codes, scale = torch.zeros((8, 2, 2, 128), dtype=torch.int8), torch.ones((2, 128))
    for c, s in ((codes.float(), scale), (codes[:, :, :1], scale), (codes[..., :64], scale), (codes, scale.double()), (codes, scale[:1]),
                 (codes, torch.ones((128, 2)).t()), (codes[0], scale)):
        with pytest.raises(ValueError):
            pk.KeyBounds(c, s)
    b = pk.KeyBounds.of(_cache(pk), 0.03)
    assert b.codes.shape == (8, 2, 2, 128) and b.scale.shape == (2, 128) and b.scale.is_contiguous() and not b.codes.any()
    assert torch.equal(pk.KeyBounds.of(_cache(pk), torch.arange(2.0)[:, None]).scale[1], torch.ones(128))


def test_calls_on_host_plans_and_mismatched_bounds_are_refused(pk):
    L, p, cache = pk._lib.lib(), _plan(pk, [100, 50], 4), _cache(pk, P=11)
    b = pk.KeyBounds.of(cache, 0.03)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    i32 = torch.zeros((2, 2, 4), dtype=torch.int32)
    assert L.pkv_token_map(p._h, None, i32.data_ptr(), i32.data_ptr(), None) == -1
    assert L.pkv_key_bounds_update(p._h, C.byref(cache.struct), b.codes.data_ptr(), b.scale.data_ptr(), 0, None) == -1
    assert L.pkv_block_select(p._h, q.data_ptr(), b.codes.data_ptr(), b.scale.data_ptr(), 11, 1, 1, i32.data_ptr(), None) == -1
    assert L.pkv_attn_decode_run_blocks(p._h, q.data_ptr(), C.byref(cache.struct), i32.data_ptr(), q.data_ptr(), None, None) == -1
    for f, a in ((L.pkv_token_map, (None, None, None)), (L.pkv_key_bounds_update, (C.byref(cache.struct), None, None, 0)),
                 (L.pkv_block_select, (None, None, None, 0, 0, 1, None)),
                 (L.pkv_attn_decode_run_blocks, (None, C.byref(cache.struct), None, None, None))):
        assert f(None, *a, None) == -1
    with pytest.raises(ValueError, match="workspace"):
        p.token_map()
    with pytest.raises(ValueError, match="geometry"):
        p.bound_keys(_cache(pk, P=12), b)
    with pytest.raises(ValueError, match="geometry"):
        p.bound_keys(_cache(pk, P=11, H=1), b)
    with pytest.raises(ValueError, match="CUDA device"):
        p.bound_keys(cache, b)
    with pytest.raises(ValueError, match="num_blocks"):
        _plan(pk, [100, 50], 0).select(q, b)
    with pytest.raises(ValueError, match="num_blocks"):
        _plan(pk, [100, 50], 0).run(q, cache, blocks=i32)
    with pytest.raises(ValueError, match="blocks"):
        p.run(q, cache, blocks=i32.long())
    with pytest.raises(ValueError, match="blocks"):
        p.run(q, cache, blocks=i32[..., :3])
    with pytest.raises(ValueError, match="q must"):
        p.select(q[:1], b)
    with pytest.raises(ValueError, match="heads"):
        p.select(q, pk.KeyBounds.of(_cache(pk, H=1), 1.0))
    with pytest.raises(ValueError, match="CUDA device"):
        p.select(q, b)


# ---- the compiled calls ----
def test_compiled_calls_refuse_other_kinds_and_keep_no_reference(pk):
    p, cache = _plan(pk, [100, 50], 4), _cache(pk, P=11)
    b, q = pk.KeyBounds.of(cache, 0.03), torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    i32 = torch.zeros((2, 2, 4), dtype=torch.int32)
    refused = [lambda: p.select([1], b), lambda: p.select(None, b),
               lambda: p.select(q, b, num_sink=1.5), lambda: p.select(q, b, num_recent="1"), lambda: p.run("q", cache, blocks=i32),
               lambda: p.run(q, cache, blocks=i32, out=3), lambda: pk._lib.binding().select(1, 2),
               lambda: pk._lib.binding().select(*[None] * 13), lambda: pk._lib.binding().attach()]
    held = [q, i32, b.codes, b.scale, p, p._streams, p._blocks_shape, p._blocks_shape[2]]
    before = [sys.getrefcount(x) for x in held]
    for _ in range(50):
        for f in refused:
            with pytest.raises(TypeError):
                f()
        for f in (lambda: p.select(q, b), lambda: p.run(q, cache, blocks=i32), lambda: p.run(q, cache, blocks=i32, out=q),
                  lambda: p.select(q, b, blocks=i32), lambda: p.select(q, b, num_sink=2 ** 31), lambda: p.select(q, b, num_recent=-2 ** 40)):
            with pytest.raises(ValueError):
                f()
    assert [sys.getrefcount(x) for x in held] == before


def test_a_missing_binding_fails_loudly(pk, monkeypatch):
    pk._lib.binding()
    monkeypatch.setattr(pk._lib, "_binding", None)
    monkeypatch.delattr(pk, "_binding")
    monkeypatch.setitem(sys.modules, pk.__name__ + "._binding", None)
    with pytest.raises(RuntimeError, match="_binding.so"):
        pk._lib.binding()
