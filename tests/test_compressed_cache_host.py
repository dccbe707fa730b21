"""The compressed cache on the host (no GPU): the oracle's NVFP4 codec and eviction pinned to closed forms,
and every refusal of the entry points that write, read, score and evict it."""

import ctypes as C

import numpy as np
import pytest
import torch

from oracle import eviction as OE
from oracle import fp8 as OF
from oracle import nvfp4 as O4


@pytest.fixture(scope="module")
def pk():
    from paged_kv_attention_slot_gb300 import build as B

    B.build()
    import paged_kv_attention_slot_gb300 as pk

    pk._lib.lib()
    return pk


# ---- oracle: the codec ----
def test_e2m1_codes_round_to_nearest_and_halfway_to_even():
    codes = np.arange(16, dtype=np.uint8)
    v = O4.decode_e2m1(codes)
    assert v.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert np.array_equal(O4.encode_e2m1(v), codes)  # the sign of zero included
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert O4.decode_e2m1(O4.encode_e2m1(ties)).tolist() == [0, 1, 1, 2, 2, 4, 4]
    eps = 1e-9
    assert O4.decode_e2m1(O4.encode_e2m1(ties + eps)).tolist() == [.5, 1, 1.5, 2, 3, 4, 6]
    assert O4.decode_e2m1(O4.encode_e2m1(ties - eps)).tolist() == [0, .5, 1, 1.5, 2, 3, 4]
    assert O4.decode_e2m1(O4.encode_e2m1([7.0, np.inf, -np.inf])).tolist() == [6, 6, -6]


def test_pack_and_unpack_are_inverse():
    c = np.random.RandomState(0).randint(0, 16, (3, 32)).astype(np.uint8)
    p = O4.pack(c)
    assert p.shape == (3, 16) and int(p[0, 0]) == int(c[0, 0]) + 16 * int(c[0, 1])
    assert np.array_equal(O4.unpack(p), c)


def test_quantize_of_representable_rows_is_exact():
    # values code * scale with a block maximum of 6 * s come back bit for bit
    r = np.random.RandomState(1)
    s = np.exp2(r.randint(-6, 8, (5, 8)).astype(np.float64))
    codes = r.randint(0, 16, (5, 8, 16)).astype(np.uint8)
    codes[..., 3] = 7
    x = (O4.decode_e2m1(codes) * s[..., None]).reshape(5, 128)
    q, sf = O4.quantize(x.astype(np.float32), 1.0)
    assert np.array_equal(OF.decode(sf), s)
    assert np.array_equal(O4.dequantize(q, sf, 1.0), x)


def test_quantize_error_is_bounded_by_the_formats():
    # |x - value|: half of the coarsest E2M1 step (1) times the block scale, plus what an E4M3 scale
    # rounded down (2^-4 relative) cuts off the block maximum
    x = np.random.RandomState(2).randn(64, 128).astype(np.float32)
    q, sf = O4.quantize(x, 1.0)
    err = np.abs(O4.dequantize(q, sf, 1.0) - x).reshape(64, 8, 16).max(-1)
    s = OF.decode(sf)
    assert np.all(err <= s * (1.0 + 6.0 * 2.0 ** -4))


def test_quantize_special_blocks():
    x = np.zeros((1, 128), np.float32)
    x[0, 16] = np.nan
    x[0, 32] = np.inf
    x[0, 48] = 1e-30
    x[0, 64] = 1e30
    q, sf = O4.quantize(x, 1.0)
    v = O4.dequantize(q, sf, 1.0)
    assert np.all(v[0, :16] == 0) and np.all(np.isnan(v[0, 16:32]))
    assert v[0, 32] == 2688.0 and np.all(v[0, 33:48] == 0)
    assert v[0, 48] == 0.0 and v[0, 64] == 2688.0


# ---- oracle: weights and eviction ----
def test_weights_sum_to_the_query_heads():
    r = np.random.RandomState(3)
    w = OE.key_weights(r.randn(8, 64), r.randn(50, 2, 64), 10, 49, 0.125, 4)
    assert np.all(w[:10] == 0) and np.allclose(w.sum(0), 4.0, atol=1e-12)


def test_uniform_scores_give_equal_weights():
    w = OE.key_weights(np.zeros((4, 64)), np.random.RandomState(4).randn(20, 1, 64), 0, 19, 0.125, 4)
    assert np.allclose(w, 4.0 / 20)


def test_kept_positions_worked_example():
    # 10 keys, keep 6: first 1, last 2, the 3 largest of positions 1..7
    s = [0.0, 5.0, 1.0, 7.0, 2.0, 9.0, 3.0, 0.0, 8.0, 8.0]
    # survivors 1, 3, 5; the front is 0..3: 1 and 3 stay, the hole at 2 takes 5; 8 and 9 follow
    assert OE.kept_positions(s, 6, 1, 2) == [0, 1, 5, 3, 8, 9]
    assert OE.kept_positions(s, 10, 1, 2) == list(range(10))
    assert OE.kept_positions(s, 3, 1, 2) == [0, 8, 9]
    assert OE.kept_positions([1.0] * 6, 3, 0, 0) == [0, 1, 2]  # ties: the lower position
    assert OE.kept_positions([np.nan, -np.inf, 0.0, -1.0], 3, 0, 0) == [3, 1, 2]  # a NaN ranks last


def test_evict_keeps_the_same_set_and_moves_the_fewest_rows():
    r = np.random.RandomState(5)
    for _ in range(200):
        L = int(r.randint(1, 40))
        b = int(r.randint(1, 40))
        S = int(r.randint(0, b + 1))
        R = int(r.randint(0, b - S + 1))
        s = r.randint(0, 6, L).astype(float)
        got = OE.kept_positions(s, b, S, R)
        assert len(got) == min(L, b) == len(set(got))
        if L > b:
            assert got[:S] == list(range(S)) and got[b - R:] == list(range(L - R, L))
            body = sorted(set(got) - set(range(S)) - set(range(L - R, L)))
            out = sorted(set(range(S, L - R)) - set(body))
            if body and out:
                assert min(s[body]) >= max(s[out])
            assert all(p == j or p >= b - R for j, p in enumerate(got))


# ---- refusals: the cache ----
def _fp4(pk, P=4, ps=16, H=2, D=128, **kw):
    c = torch.zeros((P, ps, H, D // 2), dtype=torch.uint8)
    f = torch.zeros((P, ps, H, D // 16), dtype=torch.uint8)
    return pk.KVCache(c, c.clone(), 0.5, 0.5, k_sf=f, v_sf=f.clone(), **kw)


def test_nvfp4_cache_geometry(pk):
    c = _fp4(pk)
    assert c.head_dim == 128 and c.dtype == pk._lib.PKV_NVFP4 and c.struct.head_dim == 128
    d = pk.KVCache.nvfp4(3, 16, 2, 128, 0.25, 0.5, device="cpu")
    assert d.k.shape == (3, 16, 2, 64) and d.k.stride() == (2048, 64, 1024, 1) and d.k_sf.stride() == (256, 8, 128, 1)


def test_nvfp4_cache_rejects_malformed_pools(pk):
    c = torch.zeros((4, 16, 2, 64), dtype=torch.uint8)
    f = torch.zeros((4, 16, 2, 8), dtype=torch.uint8)
    bad = [
        dict(k=c, v=c, k_sf=f),                                              # one scale pool missing
        dict(k=c, v=c, k_sf=f, v_sf=f[:3]),                                  # shapes differ
        dict(k=c, v=c, k_sf=f[..., :4], v_sf=f[..., :4]),                    # 4 scales for 128 elements
        dict(k=c, v=c, k_sf=f.float(), v_sf=f.float()),                      # scale type
        dict(k=c, v=c, k_sf=f, v_sf=f.permute(0, 1, 2, 3).transpose(1, 2).contiguous().transpose(1, 2)),  # strides differ
        dict(k=c.to(torch.bfloat16), v=c.to(torch.bfloat16), k_sf=f, v_sf=f),  # code type
        dict(k=c, v=c[..., ::2], k_sf=f, v_sf=f),                            # pools differ
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            pk.KVCache(**kw)
    with pytest.raises(ValueError):
        pk.KVCache.nvfp4(3, 16, 2, 100, device="cpu")


def _store_status(pk, cache, **over):
    """pkv_kv_store's status for host arguments it must refuse (nothing is launched)."""
    st = pk._lib.pkv_cache.from_buffer_copy(cache.struct)
    for k, v in over.items():
        setattr(st, k, v)
    x = torch.zeros((1, 2, 128), dtype=torch.bfloat16)
    s = torch.zeros(1, dtype=torch.int64)
    a = pk._lib.lib().pkv_kv_store(x.data_ptr(), x.data_ptr(), s.data_ptr(), 1, C.byref(st), None)
    b = pk._lib.lib().pkv_kv_load(s.data_ptr(), 1, C.byref(st), x.data_ptr(), x.data_ptr(), None)
    assert a == b
    return a, pk._lib.lib().pkv_last_error().decode()


@pytest.mark.parametrize("over, word", [
    (dict(k_scale=0.0), "scales"), (dict(v_scale=float("nan")), "scales"), (dict(k_scale=float("inf")), "scales"),
    (dict(k_scale=1e-40), "reciprocal"), (dict(k_sf=None), "k_sf"), (dict(v_sf=None), "v_sf"),
    (dict(sf_stride_page=-8), "positive"), (dict(sf_stride_token=0), "positive"), (dict(sf_stride_head=12), "multiples of 8"),
    (dict(head_dim=64), "head_dim"), (dict(dtype=3), "dtype"), (dict(stride_token=36), "strides"),
])
def test_store_and_load_refuse_bad_nvfp4_pools(pk, over, word):
    st, msg = _store_status(pk, _fp4(pk), **over)
    assert st in (pk._lib.PKV_EINVAL, pk._lib.PKV_EUNSUPPORTED) and word in msg, msg


def test_store_and_load_refuse_misaligned_pointers(pk):
    c = _fp4(pk)
    assert _store_status(pk, c, k_sf=c.k_sf.data_ptr() + 4)[0] == pk._lib.PKV_EINVAL
    assert _store_status(pk, c, k=c.k.data_ptr() + 4)[0] == pk._lib.PKV_EINVAL
    L = pk._lib.lib()
    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    s = torch.zeros(1, dtype=torch.int64)
    ref = C.byref(c.struct)
    assert L.pkv_kv_load(s.data_ptr(), 1, ref, x.data_ptr() + 2, x.data_ptr(), None) == pk._lib.PKV_EINVAL
    assert L.pkv_kv_load(None, 1, ref, x.data_ptr(), x.data_ptr(), None) == pk._lib.PKV_EINVAL
    assert L.pkv_kv_load(s.data_ptr(), -1, ref, x.data_ptr(), x.data_ptr(), None) == pk._lib.PKV_EINVAL
    assert L.pkv_kv_load(None, 0, ref, None, None, None) == pk._lib.PKV_OK
    assert L.pkv_kv_store_scored(x.data_ptr(), x.data_ptr(), s.data_ptr(), 1, ref, s.data_ptr() + 2, None) == pk._lib.PKV_EINVAL


def test_binding_refuses_bad_store_load_and_score_arguments(pk):
    c = _fp4(pk)
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int64)
    good = torch.zeros((4, 2, 16))
    for scores in (good.double(), good.transpose(1, 2), good[:3], good.transpose(0, 2).contiguous(), good):
        with pytest.raises(ValueError):  # the last one is well formed but not on a CUDA device
            pk.kv_store(x, x, s, c, scores=scores)
    with pytest.raises(ValueError):
        pk.kv_store(x, x, s, c)  # an NVFP4 pool on the host
    for slots, kw in ((s.int(), {}), (s.view(3, 1), {}), (torch.zeros(6, dtype=torch.int64)[::2], {}),
                      (s, dict(k=x.float())), (s, dict(v=x[:2])), (s, dict(k=x.transpose(0, 1))), (s, {})):
        with pytest.raises(ValueError):
            pk.kv_load(slots, c, **kw)


# ---- refusals: plans, scored runs, eviction ----
def _plan(pk, idx=(0, 1, 2, 3), indptr=(0, 2, 4), qo=(0, 1, 2), last=(5, 16), **kw):
    a = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_sms=152, host_only=True)
    a.update(kw)
    return pk.Plan().plan(qo, indptr, idx, last, **a)


def test_nvfp4_plans_are_decode_only_and_need_head_dim_128(pk):
    assert _plan(pk, kv_dtype="nvfp4").info()["num_work"] > 0
    with pytest.raises(pk.PkvError, match="head_dim 128"):
        _plan(pk, kv_dtype="nvfp4", head_dim=64)
    for mode in ("prefill", "ragged", "paged_ragged"):
        with pytest.raises(pk.PkvError, match="bf16"):
            _plan(pk, kv_dtype="nvfp4", mode=mode)
    with pytest.raises(pk.PkvError, match="bf16"):
        _plan(pk, kv_dtype="nvfp4", mode="mixed", qo=(0, 1, 3))
    assert _plan(pk, kv_dtype="nvfp4", mode="mixed").info()["num_decodes"] == 2


def test_nvfp4_plans_split_like_the_other_types(pk):
    # the partition covers every key of every KV head once, whatever the pool's type
    kw = dict(idx=np.arange(400, dtype=np.int32), indptr=(0, 300, 400), last=(3, 16))
    p = _plan(pk, kv_dtype="nvfp4", **kw)
    w = p.work_items()
    spans = {(r[0], r[1], r[3], r[4]) for r in w.tolist()}
    assert spans == {(i, h, 0, L) for i, L in ((0, 299 * 16 + 3), (1, 1600)) for h in (0, 1)}


@pytest.mark.parametrize("idx", [(0, 1, 2, 0), (5, 5, 2, 3), (100000, 1, 2, 100000)])
def test_scored_plans_refuse_a_page_listed_twice(pk, idx):
    _plan(pk, idx=idx)  # fine without scores
    with pytest.raises(pk.PkvError, match="listed twice"):
        _plan(pk, idx=idx, scored=True)


def test_scored_plans_need_decode_rows(pk):
    assert _plan(pk, scored=True).scored and _plan(pk, mode="mixed", scored=True).scored
    assert _plan(pk, idx=(7, 100000, 2, 3), scored=True).scored
    with pytest.raises(pk.PkvError, match="DECODE"):
        _plan(pk, mode="prefill", scored=True)
    n = C.c_size_t(0)
    assert pk._lib.lib().pkv_attn_scored_scratch_size(None, C.byref(n)) == pk._lib.PKV_EINVAL
    assert pk._lib.lib().pkv_attn_scored_scratch_size(_plan(pk)._h, None) == pk._lib.PKV_EINVAL
    assert pk._lib.lib().pkv_attn_scored_scratch_size(_plan(pk)._h, C.byref(n)) == pk._lib.PKV_OK
    assert n.value == 4 * 16 * 8 * 4 + 2 * 8 * 4


def test_scored_scratch_check_follows_a_replan(pk):
    p = _plan(pk, scored=True)
    with pytest.raises(pk.PkvError, match="listed twice"):
        p.plan((0, 1, 2), (0, 2, 4), (0, 1, 2, 1), (5, 16), num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
               num_sms=152, host_only=True, scored=True)
    assert not p.scored


def test_scored_run_and_evict_refuse_host_only_plans_and_null_arguments(pk):
    L, p, c = pk._lib.lib(), _plan(pk), _fp4(pk)
    ref = C.byref(c.struct)
    assert L.pkv_attn_decode_run_scored(p._h, None, ref, None, None, None, None, 0, None) == pk._lib.PKV_EINVAL
    assert "host-only" in L.pkv_last_error().decode()
    assert L.pkv_attn_decode_run_scored(None, None, ref, None, None, None, None, 0, None) == pk._lib.PKV_EINVAL
    assert L.pkv_kv_evict(None, ref, None, 4, 0, 0, None, None) == pk._lib.PKV_EINVAL
    assert L.pkv_kv_evict(p._h, ref, None, 4, 0, 0, None, None) == pk._lib.PKV_EINVAL
    assert "host-only" in L.pkv_last_error().decode()


def test_binding_refuses_bad_scored_runs_and_evictions(pk):
    c = _fp4(pk)
    s = torch.zeros((4, 2, 16))
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="scored=True"):
        _plan(pk).run(q, c, scores=s)
    with pytest.raises(ValueError, match="scored=True"):
        _plan(pk, mode="prefill").run(q, c, out=q, lse=s, merge_into=True, scores=s)
    with pytest.raises(ValueError):
        _plan(pk, scored=True).run(q, c, scores=s.double())
    with pytest.raises(ValueError):
        _plan(pk).evict(c, s[:2], 4)
    with pytest.raises(ValueError):
        _plan(pk).evict(c, s, 4)  # scores on the host


def test_binding_refuses_nvfp4_runs_off_the_device_and_outputs_of_another_shape(pk):
    c, p = _fp4(pk), _plan(pk, kv_dtype="nvfp4")
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    lse = torch.zeros((2, 8))
    for out in (q[:1], q.float(), q.transpose(0, 1), q.view(2, 1024)):
        with pytest.raises(ValueError, match="out must be"):
            p.run(q, c, out=out)
    for bad in (lse[:1], lse.double(), lse[:, :4], torch.zeros((8, 2)).t()):
        with pytest.raises(ValueError, match="lse must be"):
            p.run(q, c, out=q.clone(), lse=bad)
    with pytest.raises(ValueError, match="current CUDA device"):
        p.run(q, c)  # a cache and a q on the host
