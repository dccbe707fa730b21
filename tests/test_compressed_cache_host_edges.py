"""Refusals of the compressed cache's entry points at the edges of their ranges, on the host (no GPU)."""

import ctypes as C

import pytest


@pytest.fixture(scope="module")
def pk():
    from paged_kv_attention_slot_gb300 import build as B

    B.build()
    import paged_kv_attention_slot_gb300 as pk

    pk._lib.lib()
    return pk


def _plan(pk, heads, **kw):
    return pk.Plan().plan([0, 1], [0, 1], [0], [5], num_qo_heads=heads, num_kv_heads=1, head_dim=128, page_size=16, num_sms=152,
                          host_only=True, **kw)


def test_scored_plans_refuse_more_query_heads_than_their_second_kernel_holds(pk):
    # it keeps a float32 log-sum-exp per query head of a KV head in 48 KB; beyond, its launch would fail after
    # the decode had been enqueued
    assert _plan(pk, 12288, scored=True).scored
    p = _plan(pk, 12289)
    with pytest.raises(pk.PkvError, match="12288 query heads") as e:
        _plan(pk, 12289, scored=True)
    assert e.value.status == pk._lib.PKV_EUNSUPPORTED
    n = C.c_size_t(0)
    assert pk._lib.lib().pkv_attn_scored_scratch_size(p._h, C.byref(n)) == pk._lib.PKV_EUNSUPPORTED
