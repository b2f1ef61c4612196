"""Refusals of dcpa_latent_attn, which makes the checks of the expansion and of the attention over it before it enqueues
either (no GPU; only rejected and empty calls are made)."""
import pytest

from lse_weighted_merge_dcp_amd import attn
from test_attn_host import ALIGN, ATTN, BASE, DTYPE, HEADS, NULL, OK, SHAPE, STRIDE, VALUE, WORKSPACE, pack
from test_latent_host import A, EXPAND, packed

ROWS = dict(ATTN, B=2, q_T=768, q_H=192, Hq=4, k=0, v=0, block_table=0, kv_len=0, o_T=512, o_H=128, l_T=4, Hkv=0, Dk=0,
            num_pages=0, page_size=0, max_pages=0, cache_dtype=0, k_scale=0.0, v_scale=0.0)


def both(e, a):
    return packed(attn.EXPAND_ARGS, "dcpa_expand_args", dict(EXPAND, **e)), pack(attn.ATTN_ARGS, "dcpa_attn_args", dict(ROWS, **a))


def call(e={}, **a):
    return attn.lib().dcpa_latent_attn(*both(e, a), None)


def size(e={}, **a):
    return attn.lib().dcpa_latent_attn_workspace(*both(e, a))


ROUNDED = dict(k_rest=0, v_rest=0)


@pytest.mark.parametrize("parts", [True, False])
@pytest.mark.parametrize("e,want", [
    (dict(dtype=0), DTYPE), (dict(cache_dtype=1), DTYPE), (dict(dtype=1, cache_dtype=1), DTYPE), (dict(B=3), SHAPE), (dict(H=0), SHAPE),
    (dict(Dn=520), SHAPE), (dict(Dn=256), SHAPE), (dict(Dv=264), SHAPE), (dict(Dc=12), SHAPE), (dict(max_keys=-1), SHAPE), (dict(k_scale=0.0), VALUE),
    (dict(k_scale=float("nan")), VALUE), (dict(c_P=-8), STRIDE), (dict(k_B=49160), STRIDE), (dict(v_B=32760), STRIDE),
    (dict(H=3), HEADS)])
def test_shapes_are_refused_by_the_call_and_the_size_query(e, want, parts):
    e = dict(e, **({} if parts else ROUNDED))
    assert call(e) == want and size(e) == want


@pytest.mark.parametrize("parts", [True, False])
@pytest.mark.parametrize("a,want", [
    (dict(lse_base=2), BASE), (dict(T=-1), SHAPE), (dict(Hq=6), HEADS), (dict(N=0), SHAPE), (dict(rank=2), SHAPE),
    (dict(scale=0.0), VALUE), (dict(scale=float("inf")), VALUE), (dict(q_T=-8), STRIDE), (dict(o_H=-2), STRIDE)])
def test_the_attention_s_own_fields(a, want, parts):
    e = {} if parts else ROUNDED
    assert call(e, **a) == want and size(e, **a) == want


@pytest.mark.parametrize("parts", [True, False])
def test_pointers_alignment_and_workspace(parts):
    e = {} if parts else ROUNDED
    need = size(e)
    assert need > 0 and size(dict(e, k=0, v=0, cache=0, w_k=0, places=0), q=0, out=0) == need
    for key in ("cache", "block_table", "kv_len", "w_k", "w_v", "k", "v", "places"):
        assert call(dict(e, **{key: 0})) == NULL
    for key in ("q", "cu_q", "seq_len", "out"):
        assert call(e, **{key: 0}) == NULL
    assert call(e, workspace=0) == WORKSPACE and call(e, workspace_bytes=need - 1) == WORKSPACE and call(e, workspace=A + 8) == WORKSPACE
    assert call(e, q=A + 8) == ALIGN and call(e, out=A + 2) == ALIGN and call(e, o_T=511) == ALIGN and call(dict(e, k=A + 8)) == ALIGN
    assert call(dict(e, places=A + 2)) == ALIGN and call(dict(e, c_S=580)) == ALIGN
    if parts:
        assert call(dict(k_rest=0)) == NULL and call(dict(v_rest=0)) == NULL
        assert call(dict(kr_B=32760)) == STRIDE and call(dict(vr_B=32760)) == STRIDE and call(dict(v_rest=A + 8)) == ALIGN


def test_nothing_to_do():
    assert attn.lib().dcpa_latent_attn(None, both({}, {})[1], None) == NULL
    assert attn.lib().dcpa_latent_attn(both({}, {})[0], None, None) == NULL
    assert attn.lib().dcpa_latent_attn_workspace(None, None) == NULL
    none = dict(k=0, v=0, k_rest=0, v_rest=0, places=0, kv_len=0)
    assert call(dict(none, B=0), B=0) == OK and size(dict(none, B=0), B=0) == 0
    assert call(dict(none, max_keys=0), T=0) == OK and size(dict(none, max_keys=0), T=0) == 0
    # (no keys and more columns in a value than in a key: still a call of its own values)
    assert call(dict(none, max_keys=0, Dn=8, Dr=8, Dv=128), T=0) == OK
