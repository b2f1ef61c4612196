"""Refusals of the calls around latent and shared caches (dcpa_project, dcpa_latent_expand, dcpa_prefix_attn,
dcpa_pair_attn), by the library and by the binding (no GPU; only rejected and empty calls are made)."""
import re

import pytest
import torch

from lse_weighted_merge_dcp_amd import attn
from test_attn_host import ALIGN, ATTN, COMMON, DTYPE, HEADER, NULL, OK, SHAPE, STRIDE, VALUE, WORKSPACE, pack

A = 0x100000


def names(struct):
    body = re.search(r"typedef struct \{((?:(?!typedef).)*?)\} " + struct, open(HEADER).read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    got = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        got += [n.strip() for n in re.sub(r"^(const )?(void\*|int32_t\*|int64_t|double) ", "", decl).split(",")]
    return got


def packed(layout, struct, values):
    n = names(struct)
    assert sorted(n) == sorted(values)
    return layout.pack(*[values[k] for k in n])


PROJECT = dict(x=A, x_T=768, x_H=192, w=A, w_H=65536, w_N=1, w_K=512, y=A, y_T=2304, y_H=576, T=9, H=4, N=512, K=128, copy=64,
               dtype=2)
EXPAND = dict(cache=A, c_P=9216, c_S=576, block_table=A, t_B=4, kv_len=A, w_k=A, wk_H=131072, wk_N=512, w_v=A, wv_H=131072,
              wv_N=512, k=A, k_B=49152, k_S=768, k_H=192, v=A, v_B=32768, v_S=512, v_H=128, k_rest=A, kr_B=32768, kr_S=512,
              kr_H=128, v_rest=A, vr_B=32768, vr_S=512, vr_H=128, places=A, p_B=64, B=2, H=4, Dn=128, Dr=64, Dv=128, Dc=512,
              max_keys=64, num_pages=9, page_size=16, max_pages=4, dtype=2, cache_dtype=2, k_scale=1.0)


def project(**over):
    return attn.lib().dcpa_project(packed(attn.PROJECT_ARGS, "dcpa_project_args", dict(PROJECT, **over)), None)


def expand(**over):
    return attn.lib().dcpa_latent_expand(packed(attn.EXPAND_ARGS, "dcpa_expand_args", dict(EXPAND, **over)), None)


@pytest.mark.parametrize("over,want", [
    (dict(dtype=0), DTYPE), (dict(dtype=3), DTYPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(T=1 << 29), SHAPE),
    (dict(H=0), SHAPE), (dict(H=(1 << 16) + 1), SHAPE), (dict(N=0), SHAPE), (dict(N=12), SHAPE), (dict(N=1032), SHAPE),
    (dict(K=4), SHAPE), (dict(K=1032), SHAPE), (dict(copy=-8), SHAPE), (dict(copy=4), SHAPE), (dict(copy=1032), SHAPE),
    (dict(w_N=512, w_K=512), STRIDE), (dict(x_T=-8), STRIDE), (dict(y_H=1 << 57), STRIDE), (dict(w_K=-1), STRIDE),
    (dict(x=0), NULL), (dict(w=0), NULL), (dict(y=0), NULL), (dict(x=A + 8), ALIGN), (dict(w=A + 2), ALIGN), (dict(y=A + 4), ALIGN),
    (dict(x_T=764), ALIGN), (dict(w_K=516), ALIGN), (dict(w_N=516, w_K=1), ALIGN), (dict(y_T=2300), ALIGN), (dict(w_H=4), ALIGN),
    (dict(T=0), OK), (dict(T=0, x=0, w=0, y=0), OK)])
def test_project_refuses(over, want):
    assert project(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(dtype=0), DTYPE), (dict(cache_dtype=1), DTYPE), (dict(cache_dtype=0), DTYPE), (dict(B=-1), SHAPE),
    (dict(B=(1 << 20) + 1), SHAPE), (dict(H=0), SHAPE), (dict(H=1 << 17), SHAPE), (dict(Dn=0), SHAPE), (dict(Dn=520), SHAPE),
    (dict(Dn=12), SHAPE), (dict(Dv=0), SHAPE), (dict(Dv=520), SHAPE), (dict(Dr=-8), SHAPE), (dict(Dr=4), SHAPE),
    (dict(Dr=72), SHAPE), (dict(Dc=0), SHAPE), (dict(Dc=516), SHAPE), (dict(Dc=576, Dr=8), SHAPE), (dict(max_keys=-1), SHAPE),
    (dict(max_keys=1 << 30), SHAPE), (dict(max_keys=1 << 29, B=2), SHAPE), (dict(page_size=0), SHAPE),
    (dict(max_pages=1 << 26), SHAPE), (dict(num_pages=-1), SHAPE), (dict(k_scale=0.0), VALUE), (dict(k_scale=-1.0), VALUE),
    (dict(k_scale=float("nan")), VALUE), (dict(k_scale=float("inf")), VALUE), (dict(c_P=-8), STRIDE), (dict(k_B=1 << 57), STRIDE),
    (dict(vr_S=-8), STRIDE), (dict(p_B=-1), STRIDE), (dict(cache=0), NULL), (dict(block_table=0), NULL), (dict(kv_len=0), NULL),
    (dict(w_k=0), NULL), (dict(w_v=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(k_rest=0), NULL), (dict(v_rest=0), NULL),
    (dict(cache=A + 8), ALIGN), (dict(k_rest=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(places=A + 2), ALIGN),
    (dict(wk_N=516), ALIGN), (dict(c_S=580), ALIGN), (dict(kr_H=132), ALIGN), (dict(B=0), OK), (dict(max_keys=0), OK)])
def test_expand_refuses(over, want):
    assert expand(**over) == want


def prefix(cu=A, same=A, groups=2, **over):
    return attn.lib().dcpa_prefix_attn(pack(attn.ATTN_ARGS, "dcpa_attn_args", dict(ATTN, **over)), cu, same, groups, None)


def pairs(k=A, ks=(8192, 512, 128), Dr=128, v=A, vs=(8192, 512, 128), **over):
    return attn.lib().dcpa_pair_attn(pack(attn.ATTN_ARGS, "dcpa_attn_args", dict(ATTN, **over)), k, *ks, Dr, v, *vs, None)


@pytest.mark.parametrize("over,want", COMMON)
def test_both_refuse_what_the_attention_refuses(over, want):
    h, args = attn.lib(), pack(attn.ATTN_ARGS, "dcpa_attn_args", dict(ATTN, **over))
    assert prefix(**over) == want and h.dcpa_prefix_attn_workspace(args, 2) == want
    assert pairs(**over) == want and h.dcpa_pair_attn_workspace(args) == want


def test_prefix_refuses():
    one = dict(B=3, T=8)
    assert prefix(**one, groups=-1) == SHAPE and prefix(**one, groups=(1 << 20) + 1) == SHAPE
    assert prefix(**one, cu=0) == NULL and prefix(**one, same=0) == NULL and prefix(**one, kv_len=0) == NULL
    assert prefix(**one, out=0) == NULL and prefix(**one, cu=A + 2) == ALIGN and prefix(**one, same=A + 1) == ALIGN
    assert prefix(**one, v=A + 8) == ALIGN and prefix(**one, o_T=1023) == ALIGN
    need = attn.lib().dcpa_prefix_attn_workspace(pack(attn.ATTN_ARGS, "dcpa_attn_args", dict(ATTN, **one)), 2)
    assert need > 0
    assert prefix(**one, workspace_bytes=need - 1) == WORKSPACE and prefix(**one, workspace=0) == WORKSPACE
    assert prefix(**one, workspace=A + 8) == WORKSPACE
    assert prefix(B=0, cu=0) == OK and prefix(B=3, T=0, cu=0) == OK
    assert attn.lib().dcpa_prefix_attn(None, A, A, 1, None) == NULL


def test_pairs_refuse():
    one = dict(B=3, T=8)
    assert pairs(**one, cache_dtype=3) == DTYPE
    assert pairs(**one, v=0) == NULL and pairs(**one, k=0) == NULL
    args = dict(ATTN, **one)
    args["v"] = 0
    assert attn.lib().dcpa_pair_attn(pack(attn.ATTN_ARGS, "dcpa_attn_args", args), A, 8192, 512, 128, 128, A, 8192, 512, 128, None) == NULL
    for Dr in (0, 4, 132, 136):
        assert pairs(**one, Dr=Dr) == SHAPE
    assert pairs(**one, ks=(-8, 512, 128)) == STRIDE and pairs(**one, vs=(8192, 1 << 57, 128)) == STRIDE
    assert pairs(**one, ks=(8192, 516, 128)) == ALIGN and pairs(**one, k=A + 8) == ALIGN and pairs(**one, v=A + 2) == ALIGN
    assert pairs(**one, workspace=0) == WORKSPACE and pairs(**one, out=0) == NULL
    assert pairs(B=0) == OK and pairs(T=0) == OK


def test_binding_checks():
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)        # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)           # noqa: E731
    with pytest.raises(ValueError, match="w_uk"):
        attn.latent_queries(b(3, 4, 192), b(5, 128, 512))
    with pytest.raises(ValueError, match="w_uk"):
        attn.latent_queries(b(3, 4, 100), b(4, 128, 512))
    with pytest.raises(ValueError, match="w_uv"):
        attn.latent_values(b(3, 4, 512), b(4, 128, 256))
    with pytest.raises(ValueError, match="device tensors"):
        attn.latent_values(b(3, 4, 512), b(4, 128, 512))
    with pytest.raises(ValueError, match="device tensors"):
        attn.latent_expand(b(9, 16, 1, 576), b(4, 128, 512), b(4, 128, 512), i(2, 4), i(2), 64)
    with pytest.raises(ValueError, match="contiguous"):
        attn.dcp_latent_attn(b(3, 4, 192), b(9, 16, 1, 576), b(4, 128, 512), b(4, 128, 512), i(2, 4), i(3), i(2), 64,
                             k_out=b(2, 64, 4, 200)[..., :192])
    with pytest.raises(ValueError, match="rest"):
        attn.dcp_latent_attn(b(3, 4, 192), b(9, 16, 1, 576), b(4, 128, 512), b(4, 128, 512), i(2, 4), i(3), i(2), 64,
                             rounded=True, k_rest=b(2, 64, 4, 128))
    with pytest.raises(ValueError, match="q \\[T"):
        attn.dcp_latent_attn(b(3, 4, 128), b(9, 16, 1, 576), b(4, 128, 512), b(4, 128, 512), i(2, 4), i(3), i(2), 64)
    with pytest.raises(ValueError, match="device tensors"):
        attn.dcp_prefix_attn(b(3, 4, 64), b(9, 16, 1, 64), b(9, 16, 1, 64), i(2, 4), i(3), i(2), i(2), i(1))


def test_all_tensors_of_the_expanded_form_are_on_one_device(monkeypatch):
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)        # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)           # noqa: E731
    seen = []

    class Seen(Exception):
        pass

    def on_gpu(*ts):
        seen.extend(ts)
        raise Seen

    k, v = b(2, 64, 4, 192), b(2, 64, 4, 128)
    rests, places, cu, kv, seq = (b(2, 64, 4, 128), b(2, 64, 4, 128)), i(2, 64), i(3), i(2), i(2)
    q, work = b(3, 4, 192), torch.zeros(64, dtype=torch.uint8)
    out, lse = b(3, 4, 128), torch.zeros(3, 4)
    monkeypatch.setattr(attn, "latent_expand", lambda *a, **kw: (k, v))     # (which checks its own)
    monkeypatch.setattr(attn, "_on_gpu", on_gpu)
    with pytest.raises(Seen):
        attn.dcp_latent_attn(q, b(9, 16, 1, 576), b(4, 128, 512), b(4, 128, 512), i(2, 4), cu, kv, 64, seq_len=seq, k_out=k,
                             v_out=v, k_rest=rests[0], v_rest=rests[1], places=places, out=out, out_lse=lse, workspace=work)
    at = {t.data_ptr() for t in seen if t is not None}
    for t in (q, k, v, *rests, places, cu, kv, seq, out, lse, work):
        assert t.data_ptr() in at
