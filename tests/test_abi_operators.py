"""Refusals of the tree attention, path commit, attention-weight and eviction entry points.  No GPU
needed: every call below returns during validation, before the CUDA runtime is touched (the
pointers are never read)."""
import ctypes

import pytest
import torch

from compressed_decode_attention_zkv_b200 import build as B
from compressed_decode_attention_zkv_b200 import zkv

P = 4096   # a non-null, aligned pointer that nothing reads


@pytest.fixture(scope="module")
def L():
    B.build()
    return zkv.lib()


def _fill(p, **kw):
    """Every pointer but the optional ones set, then the given fields."""
    optional = {"mask", "n_draft", "lse", "error_flag", "k_smooth", "block_table", "kept", "block_table_out"}
    for name, ctype in p._fields_:
        if ctype is ctypes.c_void_p and name not in optional:
            setattr(p, name, P)
    for name, v in kw.items():
        setattr(p, name, v)
    return p


def tree(**kw):
    base = dict(B=2, N=4, Hq=8, Hkv=2, d=128, Sk=4, Sv=4, Tcap=64, Wcap=16, max_comp_len=64, q_sb=4096, q_sn=1024,
                q_sh=128, k_sb=1024, k_sn=256, k_sh=128, v_sb=1024, v_sn=256, v_sh=128)
    return _fill(zkv.TreeParams(), **{**base, **kw})


def commit(**kw):
    base = dict(B=2, N=4, M=3, Hkv=2, d=128, Sk=4, Sv=4, Tcap=64, Wcap=16, k_sb=1024, k_sn=256, k_sh=128, v_sb=1024,
                v_sn=256, v_sh=128)
    return _fill(zkv.TreeCommitParams(), **{**base, **kw})


def weights(**kw):
    base = dict(B=2, N=1, Hq=8, Hkv=2, d=128, Sk=4, Tcap=64, max_comp_len=64, q_sb=1024, q_sn=1024, q_sh=128)
    p = _fill(zkv.WeightsParams(), **{**base, **kw})
    if "lse" not in kw:
        p.lse = P
    return p


def evict(**kw):
    base = dict(B=2, Hkv=2, Sk=4, Sv=4, Tcap=64, Tcap_out=32, keep=32, recent=8, k_out=2 * P, v_out=3 * P, acc_out=4 * P)
    return _fill(zkv.EvictParams(), **{**base, **kw})


INVALID, UNSUPPORTED, WORKSPACE = zkv.ZKV_ERR_INVALID_ARG, zkv.ZKV_ERR_UNSUPPORTED, zkv.ZKV_ERR_WORKSPACE
PAGED = dict(block_table=P, page_tokens=32, max_pages=2, n_pages=4)

SHAPES = [   # (change, status) that the tree attention and its size query refuse
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(Hq=7), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(Sk=0), UNSUPPORTED), (dict(Sv=9), UNSUPPORTED), (dict(Hq=18), UNSUPPORTED), (dict(N=257), UNSUPPORTED),
    (dict(B=70000), UNSUPPORTED), (dict(B=65535, Hkv=2, N=256), UNSUPPORTED), (dict(Tcap=60), INVALID),
    (dict(max_comp_len=65), INVALID), (dict(max_comp_len=-1), INVALID), (dict(Wcap=-1), INVALID),
    (dict(Tcap=1 << 29), UNSUPPORTED), ({**PAGED, "page_tokens": 48}, INVALID), ({**PAGED, "max_pages": 3}, INVALID),
    ({**PAGED, "n_pages": 0}, INVALID),
]


@pytest.mark.parametrize("change,status", SHAPES)
def test_tree_shapes(L, change, status):
    p = tree(**change)
    assert L.zkv_rvq_tree_attn(ctypes.byref(p), P, 1 << 40, None) == status
    assert L.zkv_tree_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("change", [dict(q=None), dict(draft_k=None), dict(draft_v=None), dict(out=None), dict(k_codes=None),
                                    dict(v_codebooks=None), dict(win_k=None), dict(win_len=None), dict(q=P + 2),
                                    dict(q_sn=1023), dict(k_sh=-128), dict(v_sb=4), dict(mask=P, m_sb=-1)])
def test_tree_pointers_and_strides(L, change):
    assert L.zkv_rvq_tree_attn(ctypes.byref(tree(**change)), P, 1 << 40, None) == INVALID


def test_null_params(L):
    for f in (L.zkv_rvq_tree_attn, L.zkv_rvq_accumulate_weights):
        assert f(None, P, 1 << 40, None) == INVALID
    for f in (L.zkv_rvq_tree_commit, L.zkv_rvq_evict):
        assert f(None, None) == INVALID
    assert L.zkv_tree_workspace_size(None) == 0 and L.zkv_weights_workspace_size(None) == 0


def test_workspaces(L):
    for p, size, call in ((tree(), L.zkv_tree_workspace_size, L.zkv_rvq_tree_attn),
                          (weights(), L.zkv_weights_workspace_size, L.zkv_rvq_accumulate_weights)):
        need = size(ctypes.byref(p))
        assert need > 0
        assert call(ctypes.byref(p), None, need, None) == WORKSPACE
        assert call(ctypes.byref(p), P, need - 1, None) == WORKSPACE
        assert call(ctypes.byref(p), P + 16, need, None) == WORKSPACE


@pytest.mark.parametrize("change,status", [
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(Wcap=0), INVALID), (dict(d=32), UNSUPPORTED), (dict(Sk=9), UNSUPPORTED),
    (dict(M=257), UNSUPPORTED), (dict(path=None), INVALID), (dict(n_accept=None), INVALID), (dict(win_head=None), INVALID),
    (dict(k_sn=100), INVALID), (dict(draft_v=P + 8), INVALID), ({**PAGED, "page_tokens": 16}, INVALID),
    (dict(B=0), INVALID), (dict(Tcap=-16), INVALID), (dict(Wcap=(1 << 28) + 1), UNSUPPORTED)])
def test_commit(L, change, status):
    assert L.zkv_rvq_tree_commit(ctypes.byref(commit(**change)), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(N=0), INVALID), (dict(Hq=9), INVALID), (dict(d=100), UNSUPPORTED), (dict(Sk=9), UNSUPPORTED), (dict(Hq=18), UNSUPPORTED),
    (dict(N=300), UNSUPPORTED), (dict(B=40000), UNSUPPORTED), (dict(Tcap=40), INVALID), (dict(max_comp_len=80), INVALID),
    (dict(lse=None), INVALID), (dict(acc=None), INVALID), (dict(q_sh=3), INVALID), (dict(k_codes=P + 4), INVALID)])
def test_weights(L, change, status):
    assert L.zkv_rvq_accumulate_weights(ctypes.byref(weights(**change)), P, 1 << 40, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(keep=0), INVALID), (dict(keep=33), INVALID), (dict(recent=33), INVALID), (dict(recent=-1), INVALID), (dict(Sk=0), UNSUPPORTED),
    (dict(Tcap=zkv.EVICT_MAX_TOKENS + 1), UNSUPPORTED), (dict(acc_out=None), INVALID), (dict(len_out=None), INVALID),
    (dict(k_out=P), INVALID),                       # in place with another capacity
    (dict(acc_out=P), INVALID), ({**PAGED, "max_pages": 1}, INVALID),
    (dict(k_out=P, v_out=P, acc_out=P, Tcap_out=64, **PAGED), INVALID),     # in place with another table
    (dict(block_table_out=P, page_tokens_out=32, max_pages_out=2, n_pages_out=1), INVALID), (dict(k_out=2 * P + 1), INVALID)])
def test_evict(L, change, status):
    assert L.zkv_rvq_evict(ctypes.byref(evict(**change)), None) == status


def test_binding_constant():
    from test_abi import _header_define
    assert zkv.EVICT_MAX_TOKENS == _header_define("ZKV_EVICT_MAX_TOKENS")


def test_the_binding_refuses_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        zkv.rvq_tree_attn(z(1, 1, 1, 64).half(), z(1, 1, 1, 64).half(), z(1, 1, 1, 64).half(), z(1, 1, 16, 1).byte(),
                          z(1, 1, 16, 1).byte(), z(1).int(), z(1, 1, 256, 64), z(1, 1, 256, 64), z(1, 1, 1, 64).half(),
                          z(1, 1, 1, 64).half(), z(1).int())
    with pytest.raises(ValueError, match="CUDA"):
        zkv.rvq_evict(z(1, 1, 16, 1).byte(), z(1, 1, 16, 1).byte(), z(1).int(), z(1, 1, 16), 4)
