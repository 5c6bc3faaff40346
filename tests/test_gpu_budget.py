"""Attention-weight totals and eviction over the compressed cache against plain float64 / integer
forms, and a serving loop that verifies, commits, adds up weights and evicts."""
import math

import numpy as np
import pytest
import torch

from compressed_decode_attention_zkv_b200 import build as B
from compressed_decode_attention_zkv_b200 import zkv
from oracle import zkv_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.build()
    zkv.lib()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def hadamard(d):
    h = np.ones((1, 1))
    while len(h) < d:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(d)


def paginate(codes, P, perm, n_pages):
    Bn, Hkv, Tcap, S = codes.shape
    pool = np.full((n_pages, Hkv, P, S), 255, np.uint8)
    for b in range(Bn):
        for p in range(Tcap // P):
            pool[perm[b, p]] = codes[b, :, p * P:(p + 1) * P]
    return pool


def weights_case(seed, B, N, Hq, Hkv, d, S, Tcap, comp, ck=0.3):
    rng = np.random.default_rng(seed)
    c = dict(B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, S=S, Tcap=Tcap, lam=None)
    c["q"] = rng.standard_normal((B, N, Hq, d)).astype(np.float16)
    c["kc"] = rng.integers(0, 256, (B, Hkv, Tcap, S)).astype(np.uint8)
    c["Ck"] = (rng.standard_normal((Hkv, S, 256, d)) * ck).astype(np.float32)
    c["comp"] = np.asarray(comp, np.int32)
    c["lse"] = (3 + rng.standard_normal((B, N, Hq))).astype(np.float32)
    c["acc"] = rng.random((B, Hkv, Tcap)).astype(np.float32)
    return c


def weights_plain(c):
    """The totals in float64, and the largest relative error of the float32 form's additions."""
    B, N, Hq, d = c["q"].shape
    G = Hq // c["Hkv"]
    H = hadamard(d)
    acc = c["acc"].astype(np.float64)
    tol = 0.0
    for b in range(B):
        n = int(c["comp"][b])
        for h in range(c["Hkv"]):
            k = sum(c["Ck"][h, s].astype(np.float64)[c["kc"][b, h, :n, s]] for s in range(c["S"])) @ H
            if c["lam"] is not None:
                k = k * c["lam"][h].astype(np.float64)
            for i in range(N):
                for g in range(h * G, (h + 1) * G):
                    l = float(c["lse"][b, i, g])
                    if not math.isfinite(l):
                        continue
                    q = c["q"][b, i, g].astype(np.float64)
                    acc[b, h, :n] += np.exp(k @ q / math.sqrt(d) - l)
                    ql = q if c["lam"] is None else q * c["lam"][h]
                    mag = np.linalg.norm(ql) * sum(np.linalg.norm(c["Ck"][h, s].astype(np.float64), axis=-1).max() for s in range(c["S"]))
                    # products and sums of d terms, butterflies, stages, base change; |lse| to U
                    tol = max(tol, (d + 8 + c["S"] + 8) * U * (mag / math.sqrt(d) + abs(l)))
    return acc, math.expm1(tol) + 2.0 ** -22 + (N * G + 4) * U


def weights_check(c, acc):
    want, rel = weights_plain(c)
    got = acc.cpu().numpy()
    for b in range(c["B"]):
        n = int(c["comp"][b])
        assert np.array_equal(got[b, :, n:], c["acc"][b, :, n:])       # behind the prefix: untouched
        if n:
            assert (np.abs(got[b, :, :n] - want[b, :, :n]) <= rel * want[b, :, :n]).all()


WEIGHTS = {
    "one": dict(B=1, N=1, Hq=1, Hkv=1, d=128, S=4, Tcap=16, comp=[1]),
    "ragged": dict(B=4, N=1, Hq=8, Hkv=2, d=128, S=4, Tcap=9008, comp=[9008, 0, 4097, 513]),
    "groups of 7": dict(B=2, N=1, Hq=14, Hkv=2, d=64, S=2, Tcap=608, comp=[600, 37]),
    "groups of 3, two queries": dict(B=2, N=2, Hq=3, Hkv=1, d=64, S=3, Tcap=160, comp=[160, 1]),
    "five queries": dict(B=1, N=5, Hq=16, Hkv=2, d=256, S=1, Tcap=320, comp=[317]),
    "one stage": dict(B=1, N=1, Hq=3, Hkv=1, d=64, S=1, Tcap=320, comp=[317]),
    "two stages": dict(B=1, N=1, Hq=2, Hkv=1, d=64, S=2, Tcap=320, comp=[317]),
    "eight stages": dict(B=1, N=2, Hq=8, Hkv=1, d=64, S=8, Tcap=320, comp=[317]),
    "eight stages, one head": dict(B=1, N=1, Hq=1, Hkv=1, d=64, S=8, Tcap=320, comp=[317]),
    "six stages": dict(B=1, N=3, Hq=2, Hkv=2, d=128, S=6, Tcap=64, comp=[50]),
}


@pytest.mark.parametrize("name", WEIGHTS)
def test_weights(name):
    c = weights_case(41, **WEIGHTS[name])
    acc = _cuda(c["acc"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    zkv.rvq_accumulate_weights(*[_cuda(c[k]) for k in ("q", "lse", "kc", "comp", "Ck")], acc, error_flag=err)
    weights_check(c, acc)
    assert err.item() == 0


def test_weights_queries_that_count_for_nothing():
    c = weights_case(42, B=2, N=3, Hq=4, Hkv=2, d=64, S=2, Tcap=64, comp=[64, 30])
    c["lse"][0, 1] = np.inf
    c["lse"][1, 0] = -np.inf
    c["lse"][1, 2, 3] = np.nan
    c["q"][0, 1] = np.nan                   # a rejected draft's query may hold anything
    acc = _cuda(c["acc"])
    zkv.rvq_accumulate_weights(*[_cuda(c[k]) for k in ("q", "lse", "kc", "comp", "Ck")], acc)
    weights_check(c, acc)


@pytest.mark.parametrize("P", [32, 128])
def test_weights_pages_views_and_smoothing(P):
    c = weights_case(43, B=2, N=2, Hq=4, Hkv=2, d=128, S=4, Tcap=640, comp=[640, 333])
    c["lam"] = np.exp(np.random.default_rng(2).standard_normal((2, 128)) * 0.2).astype(np.float32)
    lam = _cuda(c["lam"])
    a1 = zkv.rvq_accumulate_weights(*[_cuda(c[k]) for k in ("q", "lse", "kc", "comp", "Ck")], _cuda(c["acc"]), k_smooth=lam)
    weights_check(c, a1)
    mp = 640 // P
    perm = np.random.default_rng(3).permutation(2 * mp + 2)[:2 * mp].reshape(2, mp).astype(np.int32)
    q = torch.zeros(2, 2, 9, 128, dtype=torch.float16, device="cuda")
    q[:, :, 3:7] = _cuda(c["q"])
    a2 = zkv.rvq_accumulate_weights(q[:, :, 3:7], _cuda(c["lse"]), _cuda(paginate(c["kc"], P, perm, 2 * mp + 2)),
                                    _cuda(c["comp"]), _cuda(c["Ck"]), _cuda(c["acc"]), k_smooth=lam,
                                    block_table=_cuda(perm))
    assert torch.equal(a1, a2)


def test_weights_bound_and_errors():
    c = weights_case(44, B=2, N=1, Hq=2, Hkv=1, d=64, S=2, Tcap=64, comp=[64, 0])
    args = [_cuda(c[k]) for k in ("q", "lse", "kc", "comp", "Ck")]
    acc = _cuda(c["acc"])
    zkv.rvq_accumulate_weights(*args, acc, max_comp_len=0)
    assert np.array_equal(acc.cpu().numpy(), c["acc"])
    zkv.rvq_accumulate_weights(*args, acc, max_comp_len=30)
    weights_check({**c, "comp": np.array([30, 0], np.int32)}, acc)
    args[3] = _cuda(np.array([65, -2], np.int32))
    acc = _cuda(c["acc"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    zkv.rvq_accumulate_weights(*args, acc, error_flag=err)
    assert err.item() == zkv.ZKV_DEVERR_COMP_LEN
    weights_check(c, acc)


def test_weights_repeat_and_replay():
    c = weights_case(45, B=2, N=1, Hq=8, Hkv=2, d=128, S=4, Tcap=5008, comp=[5000, 4200])
    args = [_cuda(c[k]) for k in ("q", "lse", "kc", "comp", "Ck")]
    acc, acc2 = _cuda(c["acc"]), _cuda(c["acc"])
    for _ in range(3):
        zkv.rvq_accumulate_weights(*args, acc)
    step = zkv.PreparedAccumulate(*args, acc2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(acc, acc2)


# ---------------------------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------------------------

def evict_case(seed, B, Hkv, Sk, Sv, Tcap, comp, ties=False):
    rng = np.random.default_rng(seed)
    c = dict(kc=rng.integers(0, 256, (B, Hkv, Tcap, Sk)).astype(np.uint8),
             vc=rng.integers(0, 256, (B, Hkv, Tcap, Sv)).astype(np.uint8),
             comp=np.asarray(comp, np.int32))
    acc = rng.integers(0, 4, (B, Hkv, Tcap)).astype(np.float32) if ties else \
        np.exp(3 * rng.standard_normal((B, Hkv, Tcap))).astype(np.float32)
    c["acc"] = acc
    return c


def evict_plain(c, keep, recent, out=None):
    """(k, v, acc, len, kept): copies of `out` (the destination's contents; the source's if None)."""
    kc, vc, acc = c["kc"], c["vc"], c["acc"]
    ko, vo, ao = (x.copy() for x in (out or (kc, vc, acc)))
    B, Hkv, Tcap = acc.shape
    kept = np.full((B, Hkv, keep), -1, np.int32)
    ln = np.zeros(B, np.int32)
    for b in range(B):
        n = min(max(int(c["comp"][b]), 0), Tcap)
        ln[b] = min(n, keep)
        for h in range(Hkv):
            if n <= keep:
                idx = np.arange(n)
            else:
                old = n - recent
                a = acc[b, h, :old].astype(np.float64)
                a = np.where(np.isnan(a), -np.inf, a)
                nan = np.isnan(acc[b, h, :old])
                order = np.lexsort((np.arange(old), nan, -a))     # NaN behind -inf
                idx = np.concatenate([np.sort(order[:keep - recent]), np.arange(old, n)])
            m = len(idx)
            ko[b, h, :m], vo[b, h, :m], ao[b, h, :m] = kc[b, h, idx], vc[b, h, idx], acc[b, h, idx]
            ao[b, h, m:n] = 0
            kept[b, h, :m] = idx
    return ko, vo, ao, ln, kept


def same(got, want):
    for g, w in zip(got, want):
        g = g.cpu().numpy()
        assert g.dtype == w.dtype and np.array_equal(g, w, equal_nan=g.dtype.kind == "f")


EVICT = {
    "one of one": dict(case=dict(B=1, Hkv=1, Sk=2, Sv=2, Tcap=1, comp=[1]), keep=1, recent=0),
    "one of many": dict(case=dict(B=2, Hkv=2, Sk=4, Sv=4, Tcap=100, comp=[100, 2]), keep=1, recent=0),
    "only the newest": dict(case=dict(B=2, Hkv=1, Sk=1, Sv=8, Tcap=333, comp=[333, 40]), keep=40, recent=40),
    "half": dict(case=dict(B=4, Hkv=2, Sk=3, Sv=5, Tcap=960, comp=[960, 0, 500, 501]), keep=500, recent=64),
    "ties": dict(case=dict(B=2, Hkv=2, Sk=4, Sv=2, Tcap=5000, comp=[5000, 4097], ties=True), keep=1234, recent=100),
    "all but one": dict(case=dict(B=1, Hkv=1, Sk=7, Sv=6, Tcap=9000, comp=[8999]), keep=8998, recent=1),
    "a cluster of 8": dict(case=dict(B=1, Hkv=2, Sk=4, Sv=4, Tcap=40000, comp=[39999]), keep=10001, recent=256),
    "few in a large one": dict(case=dict(B=2, Hkv=1, Sk=4, Sv=4, Tcap=40000, comp=[600, 31000]), keep=500, recent=3),
    "the largest": dict(case=dict(B=1, Hkv=1, Sk=1, Sv=6, Tcap=262144, comp=[262143]), keep=100001, recent=500),
    "the largest, ties": dict(case=dict(B=1, Hkv=1, Sk=8, Sv=1, Tcap=262144, comp=[200000], ties=True), keep=150000, recent=0),
    "ties over ctas": dict(case=dict(B=1, Hkv=1, Sk=2, Sv=2, Tcap=30000, comp=[30000], ties=True), keep=20000, recent=7),
}


@pytest.mark.parametrize("where", ["apart", "in place"])
@pytest.mark.parametrize("name", EVICT)
def test_evict(name, where):
    e = EVICT[name]
    c = evict_case(51, **e["case"])
    keep, recent = e["keep"], e["recent"]
    k, v, n, acc = (_cuda(c[x]) for x in ("kc", "vc", "comp", "acc"))
    B_, H_, T_ = c["acc"].shape
    kept = torch.full((B_, H_, keep), 9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if where == "in place":
        zkv.rvq_evict(k, v, n, acc, keep, recent, kept=kept, error_flag=err)
        same((k, v, acc, n, kept), evict_plain(c, keep, recent))
    else:
        cap = keep + 5
        out = [np.full((B_, H_, cap, c["kc"].shape[3]), 3, np.uint8), np.full((B_, H_, cap, c["vc"].shape[3]), 4, np.uint8),
               np.full((B_, H_, cap), 5, np.float32)]
        t = [_cuda(x) for x in out]
        ln = torch.zeros(B_, dtype=torch.int32, device="cuda")
        zkv.rvq_evict(k, v, n, acc, keep, recent, k_out=t[0], v_out=t[1], acc_out=t[2], len_out=ln, kept=kept, error_flag=err)
        want = evict_plain({**c, "comp": np.minimum(c["comp"], T_)}, keep, recent,
                           (out[0], out[1], out[2]))
        want[2][...] = want[2]
        same((t[0], t[1], t[2], ln, kept), want)
        same((k, v, acc, n), (c["kc"], c["vc"], c["acc"], c["comp"]))
    assert err.item() == 0


def test_evict_strange_totals():
    c = evict_case(52, B=1, Hkv=1, Sk=2, Sv=2, Tcap=64, comp=[64])
    a = c["acc"][0, 0]
    a[:] = 1.0
    a[3], a[5], a[7], a[9] = np.inf, -np.inf, np.nan, -1.0
    a[10], a[11], a[12], a[13] = 0.0, -0.0, 1e-45, -np.nan
    a[20:30] = np.nan
    for keep in (1, 40, 47, 50, 51, 52, 53, 54, 60):
        t = [_cuda(c[x]) for x in ("kc", "vc", "comp", "acc")]
        zkv.rvq_evict(*t, keep, 0)
        k, v, acc, n, _ = evict_plain(c, keep, 0)
        same(t, (k, v, n, acc))


def test_evict_errors_and_short_destinations():
    c = evict_case(53, B=3, Hkv=1, Sk=2, Sv=2, Tcap=64, comp=[70, -1, 64])
    t = [_cuda(c[x]) for x in ("kc", "vc", "comp", "acc")]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    zkv.rvq_evict(*t, 30, 10, error_flag=err)
    assert err.item() == zkv.ZKV_DEVERR_COMP_LEN
    k, v, acc, n, _ = evict_plain(c, 30, 10)
    same(t, (k, v, n, acc))


@pytest.mark.parametrize("P,Pout", [(32, 32), (64, 32), (32, 128)])
def test_evict_pages(P, Pout):
    c = evict_case(54, B=2, Hkv=2, Sk=4, Sv=3, Tcap=1280, comp=[1280, 700])
    mp = 1280 // P
    perm = np.random.default_rng(5).permutation(2 * mp + 1)[:2 * mp].reshape(2, mp).astype(np.int32)
    pools = [paginate(c[x], P, perm, 2 * mp + 1) for x in ("kc", "vc")]
    want = evict_plain(c, 300, 20)
    # in place
    t = [_cuda(pools[0]), _cuda(pools[1]), _cuda(c["comp"]), _cuda(c["acc"])]
    zkv.rvq_evict(*t, 300, 20, block_table=_cuda(perm))
    same(t, (paginate(want[0], P, perm, 2 * mp + 1), paginate(want[1], P, perm, 2 * mp + 1), want[3], want[2]))
    # to pages of another size
    mo = 384 // Pout
    po = np.random.default_rng(6).permutation(2 * mo + 1)[:2 * mo].reshape(2, mo).astype(np.int32)
    zero = [np.zeros((2, 2, 384, 4), np.uint8), np.zeros((2, 2, 384, 3), np.uint8), np.zeros((2, 2, 384), np.float32)]
    t = [_cuda(paginate(zero[0], Pout, po, 2 * mo + 1)), _cuda(paginate(zero[1], Pout, po, 2 * mo + 1)), _cuda(zero[2])]
    ln = torch.zeros(2, dtype=torch.int32, device="cuda")
    zkv.rvq_evict(_cuda(pools[0]), _cuda(pools[1]), _cuda(c["comp"]), _cuda(c["acc"]), 300, 20, k_out=t[0], v_out=t[1],
                  acc_out=t[2], len_out=ln, block_table=_cuda(perm), block_table_out=_cuda(po))
    w = evict_plain(c, 300, 20, tuple(zero))
    same((t[0], t[1], t[2], ln), (paginate(w[0], Pout, po, 2 * mo + 1), paginate(w[1], Pout, po, 2 * mo + 1), w[2], w[3]))


def test_evict_bad_pages():
    c = evict_case(55, B=1, Hkv=1, Sk=2, Sv=2, Tcap=128, comp=[128])
    perm = np.arange(4).reshape(1, 4).astype(np.int32)
    pools = [paginate(c[x], 32, perm, 4) for x in ("kc", "vc")]
    bad = perm.copy()
    bad[0, 1] = 99
    out = [torch.full((4, 1, 32, 2), 7, dtype=torch.uint8, device="cuda") for _ in range(2)]
    acc_out, ln = torch.zeros(1, 1, 128, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    zkv.rvq_evict(_cuda(pools[0]), _cuda(pools[1]), _cuda(c["comp"]), _cuda(c["acc"]), 128, 0, k_out=out[0], v_out=out[1],
                  acc_out=acc_out, len_out=ln, block_table=_cuda(bad), block_table_out=_cuda(np.array([[0, -1, 2, 3]], np.int32)),
                  error_flag=err)
    assert err.item() == zkv.ZKV_DEVERR_PAGE
    k = out[0].cpu().numpy()[:, 0]
    assert (k[1] == 7).all() and np.array_equal(k[0], c["kc"][0, 0, :32]) and np.array_equal(k[2:].reshape(64, 2), c["kc"][0, 0, 64:])


def test_evict_codes_in_place_and_totals_apart():
    c = evict_case(57, B=2, Hkv=2, Sk=4, Sv=8, Tcap=5008, comp=[5000, 300])
    k, v, n, acc = (_cuda(c[x]) for x in ("kc", "vc", "comp", "acc"))
    acc_out, ln = torch.full_like(acc, 5), torch.zeros_like(n)
    zkv.rvq_evict(k, v, n, acc, 700, 50, acc_out=acc_out, len_out=ln)
    ko, vo, ao, lo, _ = evict_plain(c, 700, 50, (c["kc"], c["vc"], np.full_like(c["acc"], 5)))
    same((k, v, acc_out, ln, acc, n), (ko, vo, ao, lo, c["acc"], c["comp"]))


def test_budget_binding_refusals():
    c = evict_case(58, B=1, Hkv=1, Sk=2, Sv=2, Tcap=64, comp=[64])
    k, v, n, acc = (_cuda(c[x]) for x in ("kc", "vc", "comp", "acc"))
    for kw in (dict(keep=0), dict(keep=65), dict(keep=4, recent=5)):
        with pytest.raises(zkv.ZkvError):
            zkv.rvq_evict(k, v, n, acc, **kw)
    for kw in (dict(k_out=k), dict(acc_out=acc[:, :, :32]), dict(kept=torch.zeros(1, 1, 3, dtype=torch.int32, device="cuda")),
               dict(k_out=k[:, :, :32].contiguous(), v_out=v[:, :, :32].contiguous()),
               dict(block_table_out=torch.zeros(1, 1, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            zkv.rvq_evict(k, v, n, acc, 4, **kw)
    w = weights_case(59, **WEIGHTS["one"])
    args = [_cuda(w[x]) for x in ("q", "lse", "kc", "comp", "Ck")]
    with pytest.raises(ValueError):
        zkv.rvq_accumulate_weights(*args, torch.zeros(1, 1, 8, device="cuda"))
    with pytest.raises(TypeError):
        zkv.rvq_accumulate_weights(args[0], args[1].double(), *args[2:], _cuda(w["acc"]))


def test_evict_is_replayed():
    c = evict_case(56, B=2, Hkv=2, Sk=4, Sv=4, Tcap=9000, comp=[9000, 5000])
    t = [_cuda(c[x]) for x in ("kc", "vc", "comp", "acc")]
    zkv.rvq_evict(*[x.clone() for x in t], 3000, 100)
    step = zkv.PreparedEvict(*t, 3000, recent=100)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    torch.cuda.synchronize()
    k, v, acc, n, _ = evict_plain(c, 3000, 100)
    same(t, (k, v, n, acc))
    g.replay()                               # nothing is left to evict
    torch.cuda.synchronize()
    same(t, (k, v, n, acc))


# ---------------------------------------------------------------------------------------------
# The operators as a serving loop uses them
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("d,Hq,Hkv,S", [(128, 8, 2, 4), (64, 3, 1, 2)])
def test_serving_loop(d, Hq, Hkv, S):
    """prefill, then rounds of verify, commit, note_weights and evict, each round against float64
    attention over the cache's own contents."""
    rng = np.random.default_rng(61)
    Bn, W, N, M, T = 2, 16, 6, 3, 900
    G = Hq // Hkv
    Ck = (rng.standard_normal((Hkv, S, 256, d)) * 0.4).astype(np.float32)
    Cv = (rng.standard_normal((Hkv, S, 256, d)) * 0.4).astype(np.float32)
    Ck[:, :, 0], Cv[:, :, 0] = 0, 0
    cache = zkv.RVQKVCache(_cuda(Ck), _cuda(Cv), batch=Bn, capacity=1024, window=W)
    new = lambda *s: rng.standard_normal(s).astype(np.float16)   # noqa: E731
    cache.prefill(_cuda(new(Bn, Hkv, T, d)), _cuda(new(Bn, Hkv, T, d)))
    H = hadamard(d)
    with pytest.raises(ValueError):
        cache.evict(10)
    for step in range(4):
        q, dk, dv = new(Bn, N, Hq, d), new(Bn, N, Hkv, d), new(Bn, N, Hkv, d)
        mask = np.tril(rng.random((N, N)) < 0.6) | np.eye(N, dtype=bool)
        comp, win = cache.comp_len.cpu().numpy(), cache.win_len.cpu().numpy()
        kc, vc = cache.k_codes.cpu().numpy(), cache.v_codes.cpu().numpy()
        wk, wv = cache.win_k.cpu().numpy(), cache.win_v.cpu().numpy()
        out, lse = cache.verify(_cuda(q), _cuda(dk), _cuda(dv), mask=_cuda(mask))
        before = np.zeros((Bn, Hkv, cache.Tcap)) if cache.acc is None else cache.acc.double().cpu().numpy()
        cache.note_weights(_cuda(q), lse)
        acc = cache.acc.cpu().numpy()
        o, l = out.cpu().numpy(), lse.cpu().numpy()
        for b in range(Bn):
            n, w = comp[b], win[b]
            for h in range(Hkv):
                k = np.concatenate([sum(Ck[h, s].astype(np.float64)[kc[b, h, :n, s]] for s in range(S)) @ H, wk[b, h, :w], dk[b, :, h]])
                v = np.concatenate([sum(Cv[h, s].astype(np.float64)[vc[b, h, :n, s]] for s in range(S)) @ H, wv[b, h, :w], dv[b, :, h]])
                got = np.zeros(n)
                for g in range(h * G, (h + 1) * G):
                    x = q[b, :, g].astype(np.float64) @ k.T / math.sqrt(d)
                    x[:, n + w:][~mask] = -np.inf
                    ll = np.log(np.exp(x - x.max(1, keepdims=True)).sum(1)) + x.max(1)
                    p = np.exp(x - ll[:, None])
                    # magnitudes below 12 in the scores: (d + 24) U 12 < 1.2e-4, twice for a weight
                    assert np.abs(l[b, :, g] - ll).max() < 1.5e-4
                    assert np.abs(o[b, :, g] - p @ v).max() < 3e-4 * np.abs(v).max() * 2
                    got += p[:, :n].sum(0)
                assert np.abs(acc[b, h, :n] - before[b, h, :n] - got).max() < 3e-4 * (1 + np.abs(acc[b, h]).max())
        path = np.stack([np.sort(rng.permutation(N)[:M]) for _ in range(Bn)]).astype(np.int32)
        n_accept = np.array([M - step % 3, 1 + step % 3], np.int32)
        cache.commit(_cuda(dk), _cuda(dv), _cuda(path), _cuda(n_accept))
        assert np.array_equal(cache.comp_len.cpu().numpy(), comp + n_accept)      # the window is full
        for b in range(Bn):
            head = (cache.win_head[b].item() - n_accept[b]) % W
            for i in range(n_accept[b]):
                slot = (head + i) % W
                assert np.array_equal(cache.win_k[b, :, slot].cpu().numpy(), dk[b, path[b, i]])
                for h in range(Hkv):
                    assert np.array_equal(cache.k_codes[b, h, comp[b] + i].cpu().numpy(), O.rvq_encode(wk[b, h, slot][None], Ck[h])[0][0])
        if step % 2:
            keep = 400 - 100 * (step // 2)
            kept = torch.zeros(Bn, Hkv, keep, dtype=torch.int32, device="cuda")
            c = dict(kc=cache.k_codes.cpu().numpy(), vc=cache.v_codes.cpu().numpy(), comp=cache.comp_len.cpu().numpy(),
                     acc=cache.acc.cpu().numpy())
            cache.evict(keep, recent=32, kept=kept)
            same((cache.k_codes, cache.v_codes, cache.acc, cache.comp_len, kept), evict_plain(c, keep, 32))
            assert cache.max_comp_len == keep
    out, lse = cache.attend(_cuda(new(Bn, Hq, d)))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all() and cache.error_flag.item() == 0


def _filled_cache(rng, W=16, T=700):
    Bn, Hq, Hkv, d, S = 2, 8, 2, 128, 4
    books = [_cuda((rng.standard_normal((Hkv, S, 256, d)) * 0.4).astype(np.float32)) for _ in range(2)]
    cache = zkv.RVQKVCache(*books, batch=Bn, capacity=1024, window=W)
    new = lambda *s: _cuda(rng.standard_normal(s).astype(np.float16))   # noqa: E731
    cache.prefill(new(Bn, Hkv, T, d), new(Bn, Hkv, T, d))
    drafts = lambda N: (new(Bn, N, Hq, d), new(Bn, N, Hkv, d), new(Bn, N, Hkv, d))   # noqa: E731
    return cache, drafts


def test_captured_verify_outlives_a_wider_one():
    """A graph of verify() and attend() keeps its workspaces when later calls need larger ones."""
    cache, drafts = _filled_cache(np.random.default_rng(62))
    few, many = drafts(2), drafts(40)
    q1 = few[0][:, 0].contiguous()
    out, lse = cache.verify(*few)
    first, _ = cache.attend(q1)
    g = torch.cuda.CUDAGraph()
    got, alone = torch.zeros_like(out), torch.zeros_like(first)
    with torch.cuda.graph(g):
        cache.verify(*few, out=got)
        cache.attend(q1, out=alone)
    sizes = [w.numel() for w in cache._tree_ws] + [cache._ws.numel()]
    cache.verify(*many)
    cache.note_weights(many[0], torch.zeros(many[0].shape[:3], device="cuda"))
    # memory that the calls above may have given back, filled
    fill = [torch.full((n,), 165, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out) and torch.equal(alone, first)
    for f in fill:
        assert (f == 165).all()


def test_totals_are_not_made_in_a_capture():
    cache, drafts = _filled_cache(np.random.default_rng(63))
    q, dk, dv = drafts(2)
    out, lse = cache.verify(q, dk, dv)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError):
            cache.note_weights(q, lse)
        cache.verify(q, dk, dv)
    once = cache.note_weights(q, lse).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.note_weights(q, lse)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.acc, 2 * once)
