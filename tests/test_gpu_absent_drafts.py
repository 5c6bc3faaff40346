"""Totals of received attention where sequences have fewer drafts than the batch: rows behind
n_draft add nothing, whatever their queries and their lse hold."""
import math

import numpy as np
import pytest
import torch

from compressed_decode_attention_zkv_b200 import build as B
from compressed_decode_attention_zkv_b200 import zkv
from test_gpu_budget import _filled_cache, hadamard, weights_case, weights_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.build()
    zkv.lib()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _totals(cache, q, dk, nd, before, counts=None):
    """float64 totals after the attention of the present drafts (a chain) over the cache; of those
    that ``counts`` [B, N] names, if it is given."""
    q, dk = q.double().cpu().numpy(), dk.double().cpu().numpy()
    kc, wk = cache.k_codes.cpu().numpy(), cache.win_k.double().cpu().numpy()
    comp, win = cache.comp_len.cpu().numpy(), cache.win_len.cpu().numpy()
    Ck = cache.Ck.double().cpu().numpy()
    G, d = q.shape[2] // cache.Hkv, cache.d
    H = hadamard(d)
    acc = before.copy()
    for b in range(cache.B):
        n, w, m = comp[b], win[b], nd[b]
        for h in range(cache.Hkv):
            k = sum(Ck[h, s][kc[b, h, :n, s]] for s in range(cache.Sk)) @ H
            k = np.concatenate([k, wk[b, h, :w], dk[b, :m, h]])
            for g in range(h * G, (h + 1) * G):
                x = q[b, :m, g] @ k.T / math.sqrt(d)
                x[:, n + w:][np.arange(m)[None] > np.arange(m)[:, None]] = -np.inf
                p = np.exp(x - x.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                acc[b, h, :n] += p[slice(None) if counts is None else counts[b, :m], :n].sum(0)
    return acc


@pytest.mark.parametrize("given", ["lse of the call", "lse of an old step"])
def test_totals_after_a_verify_with_absent_drafts(given):
    """Two rounds of verify(n_draft), note_weights, commit; NaN wherever no draft is."""
    cache, drafts = _filled_cache(np.random.default_rng(71))
    acc = np.zeros((cache.B, cache.Hkv, cache.Tcap))
    lse = torch.full((2, 6, 8), 0.25, device="cuda") if given == "lse of an old step" else None
    for nd in ([3, 6], [0, 5]):
        q, dk, dv = drafts(6)
        for b in range(2):
            q[b, nd[b]:], dk[b, nd[b]:], dv[b, nd[b]:] = math.nan, math.nan, math.nan
        n_draft = torch.tensor(nd, dtype=torch.int32, device="cuda")
        out, got = cache.verify(q, dk, dv, n_draft=n_draft, lse=lse)
        acc = _totals(cache, q, dk, nd, acc)
        if lse is None:
            cache.note_weights(q, got)
        else:
            cache.note_weights(q, got, n_draft=n_draft)
        # scores below 12 in magnitude: 2 (d + 24) 2^-24 12 of a weight
        assert np.abs(cache.acc.double().cpu().numpy() - acc).max() < 3e-4 * (1 + acc.max())
        cache.commit(dk, dv, torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device="cuda"),
                     torch.tensor([min(nd[0], 2), 2], dtype=torch.int32, device="cuda"))
    assert cache.error_flag.item() == 0


@pytest.mark.parametrize("N,Hq", [(3, 1), (3, 3), (9, 8)])
def test_weights_of_the_present_queries_only(N, Hq):
    c = weights_case(72, B=4, N=N, Hq=Hq, Hkv=1, d=64, S=2, Tcap=640, comp=[640, 37, 0, 300])
    nd = np.array([N, 1, 2, 0], np.int32)
    behind = np.arange(N)[None] >= nd[:, None]
    q, lse = c["q"].copy(), c["lse"].copy()
    q[behind], lse[behind] = np.nan, 0.0
    c["lse"][behind] = np.nan                  # the plain form leaves these rows out
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for given, flag in ((nd, 0), (np.array([N + 1, 1, 2, -1], np.int32), zkv.ZKV_DEVERR_DRAFT)):
        acc = _cuda(c["acc"])
        zkv.rvq_accumulate_weights(_cuda(q), _cuda(lse), *[_cuda(c[k]) for k in ("kc", "comp", "Ck")], acc,
                                   n_draft=_cuda(given), error_flag=err)
        weights_check(c, acc)                  # (counts outside 0..N are clamped and reported)
        assert err.item() == flag


def test_absent_drafts_of_a_call_without_arrays():
    """Arrays that the call makes: rows behind the drafts are an output of zero with lse -inf, which
    adds nothing to totals and counts for nothing in a merge."""
    cache, drafts = _filled_cache(np.random.default_rng(73))
    out, lse = cache.verify(*drafts(4), n_draft=torch.tensor([1, 4], dtype=torch.int32, device="cuda"))
    assert (lse[0, 1:] == -math.inf).all() and (out[0, 1:] == 0).all()
    assert torch.isfinite(lse[0, :1]).all() and torch.isfinite(lse[1]).all()


def test_n_draft_is_checked():
    c = weights_case(74, B=2, N=2, Hq=2, Hkv=1, d=64, S=2, Tcap=64, comp=[64, 3])
    args = [_cuda(c[k]) for k in ("q", "lse", "kc", "comp", "Ck", "acc")]
    with pytest.raises(ValueError):
        zkv.rvq_accumulate_weights(*args, n_draft=torch.ones(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        zkv.rvq_accumulate_weights(*args, n_draft=torch.ones(2, device="cuda"))


def test_accepted_drafts_alone_count():
    """verify, note_weights of the accepted rows, commit, evict, as a serving loop runs them."""
    cache, drafts = _filled_cache(np.random.default_rng(75))
    acc = np.zeros((cache.B, cache.Hkv, cache.Tcap))
    path = torch.tensor([[0, 2, 3], [0, 1, 0]], dtype=torch.int32, device="cuda")
    n_accept = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    accepted = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    accepted[0, [0, 2, 3]] = accepted[1, [0, 1]] = True
    for _ in range(3):
        q, dk, dv = drafts(4)
        out, lse = cache.verify(q, dk, dv)
        acc = _totals(cache, q, dk, [4, 4], acc, accepted.cpu().numpy())
        cache.note_weights(q, lse.masked_fill(~accepted[:, :, None], float("inf")))
        assert np.abs(cache.acc.double().cpu().numpy() - acc).max() < 3e-4 * (1 + acc.max())
        cache.commit(dk, dv, path, n_accept)
    old = cache.comp_len.cpu().numpy()
    kept = torch.zeros(2, cache.Hkv, 300, dtype=torch.int32, device="cuda")
    cache.evict(300, recent=50, kept=kept)
    kept = kept.cpu().numpy()
    for b in range(2):
        for h in range(cache.Hkv):
            t = np.setdiff1d(np.arange(old[b] - 50), kept[b, h])      # an old token that went is no heavier
            k = kept[b, h][kept[b, h] < old[b] - 50]
            assert len(k) == 250 and acc[b, h, t].max() <= acc[b, h, k].min() + 6e-4 * (1 + acc.max())
