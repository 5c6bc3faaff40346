"""Tree attention and path commit over the compressed cache against plain float64 / integer forms,
at the sizes, masks, layouts and states where they can go wrong."""
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


def make(seed, B, N, Hq, Hkv, d, Sk, Sv, Tcap, comp, W, win, ck=0.3, cv=0.5):
    rng = np.random.default_rng(seed)
    c = dict(B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, Sk=Sk, Sv=Sv, Tcap=Tcap, W=W, rng=rng)
    c["q"] = rng.standard_normal((B, N, Hq, d)).astype(np.float16)
    c["dk"] = rng.standard_normal((B, N, Hkv, d)).astype(np.float16)
    c["dv"] = rng.standard_normal((B, N, Hkv, d)).astype(np.float16)
    c["kc"] = rng.integers(0, 256, (B, Hkv, Tcap, Sk)).astype(np.uint8)
    c["vc"] = rng.integers(0, 256, (B, Hkv, Tcap, Sv)).astype(np.uint8)
    c["Ck"] = (rng.standard_normal((Hkv, Sk, 256, d)) * ck).astype(np.float32)
    c["Cv"] = (rng.standard_normal((Hkv, Sv, 256, d)) * cv).astype(np.float32)
    c["wk"] = rng.standard_normal((B, Hkv, W, d)).astype(np.float16)
    c["wv"] = rng.standard_normal((B, Hkv, W, d)).astype(np.float16)
    c["comp"] = np.asarray(comp, np.int32)
    c["win"] = np.asarray(win, np.int32)
    c["nd"] = np.full(B, N, np.int32)
    c["mask"] = None
    c["lam"] = None
    c["scale"] = None
    return c


def hadamard(d):
    h = np.ones((1, 1))
    while len(h) < d:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(d)


def vectors(codes, books):
    return sum(books[s][codes[:, s]] for s in range(books.shape[0])).astype(np.float64) \
        if len(codes) else np.zeros((0, books.shape[-1]))


def plain(c):
    """out [B, N, Hq, d] and lse [B, N, Hq] in float64; rows behind the drafts are NaN.  Also the
    largest error that float32 arithmetic of the kernel's form can make in out and in lse."""
    B, N, Hq, d = c["q"].shape
    G = Hq // c["Hkv"]
    H = hadamard(d)
    scale = c["scale"] or 1 / math.sqrt(d)
    out, lse = np.full((B, N, Hq, d), np.nan), np.full((B, N, Hq), np.nan)
    tol = 0.0
    vmax = 1e-30
    books = c["Ck"].astype(np.float64), c["Cv"].astype(np.float64)
    for b in range(B):
        n, w, m = int(c["comp"][b]), int(c["win"][b]), int(c["nd"][b])
        for h in range(c["Hkv"]):
            k = vectors(c["kc"][b, h, :n], books[0][h]) @ H
            if c["lam"] is not None:
                k = k * c["lam"][h].astype(np.float64)
            k = np.concatenate([k, c["wk"][b, h, :w].astype(np.float64), c["dk"][b, :m, h].astype(np.float64)])
            v = np.concatenate([vectors(c["vc"][b, h, :n], books[1][h]) @ H,
                                c["wv"][b, h, :w].astype(np.float64), c["dv"][b, :m, h].astype(np.float64)])
            if np.isfinite(v).any():
                vmax = max(vmax, np.abs(v[np.isfinite(v)]).max())
            for i in range(m):
                see = np.ones(n + w + m, bool)
                see[n + w:] = (np.arange(m) <= i) if c["mask"] is None else (c["mask"][b, i, :m] != 0)
                for g in range(h * G, (h + 1) * G):
                    q = c["q"][b, i, g].astype(np.float64)
                    if not see.any():
                        out[b, i, g], lse[b, i, g] = 0, -np.inf
                        continue
                    x = k[see] @ q * scale
                    top = x.max()
                    e = np.exp(x - top)
                    out[b, i, g] = e @ v[see] / e.sum()
                    lse[b, i, g] = top + math.log(e.sum())
                    # |score error| <= (d products and sums, log2 d butterflies, S stage sums, the
                    # scale, the base change and the reference) U times the sum of the magnitudes
                    ql = q if c["lam"] is None else q * c["lam"][h]
                    mag = max(np.linalg.norm(ql) * sum(np.linalg.norm(books[0][h][s], axis=-1).max()
                                                       for s in range(c["Sk"])),
                              np.linalg.norm(q) * (np.linalg.norm(k[n:], axis=1).max() if w + m else 0))
                    tol = max(tol, (d + 8 + c["Sk"] + 8) * U * mag * scale)
    # weights: e^x to 2^-22 and the score error on numerator and denominator, 2^-20 for the
    # counters' unit, the sums of (stage, codeword) terms and keys, the rotation back
    rel = 2 * math.expm1(tol) + 2.0 ** -20 + (c["Sv"] * 256 + c["W"] + c["N"] + d) * U
    return out, lse, vmax * c["Sv"] * rel, tol + 2.0 ** -20 + 300 * U


def gpu_args(c):
    return [_cuda(c[k]) for k in ("q", "dk", "dv", "kc", "vc", "comp", "Ck", "Cv", "wk", "wv", "win")]


def gpu_kw(c):
    return dict(mask=None if c["mask"] is None else _cuda(c["mask"]), n_draft=_cuda(c["nd"]),
                k_smooth=None if c["lam"] is None else _cuda(c["lam"]), softmax_scale=c["scale"])


def check(c, out, lse, want=None):
    wo, wl, to, tl = want or plain(c)
    live = np.arange(c["N"])[None] < c["nd"][:, None]
    o, l = out.cpu().numpy(), lse.cpu().numpy()
    assert np.abs(o[live] - wo[live]).max() <= to
    a, b = l[live], wl[live]
    assert np.array_equal(np.isinf(a), np.isinf(b))
    fin = np.isfinite(b)
    assert not fin.any() or np.abs(a[fin] - b[fin]).max() <= tl * np.maximum(1, np.abs(b[fin])).max()


def tree_mask(rng, B, N):
    m = np.zeros((B, N, N), bool)
    for b in range(B):
        for i in range(N):
            if i:
                m[b, i] = m[b, rng.integers(0, i)]
            m[b, i, i] = True
    return m


CASES = {
    "one draft, empty prefix and window": dict(B=1, N=1, Hq=1, Hkv=1, d=128, Sk=4, Sv=4, Tcap=16, comp=[0], W=1, win=[0]),
    "one token": dict(B=2, N=2, Hq=2, Hkv=1, d=64, Sk=1, Sv=1, Tcap=16, comp=[1, 0], W=3, win=[0, 1]),
    "unit borders": dict(B=6, N=3, Hq=3, Hkv=3, d=64, Sk=2, Sv=2, Tcap=1040, comp=[127, 128, 129, 511, 513, 1040], W=5, win=[5, 4, 3, 2, 1, 0]),
    "groups of 7": dict(B=2, N=5, Hq=14, Hkv=2, d=128, Sk=2, Sv=4, Tcap=1600, comp=[1600, 701], W=17, win=[17, 9]),
    "three stages": dict(B=2, N=4, Hq=8, Hkv=2, d=128, Sk=3, Sv=3, Tcap=800, comp=[799, 33], W=33, win=[33, 31]),
    "eight and one": dict(B=2, N=3, Hq=4, Hkv=2, d=64, Sk=8, Sv=1, Tcap=1600, comp=[1599, 1025], W=4, win=[4, 0]),
    "five and seven": dict(B=1, N=2, Hq=3, Hkv=1, d=64, Sk=5, Sv=7, Tcap=320, comp=[301], W=8, win=[8]),
    "one and eight": dict(B=1, N=9, Hq=2, Hkv=2, d=64, Sk=1, Sv=8, Tcap=320, comp=[320], W=64, win=[40]),
    "two and six": dict(B=1, N=2, Hq=2, Hkv=1, d=64, Sk=2, Sv=6, Tcap=160, comp=[150], W=8, win=[8]),
    "four and two": dict(B=1, N=2, Hq=8, Hkv=1, d=256, Sk=4, Sv=2, Tcap=640, comp=[639], W=40, win=[40]),
    "many rows": dict(B=1, N=67, Hq=8, Hkv=1, d=64, Sk=4, Sv=4, Tcap=640, comp=[600], W=16, win=[16]),
    "many rows, d 128": dict(B=9, N=9, Hq=6, Hkv=2, d=128, Sk=3, Sv=2, Tcap=320, comp=[300, 0, 5, 320, 200, 128, 127, 1, 77], W=16, win=[16] * 9),
    "many rows, d 256": dict(B=1, N=50, Hq=4, Hkv=1, d=256, Sk=2, Sv=5, Tcap=320, comp=[311], W=16, win=[16]),
    "256 drafts": dict(B=1, N=256, Hq=2, Hkv=1, d=64, Sk=2, Sv=2, Tcap=160, comp=[150], W=16, win=[16]),
    "a wide window": dict(B=2, N=3, Hq=6, Hkv=2, d=128, Sk=2, Sv=2, Tcap=160, comp=[150, 0], W=1000, win=[1000, 777]),
    "longer": dict(B=2, N=2, Hq=4, Hkv=2, d=128, Sk=4, Sv=4, Tcap=20000, comp=[20000, 9001], W=16, win=[16, 16]),
}


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_tree_attention(name, tree):
    c = make(11, **CASES[name])
    if tree:
        c["mask"] = tree_mask(c["rng"], c["B"], c["N"])
    c["nd"] = np.array([max(0, c["N"] - b) for b in range(c["B"])], np.int32)
    keep = torch.full((c["B"], c["N"], c["Hq"], c["d"]), 7.0, device="cuda")
    keep_l = torch.full((c["B"], c["N"], c["Hq"]), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **gpu_kw(c), out=keep, lse=keep_l, error_flag=err)
    check(c, out, lse)
    assert err.item() == 0
    behind = np.arange(c["N"])[None] >= c["nd"][:, None]     # left as they were
    assert (out.cpu().numpy()[behind] == 7).all() and (lse.cpu().numpy()[behind] == 7).all()


def test_tree_rows_without_any_key():
    c = make(12, B=2, N=4, Hq=4, Hkv=2, d=128, Sk=2, Sv=2, Tcap=32, comp=[0, 20], W=4, win=[0, 0])
    c["mask"] = np.zeros((2, 4, 4), bool)
    c["mask"][:, 2, 2] = True
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **gpu_kw(c))
    check(c, out, lse)
    assert (out[0, 0] == 0).all() and torch.isinf(lse[0, 0]).all()


def test_tree_does_not_read_what_the_masks_hide():
    """NaN in drafts that a row does not see, behind the lengths and behind the drafts."""
    c = make(13, B=2, N=4, Hq=4, Hkv=2, d=64, Sk=2, Sv=2, Tcap=64, comp=[40, 0], W=8, win=[5, 0])
    c["mask"] = np.eye(4, dtype=bool)[None].repeat(2, 0)
    c["nd"] = np.array([3, 4], np.int32)
    c["wk"][:, :, 5:], c["wv"][:, :, 5:] = np.nan, np.inf
    c["wk"][1], c["wv"][1] = np.nan, np.nan
    c["dk"][0, 3], c["dv"][0, 3], c["q"][0, 3] = np.nan, np.nan, np.nan
    c["dk"][1, 2], c["dv"][1, 2] = np.inf, np.nan           # seen by row 2 alone
    want = plain({**c, "nd": np.array([3, 2], np.int32)})
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **gpu_kw(c))
    o = out.cpu().numpy()
    assert np.abs(o[0, :3] - want[0][0, :3]).max() <= want[2]
    assert np.abs(o[1, :2] - want[0][1, :2]).max() <= want[2]
    assert np.isnan(o[1, 2]).any() and np.isfinite(o[1, 3]).all()


def test_tree_a_nan_query_spoils_its_own_rows_only():
    c = make(14, B=1, N=4, Hq=4, Hkv=1, d=64, Sk=2, Sv=2, Tcap=640, comp=[640], W=8, win=[5])
    c["q"][0, 1, 2] = np.nan
    with np.errstate(invalid="ignore"):
        wo, wl, _, _ = plain(c)
    clean = make(14, B=1, N=4, Hq=4, Hkv=1, d=64, Sk=2, Sv=2, Tcap=640, comp=[640], W=8, win=[5])
    to = plain(clean)[2]
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **gpu_kw(c))
    o = out.cpu().numpy()
    assert np.isnan(o[0, 1, 2]).all() and np.isnan(lse[0, 1, 2].item())
    o[0, 1, 2] = wo[0, 1, 2] = 0
    assert np.abs(o - wo).max() <= to


@pytest.mark.parametrize("rise", [3.0, 60.0, 300.0])
def test_tree_scores_that_rise_along_the_context(rise):
    """Scores that grow from tile to tile by more than the counters hold, and by more than a
    float32's range."""
    c = make(15, B=1, N=2, Hq=2, Hkv=1, d=64, Sk=2, Sv=2, Tcap=4096, comp=[4096], W=4, win=[4], ck=0.01)
    H = hadamard(64)
    c["q"][:] = c["q"][0, 0, 0]
    qt = H @ c["q"][0, 0, 0].astype(np.float64)
    for z in range(256):                     # codeword z of stage 0 scores about z rise / 255
        c["Ck"][0, 0, z] = (qt / (qt @ qt) * math.sqrt(64) * rise * z / 255).astype(np.float32)
    c["kc"][0, 0, :, 0] = np.arange(4096) * 256 // 4096
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **gpu_kw(c))
    check(c, out, lse)


def test_tree_smoothed_keys_and_scale():
    c = make(16, B=2, N=3, Hq=4, Hkv=2, d=128, Sk=3, Sv=2, Tcap=320, comp=[300, 320], W=8, win=[8, 2])
    c["lam"] = np.exp(c["rng"].standard_normal((2, 128)) * 0.3).astype(np.float32)
    c["scale"] = 0.05
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **gpu_kw(c))
    check(c, out, lse)


def paginate(codes, P, perm, n_pages):
    Bn, Hkv, Tcap, S = codes.shape
    pool = np.full((n_pages, Hkv, P, S), 255, np.uint8)
    for b in range(Bn):
        for p in range(Tcap // P):
            pool[perm[b, p]] = codes[b, :, p * P:(p + 1) * P]
    return pool


@pytest.mark.parametrize("P,Sk,Sv", [(32, 4, 4), (64, 3, 1), (256, 2, 5)])
def test_tree_pages_and_views_give_the_same_bits(P, Sk, Sv):
    c = make(17, B=3, N=5, Hq=8, Hkv=2, d=128, Sk=Sk, Sv=Sv, Tcap=1280, comp=[1280, 700, 31], W=16, win=[16, 3, 0])
    c["mask"] = tree_mask(c["rng"], 3, 5)
    a = gpu_args(c)
    o1, l1 = zkv.rvq_tree_attn(*a, **gpu_kw(c))
    check(c, o1, l1)
    perm = c["rng"].permutation(3 * 1280 // P + 3)[:3 * 1280 // P].reshape(3, -1)
    n_pages = 3 * 1280 // P + 3
    kp, vp = _cuda(paginate(c["kc"], P, perm, n_pages)), _cuda(paginate(c["vc"], P, perm, n_pages))
    table = _cuda(perm.astype(np.int32))
    # drafts out of a fused [B, N, (q k v), d] projection, the mask out of a larger array
    fused = torch.cat([a[0], a[1], a[2]], 2)
    big = torch.zeros(4, 9, 11, dtype=torch.bool, device="cuda")
    big[:3, :5, 2:7] = _cuda(c["mask"])
    kw = gpu_kw(c)
    kw["mask"] = big[:3, :5, 2:7]
    o2, l2 = zkv.rvq_tree_attn(fused[:, :, :8], fused[:, :, 8:10], fused[:, :, 10:], kp, vp, *a[5:],
                               **kw, block_table=table)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_tree_one_mask_for_all_and_short_bound():
    c = make(18, B=2, N=4, Hq=4, Hkv=2, d=64, Sk=2, Sv=2, Tcap=640, comp=[600, 640], W=4, win=[4, 4])
    m = tree_mask(c["rng"], 1, 4)
    kw = gpu_kw(c)
    kw["mask"] = _cuda(m[0]).to(torch.uint8) * 3
    c["mask"] = m.repeat(2, 0)
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **kw)
    check(c, out, lse)
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **kw, max_comp_len=130)    # tokens beyond are not read
    check({**c, "comp": np.array([130, 130], np.int32)}, out, lse)


def test_tree_device_errors_are_reported():
    c = make(19, B=4, N=3, Hq=2, Hkv=1, d=64, Sk=2, Sv=2, Tcap=64, comp=[64, 64, 64, 10], W=4, win=[4, 4, 4, 4])
    a = gpu_args(c)
    a[5] = _cuda(np.array([70, 64, 64, -3], np.int32))
    a[10] = _cuda(np.array([4, 9, 4, 4], np.int32))
    kw = gpu_kw(c)
    kw["n_draft"] = _cuda(np.array([3, 3, 5, 3], np.int32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = zkv.rvq_tree_attn(*a, **kw, error_flag=err)
    assert err.item() == zkv.ZKV_DEVERR_COMP_LEN | zkv.ZKV_DEVERR_WIN_LEN | zkv.ZKV_DEVERR_DRAFT
    c["comp"] = np.array([64, 64, 64, 0], np.int32)
    check(c, out, lse)


def test_tree_bad_page_reads_as_code_zero():
    c = make(20, B=1, N=2, Hq=2, Hkv=1, d=64, Sk=2, Sv=2, Tcap=128, comp=[128], W=4, win=[4])
    perm = np.arange(4).reshape(1, 4)
    kp, vp = _cuda(paginate(c["kc"], 32, perm, 4)), _cuda(paginate(c["vc"], 32, perm, 4))
    perm = perm.astype(np.int32).copy()
    perm[0, 2] = 4
    a = gpu_args(c)
    a[3], a[4] = kp, vp
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = zkv.rvq_tree_attn(*a, **gpu_kw(c), block_table=_cuda(perm), error_flag=err)
    assert err.item() == zkv.ZKV_DEVERR_PAGE
    c["kc"][:, :, 64:96], c["vc"][:, :, 64:96] = 0, 0
    check(c, out, lse)


def test_tree_graphs_streams_and_repeats_agree():
    c = make(21, B=3, N=4, Hq=8, Hkv=2, d=128, Sk=4, Sv=4, Tcap=4000, comp=[4000, 0, 1111], W=16, win=[16, 3, 0])
    a = gpu_args(c)
    step = zkv.PreparedTreeAttn(*a, **gpu_kw(c))
    o, l = (t.clone() for t in step())
    for _ in range(3):
        o2, l2 = step()
        assert torch.equal(o, o2) and torch.equal(l, l2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o3, l3 = zkv.rvq_tree_attn(*a, **gpu_kw(c))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o3) and torch.equal(l, l3)
    # two graphs with workspaces of their own, replayed at once on two streams; new inputs in place
    other = make(22, B=3, N=4, Hq=8, Hkv=2, d=128, Sk=4, Sv=4, Tcap=4000, comp=[100, 4000, 5], W=16, win=[1, 2, 16])
    step2 = zkv.PreparedTreeAttn(*gpu_args(other), **gpu_kw(other))
    w2 = [t.clone() for t in step2()]
    graphs = []
    for s in (step, step2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s()
        graphs.append(g)
    for s in (step, step2):
        s.out.zero_(), s.lse.zero_()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, o) and torch.equal(step.lse, l)
    assert torch.equal(step2.out, w2[0]) and torch.equal(step2.lse, w2[1])
    new = make(23, B=3, N=4, Hq=8, Hkv=2, d=128, Sk=4, Sv=4, Tcap=4000, comp=[2000, 129, 4000], W=16, win=[3, 0, 7])
    for dst, src in zip(a, gpu_args(new)):
        dst.copy_(src)
    graphs[0].replay()
    torch.cuda.synchronize()
    check(new, step.out, step.lse)


def test_tree_many_rows_repeat():
    """128-row tables, several segments per row group: the same bits each time."""
    c = make(24, B=2, N=26, Hq=32, Hkv=4, d=128, Sk=4, Sv=4, Tcap=9008, comp=[9001, 5000], W=16, win=[16, 3])
    step = zkv.PreparedTreeAttn(*gpu_args(c), **gpu_kw(c))
    o, l = (t.clone() for t in step())
    for _ in range(5):
        o2, l2 = step()
        assert torch.equal(o, o2) and torch.equal(l, l2)
    few = {**c, "q": c["q"][:, :2], "dk": c["dk"][:, :2], "dv": c["dv"][:, :2], "N": 2, "nd": np.array([2, 2], np.int32)}
    check(few, o[:, :2], l[:, :2])          # (a chain: the first drafts do not see the others)


def test_tree_shares_a_workspace_in_stream_order():
    a, b = make(25, **CASES["groups of 7"]), make(26, **CASES["many rows, d 128"])
    need = max(zkv.tree_workspace_size(*gpu_args(c)) for c in (a, b))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")     # no initial contents are needed
    sa = zkv.PreparedTreeAttn(*gpu_args(a), **gpu_kw(a), workspace=ws)
    sb = zkv.PreparedTreeAttn(*gpu_args(b), **gpu_kw(b), workspace=ws)
    wa, wb = plain(a), plain(b)
    for _ in range(2):
        sa()
        sb()
    check(a, sa.out, sa.lse, wa)
    check(b, sb.out, sb.lse, wb)


def test_binding_refusals():
    c = make(27, **CASES["groups of 7"])
    a, kw = gpu_args(c), gpu_kw(c)

    def bad(i=None, t=None, error=ValueError, **k):
        args = list(a)
        if i is not None:
            args[i] = t
        with pytest.raises(error):
            zkv.rvq_tree_attn(*args, **{**kw, **k})

    bad(0, a[0][0])                                        # q without its batch axis
    bad(0, a[0].float(), TypeError)
    bad(0, a[0].transpose(2, 3))                           # rows not contiguous
    bad(1, a[1][:, :3])                                    # fewer drafts than queries
    bad(5, a[5][:1])                                       # one length
    bad(5, a[5].long(), TypeError)
    bad(6, a[6][:, :1])                                    # codebooks of other stages
    bad(8, a[8][:1])
    bad(mask=torch.ones(3, 3, dtype=torch.bool, device="cuda"))
    bad(mask=torch.ones(5, 5, device="cuda"), error=TypeError)
    bad(out=torch.zeros(1, device="cuda"))
    bad(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"), error=zkv.ZkvError)
    bad(max_comp_len=c["Tcap"] + 1, error=zkv.ZkvError)
    bad(0, a[0].cpu())
    with pytest.raises(zkv.ZkvError):                      # rows of 8 bytes apart
        q = torch.zeros(2 * 5 * 14 * 132, dtype=torch.float16, device="cuda").as_strided((2, 5, 14, 128), (9240, 1848, 132, 1))
        zkv.rvq_tree_attn(q, *a[1:], **kw)


# ---------------------------------------------------------------------------------------------
# Path commit
# ---------------------------------------------------------------------------------------------

def commit_case(seed, B, N, M, Hkv, d, Sk, Sv, Tcap, W, state, accept, lam=False):
    rng = np.random.default_rng(seed)
    c = dict(B=B, N=N, M=M, Hkv=Hkv, d=d, Sk=Sk, Sv=Sv, Tcap=Tcap, W=W)
    c["dk"] = rng.standard_normal((B, N, Hkv, d)).astype(np.float16)
    c["dv"] = rng.standard_normal((B, N, Hkv, d)).astype(np.float16)
    c["wk"] = rng.standard_normal((B, Hkv, W, d)).astype(np.float16)
    c["wv"] = rng.standard_normal((B, Hkv, W, d)).astype(np.float16)
    c["kc"] = rng.integers(0, 256, (B, Hkv, Tcap, Sk)).astype(np.uint8)
    c["vc"] = rng.integers(0, 256, (B, Hkv, Tcap, Sv)).astype(np.uint8)
    c["Ck"] = (rng.standard_normal((Hkv, Sk, 256, d)) * 0.6).astype(np.float32)
    c["Cv"] = (rng.standard_normal((Hkv, Sv, 256, d)) * 0.6).astype(np.float32)
    c["path"] = np.stack([rng.permutation(N)[:M] if M <= N else rng.integers(0, N, M) for _ in range(B)]).astype(np.int32)
    c["comp"], c["win"], c["head"] = (np.array(x, np.int32) for x in zip(*state))
    c["n"] = np.asarray(accept, np.int32)
    c["lam"] = np.exp(rng.standard_normal((Hkv, d)) * 0.2).astype(np.float32) if lam else None
    return c


def commit_plain(c, skip=()):
    """One append after another, sequence by sequence."""
    r = {k: c[k].copy() for k in ("wk", "wv", "kc", "vc", "comp", "win", "head")}
    for b in range(c["B"]):
        if b in skip:
            continue
        for i in range(c["n"][b]):
            slot = r["win"][b]
            if slot == c["W"]:
                slot = r["head"][b]
                for h in range(c["Hkv"]):
                    lam = None if c["lam"] is None else c["lam"][h]
                    r["kc"][b, h, r["comp"][b]] = O.rvq_encode(r["wk"][b, h, slot][None], c["Ck"][h], smooth=lam)[0][0]
                    r["vc"][b, h, r["comp"][b]] = O.rvq_encode(r["wv"][b, h, slot][None], c["Cv"][h])[0][0]
                r["comp"][b] += 1
                r["head"][b] = (slot + 1) % c["W"]
            else:
                r["win"][b] += 1
            r["wk"][b, :, slot] = c["dk"][b, c["path"][b, i]]
            r["wv"][b, :, slot] = c["dv"][b, c["path"][b, i]]
    return r


def commit_gpu(c, paged=None):
    t = {k: _cuda(c[k]) for k in ("dk", "dv", "path", "n", "wk", "wv", "win", "head", "comp", "kc", "vc", "Ck", "Cv")}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {}
    if paged is not None:
        t["kc"], t["vc"], kw["block_table"] = paged
    zkv.rvq_tree_commit(*t.values(), error_flag=err, k_smooth=None if c["lam"] is None else _cuda(c["lam"]), **kw)
    return {k: t[k].cpu().numpy() for k in ("wk", "wv", "kc", "vc", "comp", "win", "head")}, err.item()


COMMITS = {
    "one of one": dict(B=1, N=1, M=1, Hkv=1, d=128, Sk=2, Sv=2, Tcap=16, W=4, state=[(3, 4, 2)], accept=[1]),
    "none and free slots": dict(B=3, N=4, M=4, Hkv=2, d=64, Sk=4, Sv=1, Tcap=32, W=8, state=[(0, 8, 7), (5, 3, 0), (0, 0, 0)], accept=[0, 4, 2]),
    "fills, then evicts": dict(B=3, N=6, M=6, Hkv=1, d=128, Sk=3, Sv=4, Tcap=32, W=8, state=[(2, 5, 0), (9, 7, 0), (1, 8, 6)], accept=[6, 5, 6]),
    "a window of one": dict(B=2, N=5, M=5, Hkv=2, d=64, Sk=1, Sv=2, Tcap=16, W=1, state=[(4, 1, 0), (0, 0, 0)], accept=[5, 4]),
    "round the window twice": dict(B=2, N=9, M=9, Hkv=1, d=64, Sk=2, Sv=2, Tcap=32, W=3, state=[(7, 3, 2), (0, 1, 0)], accept=[9, 8]),
    "free slots behind a moved head": dict(B=2, N=6, M=6, Hkv=1, d=64, Sk=2, Sv=2, Tcap=32, W=5, state=[(7, 3, 2), (0, 4, 4)], accept=[6, 5]),
    "the same draft twice": dict(B=1, N=2, M=5, Hkv=1, d=64, Sk=2, Sv=2, Tcap=32, W=2, state=[(7, 2, 1)], accept=[5]),
    "many sequences": dict(B=37, N=5, M=5, Hkv=2, d=64, Sk=2, Sv=2, Tcap=32, W=4, state=[(i % 20, min(4, i % 6), i % 4 if i % 6 >= 4 else 0) for i in range(37)], accept=[(3 * i) % 6 for i in range(37)]),
    "blocks of 32 evictions": dict(B=150, N=5, M=5, Hkv=4, d=64, Sk=2, Sv=1, Tcap=32, W=4, state=[(i % 20, 4, i % 4) for i in range(150)], accept=[(7 * i) % 6 for i in range(150)]),
    "blocks of 32, d 256": dict(B=90, N=4, M=4, Hkv=4, d=256, Sk=1, Sv=2, Tcap=16, W=3, state=[(i % 12, 3, i % 3) for i in range(90)], accept=[(3 * i) % 5 for i in range(90)]),
    "blocks of 32, d 128": dict(B=70, N=4, M=3, Hkv=6, d=128, Sk=3, Sv=2, Tcap=16, W=2, state=[(i % 12, 2, i % 2) for i in range(70)], accept=[(3 * i) % 4 for i in range(70)]),
    "eight stages": dict(B=2, N=3, M=3, Hkv=1, d=256, Sk=8, Sv=5, Tcap=16, W=2, state=[(7, 2, 1), (1, 2, 0)], accept=[3, 1]),
    "filled to the brim": dict(B=2, N=3, M=3, Hkv=1, d=64, Sk=2, Sv=2, Tcap=16, W=2, state=[(13, 2, 1), (16, 0, 0)], accept=[3, 2]),
}


@pytest.mark.parametrize("name", COMMITS)
def test_commit(name):
    c = commit_case(31, **COMMITS[name], lam=name == "fills, then evicts")
    got, err = commit_gpu(c)
    want = commit_plain(c)
    assert err == 0
    for k in want:
        assert np.array_equal(got[k], want[k]), k


def test_commit_more_than_256_sequences():
    c = commit_case(32, B=300, N=2, M=2, Hkv=1, d=64, Sk=1, Sv=1, Tcap=16, W=2,
                    state=[(i % 8, 2, i % 2) for i in range(300)], accept=[i % 3 for i in range(300)])
    got, err = commit_gpu(c)
    want = commit_plain(c)
    assert err == 0
    for k in want:
        assert np.array_equal(got[k], want[k]), k


def test_commit_leaves_bad_sequences_alone():
    c = commit_case(33, B=9, N=4, M=3, Hkv=1, d=64, Sk=2, Sv=2, Tcap=16, W=2,
                    state=[(3, 2, 0), (3, 2, 0), (3, 2, 0), (3, 3, 0), (3, -1, 0), (3, 2, 2), (14, 2, 0), (-1, 2, 0), (5, 2, 1)],
                    accept=[4, -1, 3, 1, 1, 1, 3, 1, 3])
    c["path"][2, 2] = 4
    c["path"][8] = [3, 0, 1]
    for b, bit in [(0, zkv.ZKV_DEVERR_DRAFT), (1, zkv.ZKV_DEVERR_DRAFT), (2, zkv.ZKV_DEVERR_DRAFT),
                   (3, zkv.ZKV_DEVERR_WIN_LEN), (4, zkv.ZKV_DEVERR_WIN_LEN), (5, zkv.ZKV_DEVERR_WIN_LEN),
                   (6, zkv.ZKV_DEVERR_COMP_LEN), (7, zkv.ZKV_DEVERR_COMP_LEN)]:
        one = {**c, "n": np.where(np.arange(9) == b, c["n"], np.where(np.arange(9) == 8, 3, 0)).astype(np.int32)}
        got, err = commit_gpu(one)
        want = commit_plain(one, skip=[b])
        # sequences with a bad window length report it even when they accept nothing
        assert err & bit
        for k in want:
            assert np.array_equal(got[k], want[k]), (b, k)


@pytest.mark.parametrize("P", [32, 64])
def test_commit_pages(P):
    c = commit_case(34, B=3, N=6, M=6, Hkv=2, d=64, Sk=2, Sv=3, Tcap=128, W=4,
                    state=[(30, 4, 1), (61, 4, 0), (122, 2, 0)], accept=[6, 5, 6])
    mp = 128 // P
    perm = np.random.default_rng(1).permutation(3 * mp + 2)[:3 * mp].reshape(3, mp).astype(np.int32)
    kp, vp = (_cuda(paginate(c[k], P, perm, 3 * mp + 2)) for k in ("kc", "vc"))
    got, err = commit_gpu(c, (kp, vp, _cuda(perm)))
    want = commit_plain(c)
    assert err == 0
    for k in ("wk", "wv", "comp", "win", "head"):
        assert np.array_equal(got[k], want[k]), k
    for k in ("kc", "vc"):
        assert np.array_equal(got[k], paginate(want[k], P, perm, 3 * mp + 2)), k
    bad = perm.copy()
    bad[0, 32 // P] = -1                     # the page that sequence 0 runs into
    kp, vp = (_cuda(paginate(c[k], P, perm, 3 * mp + 2)) for k in ("kc", "vc"))
    got, err = commit_gpu(c, (kp, vp, _cuda(bad)))
    want = commit_plain(c, skip=[0])
    assert err == zkv.ZKV_DEVERR_PAGE
    for k in ("wk", "wv", "comp", "win", "head"):
        assert np.array_equal(got[k], want[k]), k
    for k in ("kc", "vc"):
        assert np.array_equal(got[k], paginate(want[k], P, perm, 3 * mp + 2)), k


def test_commit_is_captured_and_replayed():
    c = commit_case(35, B=3, N=4, M=4, Hkv=2, d=128, Sk=4, Sv=4, Tcap=64, W=4,
                    state=[(10, 4, 1), (0, 2, 0), (5, 4, 3)], accept=[4, 3, 2])
    t = {k: _cuda(c[k]) for k in ("dk", "dv", "path", "n", "wk", "wv", "win", "head", "comp", "kc", "vc", "Ck", "Cv")}
    zkv.rvq_tree_commit(*[x.clone() for x in t.values()])      # sets the kernel's attributes
    step = zkv.PreparedTreeCommit(*t.values())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    want = c
    for _ in range(3):
        g.replay()
        want = {**want, **commit_plain(want)}
    torch.cuda.synchronize()
    for k in ("wk", "wv", "kc", "vc", "comp", "win", "head"):
        assert np.array_equal(t[k].cpu().numpy(), want[k]), k
