"""Measured cases of the operators around a compressed cache that is verified in trees and kept small.

Four operators of one serving loop over an RVQ-compressed KV cache:

  tree     attention of a tree (or chain) of drafted tokens over the compressed prefix, the fp16
           window and the drafts themselves: what verifying a speculated continuation costs
  commit   the accepted path of the tree enters the cache: window insert, eviction and RVQ encode
           of as many tokens as each sequence accepted
  weights  attention weight that each compressed token received, added to a running total
  evict    the compressed prefix shrinks to the tokens with the largest totals

``run`` computes a case in plain torch operations (``own`` false) or through the package's entry
points (``own`` true) on the same state.  Shapes are the package's workloads (one head in a small
cache, 8 sequences at 32K, one at 128K, 64 ragged sequences) and the ranges around them.
"""
import math

import numpy as np
import torch

own = False

CODEWORDS = 256
DEV = "cuda"


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # a small single-head cache, eight drafted tokens: the latency of one call
        dict(name="tree-1x1k", op="tree", B=1, Hq=1, Hkv=1, d=128, Sk=2, Sv=2, T=960, lo=960, W=64,
             N=8, chain=False, page=0),
        # a batch of 8 long sequences with grouped heads, a tree of 16 drafts each
        dict(name="tree-8x32k", op="tree", B=8, Hq=32, Hkv=8, d=128, Sk=4, Sv=4, T=32640, lo=32640,
             W=128, N=16, chain=False, page=0),
        # one very long sequence, groups of 7 heads, fewer key stages, an odd number of drafts
        dict(name="tree-1x128k", op="tree", B=1, Hq=28, Hkv=4, d=128, Sk=2, Sv=4, T=130816,
             lo=130816, W=256, N=25, chain=False, page=0),
        # 64 ragged sequences in pages, a chain of five drafts (a small draft model's guesses)
        dict(name="tree-64xragged", op="tree", B=64, Hq=32, Hkv=8, d=128, Sk=4, Sv=4, T=16384,
             lo=1024, W=128, N=5, chain=True, page=256),
        # one sequence accepts a few of its eight drafts
        dict(name="commit-1", op="commit", B=1, Hkv=1, d=128, Sk=2, Sv=2, T=960, W=64, N=8, M=4),
        # every sequence of the 32K batch accepts up to six of 16 drafts
        dict(name="commit-8", op="commit", B=8, Hkv=8, d=128, Sk=4, Sv=4, T=32640, W=128, N=16, M=6),
        # the ragged batch accepts up to five of five
        dict(name="commit-64", op="commit", B=64, Hkv=8, d=128, Sk=4, Sv=4, T=4096, W=128, N=5, M=5),
        # weights of one decode step of the 32K batch, and of the 128K sequence
        dict(name="weights-8x32k", op="weights", B=8, Hq=32, Hkv=8, d=128, Sk=4, T=32640, lo=32640,
             N=1, page=0),
        dict(name="weights-1x128k", op="weights", B=1, Hq=28, Hkv=4, d=128, Sk=2, T=130816,
             lo=130816, N=1, page=0),
        # a small cache keeps about half; a 32K batch keeps an eighth; 128K keeps a quarter
        dict(name="evict-1x1k", op="evict", B=1, Hkv=1, Sk=2, Sv=2, T=960, lo=960, keep=500, recent=64),
        dict(name="evict-8x32k", op="evict", B=8, Hkv=8, Sk=4, Sv=4, T=32640, lo=32640, keep=4096,
             recent=256),
        dict(name="evict-1x128k", op="evict", B=1, Hkv=4, Sk=2, Sv=4, T=130816, lo=130816, keep=32768,
             recent=1024),
    ]


def draw(rng):
    def logu(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["tree", "tree", "commit", "weights", "evict"])
    B = logu(1, 64)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    d = rng.choice([64, 128, 128, 128, 256])
    Sk, Sv = rng.choice([1, 2, 3, 4, 4, 8]), rng.choice([1, 2, 3, 4, 4, 8])
    T = logu(1, 131072)
    while B * Hkv * T * max(Sk, Sv) > 8 * 8 * 32640 * 4:   # codes no larger than the 32K batch's
        if B > 1 and rng.random() < 0.5:
            B = max(1, B // 2)
        else:
            T = max(1, T // 2)
    lo = rng.choice([T, max(1, T // 16), 0])
    page = rng.choice([0, 0, 32, 64, 256])
    if op == "tree":
        N = logu(1, 64)
        while B * Hkv * G * N * T * d > 8 * 32 * 16 * 32640 * 128:
            N = max(1, N // 2)
            T = max(1, T // 2) if N == 1 else T
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, Sk=Sk, Sv=Sv, T=T, lo=min(lo, T),
                    W=rng.choice([1, 17, 64, 128, 256]), N=N, chain=rng.random() < 0.3, page=page)
    if op == "commit":
        N = logu(1, 32)
        W = rng.choice([1, 16, 64, 128])
        T = min(T, 16384)
        return dict(op=op, B=B, Hkv=Hkv, d=d, Sk=Sk, Sv=Sv, T=T, W=W, N=N, M=rng.randint(1, min(N, 8)))
    if op == "weights":
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, Sk=Sk, T=T, lo=min(lo, T),
                    N=rng.choice([1, 1, 1, 2, 5]), page=page)
    keep = rng.randint(1, T)
    return dict(op=op, B=B, Hkv=Hkv, Sk=Sk, Sv=Sv, T=T, lo=min(lo, T), keep=keep,
                recent=rng.choice([0, keep // 8, keep // 2]))


def work(case):
    c = case
    if c["op"] == "tree":
        n = (c["lo"] + c["T"]) / 2                       # mean compressed length
        pairs, rows = c["B"] * c["Hkv"], c["N"] * c["Hq"] // c["Hkv"]
        dense = c["W"] + c["N"]
        byts = pairs * (n * (c["Sk"] + c["Sv"]) + dense * c["d"] * 4)
        byts += c["Hkv"] * (c["Sk"] + c["Sv"]) * CODEWORDS * c["d"] * 4
        byts += c["B"] * c["N"] * c["Hq"] * (c["d"] * (2 + 4) + 4)
        # products of the queries with the keys and of the weights with the values
        return {"bytes": byts, "flops": 4.0 * pairs * rows * (n + dense) * c["d"]}
    if c["op"] == "commit":
        m = c["B"] * (c["M"] + 1) / 2                    # mean accepted tokens of the batch
        rows = m * c["Hkv"]
        books = c["Hkv"] * (c["Sk"] + c["Sv"]) * CODEWORDS * c["d"] * 4
        byts = books + rows * (3 * c["d"] * 2 * 2 + c["Sk"] + c["Sv"])
        return {"bytes": byts, "flops": rows * (c["Sk"] + c["Sv"]) * CODEWORDS * c["d"] * 2.0}
    if c["op"] == "weights":
        n = (c["lo"] + c["T"]) / 2
        pairs, rows = c["B"] * c["Hkv"], c["N"] * c["Hq"] // c["Hkv"]
        byts = pairs * n * (c["Sk"] + 8) + c["Hkv"] * c["Sk"] * CODEWORDS * c["d"] * 4
        byts += c["B"] * c["N"] * c["Hq"] * (c["d"] * 2 + 4)
        return {"bytes": byts, "flops": 2.0 * pairs * rows * n * c["d"]}
    n = (c["lo"] + c["T"]) / 2
    kept = min(n, c["keep"])
    pairs = c["B"] * c["Hkv"]
    # totals read once; kept codes read and written, kept totals and positions written
    byts = pairs * (n * 4 + kept * 2 * (c["Sk"] + c["Sv"]) + kept * 4 + kept * 4)
    return {"bytes": byts, "flops": 0.0}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _capacity(case):
    t = case["T"]
    page = case.get("page", 0)
    return (t + page - 1) // page * page if page else (t + 15) // 16 * 16


def _codebooks(g, Hkv, S, d, first, smooth=0.6):
    # Gaussian codewords whose energy falls from stage to stage, codeword 0 the zero vector
    scale = first * smooth ** torch.arange(S, device=DEV, dtype=torch.float32)
    c = torch.randn((Hkv, S, CODEWORDS, d), generator=g, device=DEV) * scale[None, :, None, None]
    c[:, :, 0] = 0
    return c


def _codes(g, shape):
    # an uneven use of the codewords, as trained codebooks have it
    w = 1.0 / (torch.arange(CODEWORDS, device=DEV, dtype=torch.float32) + 8.0) ** 0.9
    w = w[torch.randperm(CODEWORDS, generator=g, device=DEV)]
    cdf = torch.cumsum(w / w.sum(), 0)
    u = torch.rand(shape, generator=g, device=DEV)
    return torch.searchsorted(cdf, u).clamp_(max=CODEWORDS - 1).to(torch.uint8)


def _heads(g, Hkv, d):
    # channel scales of the keys: lognormal, eight outlier channels ten times larger
    s = torch.exp(0.5 * torch.randn((Hkv, d), generator=g, device=DEV))
    s[:, :8] *= 10.0
    return s


def _lengths(g, B, lo, T):
    n = torch.randint(lo, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    return n if lo < T else torch.full_like(n, T)


def _paged(codes, page, g):
    """The contiguous codes [B, Hkv, T, S] as a shuffled pool of pages and its block table."""
    B, Hkv, T, S = codes.shape
    n = T // page
    perm = torch.randperm(B * n, generator=g, device=DEV)
    pages = codes.view(B, Hkv, n, page, S).permute(0, 2, 1, 3, 4).reshape(B * n, Hkv, page, S)
    pool = torch.empty_like(pages)
    pool[perm] = pages
    return pool, perm.view(B, n).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "tree":
        B, Hq, Hkv, d, N, W = c["B"], c["Hq"], c["Hkv"], c["d"], c["N"], c["W"]
        cap = _capacity(c)
        sc = _heads(g, Hkv, d)
        s["q"] = torch.randn((B, N, Hq, d), generator=g, device=DEV).half()
        s["draft_k"] = (torch.randn((B, N, Hkv, d), generator=g, device=DEV) * sc).half()
        s["draft_v"] = torch.randn((B, N, Hkv, d), generator=g, device=DEV).half()
        s["win_k"] = (torch.randn((B, Hkv, W, d), generator=g, device=DEV) * sc[:, None]).half()
        s["win_v"] = torch.randn((B, Hkv, W, d), generator=g, device=DEV).half()
        s["win_len"] = torch.randint(W // 2, W + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["comp_len"] = _lengths(g, B, c["lo"], c["T"])
        s["Ck"] = _codebooks(g, Hkv, c["Sk"], d, 2.4)
        s["Cv"] = _codebooks(g, Hkv, c["Sv"], d, 0.8)
        kc, vc = _codes(g, (B, Hkv, cap, c["Sk"])), _codes(g, (B, Hkv, cap, c["Sv"]))
        s["table"] = None
        if c["page"]:
            g2 = torch.Generator(device=DEV)
            g2.manual_seed(seed + 1)
            vc, s["table"] = _paged(vc, c["page"], g2)
            g2.manual_seed(seed + 1)
            kc, s["table"] = _paged(kc, c["page"], g2)
        s["k_codes"], s["v_codes"] = kc, vc
        s["n_draft"] = torch.randint(max(1, N - 2), N + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["mask"] = None
        if not c["chain"]:
            # every draft but the first hangs below an earlier one; it sees its ancestors and itself
            parent = (torch.rand((B, N), generator=g, device=DEV)
                      * torch.arange(N, device=DEV)).long().clamp_(min=0)
            mask = torch.zeros((B, N, N), dtype=torch.bool, device=DEV)
            row = torch.arange(B, device=DEV)
            for i in range(N):
                if i:
                    mask[:, i] = mask[row, parent[:, i]]
                mask[:, i, i] = True
            s["mask"] = mask
        # rows behind a sequence's drafts are left as they are
        s["out"] = torch.zeros((B, N, Hq, d), device=DEV)
        s["lse"] = torch.zeros((B, N, Hq), device=DEV)
        return s
    if c["op"] == "commit":
        B, Hkv, d, N, M, W = c["B"], c["Hkv"], c["d"], c["N"], c["M"], c["W"]
        cap = (c["T"] + M + 15) // 16 * 16
        sc = _heads(g, Hkv, d)
        s["draft_k"] = (torch.randn((B, N, Hkv, d), generator=g, device=DEV) * sc).half()
        s["draft_v"] = torch.randn((B, N, Hkv, d), generator=g, device=DEV).half()
        s["win_k"] = (torch.randn((B, Hkv, W, d), generator=g, device=DEV) * sc[:, None]).half()
        s["win_v"] = torch.randn((B, Hkv, W, d), generator=g, device=DEV).half()
        s["Ck"] = _codebooks(g, Hkv, c["Sk"], d, 2.4)
        s["Cv"] = _codebooks(g, Hkv, c["Sv"], d, 0.8)
        s["k_codes"], s["v_codes"] = _codes(g, (B, Hkv, cap, c["Sk"])), _codes(g, (B, Hkv, cap, c["Sv"]))
        # an accepted path: rising draft indices, as many as the sequence accepted
        s["path"] = torch.rand((B, N), generator=g, device=DEV).argsort(1)[:, :M].sort(1).values.int().contiguous()
        s["n_accept"] = torch.randint(1, M + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        # most windows are full, a few still have free slots
        full = torch.rand((B,), generator=g, device=DEV) < 0.8
        part = torch.randint(max(0, W - M), W + 1, (B,), generator=g, device=DEV)
        wl = torch.where(full, torch.full_like(part, W), part)
        head = torch.where(wl == W, torch.randint(0, W, (B,), generator=g, device=DEV), torch.zeros_like(wl))
        comp = torch.randint(c["T"] // 2, c["T"] + 1, (B,), generator=g, device=DEV)
        s["before"] = torch.stack([comp, wl, head]).int().contiguous()
        s["lengths"] = s["before"].clone()
        return s
    if c["op"] == "weights":
        B, Hq, Hkv, d, N = c["B"], c["Hq"], c["Hkv"], c["d"], c["N"]
        cap = _capacity(c)
        s["q"] = torch.randn((B, N, Hq, d), generator=g, device=DEV).half()
        s["comp_len"] = _lengths(g, B, c["lo"], c["T"])
        s["Ck"] = _codebooks(g, Hkv, c["Sk"], d, 2.4)
        kc = _codes(g, (B, Hkv, cap, c["Sk"]))
        s["table"] = None
        if c["page"]:
            kc, s["table"] = _paged(kc, c["page"], g)
        s["k_codes"] = kc
        # about the log-sum-exp that a context of this length has with such keys
        var = s["q"].float().square().mean(-1) * s["Ck"].square().mean((2, 3)).sum(1).repeat_interleave(Hq // Hkv)
        s["lse"] = (torch.log(s["comp_len"].float().clamp(min=1) + 64)[:, None, None] + 0.5 * var).contiguous()
        s["acc"] = torch.rand((B, Hkv, cap), generator=g, device=DEV) * 0.01
        return s
    B, Hkv = c["B"], c["Hkv"]
    cap, out = _capacity(c), (c["keep"] + 15) // 16 * 16
    s["k_codes"], s["v_codes"] = _codes(g, (B, Hkv, cap, c["Sk"])), _codes(g, (B, Hkv, cap, c["Sv"]))
    s["comp_len"] = _lengths(g, B, c["lo"], c["T"])
    # totals over many orders of magnitude; some tokens never received any
    acc = torch.exp(2.5 * torch.randn((B, Hkv, cap), generator=g, device=DEV))
    s["acc"] = torch.where(torch.rand((B, Hkv, cap), generator=g, device=DEV) < 0.9, acc, torch.zeros_like(acc))
    # the buffers that the kept tokens go to; what lies behind them stays as it is
    s["k_out"] = torch.zeros((B, Hkv, out, c["Sk"]), dtype=torch.uint8, device=DEV)
    s["v_out"] = torch.zeros((B, Hkv, out, c["Sv"]), dtype=torch.uint8, device=DEV)
    s["acc_out"] = torch.zeros((B, Hkv, out), device=DEV)
    s["len_out"] = torch.zeros((B,), dtype=torch.int32, device=DEV)
    s["kept"] = torch.zeros((B, Hkv, c["keep"]), dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------

def _hadamard(d, dtype):
    i = torch.arange(d, device=DEV)
    both = i[:, None] & i[None, :]
    parity = ((both[..., None] >> torch.arange(8, device=DEV)) & 1).sum(-1) & 1
    return 1 - 2 * parity.to(dtype)


def _flat(codes, table):
    if table is None:
        return codes
    B, n = table.shape
    _, H, P, S = codes.shape
    return codes[table.long()].permute(0, 2, 1, 3, 4).reshape(B, H, n * P, S)


def _vectors(codes, books):
    """Reconstructed vectors [B, H, T, d] in the rotated domain."""
    H, S = books.shape[:2]
    h = torch.arange(H, device=DEV)[:, None, None]
    st = torch.arange(S, device=DEV)
    return books[h, st, codes.long()].sum(-2)


def _tree(s):
    B, N, Hq, d = s["q"].shape
    Hkv, W = s["win_k"].shape[1:3]
    G = Hq // Hkv
    H = _hadamard(d, torch.float32) / math.sqrt(d)
    q = s["q"].float().view(B, N, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, d)
    dk, dv = s["draft_k"].float().transpose(1, 2), s["draft_v"].float().transpose(1, 2)
    k = _vectors(_flat(s["k_codes"], s["table"]), s["Ck"])
    T = k.shape[2]
    sp = torch.where((torch.arange(T, device=DEV) < s["comp_len"][:, None])[:, None, None],
                     (q @ H) @ k.transpose(-1, -2), -math.inf)
    sw = torch.where((torch.arange(W, device=DEV) < s["win_len"][:, None])[:, None, None],
                     q @ s["win_k"].float().transpose(-1, -2), -math.inf)
    j = torch.arange(N, device=DEV)
    see = (j[None, :] <= j[:, None]).expand(B, N, N) if s["mask"] is None else s["mask"]
    see = (see & (j < s["n_draft"][:, None])[:, None]).repeat_interleave(G, 1)[:, None]
    sd = torch.where(see, q @ dk.transpose(-1, -2), -math.inf)
    x = torch.cat([sp, sw, sd], -1) / math.sqrt(d)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    v = _vectors(_flat(s["v_codes"], s["table"]), s["Cv"])
    o = (p[..., :T] @ v) @ H + p[..., T:T + W] @ s["win_v"].float() + p[..., T + W:] @ dv
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.view(B, Hkv, N, G, d).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, d)
    lse = lse.view(B, Hkv, N, G).permute(0, 2, 1, 3).reshape(B, N, Hq)
    live = (j < s["n_draft"][:, None])[..., None]
    return torch.where(live[..., None], o, s["out"]), torch.where(live, lse, s["lse"])


def _encode(x, books):
    """Greedy residual codes of x [R, H, d] (fp16): nearest codeword per stage, decided in float64."""
    d = x.shape[-1]
    r = (x.double() @ _hadamard(d, torch.float64) / math.sqrt(d)).float()
    codes = []
    for s in range(books.shape[1]):
        c = books[:, s].double()
        dist = c.square().sum(-1)[None] - 2 * torch.einsum("rhd,hcd->rhc", r.double(), c)
        z = dist.argmin(-1)
        r = r - books[torch.arange(x.shape[1], device=DEV), s, z]
        codes.append(z.to(torch.uint8))
    return torch.stack(codes, -1)


def _commit(s):
    c = s["case"]
    B, M, W = c["B"], c["M"], c["W"]
    comp, wl, head = s["lengths"].long()
    i = torch.arange(M, device=DEV)
    new = i < s["n_accept"][:, None]                        # accepted tokens [B, M]
    slot = torch.where(wl[:, None] + i < W, wl[:, None] + i, (head[:, None] + wl[:, None] + i - W) % W)
    ev = new & (wl[:, None] + i >= W)                       # the token whose slot was taken is evicted
    age = wl[:, None] + i - W                               # how many evictions came before it
    n = ev.sum(1)
    # an entry that evicts nothing writes back what it finds behind the new codes
    pos = comp[:, None] + torch.where(ev, age, n[:, None] + i - (ev.cumsum(1) - ev.long()))
    b = torch.arange(B, device=DEV)[:, None]
    # what the slot held: an earlier accepted token of this call, or the window's own token
    same = (slot[:, None, :] == slot[:, :, None]) & new[:, None, :]
    last = torch.where(same & (i[None, :] < i[:, None]), i + 1, 0).amax(-1)
    # the last accepted token that each slot of the window takes
    takes = torch.where((slot[:, None, :] == torch.arange(W, device=DEV)[:, None]) & new[:, None, :], i + 1, 0).amax(-1)
    for kind in ("k", "v"):
        win, codes, books = s["win_" + kind], s[kind + "_codes"], s["C" + kind]
        tok = s["draft_" + kind][b, s["path"].long()]       # [B, M, Hkv, d]
        src = torch.where((last > 0)[..., None, None], tok[b, (last - 1).clamp(min=0)], win[b, :, slot])
        z = _encode(src.flatten(0, 1), books).view(B, M, -1, books.shape[1])
        codes[b, :, pos] = torch.where(ev[..., None, None], z, codes[b, :, pos])
        into = tok[b, (takes - 1).clamp(min=0)].transpose(1, 2)
        win.copy_(torch.where((takes > 0)[:, None, :, None], into, win))
    s["lengths"].copy_(torch.stack([comp + n, torch.minimum(wl + s["n_accept"], torch.full_like(wl, W)),
                                    (head + n) % W]))
    return [s[k] for k in ("k_codes", "v_codes", "win_k", "win_v", "lengths")]


def _weights(s):
    B, N, Hq, d = s["q"].shape
    Hkv = s["acc"].shape[1]
    G = Hq // Hkv
    H = _hadamard(d, torch.float32) / math.sqrt(d)
    q = s["q"].float().view(B, N, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, d)
    k = _vectors(_flat(s["k_codes"], s["table"]), s["Ck"])
    lse = s["lse"].view(B, N, Hkv, G).permute(0, 2, 1, 3).reshape(B, Hkv, N * G, 1)
    p = torch.exp((q @ H) @ k.transpose(-1, -2) / math.sqrt(d) - lse).sum(2)
    live = torch.arange(k.shape[2], device=DEV) < s["comp_len"][:, None]
    s["acc"] += torch.where(live[:, None], p, 0.0)
    return s["acc"]


def _evict(s):
    c = s["case"]
    keep, recent = c["keep"], c["recent"]
    B, Hkv, cap = s["acc"].shape
    t = torch.arange(cap, device=DEV)
    n = s["comp_len"].long()[:, None, None]
    key = torch.where(t < n, s["acc"], -math.inf)
    key = torch.where((t < n) & (t >= n - recent), math.inf, key)   # the newest are always kept
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    m = torch.minimum(n, torch.full_like(n, keep))
    j = torch.arange(order.shape[-1], device=DEV)
    kept = torch.where(j < m, order, cap).sort(-1).values
    live = j < m
    at = torch.where(live, kept, 0)

    def move(src, dst):
        w = (live if src.dim() == 3 else live[..., None])
        i = at if src.dim() == 3 else at[..., None].expand(*at.shape, src.shape[-1])
        dst[:, :, :keep] = torch.where(w, torch.gather(src, 2, i), dst[:, :, :keep])

    move(s["k_codes"], s["k_out"])
    move(s["v_codes"], s["v_out"])
    move(torch.where(t < n, s["acc"], 0.0), s["acc_out"])
    s["acc_out"] *= torch.arange(s["acc_out"].shape[-1], device=DEV) < m   # tokens to come start at zero
    s["len_out"].copy_(m[:, 0, 0])
    s["kept"].copy_(torch.where(live, kept, -1))
    return [s[k] for k in ("k_out", "v_out", "acc_out", "len_out", "kept")]


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------

def _step(s):
    """The package's call of this case with its arguments set up once, as a serving loop keeps it."""
    if "step" not in s:
        from compressed_decode_attention_zkv_b200 import zkv
        c = s["case"]
        for x in ("k_codes", "v_codes"):     # the package takes pools whose pages lie one by one
            s[x + "_pool"] = s[x].contiguous() if x in s else None
        if c["op"] == "tree":
            s["step"] = zkv.PreparedTreeAttn(
                s["q"], s["draft_k"], s["draft_v"], s["k_codes_pool"], s["v_codes_pool"], s["comp_len"], s["Ck"],
                s["Cv"], s["win_k"], s["win_v"], s["win_len"], mask=s["mask"], n_draft=s["n_draft"],
                out=s["out"], lse=s["lse"], max_comp_len=c["T"], block_table=s["table"])
        elif c["op"] == "commit":
            comp, wl, head = s["lengths"]
            s["step"] = zkv.PreparedTreeCommit(
                s["draft_k"], s["draft_v"], s["path"], s["n_accept"], s["win_k"], s["win_v"], wl, head,
                comp, s["k_codes"], s["v_codes"], s["Ck"], s["Cv"])
        elif c["op"] == "weights":
            s["step"] = zkv.PreparedAccumulate(
                s["q"], s["lse"], s["k_codes_pool"], s["comp_len"], s["Ck"], s["acc"], max_comp_len=c["T"],
                block_table=s["table"])
        else:
            s["step"] = zkv.PreparedEvict(
                s["k_codes"], s["v_codes"], s["comp_len"], s["acc"], c["keep"], recent=c["recent"],
                k_out=s["k_out"], v_out=s["v_out"], len_out=s["len_out"], acc_out=s["acc_out"],
                kept=s["kept"])
    return s["step"]


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "commit":
        s["lengths"].copy_(s["before"])      # the loop goes back to where the drafts were made
    if own:
        step = _step(s)
        for x in ("k_codes", "v_codes"):     # pools that lie otherwise are laid out in every pass
            if x in s and not s[x].is_contiguous():
                s[x + "_pool"].copy_(s[x])
        step()
    if op == "tree":
        return (s["out"], s["lse"]) if own else _tree(s)
    if op == "commit":
        return [s[k] for k in ("k_codes", "v_codes", "win_k", "win_v", "lengths")] if own else _commit(s)
    if op == "weights":
        return s["acc"] if own else _weights(s)
    return [s[k] for k in ("k_out", "v_out", "acc_out", "len_out", "kept")] if own else _evict(s)


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits (numpy and float64), sequence by sequence
# ---------------------------------------------------------------------------------------------

def _walsh(d):
    h = np.ones((1, 1))
    while len(h) < d:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(d)


def _keys64(s, kind, b, h, n):
    """The first n vectors of one sequence and head in the model's own domain, float64."""
    codes, table = s[kind + "_codes"], s["table"]
    if table is not None:
        codes = codes[table[b].long(), h].flatten(0, 1)[:n]
    else:
        codes = codes[b, h, :n]
    books = s["C" + kind][h].double()
    x = torch.zeros((n, books.shape[-1]), dtype=torch.float64, device=DEV)
    for st in range(books.shape[0]):
        x += books[st][codes[:, st].long()]
    return x @ torch.from_numpy(_walsh(books.shape[-1])).to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "tree":
        B, N, Hq, d = s["q"].shape
        G = Hq // c["Hkv"]
        out, lse = s["out"].double(), s["lse"].double()
        for b in range(B):
            n, w, m = int(s["comp_len"][b]), int(s["win_len"][b]), int(s["n_draft"][b])
            see = torch.tril(torch.ones((m, m), dtype=torch.bool, device=DEV))
            if s["mask"] is not None:
                see = s["mask"][b, :m, :m]
            see = torch.cat([torch.ones((m, n + w), dtype=torch.bool, device=DEV), see], 1)
            for h in range(c["Hkv"]):
                k = torch.cat([_keys64(s, "k", b, h, n), s["win_k"][b, h, :w].double(), s["draft_k"][b, :m, h].double()])
                v = torch.cat([_keys64(s, "v", b, h, n), s["win_v"][b, h, :w].double(), s["draft_v"][b, :m, h].double()])
                for g in range(h * G, (h + 1) * G):
                    x = s["q"][b, :m, g].double() @ k.T / math.sqrt(d)
                    x = x.masked_fill(~see, -math.inf)
                    l = torch.logsumexp(x, 1)
                    e = torch.exp(x - l[:, None])
                    out[b, :m, g] = torch.nan_to_num(e @ v, nan=0.0)
                    lse[b, :m, g] = l
        return out, lse
    if c["op"] == "weights":
        B, N, Hq, d = s["q"].shape
        G = Hq // c["Hkv"]
        acc = s["acc"].double()
        for b in range(B):
            n = int(s["comp_len"][b])
            for h in range(c["Hkv"]):
                k = _keys64(s, "k", b, h, n)
                q = s["q"][b, :, h * G:(h + 1) * G].reshape(-1, d).double()
                l = s["lse"][b, :, h * G:(h + 1) * G].reshape(-1, 1).double()
                acc[b, h, :n] += torch.exp(q @ k.T / math.sqrt(d) - l).sum(0)
        return acc
    if c["op"] == "commit":
        return [None, None, s_win(s, "k"), s_win(s, "v"), None]
    return [None, None, evicted_totals(s), None, None]


def s_win(s, kind):
    """The windows after the accepted tokens were put in one after another."""
    win = s["win_" + kind].double().cpu().numpy()
    new = s["draft_" + kind].double().cpu().numpy()
    path, count = s["path"].cpu().numpy(), s["n_accept"].cpu().numpy()
    _, wl, head = s["before"].cpu().numpy().astype(int)
    W = win.shape[2]
    for b in range(len(win)):
        for i in range(count[b]):
            if wl[b] < W:
                at = wl[b]
                wl[b] += 1
            else:
                at = head[b]
                head[b] = (head[b] + 1) % W
            win[b, :, at] = new[b, path[b, i]]
    return torch.from_numpy(win)


def evicted_totals(s):
    """The totals of the kept tokens, in their order."""
    c = s["case"]
    acc, n = s["acc"].double().cpu().numpy(), s["comp_len"].cpu().numpy()
    out = s["acc_out"].double().cpu().numpy()
    for b in range(acc.shape[0]):
        old = max(0, n[b] - c["recent"])
        heavy = max(0, min(n[b], c["keep"]) - (n[b] - old))
        for h in range(acc.shape[1]):
            best = np.lexsort((np.arange(old), -acc[b, h, :old]))[:heavy]
            kept = np.concatenate([np.sort(best), np.arange(old, n[b])])
            out[b, h, :len(kept)] = acc[b, h, kept]
    return torch.from_numpy(out)
