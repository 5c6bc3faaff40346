"""Tree attention against float64 in the 2-norm, and contexts whose border tokens carry the output.

A score is a sum of table entries; an entry's split product leaves out at most 2^-22 of |q| |c| softmax_scale
(and its sums less than that), so scores are off by eps = 2^-22 |q| sum over stages of max |c_s|
softmax_scale at most.  Errors of the scores move the weights against one another: 2 eps of the output's
norm, with 2^-20 for the roundings of weights, values and sums.  lse: eps, and four roundings of its own."""
import math

import numpy as np
import pytest
import torch

from compressed_decode_attention_zkv_b200 import build as B
from compressed_decode_attention_zkv_b200 import zkv
from test_gpu_tree import CASES, gpu_args, gpu_kw, make, plain, tree_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.build()
    zkv.lib()


def check(c):
    out, lse = zkv.rvq_tree_attn(*gpu_args(c), **gpu_kw(c))
    wo, wl, _, _ = plain(c)
    live = np.arange(c["N"])[None] < c["nd"][:, None]
    eps = 2.0 ** -22 * np.linalg.norm(c["q"].astype(np.float64), axis=-1).max() / math.sqrt(c["d"]) \
        * sum(np.linalg.norm(c["Ck"][:, s], axis=-1).max() for s in range(c["Sk"]))
    o, w = out.double().cpu().numpy()[live], wo[live]
    assert np.linalg.norm(o - w) <= (2 * eps + 2.0 ** -20) * np.linalg.norm(w)
    l, m = lse.double().cpu().numpy()[live], wl[live]
    assert np.array_equal(np.isinf(l), np.isinf(m))
    fin = np.isfinite(m)
    assert np.abs(l[fin] - m[fin]).max(initial=0) <= eps + 4 * 2.0 ** -24 * np.abs(m[fin]).max(initial=1) + 2.0 ** -20
    return o


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_norms(name, tree):
    c = make(91, **CASES[name])
    if tree:
        c["mask"] = tree_mask(c["rng"], c["B"], c["N"])
    check(c)


@pytest.mark.parametrize("what", ["window", "drafts", "first", "last", "unit"])
def test_border_tokens_carry_the_output(what):
    """Values a thousand times larger in the window, the drafts, the first or last tokens of the prefix or
    those beside a border of its units: leaving them out would change the output by tens of per cent."""
    T = (20000, 9001)
    c = make(92, B=2, N=3, Hq=4, Hkv=2, d=128, Sk=4, Sv=4, Tcap=20000, comp=T, W=16, win=[16, 11])
    c["Cv"][:, 0, 255] *= 1000
    c["vc"][..., 0] %= 255                   # the large codeword is used where it is put
    if what == "window":
        c["wv"] *= 1000
    elif what == "drafts":
        c["dv"] *= 1000
    for b in range(2):
        at = dict(first=[0], last=[T[b] - 1], unit=[127, 128, 8 * 128, T[b] // 128 * 128]).get(what, [])
        c["vc"][b][:, at, 0] = 255
    check(c)
