"""An infinity reaches every later token of its channel as in the formula, however a walk
is divided: a gate above 0 keeps it, a gate of 0 makes it NaN, a negative one turns its
sign.  Products of many small gates underflow fp32, so a map made of such a product must
not turn an infinite state into NaN.  The gates below underflow within a step of 16
tokens (1e-4), within a CTA's 128 or a segment's 64 and more (0.05 to 0.3), or not at all
(0.9); the expected values are the fp64 oracle's, where none of the products occurs.
Channels without an infinity keep the recurrence's bound."""
import numpy as np
import pytest
import torch

from oracle import rows
from test_gpu_parity import la  # noqa: F401
from test_gpu_scan import BF, F32, c, check_bwd, check_fwd, make, np64

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value encountered")]   # 0 times an infinity

# (B, T, D): two kernels with tiles, two kernels without, teams of 4, of 2 and of 1 CTA
# (fewer than 64 blocks of 64 channels; 64 to 74; 75 to 148; up to 295), one warp a walk
SHAPES = [(1, 4000, 64), (1, 3000, 33), (1, 1500, 4096), (1, 1300, 4800), (4, 600, 4096), (2, 400, 72)]
AT = 37                     # the infinity's token, counted in the direction of the walk


def gates(seed, B, T, D, size, gt):
    gen = torch.Generator().manual_seed(seed)
    a = size * (0.5 + torch.rand(B, T, D, generator=gen) / 2)
    return a.to(gt)


def classes(t):
    """-1, 1: an infinity of that sign, 2: NaN, 0: finite."""
    t = np64(t) if torch.is_tensor(t) else t
    return np.where(np.isnan(t), 2, np.where(np.isinf(t), np.sign(t), 0)).astype(int)


def picked(t, ch):
    return None if t is None else t[..., ch.to(t.device)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("size", [1e-4, 0.1, 0.3, 0.9])
@pytest.mark.parametrize("form,xt,gt", [("value", BF, F32), ("logit", BF, BF), ("signed", F32, F32)])
def test_infinity_as_in_the_formula(la, shape, size, form, xt, gt):
    B, T, D = shape
    b = B - 1
    p = make(T + D, B, T, D, xt, gt)
    a = gates(T, B, T, D, size, F32)
    gate = "logit" if form == "logit" else "value"
    tied = form == "logit"
    if form == "logit":
        p["g"] = torch.log(a / (1 - a)).to(gt)
    else:
        p["g"] = (torch.where(torch.rand(a.shape, generator=torch.Generator().manual_seed(5)) < 0.5, -a, a)
                  if form == "signed" else a).to(gt)
    inf = float("inf")
    x, dh, h0, dl, g = p["x"], p["dh"], p["h0"], p["dl"], p["g"]
    x[b, AT, 5], x[b, AT, 6], h0[b, 9] = inf, -inf, inf
    dh[b, T - 1 - AT, 5], dh[b, T - 1 - AT, 6], dl[b, 9] = inf, -inf, -inf
    if gate == "value":     # a gate of 0 long after (and, backward, long before) the infinity
        x[b, AT, 20] = dh[b, T - 1 - AT, 20] = inf
        g[b, T // 2, 20] = 0.0
    ch = torch.tensor([0, 1, 4, 5, 6, 7, 8, 9, 10, 19, 20, 21, D - 2, D - 1])
    one = lambda t: None if t is None else picked(t, ch)[b:b + 1]  # noqa: E731

    h, last = la.scan_fwd(c(x), c(g), c(h0), gate=gate, tied=tied)
    want, wl = rows.scan_fwd(one(x), one(g), one(h0), gate, tied)
    assert np.array_equal(classes(one(h)), classes(want))
    assert np.array_equal(classes(one(last)), classes(wl))
    fine = torch.from_numpy(~classes(want).any((0, 1)))
    assert int(fine.sum()) >= 8
    f = lambda t: one(t)[..., fine.to(t.device)]  # noqa: E731
    check_fwd(f(h), f(last), f(x), f(g), f(h0), gate, tied, "fwd")

    # backward, with finite stored outputs
    xf = p["x"].clone()
    xf[b, AT, 5] = xf[b, AT, 6] = xf[b, AT, 20] = 1.0
    hf0 = h0.clone()
    hf0[b, 9] = 1.0
    hs, _ = la.scan_fwd(c(xf), c(g), c(hf0), gate=gate, tied=tied)
    dx, dg, dh0 = la.scan_bwd(c(g), hs, c(dh), x=c(xf) if tied else None, h0=c(hf0), dh_last=c(dl), gate=gate, tied=tied)
    rx, rg, r0 = rows.scan_bwd(one(g), one(hs), one(dh), one(xf) if tied else None, one(hf0), one(dl), gate, tied)
    for got, ref in ((dx, rx), (dg, rg), (dh0, r0)):
        assert np.array_equal(classes(one(got)), classes(ref))
    check_bwd((f(dx), f(dg), f(dh0)), f(g), f(hs), f(dh), f(xf) if tied else None, f(hf0), f(dl), gate, tied, "bwd")
    la.check_device()


@pytest.mark.parametrize("D", [64, 33, 4096])
def test_infinity_in_packed_sequences(la, D):
    """The infinity of a sequence that spans segments and rounds ends with it."""
    lens = [40, 1700, 0, 300, 900]
    n, T = len(lens), sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64)
    p = make(D, 1, T, D)
    p["g"] = gates(3, 1, T, D, 0.2, F32)
    st = make(D + 1, n, 1, D)
    p["x"][0, 45, 5] = float("inf")
    st["h0"][4, 7] = -float("inf")
    h, last = la.scan_fwd(c(p["x"]), c(p["g"]), c(st["h0"]), cu_seqlens=cu.cuda(), max_seqlen=max(lens))
    la.check_device()
    ch = torch.tensor([4, 5, 6, 7, D - 1])
    for i in range(n):
        s = slice(int(cu[i]), int(cu[i + 1]))
        want, wl = rows.scan_fwd(p["x"][:, s][..., ch], p["g"][:, s][..., ch], st["h0"][i:i + 1][:, ch])
        assert np.array_equal(classes(h[:, s][..., ch.cuda()]), classes(want)), i
        assert np.array_equal(classes(last[i:i + 1][:, ch.cuda()]), classes(wl)), i
