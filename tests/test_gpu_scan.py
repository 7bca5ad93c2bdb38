"""The gated linear recurrence on the GPU (la_scan_fwd, la_scan_bwd, la_scan_step)
against the fp64 oracle on the same inputs, element by element.

Bounds.  With u = 2^-24 (half a step of fp32), every token adds a rounding error of
at most C u m_t to the state, where m_t = |a_t| m_{t-1} + |u_t| bounds the state and
its partial sums, and earlier errors decay as the state does:
    E_t = |a_t| E_{t-1} + C u m_t.
C counts what a token's own recurrence and its share of the composed maps cost: the
fused multiply-add, the product of gates and their composition over the levels (run,
warp, CTA, cluster), a few roundings each: C = 12.  A logit adds the error of the
sigmoid: exp(-|l|) is good to 2 + 1.173 |l| steps (the documented bound of the fast
exponential), the quotient to 2 steps; with |l| <= 9 that is at most
2 (2 + 10.6 + 2) + 4 < 36 half steps in the smaller of a and 1 - a: C = 48.
Stored results add their own rounding, eps / 2 of the output type relative to the
value.  The gradients follow the same recurrence backwards on |dh|; the products that
make dx and dg are each a handful of roundings, covered by C u once more.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import rows
from test_gpu_parity import la  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
FORMS = [(gate, tied) for gate in ("value", "logit") for tied in (False, True)]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2 if dtype is BF else 0.0


def np64(t):
    return t.detach().double().cpu().numpy()


def make(seed, B, T, D, xt=BF, gt=F32, gate="value"):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    l = (rn(B, T, D) + 2.0).clamp(-9.0, 9.0)
    g = (l if gate == "logit" else torch.sigmoid(l)).to(gt)
    return dict(x=rn(B, T, D).to(xt), g=g, h0=rn(B, D), dh=rn(B, T, D).to(xt), dl=rn(B, D))


def fwd_bound(x, g, h0, gate, tied):
    """E_t of the text for every token, and the oracle's h and h_last."""
    a, r = rows.gates(g, gate)
    x = np.abs(np64(x))
    u = r * x if tied else x
    C = 48 if gate == "logit" else 12
    m = np.abs(np64(h0)) if h0 is not None else np.zeros((x.shape[0], x.shape[2]))
    E, out = np.zeros_like(m), np.zeros_like(x)
    for t in range(x.shape[1]):
        m = np.abs(a[:, t]) * m + u[:, t]
        E = np.abs(a[:, t]) * E + C * U * m
        out[:, t] = E
    return out, E


def check_fwd(h, h_last, x, g, h0, gate, tied, what=""):
    rh, rl = rows.scan_fwd(x, g, h0, gate, tied)
    E, last = fwd_bound(x, g, h0, gate, tied)
    tol = E + half_step(h.dtype) * (np.abs(rh) + E) + 1e-37
    d = np.abs(np64(h) - rh)
    assert np.all(d <= tol), (what, float((d / tol).max()))
    if h_last is not None:
        d = np.abs(np64(h_last) - rl)
        assert np.all(d <= last + 1e-37), (what, float((d / (last + 1e-37)).max()))


def check_bwd(got, g, h, dh, x, h0, dl, gate, tied, what=""):
    dx, dg, dh0 = got
    ref = rows.scan_bwd(g, h, dh, x, h0, dl, gate, tied)
    a, r = rows.gates(g, gate)
    C = 48 if gate == "logit" else 12
    B, T, D = a.shape
    m = np.abs(np64(dl)) if dl is not None else np.zeros((B, D))
    E = np.zeros((B, D))
    hp = np.zeros((B, T, D))
    hp[:, 1:] = np.abs(np64(h))[:, :-1]
    if h0 is not None and T:
        hp[:, 0] = np.abs(np64(h0))
    if tied:
        hp = hp + np.abs(np64(x))
    for t in range(T - 1, -1, -1):
        mG = np.abs(np64(dh[:, t])) + m
        EG = E + C * U * mG
        m, E = np.abs(a[:, t]) * mG, np.abs(a[:, t]) * EG + C * U * np.abs(a[:, t]) * mG
        f = np.abs(r[:, t]) if tied else 1.0
        tol = f * (EG + C * U * mG)
        tol = tol + half_step(dx.dtype) * (np.abs(ref[0][:, t]) + tol) + 1e-37
        d = np.abs(np64(dx[:, t]) - ref[0][:, t])
        assert np.all(d <= tol), (what, "dx", t, float((d / tol).max()))
        f = np.abs(a[:, t] * r[:, t]) if gate == "logit" else 1.0
        tol = f * hp[:, t] * (EG + 2 * C * U * mG)
        tol = tol + half_step(dg.dtype) * (np.abs(ref[1][:, t]) + tol) + 1e-37
        d = np.abs(np64(dg[:, t]) - ref[1][:, t])
        assert np.all(d <= tol), (what, "dg", t, float((d / tol).max()))
    if dh0 is not None:
        d = np.abs(np64(dh0) - ref[2])
        assert np.all(d <= E + 1e-37), (what, "dh0", float((d / (E + 1e-37)).max()))


def c(t):
    return None if t is None else t.cuda()


def run_both(la, p, gate, tied, state=True, **kw):
    """Forward and backward on the GPU, checked against the oracle."""
    h0, dl = (p["h0"], p["dl"]) if state else (None, None)
    h, last = la.scan_fwd(c(p["x"]), c(p["g"]), c(h0), gate=gate, tied=tied, **kw)
    check_fwd(h, last, p["x"], p["g"], h0, gate, tied, "fwd")
    got = la.scan_bwd(c(p["g"]), h, c(p["dh"]), x=c(p["x"]) if tied else None, h0=c(h0), dh_last=c(dl),
                      gate=gate, tied=tied, **kw)
    check_bwd(got, p["g"], h, p["dh"], p["x"], h0, dl, gate, tied, "bwd")
    la.check_device()
    return h, last, got


# lengths around a run (4 or 8 tokens), a CTA's tokens (64 and more), a cluster's,
# one token and none; channel counts that are one group, odd, ragged against a CTA
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (1, 1, 64), (3, 2, 5), (2, 3, 64), (1, 4, 4), (2, 5, 8), (1, 63, 36),
                                   (2, 64, 64), (1, 65, 100), (3, 130, 33), (1, 257, 132), (2, 1000, 20),
                                   (1, 1025, 64), (5, 517, 7), (1, 4100, 4), (1, 4099, 3)])
@pytest.mark.parametrize("gate,tied", FORMS)
def test_scan_matches_oracle(la, B, T, D, gate, tied):
    run_both(la, make(B + 10 * T + D, B, T, D, gate=gate), gate, tied)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("gt", [BF, F32])
@pytest.mark.parametrize("gate,tied", FORMS)
@pytest.mark.parametrize("D", [24, 25])
def test_scan_types(la, xt, gt, gate, tied, D):
    run_both(la, make(D, 2, 300, D, xt, gt, gate), gate, tied)


@pytest.mark.parametrize("state", [False, True])
def test_scan_many_channels_walk_in_one_cta(la, state):
    """Enough channel blocks that no cluster is formed and each CTA walks its sequence."""
    run_both(la, make(3, 20, 150, 2048), "value", False, state)
    run_both(la, make(4, 40, 75, 515, gate="logit"), "logit", True, state)


def test_scan_long_sequence(la):
    """The longest cluster walk: 16 CTAs, many steps, state carried through all of them."""
    run_both(la, make(5, 1, 20000, 16), "value", False)
    run_both(la, make(6, 1, 12345, 3, F32, F32, "logit"), "logit", True)


def test_scan_without_state(la):
    p = make(7, 2, 100, 16)
    h, last = la.scan_fwd(c(p["x"]), c(p["g"]), want_state=False)
    assert last is None
    check_fwd(h, None, p["x"], p["g"], None, "value", False)
    dx, dg, dh0 = la.scan_bwd(c(p["g"]), h, c(p["dh"]), want_state=False)
    assert dh0 is None
    check_bwd((dx, dg, None), p["g"], h, p["dh"], None, None, None, "value", False)


def test_scan_no_tokens(la):
    """T = 0: the state passes through in both directions."""
    x = torch.empty(2, 0, 8, dtype=BF, device="cuda")
    g = torch.empty(2, 0, 8, device="cuda")
    s = torch.randn(2, 8, device="cuda")
    h, last = la.scan_fwd(x, g, s)
    assert h.shape == (2, 0, 8) and torch.equal(last, s)
    assert torch.equal(la.scan_fwd(x, g)[1], torch.zeros_like(s))
    dx, dg, dh0 = la.scan_bwd(g, h, x, dh_last=s)
    assert dx.shape == (2, 0, 8) and torch.equal(dh0, s)


def test_scan_split_equals_whole(la):
    """A prefix scanned, carried and continued gives the whole scan, within the bound."""
    p = make(8, 2, 700, 40)
    whole, last = la.scan_fwd(c(p["x"]), c(p["g"]), c(p["h0"]))
    for cut in (1, 64, 333):
        h1, mid = la.scan_fwd(c(p["x"][:, :cut].contiguous()), c(p["g"][:, :cut].contiguous()), c(p["h0"]))
        h2, end = la.scan_fwd(c(p["x"][:, cut:].contiguous()), c(p["g"][:, cut:].contiguous()), mid)
        E, El = fwd_bound(p["x"], p["g"], p["h0"], "value", False)
        both = np64(torch.cat([h1, h2], 1))
        assert np.all(np.abs(both - np64(whole)) <= 2 * (E + half_step(BF) * (np.abs(np64(whole)) + E)) + 1e-37)
        assert np.all(np.abs(np64(end) - np64(last)) <= 2 * El)


def test_scan_heads_and_slices(la):
    """[B,T,H,d] tensors, and slices of one projection with unaligned starts, in and out."""
    B, T, H, d = 2, 70, 3, 8
    p = make(9, B, T, H * d, BF, BF, "logit")
    v = lambda t: c(t).view(*t.shape[:-1], H, d)  # noqa: E731
    h, last = la.scan_fwd(v(p["x"]), v(p["g"]), v(p["h0"]), gate="logit", tied=True)
    assert h.shape == (B, T, H, d) and last.shape == (B, H, d)
    flat, flast = la.scan_fwd(c(p["x"]), c(p["g"]), c(p["h0"]), gate="logit", tied=True)
    assert torch.equal(h.flatten(2), flat) and torch.equal(last.flatten(1), flast)
    D = H * d
    for pad in (0, 1, 4):
        proj = torch.full((B, T, 2 * D + 3 * pad), float("nan"), dtype=BF, device="cuda")
        xs, gs = proj[..., pad:pad + D], proj[..., 2 * pad + D:2 * pad + 2 * D]
        xs.copy_(c(p["x"]))
        gs.copy_(c(p["g"]))
        out = torch.full((B, T, D + 2 * pad), 7.0, dtype=BF, device="cuda")
        hs, ls = la.scan_fwd(xs, gs, c(p["h0"]), gate="logit", tied=True, h=out[..., pad:pad + D])
        check_fwd(hs, ls, p["x"], p["g"], p["h0"], "logit", True, pad)
        if pad:
            assert torch.all(out[..., :pad] == 7.0) and torch.all(out[..., pad + D:] == 7.0)
        dout = torch.full((B, T, 2 * D + 3 * pad), 7.0, dtype=BF, device="cuda")
        got = la.scan_bwd(gs, hs, c(p["dh"]), x=xs, h0=c(p["h0"]), dh_last=c(p["dl"]), gate="logit", tied=True,
                          dx=dout[..., pad:pad + D], dg=dout[..., 2 * pad + D:2 * pad + 2 * D])
        check_bwd(got, p["g"], hs, p["dh"], p["x"], p["h0"], p["dl"], "logit", True, pad)
        if pad:
            assert torch.all(dout[..., :pad] == 7.0) and torch.all(dout[..., 2 * pad + 2 * D:] == 7.0)


LENGTHS = [1, 64, 0, 65, 200, 517, 3, 128, 0]


@pytest.mark.parametrize("D,gate,tied", [(64, "value", False), (33, "logit", True), (600, "logit", False), (4, "value", True)])
def test_scan_packed(la, D, gate, tied):
    """Packed sequences equal their own oracle runs; an empty one passes its state
    on; tokens of no sequence stay as they were."""
    n, total, extra = len(LENGTHS), sum(LENGTHS), 5
    p = make(11 + D, 1, total + extra, D, BF, F32, gate)
    st = make(12 + D, n, 1, D)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(LENGTHS)]), dtype=torch.int64)
    h = torch.full((1, total + extra, D), 9.0, dtype=BF, device="cuda")
    kw = dict(gate=gate, tied=tied, cu_seqlens=cu.cuda(), max_seqlen=max(LENGTHS))
    _, last = la.scan_fwd(c(p["x"]), c(p["g"]), c(st["h0"]), h=h, **kw)
    dx, dg = torch.full_like(h, 9.0), torch.full((1, total + extra, D), 9.0, device="cuda")
    _, _, dh0 = la.scan_bwd(c(p["g"]), h, c(p["dh"]), x=c(p["x"]) if tied else None, h0=c(st["h0"]),
                            dh_last=c(st["dl"]), dx=dx, dg=dg, **kw)
    la.check_device()
    for i in range(n):
        s = slice(int(cu[i]), int(cu[i + 1]))
        one = lambda t: t[:, s]  # noqa: E731
        h0, dl = st["h0"][i:i + 1], st["dl"][i:i + 1]
        check_fwd(h[:, s], last[i:i + 1], one(p["x"]), one(p["g"]), h0, gate, tied, i)
        check_bwd((dx[:, s], dg[:, s], dh0[i:i + 1]), one(p["g"]), h[:, s], one(p["dh"]), one(p["x"]), h0, dl,
                  gate, tied, i)
    assert torch.all(h[:, total:] == 9.0) and torch.all(dx[:, total:] == 9.0) and torch.all(dg[:, total:] == 9.0)


def test_scan_packed_bad_offsets_are_reported(la):
    """Offsets out of order or out of range, or a sequence longer than max_seqlen,
    are clamped (no access leaves the tensors) and reported."""
    p = make(13, 1, 100, 16)
    x, g = c(p["x"]), c(p["g"])
    for cu, ms in (([0, 60, 40, 100], 100), ([0, 50, 300], 100), ([-7, 50], 100), ([0, 100], 30)):
        cu = torch.tensor(cu, dtype=torch.int64, device="cuda")
        h, _ = la.scan_fwd(x, g, cu_seqlens=cu, max_seqlen=ms)
        with pytest.raises(la.LAError) as e:
            la.check_device()
        assert e.value.status == 1
        la.scan_bwd(g, h, x, cu_seqlens=cu, max_seqlen=ms)
        with pytest.raises(la.LAError):
            la.check_device()
    la.check_device()


def test_scan_state_in_place(la):
    """h_last may be h0, dh0 may be dh_last: long clusters and single CTAs."""
    for B, T, D in ((1, 3000, 8), (30, 100, 1024)):
        p = make(14, B, T, D)
        h, last = la.scan_fwd(c(p["x"]), c(p["g"]), c(p["h0"]))
        s = c(p["h0"])
        h2, l2 = la.scan_fwd(c(p["x"]), c(p["g"]), s, h_last=s)
        assert l2 is s and torch.equal(h, h2) and torch.equal(last, s)
        _, _, d0 = la.scan_bwd(c(p["g"]), h, c(p["dh"]), h0=c(p["h0"]), dh_last=c(p["dl"]))
        s = c(p["dl"])
        la.scan_bwd(c(p["g"]), h, c(p["dh"]), h0=c(p["h0"]), dh_last=s, dh0=s)
        assert torch.equal(d0, s)


@pytest.mark.parametrize("B,T,D", [(1, 2000, 8), (2, 300, 33), (30, 80, 1024)])
def test_scan_same_bits_again(la, B, T, D):
    p = make(15, B, T, D, BF, BF, "logit")
    x, g, dh = c(p["x"]), c(p["g"]), c(p["dh"])
    first = la.scan_fwd(x, g, gate="logit", tied=True)
    fb = la.scan_bwd(g, first[0], dh, x=x, gate="logit", tied=True)
    for _ in range(3):
        again = la.scan_fwd(x, g, gate="logit", tied=True)
        assert all(torch.equal(i, j) for i, j in zip(first, again))
        assert all(torch.equal(i, j) for i, j in zip(fb, la.scan_bwd(g, first[0], dh, x=x, gate="logit", tied=True)))


@pytest.mark.parametrize("D", [8, 9])
def test_scan_zero_and_open_gates(la, D):
    """a = 0 forgets, a = 1 keeps (a plain sum); logits of any size give no NaN."""
    p = make(16, 1, 500, D)
    a = torch.zeros(1, 500, D)
    a[:, 1::3] = 1.0
    p["g"] = a
    run_both(la, p, "value", False)
    run_both(la, p, "value", True)
    h, _ = la.scan_fwd(c(p["x"]), torch.zeros(1, 500, D, device="cuda"))
    assert torch.equal(h.cpu(), p["x"])
    big = torch.tensor([-1e30, -200.0, 200.0, 1e30, float("inf"), -float("inf")], device="cuda")
    g = big[torch.randint(0, 6, (1, 500, D), generator=torch.Generator().manual_seed(1))]
    h, last = la.scan_fwd(c(p["x"]), g, c(p["h0"]), gate="logit", tied=True)
    want, wl = rows.scan_fwd(p["x"], (g > 0).float(), p["h0"], "value", True)
    # sigmoid(+-200) is 1 or 0 to fp32, so the state is kept or replaced as it is
    assert np.all(np.abs(np64(h) - want) <= half_step(BF) * np.abs(want)) and np.array_equal(np64(last), wl)
    got = la.scan_bwd(g, h, c(p["dh"]), x=c(p["x"]), h0=c(p["h0"]), gate="logit", tied=True)
    assert all(torch.isfinite(t).all() for t in got)
    assert torch.all(got[1] == 0)


@pytest.mark.parametrize("D,T", [(8, 900), (9, 300), (64, 50)])
def test_scan_nan_stays_in_its_channel(la, D, T):
    """A NaN or infinity reaches its own channel, from its token on, and nothing
    else; the backward pass carries one to the tokens before it."""
    p = make(17, 2, T, D)
    clean, last = la.scan_fwd(c(p["x"]), c(p["g"]), c(p["h0"]))
    for name in ("x", "g"):
        q = {k: v.clone() for k, v in p.items()}
        q[name][1, 37, 5] = float("nan")
        h, l = la.scan_fwd(c(q["x"]), c(q["g"]), c(q["h0"]))
        assert torch.isnan(h[1, 37:, 5]).all() and torch.isnan(l[1, 5])
        h[1, 37:, 5] = clean[1, 37:, 5]
        l[1, 5] = last[1, 5]
        assert torch.equal(h, clean) and torch.equal(l, last)
    q = {k: v.clone() for k, v in p.items()}
    q["x"][1, 37, 5] = float("inf")
    h, _ = la.scan_fwd(c(q["x"]), c(q["g"]), c(q["h0"]))
    assert torch.isposinf(h[1, 37, 5]) and torch.equal(h[1, :37], clean[1, :37]) and torch.equal(h[0], clean[0])
    ref = la.scan_bwd(c(p["g"]), clean, c(p["dh"]), h0=c(p["h0"]), dh_last=c(p["dl"]))
    q = p["dh"].clone()
    q[1, 37, 5] = float("nan")
    dx, dg, d0 = la.scan_bwd(c(p["g"]), clean, c(q), h0=c(p["h0"]), dh_last=c(p["dl"]))
    assert torch.isnan(dx[1, :38, 5]).all() and torch.isnan(d0[1, 5])
    for got, want in ((dx, ref[0]), (dg, ref[1])):
        got[1, :38, 5] = want[1, :38, 5]
        assert torch.equal(got, want)


def test_scan_offsets_past_32_bits(la):
    """Rows of a wide tensor: element offsets beyond 2^31."""
    T, W, D = 300, 8_000_000, 8
    wide = torch.empty(1, T, W, dtype=BF, device="cuda")
    assert T * W > 2 ** 31
    p = make(18, 1, T, D)
    x = wide[..., W - D:]
    x.copy_(c(p["x"]))
    out = wide[..., :D]
    h, last = la.scan_fwd(x, c(p["g"]), c(p["h0"]), h=out)
    check_fwd(h, last, p["x"], p["g"], p["h0"], "value", False)
    dx = wide[..., 64:64 + D]
    got = la.scan_bwd(c(p["g"]), h, x, h0=c(p["h0"]), dx=dx)
    check_bwd(got, p["g"], h, p["x"], None, p["h0"], None, "value", False)


@pytest.mark.parametrize("gate,tied", FORMS)
@pytest.mark.parametrize("xt,gt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 64), (5, 33), (300, 1028)])
def test_step_is_the_scan_of_one_token(la, gate, tied, xt, gt, N, D):
    p = make(N + D, N, 1, D, xt, gt, gate)
    s = c(p["h0"])
    h = la.scan_step(c(p["x"][:, 0].contiguous()), c(p["g"][:, 0].contiguous()), s, gate=gate, tied=tied)
    check_fwd(h[:, None], s, p["x"], p["g"], p["h0"], gate, tied)


def test_steps_follow_the_scan(la):
    """Prefill, then tokens one by one from slices of a projection, against the whole scan."""
    p = make(20, 3, 40, 24, BF, BF, "logit")
    E, El = fwd_bound(p["x"], p["g"], p["h0"], "logit", True)
    _, s = la.scan_fwd(c(p["x"][:, :30].contiguous()), c(p["g"][:, :30].contiguous()), c(p["h0"]), gate="logit", tied=True)
    want, last = rows.scan_fwd(p["x"], p["g"], p["h0"], "logit", True)
    for t in range(30, 40):
        proj = torch.cat([p["x"][:, t], torch.zeros(3, 1, dtype=BF), p["g"][:, t]], 1).cuda()
        out = torch.full((3, 27), 5.0, dtype=BF, device="cuda")
        h = la.scan_step(proj[:, :24], proj[:, 25:], s, gate="logit", tied=True, h=out[:, 1:25])
        assert np.all(np.abs(np64(h) - want[:, t]) <= E[:, t] + half_step(BF) * (np.abs(want[:, t]) + E[:, t]) + 1e-37)
        assert torch.all(out[:, 0] == 5.0) and torch.all(out[:, 25:] == 5.0)
    assert np.all(np.abs(np64(s) - last) <= El)


def test_scan_on_another_stream(la):
    p = make(21, 1, 5000, 32)
    want, wl = la.scan_fwd(c(p["x"]), c(p["g"]), c(p["h0"]))
    s = torch.cuda.Stream()
    x, g, h0 = c(p["x"]), c(p["g"]), c(p["h0"])
    s.wait_stream(torch.cuda.current_stream())
    h, last = la.scan_fwd(x, g, h0, stream=s)
    del x, g, h0                                   # their memory is kept for the queued work
    torch.empty(1 << 22, device="cuda").fill_(float("nan"))
    dh = c(p["dh"])
    s.wait_stream(torch.cuda.current_stream())
    got = la.scan_bwd(c(p["g"]), h, dh, stream=s)
    st = la.scan_step(dh[:, 0].contiguous(), dh[:, 1].float(), last.clone(), stream=s)
    s.synchronize()
    assert torch.equal(h, want) and torch.equal(last, wl) and torch.isfinite(st).all()
    ref = la.scan_bwd(c(p["g"]), want, c(p["dh"]))
    assert all(torch.equal(i, j) for i, j in zip(got, ref))


def test_scan_captured_and_replayed(la):
    """Forward, backward and step in one graph, replayed on new inputs, two graphs at once."""
    p, q = make(22, 1, 3000, 16), make(23, 1, 3000, 16)
    graphs = []
    for _ in range(2):
        b = {k: c(v) for k, v in p.items()}
        la.scan_fwd(b["x"], b["g"], b["h0"])
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            h, last = la.scan_fwd(b["x"], b["g"], b["h0"])
            d = la.scan_bwd(b["g"], h, b["dh"], h0=b["h0"], dh_last=b["dl"])
        graphs.append((gr, b, h, last, d))
    for k in ("x", "g", "h0", "dh", "dl"):
        graphs[1][1][k].copy_(q[k])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0][0].replay()
    with torch.cuda.stream(side):
        graphs[1][0].replay()
    torch.cuda.synchronize()
    for (gr, b, h, last, d), w in zip(graphs, (p, q)):
        check_fwd(h, last, w["x"], w["g"], w["h0"], "value", False)
        check_bwd(d, w["g"], h, w["dh"], None, w["h0"], w["dl"], "value", False)


def test_scan_gradients_are_differences_of_the_gpu_forward(la):
    """Central differences of the kernel's own forward pass (fp32), against its
    backward pass.  With step e the forward pass' rounding gives at most
    2 sum |dh| E_t / (2 e).  An output is linear in x and h0 and in each single gate
    a_i, so the truncation is e^2 / 6 of sigmoid's third derivative (at most 1 / 8) times
    |h_{i-1} - x_i| <= 2 M, M the largest of |x| and |h0| (a tied state stays between
    them): e^2 / 24 M sum |dh|."""
    p = make(24, 1, 6, 4, F32, F32, "logit")
    x, g, h0, dh = (c(p[k]) for k in ("x", "g", "h0", "dh"))
    h, _ = la.scan_fwd(x, g, h0, gate="logit", tied=True)
    dx, dg, dh0 = la.scan_bwd(g, h, dh, x=x, h0=h0, gate="logit", tied=True)
    E, _ = fwd_bound(p["x"], p["g"], p["h0"], "logit", True)
    e = 2.0 ** -5
    noise = float((np.abs(np64(dh)) * E).sum()) / e
    M = max(float(np.abs(np64(x)).max()) + e, float(np.abs(np64(h0)).max()) + e)
    trunc = e * e / 24 * M * float(np.abs(np64(dh)).sum())
    loss = lambda: float((la.scan_fwd(x, g, h0, gate="logit", tied=True)[0].double() * dh.double()).sum())  # noqa: E731
    for t, d in ((x, dx), (g, dg), (h0, dh0)):
        f, df = t.view(-1), d.view(-1)
        for i in range(f.numel()):
            keep = f[i].item()
            f[i] = keep + e
            up, hi = loss(), f[i].item()
            f[i] = keep - e
            down, lo = loss(), f[i].item()
            f[i] = keep
            assert abs((up - down) / (hi - lo) - df[i].item()) <= noise + trunc


def test_scan_refuses(la):
    p = make(25, 2, 8, 8)
    x, g, s = c(p["x"]), c(p["g"]), c(p["h0"])
    for bad in (dict(x=p["x"]), dict(g=g[:, :4]), dict(h0=s.double()), dict(h0=s[:1]), dict(g=g.half()),
                dict(gate="exp"), dict(g=g[:, :1].expand(2, 8, 8)), dict(x=x.transpose(0, 1)), dict(max_seqlen=4),
                dict(x=x.transpose(1, 2)), dict(cu_seqlens=torch.tensor([0, 8], device="cuda"), max_seqlen=8),
                dict(h_last=torch.empty(2, 8, dtype=BF, device="cuda"))):
        kw = dict(x=x, g=g, h0=s)
        kw.update(bad)
        with pytest.raises(ValueError):
            la.scan_fwd(**kw)
    h, _ = la.scan_fwd(x, g)
    with pytest.raises(ValueError):
        la.scan_bwd(g, h, x, tied=True)
    with pytest.raises(ValueError):
        la.scan_bwd(g, h.float(), x)
    with pytest.raises(ValueError):
        la.scan_step(x[:, 0], g[:, 0], None)
    with pytest.raises(ValueError):
        la.scan_fwd(x[:1], g[:1], cu_seqlens=torch.tensor([0, 8], dtype=torch.int32, device="cuda"), max_seqlen=8)


# The three ways of dividing a walk (whole walks, teams, maps and then outputs) at the
# channel counts that choose them, with sequences that start and end anywhere.
@pytest.mark.parametrize("D", [4096, 4104, 8192, 19008, 20])
@pytest.mark.parametrize("gate,tied", [("value", False), ("logit", True)])
def test_scan_packed_many_channels(la, D, gate, tied):
    lens = [1, 0, 15, 16, 17, 300, 2, 1, 1, 0, 129, 128, 640]
    n, total = len(lens), sum(lens)
    p = make(31 + D, 1, total, D, BF, BF if gate == "logit" else F32, gate)
    st = make(32 + D, n, 1, D)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64)
    kw = dict(gate=gate, tied=tied, cu_seqlens=cu.cuda(), max_seqlen=max(lens))
    s = c(st["h0"])
    h, last = la.scan_fwd(c(p["x"]), c(p["g"]), s, h_last=s, **kw)       # the state in place
    e = c(st["dl"])
    dx, dg, dh0 = la.scan_bwd(c(p["g"]), h, c(p["dh"]), x=c(p["x"]) if tied else None, h0=c(st["h0"]), dh_last=e,
                              dh0=e, **kw)
    la.check_device()
    pick = torch.randperm(D, generator=torch.Generator().manual_seed(D))[:24]     # the oracle's channels
    for i in range(n):
        sl = slice(int(cu[i]), int(cu[i + 1]))
        one = lambda t: t[:, sl][..., pick.to(t.device)]  # noqa: E731
        h0, dl = st["h0"][i:i + 1][:, pick], st["dl"][i:i + 1][:, pick]
        check_fwd(one(h), last[i:i + 1][:, pick.cuda()], one(p["x"]), one(p["g"]), h0, gate, tied, (i, lens[i]))
        check_bwd((one(dx), one(dg), dh0[i:i + 1][:, pick.cuda()]), one(p["g"]), one(h), one(p["dh"]), one(p["x"]), h0,
                  dl, gate, tied, (i, lens[i]))


def test_scan_thousands_of_sequences(la):
    """More sequences than one search step sees, most of them short, some empty."""
    gen = torch.Generator().manual_seed(33)
    lens = torch.randint(0, 6, (3000,), generator=gen)
    lens[1500] = 700
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    total, D = int(cu[-1]), 12
    p, st = make(34, 1, total, D), make(35, 3000, 1, D)
    h, last = la.scan_fwd(c(p["x"]), c(p["g"]), c(st["h0"]), cu_seqlens=cu.cuda(), max_seqlen=700)
    got = la.scan_bwd(c(p["g"]), h, c(p["dh"]), h0=c(st["h0"]), dh_last=c(st["dl"]), cu_seqlens=cu.cuda(), max_seqlen=700)
    la.check_device()
    for i in [0, 1, 2, 31, 32, 33, 1023, 1024, 1499, 1500, 1501, 2998, 2999] + list(range(700, 760)):
        s = slice(int(cu[i]), int(cu[i + 1]))
        check_fwd(h[:, s], last[i:i + 1], p["x"][:, s], p["g"][:, s], st["h0"][i:i + 1], "value", False, i)
        check_bwd((got[0][:, s], got[1][:, s], got[2][i:i + 1]), p["g"][:, s], h[:, s], p["dh"][:, s], None,
                  st["h0"][i:i + 1], st["dl"][i:i + 1], "value", False, i)


@pytest.mark.parametrize("B,T,D", [(300, 1, 40), (500, 7, 64), (130, 63, 72), (90, 64, 8), (2000, 3, 5)])
def test_scan_short_dense_sequences(la, B, T, D):
    """Short dense sequences are walked as one axis."""
    run_both(la, make(36 + B, B, T, D), "value", True)
    run_both(la, make(37 + B, B, T, D, BF, BF, "logit"), "logit", False, state=False)


def test_scan_odd_channels_in_aligned_rows(la):
    """A channel count that is no multiple of a tile in rows that are multiples of 16 bytes."""
    p = make(38, 1, 900, 1001, BF, F32)
    wide = lambda t, w: torch.full((1, 900, w), 7.0, dtype=t.dtype, device="cuda")  # noqa: E731
    x, g, out, dx, dg = wide(p["x"], 1008), wide(p["g"], 1004), wide(p["x"], 1016), wide(p["x"], 1008), wide(p["g"], 1004)
    x[..., :1001] = c(p["x"])
    g[..., :1001] = c(p["g"])
    h, last = la.scan_fwd(x[..., :1001], g[..., :1001], c(p["h0"]), h=out[..., :1001])
    check_fwd(h, last, p["x"], p["g"], p["h0"], "value", False)
    got = la.scan_bwd(g[..., :1001], h, c(p["dh"]), h0=c(p["h0"]), dh_last=c(p["dl"]), dx=dx[..., :1001], dg=dg[..., :1001])
    check_bwd(got, p["g"], h, p["dh"], None, p["h0"], p["dl"], "value", False)
    for t in (out, dx, dg):
        assert torch.all(t[..., 1001:] == 7.0)


@pytest.mark.parametrize("D,T", [(4096, 700), (8, 700), (20000, 40), (8, 3)])
def test_scan_infinity_stays_in_its_sequence(la, D, T):
    """What a sequence left, infinities and NaN included, does not reach the next one; a
    NaN gate of any bits makes its channel NaN to the end of its sequence."""
    cut = T // 2
    cu = torch.tensor([0, cut, T], dtype=torch.int64, device="cuda")
    p = make(39, 1, T, D)
    x, g = c(p["x"]), c(p["g"])
    clean, cl = la.scan_fwd(x, g, cu_seqlens=cu, max_seqlen=T)
    y = x.clone()
    y[0, 0, 1], y[0, cut - 1, 2] = float("inf"), float("nan")
    gg = g.clone()
    gg.view(torch.int32)[0, 0, 3] = 0x7FA5C31D
    h, last = la.scan_fwd(y, gg, cu_seqlens=cu, max_seqlen=T)
    assert torch.equal(h[0, cut:], clean[0, cut:]) and torch.equal(last[1], cl[1])
    assert torch.isnan(h[0, :cut, 3]).all() and torch.isnan(last[0, 3]) and torch.isinf(h[0, 0, 1])
    dh = x.clone()
    dh[0, T - 1, 1], dh[0, cut, 2] = float("inf"), float("nan")
    a = la.scan_bwd(g, clean, x, cu_seqlens=cu, max_seqlen=T)
    b = la.scan_bwd(g, clean, dh, cu_seqlens=cu, max_seqlen=T)
    assert torch.equal(a[0][0, :cut], b[0][0, :cut]) and torch.equal(a[2][0], b[2][0]) and torch.isnan(b[2][1, 2])


@pytest.mark.parametrize("D", [4096, 16])
def test_scan_two_at_once(la, D):
    """Two calls on two streams, whose CTAs share the SMs: each has scratch of its own."""
    ps = [make(40 + i, 1, 4000, D, BF, BF, "logit") for i in range(2)]
    dev = [{k: c(v) for k, v in p.items()} for p in ps]
    want = [la.scan_fwd(d["x"], d["g"], d["h0"], gate="logit", tied=True) for d in dev]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(la.scan_fwd(dev[i]["x"], dev[i]["g"], dev[i]["h0"], gate="logit", tied=True, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for h, last in got[i]:
            assert torch.equal(h, want[i][0]) and torch.equal(last, want[i][1])


def test_scan_short_wait_limit_reports_timeout(la):
    """Waits that run out are reported; the boxes and a team's messages are still waited
    for, so the next call on the same context is right."""
    p = make(42, 1, 5000, 4096)
    x, g = c(p["x"]), c(p["g"])
    want, wl = la.scan_fwd(x, g)
    la.check_device()
    prev = ctypes.c_int64(0)
    L = la.lib()
    assert L.la_testing_set_wait_limit(1, ctypes.byref(prev)) == 0
    try:
        la.scan_fwd(x, g)
        with pytest.raises(la.LAError) as e:
            la.check_device()
        assert e.value.status == 5
    finally:
        assert L.la_testing_set_wait_limit(prev.value, None) == 0
    h, last = la.scan_fwd(x, g)
    la.check_device()
    assert torch.equal(h, want) and torch.equal(last, wl)


def test_recurrent_block_trains_and_serves(la):
    """Norm, gates, recurrence and norm as a block uses them: one step of gradients through
    the kernels' own backward passes against fp64 autograd, then tokens one at a time
    against the prefill.  Tolerances are those of bf16 storage between the kernels: every
    stored tensor is half a step off relative to its value, and at most six of them lie
    between an input and an output, each passed on with a gain below 4."""
    B, T, D = 2, 70, 128
    p = make(43, B, T, D, F32, F32, "logit")
    w = 1.0 + 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(2))
    x, g, dy = (c(p[k].to(BF)) for k in ("x", "g", "dh"))
    wd = c(w)
    n, mean, rstd = la.norm_fwd(x, wd, eps=1e-5)
    h, last = la.scan_fwd(n, g, gate="logit", tied=True)
    y, _, r2 = la.norm_fwd(h, wd, kind="rms", eps=1e-5)
    dh, dw2, _ = la.norm_bwd(dy, h, r2, w=wd, kind="rms", want_db=False)
    dn, dg, _ = la.scan_bwd(g, h, dh, x=n, gate="logit", tied=True)
    dx, dw, _ = la.norm_bwd(dn, x, rstd, mean=mean, w=wd, want_db=False)

    X, G, W = (t.double().cpu().requires_grad_() for t in (x, g, wd))
    m = X.mean(-1, keepdim=True)
    N = (X - m) / torch.sqrt((X - m).square().mean(-1, keepdim=True) + 1e-5) * W
    A, s, hs = torch.sigmoid(G), torch.zeros(B, D, dtype=torch.float64), []
    for t in range(T):
        s = A[:, t] * s + (1 - A[:, t]) * N[:, t]
        hs.append(s)
    H = torch.stack(hs, 1)
    Y = H / torch.sqrt(H.square().mean(-1, keepdim=True) + 1e-5) * W
    Y.backward(dy.double().cpu())
    tol = 6 * 4 * half_step(BF)
    for got, ref in ((y, Y), (dx, X.grad), (dg, G.grad), (dw + dw2, W.grad)):
        ref = ref.detach().numpy()
        assert np.linalg.norm(np64(got) - ref) <= tol * np.linalg.norm(ref)
    state = torch.zeros(B, D, device="cuda")
    for t in range(T):
        nt, _, _ = la.norm_fwd(x[:, t], wd, eps=1e-5)
        assert torch.equal(nt, n[:, t])
        ht = la.scan_step(nt, g[:, t], state, gate="logit", tied=True)
    E, El = fwd_bound(n, g, None, "logit", True)
    assert np.all(np.abs(np64(state) - np64(last)) <= 2 * El + 1e-37)
    assert np.all(np.abs(np64(ht) - np64(h[:, -1])) <= 2 * E[:, -1] + 2 * half_step(BF) * np.abs(np64(ht)) + 1e-37)
