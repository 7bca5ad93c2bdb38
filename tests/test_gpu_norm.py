"""Layer norm and RMS norm on the GPU (la_norm_fwd, la_norm_bwd) against the fp64
oracle on the same inputs, element by element.

Bounds, with u = 2^-24 (half a step of fp32).  A sum over a row is 16 additions in a
thread and at most 10 across threads, so it is off by at most 32 u times the sum of
magnitudes:
    mean   dm = 33 u mean|x|
    var    relative: twice the centred values' error against their RMS s,
           2 dm / s, and 36 u of its own;  rstd: half of it, and 6 u for the root
    y      |w| rstd (dm + u |c|) + |w xh| (relative error of rstd + 3 u) + 2 u (|y| + |b|)
    dx     rstd (34 u mean|d| + |xh| 44 u mean|d xh| + 8 u (|d| + |mean d| + |xh mean(d xh)|))
    dw, db (180 + R / 148) u sum of magnitudes: a thread adds at most R / 148 + 1 rows (or
           one where there are fewer than 148 CTAs), then at most 13 and 156 partial sums
    and the rounding of what is stored, eps / 2 of its type relative to the value.
"""
import numpy as np
import pytest
import torch

from oracle import rows
from test_gpu_parity import la  # noqa: F401
from test_gpu_scan import BF, F32, U, c, half_step, np64

pytestmark = pytest.mark.gpu
EPS = 1e-5


def make(seed, R, D, dt=BF, off=0.3):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=(rn(R, D) * (0.5 + torch.rand(R, 1, generator=gen)) + off * rn(R, 1)).to(dt),
                w=1.0 + 0.3 * rn(D), b=0.3 * rn(D), dy=rn(R, D).to(dt))


def check_fwd(got, x, w, b, kind, eps=EPS):
    y, mean, rstd = got
    ry, rm, rr = rows.norm_fwd(x, w, b, kind, eps)
    x64 = np64(x)
    dm = 33 * U * np.abs(x64).mean(1) if kind == "layer" else np.zeros(len(x64))
    rel = dm * rr + 18 * U + 6 * U
    if kind == "layer":
        assert np.all(np.abs(np64(mean) - rm) <= dm + 1e-37)
    else:
        assert mean is None
    assert np.all(np.abs(np64(rstd) - rr) <= (rel + U) * rr)
    cen = x64 - rm[:, None] if kind == "layer" else x64
    aw = np.abs(np64(w)) if w is not None else 1.0
    ab = np.abs(np64(b)) if b is not None else 0.0
    tol = aw * rr[:, None] * (dm[:, None] + U * np.abs(cen)) + aw * np.abs(cen) * rr[:, None] * (rel[:, None] + 3 * U)
    tol = tol + 2 * U * (np.abs(ry) + ab)
    tol = tol + half_step(y.dtype) * (np.abs(ry) + tol) + 1e-37
    d = np.abs(np64(y) - ry)
    assert np.all(d <= tol), float((d / tol).max())


def check_bwd(got, dy, x, rstd, mean, w, kind):
    dx, dw, db = got
    rx, rw, rb = rows.norm_bwd(dy, x, rstd, mean, w, kind)
    rs = np64(rstd)[:, None]
    xh = np.abs(((np64(x) - np64(mean)[:, None]) if kind == "layer" else np64(x)) * rs)
    d = np.abs(np64(dy)) * (np.abs(np64(w)) if w is not None else 1.0)
    md, mdx = d.mean(1, keepdims=True), (d * xh).mean(1, keepdims=True)
    tol = rs * (34 * U * md + xh * 44 * U * mdx + 8 * U * (d + md + xh * mdx))
    tol = tol + half_step(dx.dtype) * (np.abs(rx) + tol) + 1e-37
    e = np.abs(np64(dx) - rx)
    assert np.all(e <= tol), float((e / tol).max())
    n = (180 + len(d) / 148) * U
    if dw is not None:
        e, tol = np.abs(np64(dw) - rw), (n + 6 * U) * (np.abs(np64(dy)) * xh).sum(0) + 1e-37
        assert np.all(e <= tol), float((e / tol).max())
    if db is not None:
        e, tol = np.abs(np64(db) - rb), n * np.abs(np64(dy)).sum(0) + 1e-37
        assert np.all(e <= tol), float((e / tol).max())


def run_both(la, p, kind, weight=True, bias=True):
    w, b = (p["w"] if weight else None), (p["b"] if bias else None)
    got = la.norm_fwd(c(p["x"]), c(w), c(b), kind=kind, eps=EPS)
    check_fwd(got, p["x"], w, b, kind)
    _, mean, rstd = got
    back = la.norm_bwd(c(p["dy"]), c(p["x"]), rstd, mean=mean, w=c(w), kind=kind)
    check_bwd(back, p["dy"], p["x"], rstd, mean, w, kind)
    return got, back


# rows of one element up to the largest, around a thread's 16, a warp's 512, a CTA's
# 8192; even, odd and unaligned counts
@pytest.mark.parametrize("D", [1, 2, 7, 8, 16, 17, 32, 33, 64, 100, 128, 255, 256, 500, 511, 512, 513, 520, 1000,
                               1001, 1024, 2048, 2752, 4096, 4097, 8192, 8200, 8201, 16383, 16384])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_matches_oracle(la, D, dt, kind):
    run_both(la, make(D, 37, D, dt), kind)


@pytest.mark.parametrize("R", [1, 2, 31, 33, 148, 1200, 5000])
@pytest.mark.parametrize("D", [4, 128, 129, 640])
def test_norm_row_counts(la, R, D):
    run_both(la, make(R + D, R, D), "layer")
    run_both(la, make(R + D, R, D), "rms")


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("D", [96, 1025, 16384])
def test_norm_without_weight_or_bias(la, weight, bias, D):
    for kind in ("layer", "rms"):
        run_both(la, make(D, 20, D), kind, weight, bias)


def test_norm_some_gradients_only(la):
    p = make(1, 50, 200)
    _, mean, rstd = la.norm_fwd(c(p["x"]), c(p["w"]), eps=EPS)
    full = la.norm_bwd(c(p["dy"]), c(p["x"]), rstd, mean=mean, w=c(p["w"]))
    for dw, db in ((True, False), (False, True), (False, False)):
        got = la.norm_bwd(c(p["dy"]), c(p["x"]), rstd, mean=mean, w=c(p["w"]), want_dw=dw, want_db=db)
        assert torch.equal(got[0], full[0])
        assert (torch.equal(got[1], full[1]) if dw else got[1] is None)
        assert (torch.equal(got[2], full[2]) if db else got[2] is None)
    y, m, r = la.norm_fwd(c(p["x"]), c(p["w"]), eps=EPS, want_stats=False)
    assert m is None and r is None and torch.equal(y, la.norm_fwd(c(p["x"]), c(p["w"]), eps=EPS)[0])


def test_norm_no_rows(la):
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    y, mean, rstd = la.norm_fwd(x)
    assert y.shape == (0, 64) and mean.shape == (0,) and rstd.shape == (0,)
    dx, dw, db = la.norm_bwd(x, x, rstd, mean=mean)
    assert dx.shape == (0, 64) and torch.all(dw == 0) and torch.all(db == 0)


@pytest.mark.parametrize("D", [64, 33, 1000])
def test_norm_large_offset_keeps_the_deviation(la, D):
    """Rows whose mean is 1000 times their deviation: the variance is of centred values."""
    gen = torch.Generator().manual_seed(D)
    x = 1000.0 + torch.randn(9, D, generator=gen)
    check_fwd(la.norm_fwd(x.cuda(), eps=EPS), x, None, None, "layer")


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_constant_and_zero_rows(la, kind):
    x = torch.zeros(4, 96)
    x[1], x[2] = 2.0, -0.5
    x[3, 0] = 1.0
    run_both(la, dict(make(2, 4, 96, F32), x=x), kind)


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 1032])
def test_norm_slices(la, pad, dt, D):
    """Rows of wider tensors, starts that forbid wide accesses, in and out."""
    p = make(3 + D, 30, D, dt)
    wide = lambda v: torch.full((2, 15, D + 2 * pad), v, dtype=dt, device="cuda")[..., pad:pad + D]  # noqa: E731
    x, dy, y, dx = wide(float("nan")), wide(float("nan")), wide(7.0), wide(7.0)
    x.copy_(c(p["x"]).view(2, 15, D))
    dy.copy_(c(p["dy"]).view(2, 15, D))
    got = la.norm_fwd(x, c(p["w"]), c(p["b"]), eps=EPS, y=y)
    assert got[0] is y and got[1].shape == (2, 15)
    check_fwd((y.reshape(30, D), got[1].view(30), got[2].view(30)), p["x"], p["w"], p["b"], "layer")
    back = la.norm_bwd(dy, x, got[2], mean=got[1], w=c(p["w"]), dx=dx)
    check_bwd((dx.reshape(30, D), back[1], back[2]), p["dy"], p["x"], got[2].view(30), got[1].view(30), p["w"], "layer")
    for t in (y, dx):
        if pad:
            whole = t.as_strided((2, 15, D + 2 * pad), t.stride(), 0)
            assert torch.all(whole[..., :pad] == 7.0) and torch.all(whole[..., pad + D:] == 7.0)


@pytest.mark.parametrize("R,D", [(700, 128), (300, 2048), (40, 16384), (500, 77)])
def test_norm_same_bits_again(la, R, D):
    p = make(4, R, D)
    x, dy, w = c(p["x"]), c(p["dy"]), c(p["w"])
    _, mean, rstd = la.norm_fwd(x, w)
    first = la.norm_bwd(dy, x, rstd, mean=mean, w=w)
    for _ in range(3):
        assert all(torch.equal(i, j) for i, j in zip(first, la.norm_bwd(dy, x, rstd, mean=mean, w=w)))


def test_norm_nan_stays_in_its_row(la):
    for D in (64, 2048, 9000):
        p = make(5, 40, D)
        clean = la.norm_fwd(c(p["x"]), c(p["w"]), c(p["b"]))
        for bad in (float("nan"), float("inf")):
            x = p["x"].clone()
            x[17, D // 2] = bad
            y, mean, rstd = la.norm_fwd(c(x), c(p["w"]), c(p["b"]))
            assert torch.isnan(y[17]).any()
            keep = [i for i in range(40) if i != 17]
            assert torch.equal(y[keep], clean[0][keep]) and torch.equal(rstd[keep], clean[2][keep])


def test_norm_offsets_past_32_bits(la):
    W, D, R = 8_000_000, 64, 300
    wide = torch.empty(R, W, dtype=BF, device="cuda")
    p = make(6, R, D)
    x, y, dx = wide[:, W - D:], wide[:, :D], wide[:, 128:128 + D]
    x.copy_(c(p["x"]))
    got = la.norm_fwd(x, c(p["w"]), c(p["b"]), eps=EPS, y=y)
    check_fwd(got, p["x"], p["w"], p["b"], "layer")
    back = la.norm_bwd(c(p["dy"]), x, got[2], mean=got[1], w=c(p["w"]), dx=dx)
    check_bwd(back, p["dy"], p["x"], got[2], got[1], p["w"], "layer")


def test_norm_rms_is_the_output_norm(la):
    """The head-wise normalisation that la_fwd applies to its output (out_norm)."""
    import workloads
    q = workloads.make_problem("gla", 1, 70, 2, 64, 64, seed=3)
    args = [c(t) for t in (q.q, q.k, q.v, q.g)]
    w = 1.0 + 0.1 * torch.randn(64, generator=torch.Generator().manual_seed(1))
    raw, _, _ = la.fwd("gla", *args)
    fused, _, _ = la.fwd("gla", *args, out_norm=True, norm_w=c(w), norm_eps=EPS)
    y, _, rstd = la.norm_fwd(raw, c(w), kind="rms", eps=EPS)
    assert rstd.shape == (1, 70, 2)
    # the same row, each rounded once: half a step each, and the fp32 error of both
    d = np.abs(np64(y) - np64(fused))
    assert np.all(d <= (2 * half_step(BF) + 128 * U) * np.abs(np64(y)) * (1 + 4 * half_step(BF)) + 1e-30)


def test_norm_on_another_stream_and_in_graphs(la):
    """Partial sums are each call's own: two graphs replayed at once do not meet."""
    p, q = make(7, 3000, 512), make(8, 3000, 512)
    s = torch.cuda.Stream()
    b = {k: c(v) for k, v in p.items()}
    _, mean, rstd = la.norm_fwd(b["x"], b["w"])
    want = la.norm_bwd(b["dy"], b["x"], rstd, mean=mean, w=b["w"])
    s.wait_stream(torch.cuda.current_stream())
    y2, m2, r2 = la.norm_fwd(b["x"], b["w"], stream=s)
    got = la.norm_bwd(b["dy"], b["x"], r2, mean=m2, w=b["w"], stream=s)
    s.synchronize()
    assert torch.equal(r2, rstd) and all(torch.equal(i, j) for i, j in zip(got, want))
    graphs = []
    for src in (p, q):
        b = {k: c(v) for k, v in src.items()}
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f = la.norm_fwd(b["x"], b["w"], eps=EPS)
            d = la.norm_bwd(b["dy"], b["x"], f[2], mean=f[1], w=b["w"])
        graphs.append((gr, b, f, d))
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(s):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for (gr, b, f, d), src in zip(graphs, (p, q)):
            check_fwd(f, src["x"], src["w"], None, "layer")
            check_bwd(d, src["dy"], src["x"], f[2], f[1], src["w"], "layer")


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradients_are_differences_of_the_gpu_forward(la, kind):
    """Central differences of the kernel's own forward pass in fp32.  With step e the
    forward pass' rounding (the bound above, below 80 u (|y| + 1) an element on these
    rows) gives at most sum |dy| 80 u (|y| + 1) / e.  The truncation is e^2 / 6 of the
    third derivative: v = mean(c^2) has |dv| <= 2 sqrt(v / D) and |d2v| <= 2 / D, so
    r = rstd has |d3r| <= 24 r^4 / D^1.5 and |d2r| <= 4 r^3 / D, and an output's third
    derivative is at most |w| r^3 (24 |xh| / D^1.5 + 12 / D) <= |w| r^3 (|xh| + 1) at
    D = 12; the factor 2 is for r's change over the step.  dw and db are linear."""
    p = make(9, 3, 12, F32)
    p["x"] = p["x"] * 2.0
    x, w, b, dy = (c(p[k]) for k in ("x", "w", "b", "dy"))
    y, mean, rstd = la.norm_fwd(x, w, b, kind=kind, eps=EPS)
    dx, dw, db = la.norm_bwd(dy, x, rstd, mean=mean, w=w, kind=kind)
    e = 2.0 ** -6
    ay, ady = np.abs(np64(y)), np.abs(np64(dy))
    xh = np.abs(rows.norm_fwd(x, kind=kind, eps=EPS)[0])
    noise = float((ady * 80 * U * (ay + 1)).sum()) / e
    trunc = 2 * e * e / 6 * float(np64(rstd).max()) ** 3 * float((ady * np.abs(np64(w)) * (xh + 1)).sum())
    loss = lambda: float((la.norm_fwd(x, w, b, kind=kind, eps=EPS)[0].double() * dy.double()).sum())  # noqa: E731
    for t, d in ((x, dx), (w, dw), (b, db)):
        f, df = t.view(-1), d.view(-1)
        for i in range(f.numel()):
            keep = f[i].item()
            f[i] = keep + e
            up, hi = loss(), f[i].item()
            f[i] = keep - e
            down, lo = loss(), f[i].item()
            f[i] = keep
            assert abs((up - down) / (hi - lo) - df[i].item()) <= noise + trunc


def test_norm_refuses(la):
    p = make(10, 6, 32)
    x, w = c(p["x"]), c(p["w"])
    y, mean, rstd = la.norm_fwd(x, w)
    for bad in (dict(x=p["x"]), dict(x=x.half()), dict(w=w.to(BF)), dict(w=w[:16]), dict(kind="batch"),
                dict(x=x.t()), dict(x=x[:1].expand(6, 32)), dict(y=y.float()),
                dict(x=torch.zeros(2, 3, 4, 32, dtype=BF, device="cuda").transpose(0, 1))):
        kw = dict(x=x, w=w)
        kw.update(bad)
        with pytest.raises(ValueError):
            la.norm_fwd(**kw)
    for kw in (dict(mean=None), dict(mean=mean, kind="rms"), dict(mean=mean[:3])):
        with pytest.raises(ValueError):
            la.norm_bwd(y, x, rstd, w=w, **kw)
    with pytest.raises(la.LAError):
        la.norm_fwd(x, eps=0.0)
    with pytest.raises(la.LAError) as e:
        la.norm_fwd(torch.zeros(1, 16385, device="cuda"))
    assert e.value.status == 2
