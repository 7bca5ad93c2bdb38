"""Every division of a walk (csrc/scan.cuh, scan_plan) against the fp64 oracle, for every
pair of types, gate and input: teams of 4, 2 and 1 CTAs over one and several dense walks,
maps and then outputs, with tiles and without, and one warp a walk.  Which one a shape
takes on 148 SMs, by its blocks of 64 channels over all walks (more than 512 tokens):

    64 to 74     a team of 4 CTAs a block
    75 to 148    of 2
    149 to 295   of 1
    fewer        maps of segments, then outputs
    296 and more, or at most 512 tokens   one warp a walk

A few channels are compared (the first and last of blocks and of the row among them),
with the bounds of test_gpu_scan.py; the state is updated in place."""
import numpy as np
import pytest
import torch

from test_gpu_parity import la  # noqa: F401
from test_gpu_scan import BF, F32, FORMS, c, check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu

SHAPES = [
    pytest.param(2, 700, 2048, id="team4-2walks"),
    pytest.param(1, 1043, 4096, id="team4-1walk"),
    pytest.param(2, 600, 3000, id="team2-2walks-ragged"),
    pytest.param(4, 530, 4096, id="team1-4walks"),
    pytest.param(3, 2000, 64, id="segments-3walks"),
    pytest.param(1, 900, 1000, id="segments-ragged"),
    pytest.param(1, 900, 1001, id="segments-no-tiles"),
    pytest.param(2, 530, 4097, id="segments-no-tiles-many"),
    pytest.param(5, 520, 4096, id="warp-many-walks"),
    pytest.param(2, 500, 2048, id="warp-short"),
]


def channels(D):
    gen = torch.Generator().manual_seed(D)
    edges = [0, 1, 31, 32, 33, 62, 63, 64, 65, D // 2, D - 65, D - 64, D - 2, D - 1]
    return torch.unique(torch.tensor([e for e in edges if 0 <= e < D] + torch.randint(0, D, (10,), generator=gen).tolist()))


def compare(p, got, back, ch, gate, tied, b0, b1, t0, t1, dl, h0):
    """Rows [b0, b1) x tokens [t0, t1) of the picked channels, with their states h0 and dl."""
    h, last = got
    dx, dg, dh0 = back
    one = lambda t: t[b0:b1, t0:t1][..., ch.to(t.device)]  # noqa: E731
    check_fwd(one(h), last, one(p["x"]), one(p["g"]), h0, gate, tied, (b0, t0))
    check_bwd((one(dx), one(dg), dh0), one(p["g"]), one(h), one(p["dh"]), one(p["x"]), h0, dl, gate, tied, (b0, t0))


def run(la, p, h0, dl, gate, tied, **kw):
    s, e = c(h0), c(dl)
    h, last = la.scan_fwd(c(p["x"]), c(p["g"]), s, gate=gate, tied=tied, h_last=s, **kw)
    back = la.scan_bwd(c(p["g"]), h, c(p["dh"]), x=c(p["x"]) if tied else None, h0=c(h0), dh_last=e, dh0=e,
                       gate=gate, tied=tied, **kw)
    la.check_device()
    assert last is s and back[2] is e
    return (h, last), back


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("xt,gt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("gate,tied", FORMS)
def test_dense(la, B, T, D, xt, gt, gate, tied):
    p = make(B + T + D, B, T, D, xt, gt, gate)
    got, back = run(la, p, p["h0"], p["dl"], gate, tied)
    ch = channels(D)
    for b in range(B):
        pick = lambda t: t[b:b + 1][:, ch.to(t.device)]  # noqa: E731
        compare(p, (got[0], pick(got[1])), (back[0], back[1], pick(back[2])), ch, gate, tied, b, b + 1, 0, T,
                pick(p["dl"]), pick(p["h0"]))


LENS = [1, 0, 517, 16, 17, 0, 300, 2, 15, 1, 129]


@pytest.mark.parametrize("D", [pytest.param(4096, id="team4"), pytest.param(6144, id="team2"), pytest.param(10240, id="team1"),
                               pytest.param(192, id="segments"), pytest.param(191, id="no-tiles"),
                               pytest.param(18944, id="warp")])
@pytest.mark.parametrize("xt,gt", [(BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("gate,tied", [("value", False), ("logit", True)])
def test_packed(la, D, xt, gt, gate, tied):
    n, total, extra = len(LENS), sum(LENS), 7
    p, st = make(D, 1, total + extra, D, xt, gt, gate), make(D + 1, n, 1, D)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int64)
    h = torch.full((1, total + extra, D), 9.0, dtype=xt, device="cuda")
    dx, dg = torch.full_like(h, 9.0), torch.full((1, total + extra, D), 9.0, dtype=gt, device="cuda")
    kw = dict(gate=gate, tied=tied, cu_seqlens=cu.cuda(), max_seqlen=max(LENS))
    s, e = c(st["h0"]), c(st["dl"])
    la.scan_fwd(c(p["x"]), c(p["g"]), s, h=h, h_last=s, **kw)
    la.scan_bwd(c(p["g"]), h, c(p["dh"]), x=c(p["x"]) if tied else None, h0=c(st["h0"]), dh_last=e, dh0=e, dx=dx, dg=dg, **kw)
    la.check_device()
    ch = channels(D)
    for i in range(n):
        pick = lambda t: t[i:i + 1][:, ch.to(t.device)]  # noqa: E731
        compare(p, (h, pick(s)), (dx, dg, pick(e)), ch, gate, tied, 0, 1, int(cu[i]), int(cu[i + 1]), pick(st["dl"]),
                pick(st["h0"]))
    for t in (h, dx, dg):
        assert torch.all(t[:, total:] == 9.0)


@pytest.mark.parametrize("D", [4096, 6144, 10240])
def test_teams_captured_and_replayed(la, D):
    """Two graphs of teams replayed at once on two streams, on inputs of other values than at capture."""
    ps = [make(50 + i, 1, 900, D, BF, BF, "logit") for i in range(2)]
    graphs = []
    for p in ps:
        b = {k: c(v) for k, v in ps[0].items()}
        la.scan_bwd(b["g"], la.scan_fwd(b["x"], b["g"], gate="logit")[0], b["dh"], gate="logit")
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            h, last = la.scan_fwd(b["x"], b["g"], b["h0"], gate="logit")
            back = la.scan_bwd(b["g"], h, b["dh"], h0=b["h0"], dh_last=b["dl"], gate="logit")
        for k in b:
            b[k].copy_(p[k])
        graphs.append((gr, (h, last), back, b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    la.check_device()
    ch = channels(D)
    for p, (_, got, back, _) in zip(ps, graphs):
        pick = lambda t: t[:, ch.to(t.device)]  # noqa: E731
        compare(p, (got[0], pick(got[1])), (back[0], back[1], pick(back[2])), ch, "logit", False, 0, 1, 0, 900,
                pick(p["dl"]), pick(p["h0"]))
