"""A call that is refused while `stream=` is given raises the documented ValueError and
leaves the caller's current stream as it was (the recurrence's and the norms' five calls)."""
import pytest
import torch

from test_gpu_parity import la  # noqa: F401
from test_gpu_scan import BF, c, make

pytestmark = pytest.mark.gpu


def calls(la):
    p = make(1, 2, 8, 8)
    x, g, dh, s = (c(p[k]) for k in ("x", "g", "dh", "h0"))
    h, _ = la.scan_fwd(x, g)
    w = torch.ones(8, device="cuda")
    _, mean, rstd = la.norm_fwd(x, w)
    state = lambda: torch.zeros(2, 8)  # noqa: E731
    return {
        "scan_fwd h0": lambda st: la.scan_fwd(x, g, state(), stream=st),
        "scan_fwd h": lambda st: la.scan_fwd(x, g, h=torch.empty(2, 8, 8, dtype=BF), stream=st),
        "scan_fwd h_last": lambda st: la.scan_fwd(x, g, s, h_last=state(), stream=st),
        "scan_bwd h0": lambda st: la.scan_bwd(g, h, dh, h0=state(), stream=st),
        "scan_bwd dh_last": lambda st: la.scan_bwd(g, h, dh, dh_last=state(), stream=st),
        "scan_bwd dx": lambda st: la.scan_bwd(g, h, dh, dx=torch.empty(2, 8, 8, dtype=BF), stream=st),
        "scan_bwd dg": lambda st: la.scan_bwd(g, h, dh, dg=torch.empty(2, 8, 8), stream=st),
        "scan_bwd dh0": lambda st: la.scan_bwd(g, h, dh, dh0=state(), stream=st),
        "scan_step state": lambda st: la.scan_step(x[:, 0], g[:, 0], state(), stream=st),
        "scan_step h": lambda st: la.scan_step(x[:, 0], g[:, 0], s, h=torch.empty(2, 8, dtype=BF), stream=st),
        "norm_fwd w": lambda st: la.norm_fwd(x, torch.ones(8), stream=st),
        "norm_fwd b": lambda st: la.norm_fwd(x, w, torch.ones(8), stream=st),
        "norm_fwd y": lambda st: la.norm_fwd(x, w, y=torch.empty(2, 8, 8, dtype=BF), stream=st),
        "norm_bwd mean": lambda st: la.norm_bwd(dh, x, rstd, mean=mean.cpu(), w=w, stream=st),
        "norm_bwd rstd": lambda st: la.norm_bwd(dh, x, rstd.cpu(), mean=mean, w=w, stream=st),
        "norm_bwd w": lambda st: la.norm_bwd(dh, x, rstd, mean=mean, w=torch.ones(8), stream=st),
        "norm_bwd dx": lambda st: la.norm_bwd(dh, x, rstd, mean=mean, w=w, dx=torch.empty(2, 8, 8, dtype=BF), stream=st),
    }


def test_refused_calls_leave_the_current_stream(la):
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    for name, call in calls(la).items():
        for outer in (torch.cuda.default_stream(), mine):
            with torch.cuda.stream(outer):
                try:
                    with pytest.raises(ValueError):
                        call(side)
                    assert torch.cuda.current_stream() == outer, name
                finally:
                    torch.cuda.set_stream(outer)
    torch.cuda.synchronize()


def test_calls_after_a_refused_one_run_in_the_callers_order(la):
    """What the caller queues after a refusal is ordered behind what they queued before it."""
    p = make(2, 1, 2000, 64)
    x, g = c(p["x"]), c(p["g"])
    want, _ = la.scan_fwd(x, g)
    side, y = torch.cuda.Stream(), torch.zeros_like(x)
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device="cuda")
    for _ in range(10):
        big = (big @ big) * 1e-4           # the caller's stream is busy
    y.copy_(x)
    with pytest.raises(ValueError):
        la.scan_fwd(x, g, torch.zeros(1, 64), stream=side)
    got, _ = la.scan_fwd(y, g)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
