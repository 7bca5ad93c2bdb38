"""Host-side checks of la_scan_* and la_norm_* (no GPU needed, no kernel launched):
invalid arguments are refused with the documented status before anything is
launched; the pointers below are never dereferenced."""
import ctypes

import pytest
import torch

import gated_delta_rule_attn_b200 as la
from gated_delta_rule_attn_b200 import build as la_build

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    la_build.build()
    return la.lib()


def struct(cls, **kw):
    a = cls()
    a.struct_size = ctypes.sizeof(cls)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def fwd(**kw):
    return struct(la.ScanFwdArgs, **dict(dict(dtype=1, gate_dtype=0, B=2, T=8, D=16, x=FAKE, g=FAKE, h=FAKE), **kw))


def bwd(**kw):
    return struct(la.ScanBwdArgs, **dict(dict(dtype=1, gate_dtype=0, B=2, T=8, D=16, g=FAKE, h=FAKE, dh=FAKE,
                                              dx=FAKE, dg=FAKE), **kw))


def step(**kw):
    return struct(la.ScanStepArgs, **dict(dict(dtype=1, gate_dtype=0, N=2, D=16, x=FAKE, g=FAKE, state=FAKE, h=FAKE), **kw))


def nfwd(**kw):
    return struct(la.NormFwdArgs, **dict(dict(dtype=1, R=4, D=16, x=FAKE, y=FAKE, eps=1e-5), **kw))


def nbwd(**kw):
    return struct(la.NormBwdArgs, **dict(dict(dtype=1, R=4, D=16, x=FAKE, dy=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE,
                                              dw=FAKE, workspace=FAKE, workspace_bytes=1 << 30), **kw))


COMMON = [(dict(dtype=2), 1), (dict(gate_dtype=7), 1), (dict(gate=2), 1), (dict(tied=2), 1), (dict(D=0), 1),
          (dict(D=-4), 1), (dict(g=None), 1), (dict(h=None), 1), (dict(struct_size=16), 1), (dict(g_row=15), 1),
          (dict(h_row=-1), 1), (dict(g=FAKE + 2), 3), (dict(h=FAKE + 1), 3)]
SEQ = [(dict(B=0), 1), (dict(T=-1), 1), (dict(B=1 << 20, D=1 << 20), 1), (dict(h0=FAKE + 2), 3),
       (dict(cu_seqlens=FAKE + 4, max_seqlen=8), 3), (dict(cu_seqlens=FAKE, max_seqlen=9), 1),
       (dict(cu_seqlens=FAKE, max_seqlen=-1), 1)]


@pytest.mark.parametrize("kw,status", COMMON + SEQ + [(dict(x=None), 1), (dict(x=FAKE + 1), 3), (dict(x_row=3), 1),
                                                      (dict(h_last=FAKE + 1), 3)])
def test_scan_fwd_refuses(L, kw, status):
    assert L.la_scan_fwd(ctypes.byref(fwd(**kw)), None) == status
    assert L.la_last_error_message()


@pytest.mark.parametrize("kw,status", COMMON + SEQ + [(dict(tied=1), 1), (dict(x=FAKE), 1), (dict(dh=None), 1),
                                                      (dict(dx=None), 1), (dict(dg=None), 1), (dict(dg=FAKE + 2), 3),
                                                      (dict(dh_row=1), 1), (dict(dx_row=1), 1), (dict(dg_row=1), 1),
                                                      (dict(dh_last=FAKE + 2), 3), (dict(dh0=FAKE + 2), 3)])
def test_scan_bwd_refuses(L, kw, status):
    assert L.la_scan_bwd(ctypes.byref(bwd(**kw)), None) == status
    assert L.la_last_error_message()


@pytest.mark.parametrize("kw,status", COMMON + [(dict(N=0), 1), (dict(x=None), 1), (dict(state=None), 1),
                                                (dict(state=FAKE + 2), 3)])
def test_scan_step_refuses(L, kw, status):
    assert L.la_scan_step(ctypes.byref(step(**kw)), None) == status
    assert L.la_last_error_message()


ROWS = [(dict(dtype=3), 1), (dict(kind=2), 1), (dict(R=-1), 1), (dict(D=0), 1), (dict(D=16385), 2), (dict(x=None), 1),
        (dict(x=FAKE + 1), 3), (dict(x_row=8), 1), (dict(w=FAKE + 2), 3), (dict(struct_size=8), 1)]


@pytest.mark.parametrize("kw,status", ROWS + [(dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
                                              (dict(eps=float("inf")), 1), (dict(y=None), 1), (dict(y_row=1), 1),
                                              (dict(kind=1, mean=FAKE), 1), (dict(b=FAKE + 1), 3), (dict(rstd=FAKE + 1), 3)])
def test_norm_fwd_refuses(L, kw, status):
    assert L.la_norm_fwd(ctypes.byref(nfwd(**kw)), None) == status
    assert L.la_last_error_message()


@pytest.mark.parametrize("kw,status", ROWS + [(dict(dy=None), 1), (dict(dx=None), 1), (dict(rstd=None), 1),
                                              (dict(mean=None), 1), (dict(kind=1), 1), (dict(dy_row=2), 1),
                                              (dict(workspace=None), 8), (dict(workspace_bytes=8), 8),
                                              (dict(workspace=FAKE + 4), 8), (dict(dw=FAKE + 2), 3), (dict(db=FAKE + 2), 3)])
def test_norm_bwd_refuses(L, kw, status):
    assert L.la_norm_bwd(ctypes.byref(nbwd(**kw)), None) == status
    assert L.la_last_error_message()


def test_null_and_empty(L):
    for f in (L.la_scan_fwd, L.la_scan_bwd, L.la_scan_step, L.la_norm_fwd, L.la_norm_bwd):
        assert f(None, None) == 1
    n = ctypes.c_size_t(7)
    assert L.la_norm_bwd_workspace_size(None, ctypes.byref(n)) == 1
    assert L.la_norm_bwd_workspace_size(ctypes.byref(nbwd()), None) == 1
    assert L.la_norm_bwd_workspace_size(ctypes.byref(nbwd()), ctypes.byref(n)) == 0 and n.value >= 2 * 16 * 4
    assert L.la_norm_bwd_workspace_size(ctypes.byref(nbwd(dw=None)), ctypes.byref(n)) == 0 and n.value == 0
    assert L.la_norm_bwd_workspace_size(ctypes.byref(nbwd(R=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert L.la_norm_fwd(ctypes.byref(nfwd(R=0, x=None, y=None)), None) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        la.scan_fwd(x, x)
    with pytest.raises(ValueError):
        la.scan_bwd(x, x, x)
    with pytest.raises(ValueError):
        la.scan_step(x[0], x[0], x[0])
    with pytest.raises(ValueError):
        la.norm_fwd(x)
    with pytest.raises(ValueError):
        la.norm_bwd(x, x, x[..., 0], mean=x[..., 0])


@pytest.mark.parametrize("make,size", [(fwd, "la_scan_fwd_workspace_size"), (bwd, "la_scan_bwd_workspace_size")])
def test_scan_workspace(L, make, size):
    f, n = getattr(L, size), ctypes.c_size_t(7)
    assert f(None, ctypes.byref(n)) == 1 and f(ctypes.byref(make()), None) == 1
    assert f(ctypes.byref(make()), ctypes.byref(n)) == 0 and n.value == 0          # short: none
    assert f(ctypes.byref(make(B=0)), ctypes.byref(n)) == 1
    assert f(ctypes.byref(make(B=1, T=100000)), ctypes.byref(n)) == 0 and n.value > 0
    call = L.la_scan_fwd if make is fwd else L.la_scan_bwd
    for kw in (dict(), dict(workspace=FAKE, workspace_bytes=n.value - 1), dict(workspace=FAKE + 8, workspace_bytes=n.value)):
        assert call(ctypes.byref(make(B=1, T=100000, **kw)), None) == 8
    assert call(ctypes.byref(make(T=(1 << 30) + 1)), None) == 2
