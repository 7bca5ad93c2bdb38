"""Kernels that need more than the default shared memory run in every CUDA context of a
process: the primary one, one the caller created, the primary one again, and another
created after that was destroyed.  (A context has its own limits of its kernels.)

The calls go through the C ABI in a process of their own, which holds no PyTorch
context: la_fwd's chunked gated delta rule, the recurrence as a team and as maps and
outputs, and the norms' backward pass, with the same bytes as result in every context."""
import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_every_context_of_a_process():
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip().endswith("same results in 4 contexts"), r.stdout + r.stderr[-3000:]


def main():
    sys.path.insert(0, ROOT)
    import torch

    import gated_delta_rule_attn_b200 as la
    import workloads
    cu, L = ctypes.CDLL("libcuda.so.1"), la.lib()

    def ok(r, what=""):
        assert r == 0, (what, r, L.la_last_error_message())

    def up(t):
        t = t.contiguous()
        p, n = ctypes.c_uint64(), t.numel() * t.element_size()
        ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(max(n, 16))), "alloc")
        ok(cu.cuMemcpyHtoD_v2(p, ctypes.c_void_p(t.data_ptr()), ctypes.c_size_t(n)), "up")
        return p.value

    def down(p, n):
        b = ctypes.create_string_buffer(n)
        ok(cu.cuMemcpyDtoH_v2(b, ctypes.c_uint64(p), ctypes.c_size_t(n)), "down")
        return b.raw

    gen = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    bf = torch.bfloat16
    gdn = workloads.make_problem("gdn", 1, 200, 2, 128, 128, seed=3, init_state="normal")
    x, g = rn(1, 700, 4096).to(bf), torch.sigmoid(rn(1, 700, 4096))
    dy, w = rn(12, 4096).to(bf), rn(4096)
    rows = rn(12, 4096).to(bf)
    empty = lambda *s: torch.zeros(*s, dtype=bf)  # noqa: E731

    def results():
        out = []
        # the gated delta rule's chunked kernels
        a = la.FwdArgs()
        a.struct_size, a.rule, a.dtype = ctypes.sizeof(a), la.RULES["gdn"], 1
        a.B, a.T, a.H, a.dk, a.dv = 1, 200, 2, 128, 128
        a.q, a.k, a.v, a.g, a.beta, a.S0 = (up(t) for t in (gdn.q, gdn.k, gdn.v, gdn.g, gdn.beta, gdn.S0))
        a.o, a.S_out = up(empty(1, 200, 2, 128)), up(torch.zeros(1, 2, 128, 128))
        n = ctypes.c_size_t()
        ok(L.la_fwd_workspace_size(ctypes.byref(a), ctypes.byref(n)), "la_fwd size")
        a.workspace, a.workspace_bytes = up(torch.zeros(n.value, dtype=torch.uint8)), n.value
        ok(L.la_fwd(ctypes.byref(a), None), "la_fwd")
        out.append((a.o, 200 * 2 * 128 * 2))
        # a team of four CTAs, and maps and outputs
        for D in (4096, 1024):
            s = la.ScanFwdArgs(ctypes.sizeof(la.ScanFwdArgs), 1, 0, 0, 0, 1, 700, D)
            s.x, s.g, s.h = up(x[..., :D]), up(g[..., :D]), up(empty(1, 700, D))
            ok(L.la_scan_fwd_workspace_size(ctypes.byref(s), ctypes.byref(n)), "la_scan_fwd size")
            s.workspace, s.workspace_bytes = up(torch.zeros(n.value + 16, dtype=torch.uint8)), n.value
            ok(L.la_scan_fwd(ctypes.byref(s), None), "la_scan_fwd")
            out.append((s.h, 700 * D * 2))
        # the norms' backward pass, rows ahead in shared memory
        b = la.NormBwdArgs(ctypes.sizeof(la.NormBwdArgs), 1, la.NORMS["rms"], 12, 4096)
        b.x, b.dy, b.w, b.rstd, b.dx = up(rows), up(dy), up(w), up(torch.ones(12)), up(empty(12, 4096))
        b.dw = up(torch.zeros(4096))
        ok(L.la_norm_bwd_workspace_size(ctypes.byref(b), ctypes.byref(n)), "la_norm_bwd size")
        b.workspace, b.workspace_bytes = up(torch.zeros(n.value, dtype=torch.uint8)), n.value
        ok(L.la_norm_bwd(ctypes.byref(b), None), "la_norm_bwd")
        out += [(b.dx, 12 * 4096 * 2), (b.dw, 4096 * 4)]
        ok(cu.cuCtxSynchronize(), "synchronise")
        return [down(p, n) for p, n in out]

    dev, own, made = ctypes.c_int(), ctypes.c_void_p(), ctypes.c_void_p()
    ok(cu.cuInit(0))
    ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
    ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(own), dev))
    ok(cu.cuCtxSetCurrent(own))
    got = [results()]
    ok(cu.cuCtxCreate_v2(ctypes.byref(made), 0, dev), "a context")
    got.append(results())
    ok(cu.cuCtxSetCurrent(own))
    got.append(results())
    ok(cu.cuCtxDestroy_v2(made), "its end")
    ok(cu.cuCtxCreate_v2(ctypes.byref(made), 0, dev), "another context")
    got.append(results())
    assert all(r == got[0] for r in got[1:])
    assert all(any(b) for b in got[0])
    ok(cu.cuCtxDestroy_v2(made))
    ok(cu.cuCtxSetCurrent(own))
    print(f"same results in {len(got)} contexts")


if __name__ == "__main__":
    main()
