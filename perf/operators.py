"""The gated linear recurrence and the row norms: measured cases, plain forms and exact values.

Operators (one pass of ``run`` is one call):

* ``scan_fwd``   h_t = a_t h_{t-1} + u_t per channel over [B, T, D], initial state in, final state out;
* ``scan_bwd``   its gradients (inputs, gates, initial state) from the stored outputs;
* ``scan_step``  one token per sequence, fp32 state updated in place;
* ``norm_fwd``   layer norm or RMS norm of rows, with the statistics the backward pass reads;
* ``norm_bwd``   its gradients (rows, weight, bias).

The gate is given as a value (fp32, as the framework's other gates) or as the logit a projection
produces (``a = sigmoid(g)``); a tied input enters as ``u = (1 - a) x``, otherwise ``u = x``.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}
EPS = 1e-5


def _scan_case(name, op, B, T, D, x, g, gate, tied, state, nseq=0):
    c = {"op": op, "B": B, "T": T, "D": D, "x": x, "g": g, "gate": gate, "tied": tied, "state": state, "nseq": nseq}
    return dict(c, name=name) if name else c


def _norm_case(name, op, R, D, x, kind, bias):
    c = {"op": op, "R": R, "D": D, "x": x, "kind": kind, "bias": bias}
    return dict(c, name=name) if name else c


def listed():
    return [
        # serving a few sequences: one token each, latency alone counts
        _scan_case("step_n8_d2048_bf16_logit_tied", "scan_step", 8, 1, 2048, BF16, BF16, "logit", True, True),
        # a large decode batch whose states exceed L2
        _scan_case("step_n4096_d8192_bf16_value", "scan_step", 4096, 1, 8192, BF16, F32, "value", False, True),
        # prefill / training forward at the shape of the repository's own bench (B=2, 16 heads of 128, T=8192)
        _scan_case("fwd_b2_t8192_d2048_bf16_value", "scan_fwd", 2, 8192, 2048, BF16, F32, "value", False, False),
        # one long sequence (T=32768): few channels, the scan has to be split along time
        _scan_case("fwd_b1_t32768_d1024_bf16_logit_tied", "scan_fwd", 1, 32768, 1024, BF16, BF16, "logit", True, True),
        # sequences of ragged lengths packed on one axis, odd channel count, full precision
        _scan_case("fwd_packed37_t20011_d1001_f32_logit", "scan_fwd", 1, 20011, 1001, F32, F32, "logit", False, True, 37),
        # backward of a large training batch
        _scan_case("bwd_b4_t8192_d4096_bf16_value", "scan_bwd", 4, 8192, 4096, BF16, F32, "value", False, False),
        # backward of the long sequence, carrying the state and its gradient across segments
        _scan_case("bwd_b1_t32768_d1024_bf16_logit_tied", "scan_bwd", 1, 32768, 1024, BF16, BF16, "logit", True, True),
        # backward of packed sequences
        _scan_case("bwd_packed24_t16384_d2048_bf16_value", "scan_bwd", 1, 16384, 2048, BF16, F32, "value", False, True, 24),
        # the norm of a decode batch: few rows, latency alone counts
        _norm_case("norm_fwd_layer_r16_d4096_bf16", "norm_fwd", 16, 4096, BF16, "layer", True),
        # the norm before a block in training
        _norm_case("norm_fwd_layer_r16384_d4096_bf16", "norm_fwd", 16384, 4096, BF16, "layer", True),
        # its backward pass, with the weight's and the bias' gradient
        _norm_case("norm_bwd_layer_r16384_d4096_bf16", "norm_bwd", 16384, 4096, BF16, "layer", True),
        # backward of the head-wise RMS norm of an output (B=2, T=8192, 16 heads of 128)
        _norm_case("norm_bwd_rms_r262144_d128_bf16", "norm_bwd", 262144, 128, BF16, "rms", False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd", "norm_bwd"])
    x = rng.choice([BF16, BF16, F32])
    if op.startswith("norm"):
        D = rng.choice([64 * _log(rng, 1, 256), 64 * _log(rng, 1, 256), _log(rng, 1, 16384)])
        R = _log(rng, 1, min(262144, (1 << 26) // D))
        return _norm_case("", op, R, D, x, rng.choice(["layer", "rms"]), rng.random() < 0.5)
    g = F32 if x == F32 else rng.choice([BF16, F32])
    gate = rng.choice(["value", "logit"]) if g == F32 else "logit"
    D = rng.choice([64 * _log(rng, 1, 128), 64 * _log(rng, 1, 128), _log(rng, 1, 8192)])
    tied, state = rng.random() < 0.5, rng.random() < 0.5
    if op == "scan_step":
        return _scan_case("", op, _log(rng, 1, min(8192, (1 << 25) // D)), 1, D, x, g, gate, tied, True)
    T = _log(rng, 1, min(65536, (1 << 26) // D))
    if rng.random() < 0.35:
        return _scan_case("", op, 1, T, D, x, g, gate, tied, state, _log(rng, 1, 64))
    return _scan_case("", op, _log(rng, 1, max(1, min(16, (1 << 26) // (D * T)))), T, D, x, g, gate, tied, state)


def _offsets(case, gen):
    """Offsets of nseq sequences that fill T tokens, ragged (an empty one can occur)."""
    cuts = torch.randint(0, case["T"] + 1, (case["nseq"] - 1,), generator=gen, device="cuda")
    ends = torch.tensor([0, case["T"]], device="cuda")
    return torch.cat([ends[:1], cuts.sort().values, ends[1:]]).to(torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["x"]]
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"].startswith("norm"):
        R, D = case["R"], case["D"]
        scale = 0.5 + torch.rand(R, 1, generator=gen, device="cuda")
        s["x"] = (rn(R, D) * scale + 0.2 * rn(R, 1)).to(dt)
        s["w"] = 1.0 + 0.1 * rn(D)
        s["b"] = 0.1 * rn(D) if case["bias"] else None
        if case["op"] == "norm_bwd":
            s["dy"] = rn(R, D).to(dt)
            # what the forward pass left for the backward pass
            _, s["mean"], s["rstd"] = _plain_norm_fwd(s)
        return s
    B, T, D = case["B"], case["T"], case["D"]
    step = case["op"] == "scan_step"
    shape = (B, D) if step else (B, T, D)
    g = rn(*shape)
    if case["gate"] == "logit":
        g = (g + 3.0).to(_DT[case["g"]])
    else:
        g = torch.exp(-torch.nn.functional.softplus(g) / 16.0).to(_DT[case["g"]])
    s["x"], s["g"] = rn(*shape).to(dt), g
    if step:
        s["h0"] = rn(B, D)
        return s
    s["cu"], s["max_seqlen"], n = None, None, B
    if case["nseq"]:
        s["cu"], n = _offsets(case, gen), case["nseq"]
        s["max_seqlen"] = int((s["cu"][1:] - s["cu"][:-1]).max())
    s["h0"] = rn(n, D) if case["state"] else None
    if case["op"] == "scan_bwd":
        s["h"], _ = _plain_scan_fwd(s)   # the outputs that the forward pass stored
        s["dh"] = rn(*shape).to(dt)
        s["dh_last"] = rn(n, D) if case["state"] else None
        if not case["tied"]:
            s["x"] = None                # the backward pass of an untied input does not read it
    return s


# ---------------------------------------------------------------------------
# Plain forms: elementary operations in 32 bits, rounded once at the end.
# ---------------------------------------------------------------------------
def _gates(s):
    """a and the factor of x."""
    g = s["g"].float()
    if s["gate"] == "logit":
        a, r = torch.sigmoid(g), torch.sigmoid(-g)
    else:
        a, r = g, 1.0 - g
    return a, (r if s["tied"] else None)


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1 (h_{-1} = 0): pairs of tokens become one, then the odd places give the even ones."""
    T = a.shape[1]
    if T == 1:
        return u
    n, m = T // 2, (T - 1) // 2
    a1 = a[:, 1:2 * n:2]
    odd = _scan(a1 * a[:, 0:2 * n:2], a1 * u[:, 0:2 * n:2] + u[:, 1:2 * n:2])
    h = torch.empty_like(u)
    h[:, 1:2 * n:2] = odd
    h[:, 0] = u[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :m] + u[:, 2::2]
    return h


def _bounds(s):
    """First and last token of every sequence that is not empty, on axes (row, token), and which sequences those are."""
    if s["cu"] is None:
        n = torch.arange(s["B"], device="cuda")
        return n, torch.zeros_like(n), n, torch.full_like(n, s["T"] - 1), n
    full = (s["cu"][1:] > s["cu"][:-1]).nonzero()[:, 0]
    row = torch.zeros_like(full)
    return row, s["cu"][:-1][full], row, s["cu"][1:][full] - 1, full


def _plain_scan_fwd(s):
    a, r = _gates(s)
    u = s["x"].float() * r if s["tied"] else s["x"].to(torch.float32, copy=True)
    fr, ft, lr, lt, full = _bounds(s)
    n = s["B"] if s["cu"] is None else s["nseq"]
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(n, s["D"], device="cuda")
    u[fr, ft] += a[fr, ft] * h0[full]
    a = a.clone()
    a[fr, ft] = 0.0
    h = _scan(a, u)
    h_last = h0.clone()
    h_last[full] = h[lr, lt]
    return h.to(s["x"].dtype), h_last


def _plain_scan_bwd(s):
    a, r = _gates(s)
    fr, ft, lr, lt, full = _bounds(s)
    n = s["B"] if s["cu"] is None else s["nseq"]
    zero = torch.zeros(n, s["D"], device="cuda")
    h0 = s["h0"] if s["h0"] is not None else zero
    dl = s["dh_last"] if s["dh_last"] is not None else zero
    G = s["dh"].to(torch.float32, copy=True)
    G[lr, lt] += dl[full]
    nxt = torch.zeros_like(a)            # the gate of the following token of the same sequence
    nxt[:, :-1] = a[:, 1:]
    nxt[lr, lt] = 0.0
    G = _scan(nxt.flip(1), G.flip(1)).flip(1)
    prev = torch.zeros_like(a)
    prev[:, 1:] = s["h"][:, :-1].float()
    prev[fr, ft] = h0[full]
    da = G * (prev - s["x"].float()) if s["tied"] else G * prev
    if s["gate"] == "logit":
        da = da * a * torch.sigmoid(-s["g"].float())
    dx = G * r if s["tied"] else G
    dh0 = dl.clone()
    dh0[full] = a[fr, ft] * G[fr, ft]
    return dx.to(s["dh"].dtype), da.to(s["g"].dtype), dh0


def _plain_scan_step(s):
    a, r = _gates(s)
    x = s["x"].float()
    s["h0"].copy_(a * s["h0"] + (r * x if s["tied"] else x))
    return s["h0"].to(s["x"].dtype), s["h0"]


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1) if s["kind"] == "layer" else None
    xc = x - mean[:, None] if mean is not None else x
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + EPS)
    y = xc * rstd[:, None] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd if s["kind"] == "layer" else x * rstd
    d = dy * s["w"]
    dx = d - xh * (d * xh).mean(1, keepdim=True)
    if s["kind"] == "layer":
        dx = dx - d.mean(1, keepdim=True)
    dw = (dy * xh).sum(0)
    db = dy.sum(0) if s["b"] is not None else None
    return (dx * rstd).to(s["x"].dtype), dw, db


def run(s):
    op = s["op"]
    if not own:
        return {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
                "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[op](s)
    import gated_delta_rule_attn_b200 as la
    if op == "scan_fwd":
        return la.scan_fwd(s["x"], s["g"], s["h0"], gate=s["gate"], tied=s["tied"],
                           cu_seqlens=s["cu"], max_seqlen=s["max_seqlen"])
    if op == "scan_bwd":
        return la.scan_bwd(s["g"], s["h"], s["dh"], x=s["x"], h0=s["h0"], dh_last=s["dh_last"],
                           gate=s["gate"], tied=s["tied"], cu_seqlens=s["cu"], max_seqlen=s["max_seqlen"])
    if op == "scan_step":
        return la.scan_step(s["x"], s["g"], s["h0"], gate=s["gate"], tied=s["tied"]), s["h0"]
    if op == "norm_fwd":
        return la.norm_fwd(s["x"], s["w"], s["b"], kind=s["kind"], eps=EPS)
    return la.norm_bwd(s["dy"], s["x"], s["rstd"], mean=s["mean"], w=s["w"], kind=s["kind"],
                       want_db=s["b"] is not None)


def work(case):
    ex = _SIZE[case["x"]]
    if case["op"].startswith("norm"):
        R, D = case["R"], case["D"]
        stats = 8 if case["kind"] == "layer" else 4
        cols = 8 if case["bias"] else 4
        if case["op"] == "norm_fwd":
            return {"bytes": R * (2 * D * ex + stats) + D * cols, "flops": 8 * R * D}
        return {"bytes": R * (3 * D * ex + stats) + D * (4 + cols), "flops": 14 * R * D}
    eg, n = _SIZE[case["g"]], case["B"] * case["T"] * case["D"]
    if case["op"] == "scan_step":
        return {"bytes": n * (2 * ex + eg + 8), "flops": 4 * n}
    seqs = (case["nseq"] or case["B"]) * case["D"] * 4
    if case["op"] == "scan_fwd":
        return {"bytes": n * (2 * ex + eg) + seqs * (2 if case["state"] else 1), "flops": 4 * n}
    return {"bytes": n * ((4 if case["tied"] else 3) * ex + 2 * eg) + seqs * (3 if case["state"] else 1), "flops": 8 * n}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, token after token.
# ---------------------------------------------------------------------------
def _spans(s):
    if s["cu"] is None:
        return [(slice(0, s["B"]), slice(0, s["B"]), 0, s["T"])]
    cu = s["cu"].tolist()
    return [(slice(0, 1), slice(i, i + 1), cu[i], cu[i + 1]) for i in range(s["nseq"])]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op.startswith("norm"):
        x, w = s["x"].double(), s["w"].double()
        D = s["D"]
        if op == "norm_fwd":
            mean = x.sum(1) / D if s["kind"] == "layer" else None
            c = x if mean is None else x - mean[:, None]
            rstd = (c.square().sum(1) / D + EPS).rsqrt()
            y = c * (rstd[:, None] * w)
            return (y if s["b"] is None else y + s["b"].double()), mean, rstd
        c = x if s["kind"] == "rms" else x - s["mean"].double()[:, None]
        rs = s["rstd"].double()[:, None]
        dy = s["dy"].double()
        dot = torch.einsum("rd,rd,d->r", dy, c, w)[:, None] * rs
        dx = rs * (dy * w - c * rs * dot / D)
        if s["kind"] == "layer":
            dx -= rs * (torch.mv(dy, w)[:, None] / D)
        dw = torch.mm((rs * c).mul_(dy).t(), torch.ones(s["R"], 1, dtype=torch.float64, device="cuda"))[:, 0]
        return dx, dw, (dy.sum(0) if s["b"] is not None else None)
    g = s["g"].double()
    a = 1.0 / (1.0 + torch.exp(-g)) if s["gate"] == "logit" else g
    x = s["x"].double() if s["x"] is not None else None
    if op == "scan_step":
        h = a * s["h0"].double() + ((1.0 - a) * x if s["tied"] else x)
        return h, h
    n = s["B"] if s["cu"] is None else s["nseq"]
    state = torch.zeros(n, s["D"], dtype=torch.float64, device="cuda")
    if op == "scan_fwd":
        if s["h0"] is not None:
            state += s["h0"]
        out = (1.0 - a) * x if s["tied"] else x.clone()
        for rows, seqs, t0, t1 in _spans(s):
            h = state[seqs]
            for t in range(t0, t1):
                h = out[rows, t].addcmul_(a[rows, t], h)
            state[seqs] = h
        return out, state
    if s["dh_last"] is not None:
        state += s["dh_last"]
    first = s["h0"].double() if s["h0"] is not None else torch.zeros_like(state)
    G, h = s["dh"].double(), s["h"].double()
    before = torch.empty_like(h)
    for rows, seqs, t0, t1 in _spans(s):
        c = state[seqs]
        for t in range(t1 - 1, t0 - 1, -1):
            c = a[rows, t] * G[rows, t].add_(c)
        state[seqs] = c
        if t1 > t0:
            before[rows, t0] = first[seqs]
            before[rows, t0 + 1:t1] = h[rows, t0:t1 - 1]
    if s["tied"]:
        da, dx = G * (before - x), G * (1.0 - a)
    else:
        da, dx = G * before, G
    if s["gate"] == "logit":
        da = da * (a - a.square())
    return dx, da, state
