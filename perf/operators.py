"""The recurrent operators around the selective scan, as they are measured: the gated linear
recurrence and its gradient, the gradient of the selective scan, the single-token step over a
pool of states, and the parking of states in 8 or 4 bits.

``run`` computes an operator in elementary torch operations where ``own`` is false and through the
package's entry points where it is true; ``exact`` states the definition step by step in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
FWD, REV, COL, COL_REV = 0, 1, 2, 3
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one layer of a 130M-parameter model over a training batch: sigmoid gate, leaky input
        dict(name="recurrence_layer", op="recurrence", batch=8, L=2048, D=1536, io="bf16",
             form="sigmoid", complement=True, reverse=False, initial=False),
        # the prefill of one very long sequence: few rows, the work has to be split along time
        dict(name="recurrence_long", op="recurrence", batch=1, L=131072, D=5120, io="bf16",
             form="exp", complement=False, reverse=False, initial=False),
        # a small bidirectional vision layer's backward order, fp32, continued from a state
        dict(name="recurrence_short_f32", op="recurrence", batch=4, L=197, D=768, io="f32",
             form="sigmoid", complement=True, reverse=True, initial=True),
        # the gradient of the first case, as a training step needs it
        dict(name="recurrence_bwd_layer", op="recurrence_bwd", batch=8, L=2048, D=1536, io="bf16",
             form="sigmoid", complement=True, reverse=False, initial=False),
        # an odd length and width in fp32, with a carried state and its gradient
        dict(name="recurrence_bwd_f32", op="recurrence_bwd", batch=2, L=3137, D=200, io="f32",
             form="exp", complement=False, reverse=False, initial=True),
        # training one layer of a 130M-parameter selective-scan model
        dict(name="scan_bwd_layer", op="scan_bwd", batch=8, L=2048, D=1536, N=16, io="bf16",
             dirs="0", H=0, W=0, gate=True, initial=False),
        # training a bidirectional vision layer: 64 images of 196 patches and a class token
        dict(name="scan_bwd_bidirectional", op="scan_bwd", batch=64, L=197, D=768, N=16, io="bf16",
             dirs="01", H=0, W=0, gate=True, initial=False),
        # fp32 fine-tuning on short ragged chunks that continue from a state, 11 states
        dict(name="scan_bwd_f32", op="scan_bwd", batch=2, L=333, D=72, N=11, io="f32", dirs="0",
             H=0, W=0, gate=True, initial=True),
        # decoding one sequence: a token's latency, with the causal convolution's window
        dict(name="step_single", op="step", batch=1, D=1536, N=16, io="bf16", width=4, slots=4,
             padded=0, gate=True),
        # decoding a serving batch out of a pool of states, some rows padding
        dict(name="step_batch", op="step", batch=256, D=5120, N=16, io="bf16", width=4, slots=320,
             padded=3, gate=True),
        # parking and resuming the states of many sequences of one layer in 8 bits
        dict(name="state_cache_int8", op="state", rows=256, slots=300, D=5120, N=16, bits=8),
        # the same for a few sequences in 4 bits
        dict(name="state_cache_int4", op="state", rows=5, slots=9, D=1536, N=16, bits=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["recurrence", "recurrence_bwd", "scan_bwd", "step", "state"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("recurrence", "recurrence_bwd"):
        batch, L, D = _log(rng, 1, 32), _log(rng, 1, 65536), 8 * _log(rng, 1, 640)
        while batch * L * D > 1 << 25:
            batch, L = max(1, batch // 2), max(1, L * 2 // 3)
        return dict(op=op, batch=batch, L=L, D=D, io=io, form=rng.choice(["sigmoid", "exp"]),
                    complement=rng.random() < 0.5, reverse=rng.random() < 0.3,
                    initial=rng.random() < 0.5)
    if op == "scan_bwd":
        dirs = rng.choice(["0", "0", "1", "01", "0213"])
        batch, L, D, N = _log(rng, 1, 32), _log(rng, 1, 8192), 8 * _log(rng, 1, 256), rng.randint(1, 16)
        H = W = 0
        if dirs == "0213":
            H, W = rng.randint(3, 60), rng.randint(3, 60)
            L = H * W
        while batch * L * D * N * len(dirs) > 1 << 28:
            if batch > 1:
                batch //= 2
            else:
                D = 8 * max(1, D // 16)
        return dict(op=op, batch=batch, L=L, D=D, N=N, io=io, dirs=dirs, H=H, W=W,
                    gate=rng.random() < 0.7, initial=rng.random() < 0.5)
    if op == "step":
        batch = _log(rng, 1, 512)
        return dict(op=op, batch=batch, D=8 * _log(rng, 1, 640), N=rng.randint(1, 16), io=io,
                    width=rng.choice([0, 2, 3, 4]), slots=batch + rng.randint(0, 40),
                    padded=rng.randint(0, max(0, batch // 8)), gate=rng.random() < 0.8)
    rows = _log(rng, 1, 512)
    return dict(op=op, rows=rows, slots=rows + rng.randint(0, 40), D=8 * _log(rng, 1, 640),
                N=rng.randint(1, 16), bits=rng.choice([4, 8]))


# ------------------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _log_uniform(g, shape, lo, hi):
    u = torch.rand(shape, generator=g, device=DEV, dtype=torch.float64)
    return torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo)))


def prepare(case, seed):
    make = {"recurrence": _prepare_recurrence, "recurrence_bwd": _prepare_recurrence,
            "scan_bwd": _prepare_scan, "step": _prepare_step, "state": _prepare_state}
    return make[case["op"]](case, _generator(seed))


def _prepare_recurrence(c, g):
    b, L, D, io = c["batch"], c["L"], c["D"], TYPES[c["io"]]
    s = dict(case=c, x=_normal(g, (b, L, D), io))
    memory = _log_uniform(g, (D,), 8, 1000)  # steps that a channel remembers
    if c["form"] == "sigmoid":
        s["gate"] = _normal(g, (b, L, D), io)
        s["bias"] = torch.log(memory - 1).float()  # sigmoid(bias) = 1 - 1/memory
    else:
        s["gate"] = (-torch.exp(0.5 * _normal(g, (b, L, D))) / memory.float()).to(io)
        s["bias"] = None
    s["h0"] = _normal(g, (b, D)) if c["initial"] else None
    if c["op"].endswith("_bwd"):
        # what the forward pass kept, and the gradients that come in
        s["out"] = _recurrence(s)["out"]
        s["dout"] = _normal(g, (b, L, D), io)
        s["dlast"] = _normal(g, (b, D)) if c["initial"] else None
    return s


def _prepare_scan(c, g):
    b, L, D, N, K, io = c["batch"], c["L"], c["D"], c["N"], len(c["dirs"]), TYPES[c["io"]]
    delta0 = _log_uniform(g, (D,), 1e-3, 1e-1)
    s = dict(case=c, dirs=tuple(int(d) for d in c["dirs"]),
             u=_normal(g, (b, L, D), io), delta=_normal(g, (K, b, L, D), io),
             # trained decay rates: near -(n+1), no longer on it
             A=-(torch.arange(1, N + 1, device=DEV) * torch.exp(0.1 * _normal(g, (D, N)))).float(),
             B=_normal(g, (K, b, L, N), io), C=_normal(g, (K, b, L, N), io),
             D=1 + 0.1 * _normal(g, (D,)), bias=(delta0 + torch.log(-torch.expm1(-delta0))).float(),
             z=_normal(g, (b, L, D), io) if c["gate"] else None,
             h0=_normal(g, (K, b, D, N)) if c["initial"] else None,
             dout=_normal(g, (b, L, D), io),
             dlast=_normal(g, (K, b, D, N)) if c["initial"] else None)
    return s


def _prepare_step(c, g):
    b, D, N, io, S, w = c["batch"], c["D"], c["N"], TYPES[c["io"]], c["slots"], c["width"]
    delta0 = _log_uniform(g, (D,), 1e-3, 1e-1)
    slots = torch.randperm(S, generator=g, device=DEV)[:b].to(torch.int32)
    if c["padded"]:
        slots[-c["padded"]:] = -1
    s = dict(case=c, slots=slots, state=_normal(g, (S, D, N)),
             u=_normal(g, (b, D), io), delta=_normal(g, (b, D), io),
             A=-(torch.arange(1, N + 1, device=DEV) * torch.exp(0.1 * _normal(g, (D, N)))).float(),
             B=_normal(g, (b, N), io), C=_normal(g, (b, N), io), D=1 + 0.1 * _normal(g, (D,)),
             bias=(delta0 + torch.log(-torch.expm1(-delta0))).float(),
             z=_normal(g, (b, D), io) if c["gate"] else None,
             out=torch.zeros((b, D), dtype=io, device=DEV))
    s["cw"] = _normal(g, (D, w)) / math.sqrt(w) if w else None
    s["cb"] = 0.1 * _normal(g, (D,)) if w else None
    s["window"] = _normal(g, (S, w - 1, D), io) if w else None
    return s


def _prepare_state(c, g):
    S, D, N, R = c["slots"], c["D"], c["N"], c["rows"]
    # states of one channel: faster decays hold less
    live = _normal(g, (S, D, N)) * _log_uniform(g, (S, D, 1), 0.05, 20).float()
    live = live / torch.arange(1, N + 1, device=DEV).sqrt()
    pick = lambda: torch.randperm(S, generator=g, device=DEV)[:R].to(torch.int32)  # noqa: E731
    width = N if c["bits"] == 8 else (N + 1) // 2
    return dict(case=c, live=live, src=pick(), parked=pick(), dst=pick(),
                codes=torch.zeros((S, D, width), dtype=torch.int8, device=DEV),
                scales=torch.zeros((S, D), device=DEV), resumed=torch.zeros((S, D, N), device=DEV))


# ------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"recurrence": _own_recurrence, "recurrence_bwd": _own_recurrence_bwd,
                "scan_bwd": _own_scan_bwd, "step": _own_step, "state": _own_state}[op](s)
    return {"recurrence": _recurrence, "recurrence_bwd": _recurrence_bwd, "scan_bwd": _scan_bwd,
            "step": _step, "state": _state}[op](s)


def _own_recurrence(s):
    from selective_state_space_13_b200 import ops
    c = s["case"]
    out, last = ops.gated_recurrence_fwd(
        s["x"], s["gate"], gate_bias=s["bias"], initial_state=s["h0"], form=c["form"],
        complement=c["complement"], reverse=c["reverse"], return_last_state=True)
    return {"out": out, "last": last}


def _own_recurrence_bwd(s):
    from selective_state_space_13_b200 import ops
    c = s["case"]
    dx, dgate, dbias, dh0 = ops.gated_recurrence_bwd(
        s["dout"], s["x"], s["gate"], s["out"], gate_bias=s["bias"], initial_state=s["h0"],
        dlast_state=s["dlast"], form=c["form"], complement=c["complement"], reverse=c["reverse"])
    return {"dx": dx, "dgate": dgate, "dbias": dbias, "dh0": dh0}


def _own_scan_bwd(s):
    from selective_state_space_13_b200 import ops
    c = s["case"]
    return ops.selective_scan_bwd(
        s["dout"], s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
        delta_bias=s["bias"], dirs=s["dirs"], H=c["H"], W=c["W"], initial_state=s["h0"],
        dlast_state=s["dlast"])


def _own_step(s):
    from selective_state_space_13_b200 import ops
    ops.selective_scan_step(
        s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
        delta_bias=s["bias"], slots=s["slots"], conv_weight=s["cw"], conv_bias=s["cb"],
        conv_state=s["window"], out=s["out"])
    return {"out": s["out"], "state": s["state"], "window": s["window"]}


def _own_state(s):
    from selective_state_space_13_b200 import ops
    bits = s["case"]["bits"]
    ops.selective_state_store(s["live"], s["codes"], s["scales"], bits=bits, src_slots=s["src"],
                              dst_slots=s["parked"])
    ops.selective_state_load(s["codes"], s["scales"], s["resumed"], bits=bits,
                             src_slots=s["parked"], dst_slots=s["dst"])
    return {"resumed": s["resumed"], "scales": s["scales"]}


# ---------------------------------------------------------------- the plain forms: elementary torch

def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t from zero along dimension 1, by doubling: after the pass with
    distance d every step holds the composition of its last 2d maps."""
    d, L = 1, b.shape[1]
    while d < L:
        b = torch.cat([b[:, :d], torch.addcmul(b[:, d:], a[:, d:], b[:, :-d])], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1) if 2 * d < L else a
        d *= 2
    return b


def _scan_from(a, b, h0):
    """The same from the state h0 (None: zero)."""
    if h0 is not None:
        b = torch.cat([torch.addcmul(b[:, :1], a[:, :1], h0.unsqueeze(1)), b[:, 1:]], 1)
    return _linear_scan(a, b)


def _scan_back(a, b, last):
    """g_t = b_t + a_{t+1} g_{t+1} along dimension 1, with `last` added to the last step."""
    b = b.flip(1)
    if last is not None:
        b = torch.cat([b[:, :1] + last.unsqueeze(1), b[:, 1:]], 1)
    a = torch.cat([torch.zeros_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    return _linear_scan(a, b).flip(1)


def _gates(s):
    c = s["case"]
    x, gate = s["x"].float(), s["gate"].float()
    if c["reverse"]:
        x, gate = x.flip(1), gate.flip(1)
    if s["bias"] is not None:
        gate = gate + s["bias"]
    if c["form"] == "sigmoid":
        a, rest = 1 / (1 + torch.exp(-gate)), 1 / (1 + torch.exp(gate))
    else:
        a, rest = torch.exp(gate), -torch.expm1(gate)
    return x, a, rest


def _recurrence(s):
    c = s["case"]
    x, a, rest = _gates(s)
    h = _scan_from(a, rest * x if c["complement"] else x, s["h0"])
    last = h[:, -1].clone()
    return {"out": (h.flip(1) if c["reverse"] else h).to(s["x"].dtype), "last": last}


def _recurrence_bwd(s):
    c, io = s["case"], s["x"].dtype
    x, a, rest = _gates(s)
    dout, out = s["dout"].float(), s["out"].float()
    if c["reverse"]:
        dout, out = dout.flip(1), out.flip(1)
    first = torch.zeros_like(out[:, :1]) if s["h0"] is None else s["h0"].unsqueeze(1)
    before = torch.cat([first, out[:, :-1]], 1)  # the state before each step, as it was kept
    g = _scan_back(a, dout, s["dlast"])
    dx = rest * g if c["complement"] else g
    ds = g * (before - x if c["complement"] else before) * a
    if c["form"] == "sigmoid":
        ds = ds * rest
    r = {"dbias": None if s["bias"] is None else ds.sum((0, 1)),
         "dh0": None if s["h0"] is None else a[:, 0] * g[:, 0]}
    if c["reverse"]:
        dx, ds = dx.flip(1), ds.flip(1)
    return {"dx": dx.to(io), "dgate": ds.to(io), **r}


def _order(d, L, H, W):
    """The position that each step of an order visits."""
    t = torch.arange(L, device=DEV)
    if d in (COL, COL_REV):
        t = (t % H) * W + t // H
    return t.flip(0) if d in (REV, COL_REV) else t


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _scan_bwd(s):
    c, io = s["case"], s["u"].dtype
    A, Dskip = s["A"], s["D"]
    u, dout = s["u"].float(), s["dout"].float()
    z = None if s["z"] is None else s["z"].float()
    sig = None if z is None else 1 / (1 + torch.exp(-z))
    dy_at = dout if z is None else dout * z * sig
    du, y_at = torch.zeros_like(u), torch.zeros_like(u)
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(Dskip), torch.zeros_like(s["bias"])
    ddelta, dB, dC, dh0 = [], [], [], []
    for k, d in enumerate(s["dirs"]):
        p = _order(d, c["L"], c["H"], c["W"])
        raw = s["delta"][k].float() + s["bias"]
        uk, dy, Bk, Ck = u[:, p], dy_at[:, p], s["B"][k].float(), s["C"][k].float()
        step = _softplus(raw)
        a = torch.exp(step.unsqueeze(-1) * A)
        h0 = None if s["h0"] is None else s["h0"][k]
        h = _scan_from(a, (step * uk).unsqueeze(-1) * Bk.unsqueeze(2), h0)
        g = _scan_back(a, dy.unsqueeze(-1) * Ck.unsqueeze(2),
                       None if s["dlast"] is None else s["dlast"][k])
        if z is not None:
            y_at[:, p] += (h * Ck.unsqueeze(2)).sum(-1) + Dskip * uk
        dC.append((dy.unsqueeze(-1) * h).sum(2))
        dB.append((g * (step * uk).unsqueeze(-1)).sum(2))
        gB = (g * Bk.unsqueeze(2)).sum(-1)
        du[:, p] += Dskip * dy + step * gB
        first = torch.zeros_like(h[:, :1]) if h0 is None else h0.unsqueeze(1)
        ga = g * a * torch.cat([first, h[:, :-1]], 1)  # gradient of Delta A, per state
        draw = (uk * gB + (ga * A).sum(-1)) / (1 + torch.exp(-raw))
        ddelta.append(draw)
        dA += (ga * step.unsqueeze(-1)).sum((0, 1))
        dD += (dy * uk).sum((0, 1))
        dbias += draw.sum((0, 1))
        dh0.append(a[:, 0] * g[:, 0])
    stack = lambda v: torch.stack(v).to(io)  # noqa: E731
    return {"du": du.to(io), "ddelta": stack(ddelta), "dA": dA, "dB": stack(dB), "dC": stack(dC),
            "dD": dD, "dz": None if z is None else
            (dout * y_at * sig * (1 + z * (1 - sig))).to(io), "ddelta_bias": dbias,
            "dinitial_state": None if s["h0"] is None else torch.stack(dh0)}


def _step(s):
    io = s["u"].dtype
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][rows].long()
    u = s["u"][rows].float()
    if s["cw"] is not None:
        seen = torch.cat([s["window"][at], s["u"][rows].unsqueeze(1)], 1)
        s["window"][at] = seen[:, 1:]
        u = (seen.float() * s["cw"].t()).sum(1) + s["cb"]
        u = u / (1 + torch.exp(-u))
    step = _softplus(s["delta"][rows].float() + s["bias"])
    h = torch.exp(step.unsqueeze(-1) * s["A"]) * s["state"][at]
    h = h + (step * u).unsqueeze(-1) * s["B"][rows].float().unsqueeze(1)
    s["state"][at] = h
    y = (h * s["C"][rows].float().unsqueeze(1)).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"][rows].float()
        y = y * z / (1 + torch.exp(-z))
    s["out"][rows] = y.to(io)
    return {"out": s["out"], "state": s["state"], "window": s["window"]}


def _state(s):
    c, N = s["case"], s["case"]["N"]
    q = 127 if c["bits"] == 8 else 7
    h = s["live"][s["src"].long()]
    amax = h.abs().amax(-1, keepdim=True).double()
    # in 64 bits, so that values next to the border of two codes fall on the right side
    codes = torch.round(h.double() * q / amax.clamp(min=1e-300)).to(torch.int8)
    at = s["parked"].long()
    if c["bits"] == 4:  # two codes a byte, the even state in the low half
        codes = torch.nn.functional.pad(codes, (0, N % 2))
        codes = (codes[..., 0::2] & 15) | (codes[..., 1::2] << 4)
    s["codes"][at] = codes
    s["scales"][at] = (amax[..., 0] / q).float()
    codes = s["codes"][at]
    if c["bits"] == 4:
        codes = torch.stack([(codes << 4) >> 4, codes >> 4], -1).flatten(-2)[..., :N]
    s["resumed"][s["dst"].long()] = codes.float() * s["scales"][at].unsqueeze(-1)
    return {"resumed": s["resumed"], "scales": s["scales"]}


# ------------------------------------------------------------------------------------- floors

def work(c):
    e = 2 if c.get("io") == "bf16" else 4
    if c["op"].startswith("recurrence"):
        n = c["batch"] * c["L"] * c["D"]
        states = c["batch"] * c["D"] * 4 * (2 if c["initial"] else 1)
        if c["op"] == "recurrence":
            return {"bytes": 3 * n * e + states + 4 * c["D"], "flops": 8 * n}
        return {"bytes": (6 if c["complement"] else 5) * n * e + 3 * states, "flops": 16 * n}
    if c["op"] == "scan_bwd":
        K, N = len(c["dirs"]), c["N"]
        rows, n = c["batch"] * c["L"], c["batch"] * c["L"] * c["D"]
        # u, dout and du, z and dz; Delta and its gradient; B, C and theirs; parameters; states
        bytes_ = (3 + (2 if c["gate"] else 0) + 2 * K) * n * e + 4 * K * rows * N * e
        bytes_ += 2 * 4 * c["D"] * (N + 2)
        bytes_ += 3 * 4 * K * c["batch"] * c["D"] * N if c["initial"] else 0
        return {"bytes": bytes_, "flops": 22 * K * n * N}
    if c["op"] == "step":
        rows, D, N = c["batch"] - c["padded"], c["D"], c["N"]
        bytes_ = rows * D * (8 * N + (4 if c["gate"] else 3) * e) + rows * 2 * N * e
        bytes_ += rows * D * 2 * (c["width"] - 1) * e if c["width"] else 0
        bytes_ += 4 * D * (N + 2 + (c["width"] + 1 if c["width"] else 0))
        return {"bytes": max(1, bytes_), "flops": 7 * rows * D * N}
    n = c["rows"] * c["D"]
    width = c["N"] if c["bits"] == 8 else (c["N"] + 1) // 2
    return {"bytes": n * (8 * c["N"] + 2 * width + 8), "flops": 4 * n * c["N"]}


# ------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    """What run() returns, from the definition, one step after the other, in 64 bits."""
    define = {"recurrence": _exact_recurrence, "recurrence_bwd": _exact_recurrence_bwd,
              "scan_bwd": _exact_scan_bwd, "step": _exact_step, "state": _exact_state}
    return define[case["op"]](prepare(case, seed))


def _d(t):
    return None if t is None else t.double()


def _decay64(s):
    gate = _d(s["gate"])
    if s["case"]["form"] == "sigmoid":
        return torch.sigmoid(gate + _d(s["bias"])), torch.sigmoid(-gate - _d(s["bias"]))
    return torch.exp(gate), -torch.expm1(gate)


def _exact_recurrence(s):
    c = s["case"]
    a, rest = _decay64(s)
    b = _d(s["x"]).mul_(rest) if c["complement"] else _d(s["x"])
    del rest
    h = torch.zeros_like(b[:, 0]) if s["h0"] is None else _d(s["h0"])
    for t in range(c["L"] - 1, -1, -1) if c["reverse"] else range(c["L"]):
        b[:, t] += a[:, t] * h
        h = b[:, t]
    return {"out": b, "last": h.clone()}


def _exact_recurrence_bwd(s):
    c, L = s["case"], s["case"]["L"]
    a, rest = _decay64(s)
    x, out, g = _d(s["x"]), _d(s["out"]), _d(s["dout"]).clone()
    order = list(range(L - 1, -1, -1) if c["reverse"] else range(L))
    carry = torch.zeros_like(g[:, 0]) if s["dlast"] is None else _d(s["dlast"])
    before = torch.empty_like(out)
    for i in range(L - 1, -1, -1):
        t = order[i]
        g[:, t] += carry
        carry = a[:, t] * g[:, t]
        before[:, t] = out[:, order[i - 1]] if i else (0 if s["h0"] is None else _d(s["h0"]))
    lam = before - x if c["complement"] else before
    dgate = g * lam * a * (rest if c["form"] == "sigmoid" else 1)
    return {"dx": g * rest if c["complement"] else g, "dgate": dgate,
            "dbias": None if s["bias"] is None else dgate.sum((0, 1)),
            "dh0": None if s["h0"] is None else carry}


def _exact_scan_bwd(s):
    c = s["case"]
    b, L, D, N, K = c["batch"], c["L"], c["D"], c["N"], len(s["dirs"])
    u, delta, A, B, C, dout = (_d(s[n]) for n in ("u", "delta", "A", "B", "C", "dout"))
    Dskip, bias, z = _d(s["D"]), _d(s["bias"]), _d(s["z"])
    gate = torch.ones_like(u) if z is None else z * torch.sigmoid(z)
    y, du = torch.zeros_like(u), torch.zeros_like(u)
    ddelta, dB, dC = torch.zeros_like(delta), torch.zeros_like(B), torch.zeros_like(C)
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(Dskip), torch.zeros_like(bias)
    dh0 = torch.zeros(K, b, D, N, dtype=torch.float64, device=DEV)
    for k, d in enumerate(s["dirs"]):
        pos = [(t if d == FWD else L - 1 - t if d == REV else None) for t in range(L)]
        if d in (COL, COL_REV):
            walk = [i * c["W"] + j for j in range(c["W"]) for i in range(c["H"])]
            pos = walk if d == COL else walk[::-1]
        h = torch.zeros(b, D, N, dtype=torch.float64, device=DEV) if s["h0"] is None else _d(s["h0"][k])
        hs = [h]
        for t in range(L):
            dt = torch.nn.functional.softplus(delta[k, :, t] + bias, threshold=700)
            h = torch.exp(dt[..., None] * A) * h + (dt * u[:, pos[t]])[..., None] * B[k, :, t, None]
            hs.append(h)
            y[:, pos[t]] += (h * C[k, :, t, None]).sum(-1) + Dskip * u[:, pos[t]]
        g = torch.zeros_like(h) if s["dlast"] is None else _d(s["dlast"][k])
        for t in range(L - 1, -1, -1):
            p, raw = pos[t], delta[k, :, t] + bias
            dt, up = torch.nn.functional.softplus(raw, threshold=700), u[:, p]
            dy = dout[:, p] * gate[:, p]
            g = g + dy[..., None] * C[k, :, t, None]
            dC[k, :, t] = (dy[..., None] * hs[t + 1]).sum(1)
            dB[k, :, t] = (g * (dt * up)[..., None]).sum(1)
            gb = (g * B[k, :, t, None]).sum(-1)
            carry = g * torch.exp(dt[..., None] * A)
            dlog = carry * hs[t]
            dA += (dlog * dt[..., None]).sum(0)
            ddt = up * gb + (dlog * A).sum(-1)
            ddelta[k, :, t] = ddt * torch.sigmoid(raw)
            du[:, p] += Dskip * dy + dt * gb
            dD += (dy * up).sum(0)
            g = carry
        dh0[k] = g
        dbias += ddelta[k].sum((0, 1))
    dz = None
    if z is not None:
        sg = torch.sigmoid(z)
        dz = dout * y * (sg + z * sg * (1 - sg))
    return {"du": du, "ddelta": ddelta, "dA": dA, "dB": dB, "dC": dC, "dD": dD, "dz": dz,
            "ddelta_bias": dbias, "dinitial_state": None if s["h0"] is None else dh0}


def _exact_step(s):
    c, w = s["case"], s["case"]["width"]
    out, state, window = _d(s["out"]), _d(s["state"]), _d(s["window"])
    u, delta, A, B, C, D, bias, z = (_d(s[n]) for n in ("u", "delta", "A", "B", "C", "D", "bias", "z"))
    for r, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        v = u[r]
        if w:
            v = _d(s["cb"]) + _d(s["cw"][:, w - 1]) * u[r]
            for j in range(w - 1):
                v = v + _d(s["cw"][:, j]) * window[slot, j]
            window[slot] = torch.cat([window[slot, 1:], u[r][None]])
            v = v * torch.sigmoid(v)
        dt = torch.nn.functional.softplus(delta[r] + bias, threshold=700)
        h = torch.exp(dt[:, None] * A) * state[slot] + (dt * v)[:, None] * B[r]
        state[slot] = h
        y = h @ C[r] + D * v
        out[r] = y if z is None else y * z[r] * torch.sigmoid(z[r])
    return {"out": out, "state": state, "window": window}


def _exact_state(s):
    q = 127.0 if s["case"]["bits"] == 8 else 7.0
    resumed, scales = _d(s["resumed"]), _d(s["scales"])
    for src, at, dst in zip(s["src"].tolist(), s["parked"].tolist(), s["dst"].tolist()):
        h = _d(s["live"][src])
        scale = h.abs().max(1).values / q
        scales[at] = scale
        resumed[dst] = torch.round(h / torch.where(scale > 0, scale, 1)[:, None]) * scale[:, None]
    return {"resumed": resumed, "scales": scales}
