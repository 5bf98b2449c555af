"""GPU parity of the operators around the scan against plain 64-bit implementations
(tests/ops_util.py), at the sizes, options and values where they can go wrong."""

import numpy as np
import pytest
import torch

from selective_state_space_13_b200 import ops, scan
from tests import ops_util as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g).to(dtype)


def cuda(*ts):
    return tuple(None if t is None else t.cuda() for t in ts)


def bias_of(g, D):
    d0 = torch.exp(torch.empty(D).uniform_(np.log(1e-3), np.log(0.1), generator=g))
    return d0 + torch.log(-torch.expm1(-d0))


# ----------------------------------------------------------------------------- gated recurrence

def rec_inputs(seed, b, L, D, io, form, bias=True, initial=True):
    g = gen(seed)
    x = normal(g, b, L, D, dtype=io)
    memory = torch.exp(torch.empty(D).uniform_(np.log(2), np.log(500), generator=g))
    if form == "sigmoid":
        gate, gb = normal(g, b, L, D, dtype=io), torch.log(memory - 1) if bias else None
    else:
        gate, gb = (-torch.exp(normal(g, b, L, D)) / memory).to(io), None
    return dict(x=x, gate=gate, gate_bias=gb, initial_state=normal(g, b, D) if initial else None,
                dout=normal(g, b, L, D, dtype=io), dlast=normal(g, b, D) if initial else None)


def check_recurrence(t, **kw):
    x, gate, gb, h0, dout, dlast = cuda(*(t[n] for n in ("x", "gate", "gate_bias", "initial_state",
                                                         "dout", "dlast")))
    out, last = ops.gated_recurrence_fwd(x, gate, gate_bias=gb, initial_state=h0,
                                         return_last_state=True, **kw)
    r = ref.f64
    want, wlast = ref.recurrence(r(x), r(gate), r(gb), r(h0), **kw)
    ref.close(out, want, what="out")
    ref.close(last, wlast, what="last")
    dx, dgate, dbias, dh0 = ops.gated_recurrence_bwd(dout, x, gate, out, gate_bias=gb,
                                                     initial_state=h0, dlast_state=dlast, **kw)
    wx, wg, wb, w0 = ref.recurrence_grads(r(dout), r(x), r(gate), r(out), r(gb), r(h0), r(dlast),
                                          **kw)
    ref.close(dx, wx, what="dx")
    ref.close(dgate, wg, what="dgate")
    assert (dbias is None) == (gb is None) and (dh0 is None) == (h0 is None)
    if dbias is not None:
        ref.close(dbias, wb, what="dbias")
    if dh0 is not None:
        ref.close(dh0, w0, what="dh0")


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("io", [F32, BF16])
def test_recurrence_options(cuda_device, io, form, complement, reverse):
    check_recurrence(rec_inputs(1, 2, 197, 72, io, form), form=form, complement=complement,
                     reverse=reverse)


@pytest.mark.parametrize("b,L,D", [(1, 1, 8), (3, 2, 8), (1, 31, 264), (2, 63, 128), (1, 65, 16),
                                   (1, 129, 1000), (5, 333, 200), (1, 5000, 8), (1, 1025, 520),
                                   (33, 40, 136), (1, 4200, 72), (2, 2049, 128)])
@pytest.mark.parametrize("io", [F32, BF16])
def test_recurrence_sizes(cuda_device, io, b, L, D):
    # (few columns of many steps are cut into segments, from 8 clusters' rounds on)
    check_recurrence(rec_inputs(b + L + D, b, L, D, io, "sigmoid", initial=L % 2 == 1),
                     complement=True)


def test_recurrence_without_bias_or_state(cuda_device):
    check_recurrence(rec_inputs(4, 2, 100, 24, F32, "sigmoid", bias=False, initial=False))


def test_recurrence_no_steps(cuda_device):
    x = torch.zeros(2, 0, 8, device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    out, last = ops.gated_recurrence_fwd(x, x, initial_state=h0, return_last_state=True)
    assert out.shape == (2, 0, 8) and torch.equal(last, h0)
    _, last = ops.gated_recurrence_fwd(x, x, return_last_state=True)
    assert torch.equal(last, torch.zeros_like(h0))
    gb = torch.zeros(8, device="cuda")
    dx, dgate, dbias, dh0 = ops.gated_recurrence_bwd(x, x, x, x, gate_bias=gb, initial_state=h0,
                                                     dlast_state=2 * h0)
    assert torch.equal(dh0, 2 * h0) and torch.equal(dbias, gb)
    for shape in ((0, 5, 8), (2, 5, 0)):
        x = torch.zeros(shape, device="cuda")
        out, last = ops.gated_recurrence_fwd(x, x, return_last_state=True)
        assert out.shape == shape and last.shape == (shape[0], shape[2])


@pytest.mark.parametrize("form", ["sigmoid", "exp"])
def test_recurrence_gates_at_their_ends(cuda_device, form):
    # gates that close or open entirely: the state is kept or replaced exactly
    g = gen(7)
    x = normal(g, 1, 300, 16)
    gate = torch.where(torch.rand(1, 300, 16, generator=g) < 0.5, -200.0, 0.0 if form == "exp" else 200.0)
    gate[0, 7] = -float("inf")
    if form == "sigmoid":
        gate[0, 9] = float("inf")
    x, gate = cuda(x, gate)
    out = ops.gated_recurrence_fwd(x, gate, form=form, complement=True)
    want, _ = ref.recurrence(ref.f64(x), ref.f64(gate), form=form, complement=True)
    ref.close(out, want)
    dx, dgate, _, _ = ops.gated_recurrence_bwd(torch.ones_like(x), x, gate, out, form=form,
                                               complement=True)
    wx, wg, _, _ = ref.recurrence_grads(torch.ones_like(x).double().cpu(), ref.f64(x), ref.f64(gate),
                                        ref.f64(out), form=form, complement=True)
    ref.close(dx, wx)
    ref.close(dgate, wg)


def test_recurrence_nan_stays_in_its_channel(cuda_device):
    t = rec_inputs(8, 2, 500, 64, F32, "sigmoid")
    t["x"][1, 250, 5] = float("nan")
    x, gate, gb, h0 = cuda(t["x"], t["gate"], t["gate_bias"], t["initial_state"])
    out = ops.gated_recurrence_fwd(x, gate, gate_bias=gb, initial_state=h0)
    bad = torch.isnan(out)
    assert bad[1, 250:, 5].all() and bad.sum() == 250


def test_recurrence_step_by_step_is_the_sequence(cuda_device):
    t = rec_inputs(9, 2, 40, 24, F32, "sigmoid")
    x, gate, gb, h = cuda(t["x"], t["gate"], t["gate_bias"], t["initial_state"])
    whole, last = ops.gated_recurrence_fwd(x, gate, gate_bias=gb, initial_state=h, complement=True,
                                           return_last_state=True)
    for i in range(40):
        o, h = ops.gated_recurrence_fwd(x[:, i:i + 1].contiguous(), gate[:, i:i + 1].contiguous(),
                                        gate_bias=gb, initial_state=h, complement=True,
                                        return_last_state=True)
        ref.close(o[:, 0], whole[:, i])
    ref.close(h, last)


def test_recurrence_gradient_against_differences(cuda_device):
    # <gradient, v> against (f(x + e v) - f(x - e v)) / 2e of the plain 64-bit forward pass; the
    # difference quotient of the smooth f is off by e^2 f''' / 6 and by rounding, both far below
    # the bound.  The bound: an element of the gradient is off by at most 5e-5 (|g| + rms), so with
    # independent normal v the sum is off by about 1e-4 |gradient|, times a few standard deviations
    t = rec_inputs(10, 2, 90, 16, F32, "sigmoid")
    names = ("x", "gate", "gate_bias", "initial_state")
    xs = dict(zip(names, cuda(*(t[n] for n in names))))
    dout, dlast = cuda(t["dout"], t["dlast"])
    out = ops.gated_recurrence_fwd(**xs, complement=True)
    grads = ops.gated_recurrence_bwd(dout, out=out, dlast_state=dlast, complement=True, **xs)
    base = [ref.f64(xs[n]) for n in names]

    def f(args):
        o, last = ref.recurrence(*args, complement=True)
        return ((o * ref.f64(dout)).sum() + (last * ref.f64(dlast)).sum()).item()

    g = gen(11)
    for i, grad in enumerate(grads):
        v = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        e = 1e-5
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - e * v, base[i] + e * v
        want = (f(hi) - f(lo)) / (2 * e)
        got = (ref.f64(grad) * v).sum().item()
        assert abs(got - want) <= 1e-4 * grad.double().norm().item() * v.norm().item() ** 0.5, names[i]


def test_recurrence_autograd(cuda_device):
    t = rec_inputs(12, 2, 70, 24, F32, "sigmoid")
    leaves = [v.cuda().requires_grad_() for v in (t["x"], t["gate"], t["gate_bias"],
                                                  t["initial_state"])]
    out, last = ops.gated_recurrence(*leaves, complement=True)
    ((out * out).sum() + last.sum()).backward()
    plain = [ref.f64(v).requires_grad_() for v in leaves]
    o, la = ref.recurrence(*plain, complement=True)
    ((o * o).sum() + la.sum()).backward()
    for a, b in zip(leaves, plain):
        ref.close(a.grad, b.grad, tol=2e-4)  # dout itself is an fp32 state: four bounds on top


# ----------------------------------------------------------------------------- gradient of the scan

SCAN_NAMES = ("u", "delta", "A", "B", "C", "D", "z", "bias", "h0")
GRAD_OF = dict(u="du", delta="ddelta", A="dA", B="dB", C="dC", D="dD", z="dz", bias="ddelta_bias",
               h0="dinitial_state")


def scan_inputs(seed, b, L, D, N, io, dirs=(0,), gate=True, skip=True, bias=True, initial=True,
                u_per_dir=False, per_dir=False):
    g = gen(seed)
    K = len(dirs)
    lead = (K,) if per_dir else ()
    A = -torch.arange(1, N + 1).float() * torch.exp(0.2 * normal(g, *lead, D, N))
    return dict(u=normal(g, *((K,) if u_per_dir else ()), b, L, D, dtype=io),
                delta=normal(g, K, b, L, D, dtype=io), A=A, B=normal(g, K, b, L, N, dtype=io),
                C=normal(g, K, b, L, N, dtype=io), D=normal(g, *lead, D) if skip else None,
                z=normal(g, b, L, D, dtype=io) if gate else None,
                bias=bias_of(g, D * max(1, K if per_dir else 1)).view(*lead, D) if bias else None,
                h0=normal(g, K, b, D, N) if initial else None,
                dout=normal(g, b, L, D, dtype=io), dlast=normal(g, K, b, D, N) if initial else None)


def check_scan(t, dirs=(0,), H=0, W=0, softplus=True, segments=0, flags=0):
    d = dict(zip(t, cuda(*t.values())))
    got = ops.selective_scan_bwd(d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"], D=d["D"],
                                 z=d["z"], delta_bias=d["bias"], softplus=softplus, dirs=dirs, H=H,
                                 W=W, initial_state=d["h0"], dlast_state=d["dlast"],
                                 segments=segments, flags=flags)
    leaves = {n: ref.f64(t[n]).requires_grad_() for n in SCAN_NAMES if t[n] is not None}
    arg = [leaves.get(n) for n in SCAN_NAMES]
    out, last = ref.scan(*arg[:8], softplus=softplus, dirs=dirs, H=H, W=W, h0=arg[8])
    loss = (out * ref.f64(t["dout"])).sum()
    if t["dlast"] is not None:
        loss = loss + (last * ref.f64(t["dlast"])).sum()
    want = torch.autograd.grad(loss, list(leaves.values()))
    for n, w in zip(leaves, want):
        ref.close(got[GRAD_OF[n]], w, what=GRAD_OF[n])
    for n in SCAN_NAMES:
        assert (got[GRAD_OF[n]] is None) == (t[n] is None)
    return d, got


@pytest.mark.parametrize("segments", [0, 1, 2, 5])
@pytest.mark.parametrize("io", [F32, BF16])
def test_scan_bwd_one_direction(cuda_device, io, segments):
    check_scan(scan_inputs(20, 2, 150, 72, 16, io), segments=segments)


@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 16, 17, 63, 65])
def test_scan_bwd_lengths(cuda_device, L):
    check_scan(scan_inputs(21 + L, 1, L, 24, 16, F32), segments=3 if L > 16 else 0)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 11, 12, 15])
def test_scan_bwd_state_sizes(cuda_device, N):
    check_scan(scan_inputs(40 + N, 2, 45, 40, N, F32 if N % 2 else BF16), segments=2)


@pytest.mark.parametrize("D", [8, 56, 64, 72, 136, 200])
def test_scan_bwd_widths(cuda_device, D):
    check_scan(scan_inputs(60 + D, 3, 33, D, 16, BF16, initial=False))


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dirs,H,W", [((1,), 0, 0), ((0, 1), 0, 0), ((0, 2, 1, 3), 6, 9),
                                      ((3,), 8, 5), ((2, 2, 0), 7, 7)])
def test_scan_bwd_directions(cuda_device, dirs, H, W, gate):
    L = H * W or 50
    check_scan(scan_inputs(80 + L, 2, L, 40, 8, F32, dirs=dirs, gate=gate), dirs=dirs, H=H, W=W,
               segments=2)


@pytest.mark.parametrize("u_per_dir,per_dir", [(True, False), (False, True), (True, True)])
def test_scan_bwd_per_direction(cuda_device, u_per_dir, per_dir):
    dirs = (0, 3, 1)
    check_scan(scan_inputs(95, 2, 48, 24, 16, BF16, dirs=dirs, u_per_dir=u_per_dir, per_dir=per_dir),
               dirs=dirs, H=6, W=8)


def test_scan_bwd_optional_inputs(cuda_device):
    check_scan(scan_inputs(100, 2, 60, 16, 16, F32, gate=False, skip=False, bias=False,
                           initial=False))
    t = scan_inputs(101, 2, 60, 16, 16, F32, bias=False)
    t["delta"] = t["delta"].abs() * 0.3
    check_scan(t, softplus=False, segments=2)
    t = scan_inputs(102, 2, 60, 16, 16, F32)
    t["dlast"] = None
    check_scan(t)
    t = scan_inputs(103, 2, 60, 16, 16, F32)
    t["h0"] = None
    check_scan(t, flags=scan.SS_FLAG_GENERIC_A)


@pytest.mark.parametrize("io", [F32, BF16])
def test_scan_bwd_extreme_steps(cuda_device, io):
    # steps that keep the state exactly (Delta = 0), steps that forget it, and zero inputs
    t = scan_inputs(104, 2, 120, 16, 16, io)
    r = torch.rand(t["delta"].shape, generator=gen(105))
    t["delta"] = torch.where(r < 0.2, -200.0, torch.where(r > 0.8, 60.0, t["delta"].float())).to(io)
    t["u"][:, 10:20] = 0
    t["z"][0, 5] = -90.0
    t["z"][0, 6] = 90.0
    check_scan(t, segments=3)


def test_scan_bwd_empty(cuda_device):
    t = scan_inputs(106, 2, 0, 16, 4, F32)
    d = dict(zip(t, cuda(*t.values())))
    got = ops.selective_scan_bwd(d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"], D=d["D"],
                                 z=d["z"], delta_bias=d["bias"], initial_state=d["h0"],
                                 dlast_state=d["dlast"])
    assert torch.equal(got["dinitial_state"], d["dlast"])
    for n in ("dA", "dD", "ddelta_bias"):
        assert not got[n].any()
    t = scan_inputs(107, 0, 5, 16, 4, F32)
    d = dict(zip(t, cuda(*t.values())))
    got = ops.selective_scan_bwd(d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"])
    assert not got["dA"].any() and got["du"].shape == (0, 5, 16)


@pytest.mark.parametrize("seed", range(24))
def test_scan_bwd_random(cuda_device, seed):
    rng = np.random.default_rng(300 + seed)
    dirs, H, W = [((0,), 0, 0), ((1,), 0, 0), ((0, 1), 0, 0), ((0, 2, 1, 3), 5, 9)][rng.integers(4)]
    L = H * W or int(rng.integers(1, 200))
    flag = lambda: bool(rng.integers(2))  # noqa: E731
    t = scan_inputs(seed, int(rng.integers(1, 4)), L, 8 * int(rng.integers(1, 20)),
                    int(rng.integers(1, 17)), F32 if flag() else BF16, dirs=dirs, gate=flag(),
                    skip=flag(), bias=flag(), initial=flag(), u_per_dir=flag(), per_dir=flag())
    check_scan(t, dirs=dirs, H=H, W=W, segments=int(rng.integers(0, 6)))


def test_scan_bwd_against_differences(cuda_device):
    t = scan_inputs(110, 1, 40, 8, 4, F32)
    d = dict(zip(t, cuda(*t.values())))
    got = ops.selective_scan_bwd(d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"], D=d["D"],
                                 z=d["z"], delta_bias=d["bias"], initial_state=d["h0"],
                                 dlast_state=d["dlast"])
    base = {n: ref.f64(t[n]) for n in SCAN_NAMES}

    def f(**kw):
        a = dict(base, **kw)
        out, last = ref.scan(*(a[n] for n in SCAN_NAMES[:8]), h0=a["h0"])
        return ((out * ref.f64(t["dout"])).sum() + (last * ref.f64(t["dlast"])).sum()).item()

    g = gen(111)
    for n in SCAN_NAMES:
        v = torch.randn(base[n].shape, generator=g, dtype=torch.float64)
        e = 1e-5
        want = (f(**{n: base[n] + e * v}) - f(**{n: base[n] - e * v})) / (2 * e)
        grad = ref.f64(got[GRAD_OF[n]])
        assert abs((grad * v).sum().item() - want) <= 1e-4 * grad.norm().item() * v.norm().item() ** 0.5, n


def test_scan_bwd_repeats_bit_for_bit(cuda_device):
    t = scan_inputs(112, 2, 300, 136, 16, BF16)
    d, a = check_scan(t, segments=4)
    _, b = check_scan(t, segments=4)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_scan_autograd_matches_plain(cuda_device):
    # the library's forward and gradient together, as a training step runs them
    dirs = (0, 1)
    t = scan_inputs(113, 2, 60, 24, 16, F32, dirs=dirs)
    leaves = {n: t[n].cuda().requires_grad_() for n in SCAN_NAMES}
    out, last = ops.selective_scan(*(leaves[n] for n in SCAN_NAMES[:8]), dirs=dirs,
                                   initial_state=leaves["h0"])
    ((out * out).sum() + last.sin().sum()).backward()
    plain = {n: ref.f64(t[n]).requires_grad_() for n in SCAN_NAMES}
    o, la = ref.scan(*(plain[n] for n in SCAN_NAMES[:8]), dirs=dirs, h0=plain["h0"])
    ((o * o).sum() + la.sin().sum()).backward()
    for n in SCAN_NAMES:
        ref.close(leaves[n].grad, plain[n].grad, tol=2e-4, what=n)  # dout is an fp32 output itself


# ----------------------------------------------------------------------------- single-token step

def step_inputs(seed, b, D, N, io, width=0, slots=8, gate=True, skip=True, bias=True, cb=True):
    g = gen(seed)
    return dict(u=normal(g, b, D, dtype=io), delta=normal(g, b, D, dtype=io),
                A=-torch.arange(1, N + 1).float() * torch.exp(0.2 * normal(g, D, N)),
                B=normal(g, b, N, dtype=io), C=normal(g, b, N, dtype=io),
                state=normal(g, slots, D, N), D=normal(g, D) if skip else None,
                z=normal(g, b, D, dtype=io) if gate else None, bias=bias_of(g, D) if bias else None,
                cw=normal(g, D, width) if width else None,
                cb=normal(g, D) if width and cb else None,
                cs=normal(g, slots, width - 1, D, dtype=io) if width else None)


def plain_step(t, slots, softplus=True):
    """(out rows or None, state, window) in 64 bits; the first row that names a slot takes it."""
    r = {n: ref.f64(v) for n, v in t.items()}
    state, win, outs, taken = r["state"].clone(), r["cs"], [], set()
    win = None if win is None else win.clone()
    for i, s in enumerate(slots):
        if not 0 <= s < state.shape[0] or s in taken:
            outs.append(None)
            continue
        taken.add(s)
        u = r["u"][i]
        if r["cw"] is not None:
            seen = torch.cat([win[s], u[None]])
            win[s] = seen[1:]
            u = (seen * r["cw"].t()).sum(0) + (0 if r["cb"] is None else r["cb"])
            u = u * torch.sigmoid(u)
        one = lambda v: v[i][None, None, None]  # noqa: E731
        o, last = ref.scan(u[None, None], one(r["delta"]), r["A"], one(r["B"]), one(r["C"]), r["D"],
                           None if r["z"] is None else r["z"][i][None, None], r["bias"],
                           softplus=softplus, h0=state[s][None, None])
        state[s] = last[0, 0]
        outs.append(o[0, 0])
    return outs, state, win


def check_step(t, slots=None, softplus=True):
    d = dict(zip(t, cuda(*t.values())))
    b = t["u"].shape[0]
    out = torch.full(t["u"].shape, 7.0, dtype=t["u"].dtype, device="cuda")
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    want, wstate, wwin = plain_step(t, list(range(b)) if slots is None else slots, softplus)
    ops.selective_scan_step(d["u"], d["delta"], d["A"], d["B"], d["C"], d["state"], D=d["D"],
                            z=d["z"], delta_bias=d["bias"], softplus=softplus, slots=sl,
                            conv_weight=d["cw"], conv_bias=d["cb"], conv_state=d["cs"], out=out)
    ref.close(d["state"], wstate, what="state")
    for i, w in enumerate(want):
        if w is None:
            assert (out[i] == 7).all()
        else:
            ref.close(out[i], w, what="out %d" % i)
    untouched = set(range(wstate.shape[0])) - set(range(b) if slots is None else slots)
    for s in untouched:
        assert torch.equal(d["state"][s].cpu(), t["state"][s])
    if wwin is not None:
        assert torch.equal(d["cs"].double().cpu(), wwin)  # a shift copies


@pytest.mark.parametrize("width", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("io", [F32, BF16])
def test_step_with_and_without_conv(cuda_device, io, width):
    check_step(step_inputs(120 + width, 3, 72, 16, io, width=width), slots=[5, 0, 2])


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 7, 8, 11, 12, 15, 16])
def test_step_state_sizes(cuda_device, N):
    check_step(step_inputs(130 + N, 2, 40, N, F32 if N % 2 else BF16, width=4))


@pytest.mark.parametrize("D", [8, 24, 32, 136, 1000])
def test_step_widths(cuda_device, D):
    check_step(step_inputs(150 + D, 5, D, 16, BF16, width=3, slots=6), slots=[1, 2, 3, 4, 0])


def test_step_options(cuda_device):
    check_step(step_inputs(160, 2, 16, 16, F32, gate=False, skip=False, bias=False))
    t = step_inputs(161, 2, 16, 16, F32, bias=False, width=4, cb=False)
    t["delta"] = t["delta"].abs()
    check_step(t, softplus=False)


def test_step_padding_and_repeated_slots(cuda_device):
    # padded rows (negative or behind the pool) change nothing; of rows with one slot the first works
    check_step(step_inputs(162, 9, 40, 16, BF16, width=4, slots=6),
               slots=[3, -1, 3, 0, 6, 2 ** 31 - 1, 0, 5, 3])
    check_step(step_inputs(163, 300, 8, 4, F32, slots=300), slots=list(range(299)) + [0])
    check_step(step_inputs(164, 4, 8, 5, F32, slots=3), slots=[-1] * 4)


def test_step_no_rows(cuda_device):
    t = step_inputs(165, 0, 8, 4, F32)
    d = dict(zip(t, cuda(*t.values())))
    out = ops.selective_scan_step(d["u"], d["delta"], d["A"], d["B"], d["C"], d["state"])
    assert out.shape == (0, 8) and torch.equal(d["state"].cpu(), t["state"])


# ----------------------------------------------------------------------------- parked states

def check_park(h, bits, src=None, dst=None, cache=None):
    """Store and load back; compares codes and scales with exact arithmetic, and every slot that
    is not written with what was there."""
    S, D, N = h.shape
    cache = cache or S
    width = N if bits == 8 else (N + 1) // 2
    codes = torch.full((cache, D, width), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((cache, D), 99.0, device="cuda")
    back = torch.full((S, D, N), 99.0, device="cuda")
    si, di = (None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")
              for v in (src, dst))
    ops.selective_state_store(h.cuda(), codes, scales, bits=bits, src_slots=si, dst_slots=di)
    ops.selective_state_load(codes, scales, back, bits=bits, src_slots=di, dst_slots=si)
    want_codes, want_scales = codes.cpu() * 0 + 99, scales.cpu() * 0 + 99
    want_back = back.cpu() * 0 + 99
    wc, ws = ref.park(ref.f64(h), bits)
    rows = len(src or dst or range(S))
    taken, owner = set(), {}
    for r in range(rows):
        s, d = (src or range(rows))[r], (dst or range(rows))[r]
        if 0 <= s < S and 0 <= d < cache:
            if d not in taken:
                taken.add(d)
                want_codes[d] = wc[s] if bits == 8 else ref.pack4(wc[s])
                want_scales[d] = ws[s]
                owner[d] = s
    done = set()
    for r in range(rows):
        s, d = (src or range(rows))[r], (dst or range(rows))[r]
        if 0 <= s < S and 0 <= d < cache and s not in done:
            done.add(s)
            want_back[s] = wc[owner[d]].float() * ws[owner[d]][:, None]
    assert torch.equal(codes.cpu(), want_codes)
    # amax / q rounded once in fp32 against the fp64 quotient rounded to fp32: the same value
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(back.cpu(), want_back)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 9, 12, 15, 16])
def test_park_state_sizes(cuda_device, N, bits):
    g = gen(170 + N)
    check_park(normal(g, 5, 72, N) * torch.exp(3 * normal(g, 5, 72, 1)), bits)


@pytest.mark.parametrize("bits", [8, 4])
def test_park_slots(cuda_device, bits):
    h = normal(gen(171), 6, 40, 16)
    check_park(h, bits, src=[0, 5, 3], dst=[7, 2, 1], cache=9)
    check_park(h, bits, src=[0, 5, -1, 2, 6], dst=[3, 9, 1, -5, 0], cache=9)
    check_park(h, bits, src=[4, 1, 0], dst=[2, 2, 3], cache=4)  # the first of two takes slot 2
    check_park(h, bits, src=[9, 1, 0], dst=[2, 2, 3], cache=4)  # a skipped row takes nothing
    check_park(h, bits, dst=[5, 4, 3, 2, 1, 0])


@pytest.mark.parametrize("bits", [8, 4])
def test_park_borders_between_codes(cuda_device, bits):
    # values on and next to the border of two codes: ties go to the even code, and a value one
    # fp32 step off the border to its own side
    q = 127 if bits == 8 else 7
    k = torch.arange(-q, q).double() + 0.5
    amax = torch.tensor([1.0, 3.0, 0.7, 127.0, 1e-3, 254.0, 1e-42, 3e38]).float()
    mid = (k[None] * amax.double()[:, None] / q).float()
    rows = torch.cat([mid, torch.nextafter(mid, mid * 0), torch.nextafter(mid, mid * 2)], 1)
    rows = torch.minimum(rows.abs(), amax[:, None]) * rows.sign()
    n = rows.shape[1] // 6 * 6
    h = rows[:, :n].reshape(8, -1, 6)
    h = torch.cat([h, amax[:, None, None].expand(8, h.shape[1], 1)], 2)
    pad = (-h.shape[1]) % 8
    check_park(torch.nn.functional.pad(h, (0, 1, 0, pad)), bits)
    check_park(h[:, :h.shape[1] // 8 * 8].contiguous(), bits)


def test_park_zero_and_not_finite(cuda_device):
    h = normal(gen(172), 2, 8, 16)
    h[0, 0] = 0
    h[0, 1, 3] = float("inf")
    h[0, 2, 5] = float("nan")
    h[0, 3, 5] = -float("inf")
    h[0, 4] = -0.0
    for bits in (8, 4):
        codes = torch.empty((2, 8, 16 if bits == 8 else 8), dtype=torch.int8, device="cuda")
        scales, back = torch.empty((2, 8), device="cuda"), torch.empty((2, 8, 16), device="cuda")
        ops.selective_state_store(h.cuda(), codes, scales, bits=bits)
        ops.selective_state_load(codes, scales, back, bits=bits)
        back, scales = back.cpu(), scales.cpu()
        assert (back[0, 0] == 0).all() and scales[0, 0] == 0 and (back[0, 4] == 0).all()
        for c in (1, 2, 3):
            assert torch.isnan(back[0, c]).all() and torch.isnan(scales[0, c])
            assert not codes[0, c].any()
        rest = [5, 6, 7]
        # half a code step, and the rounding of scale and product
        half = h.abs().amax(-1)[..., None] / (127 if bits == 8 else 7) * (0.5 + 1e-4)
        assert ((back - h).abs() <= half)[0, rest].all() and ((back - h).abs() <= half)[1].all()


# ----------------------------------------------------------------------------- together

def test_prefill_park_resume_decode(cuda_device):
    # a request's life: the scan over its prompt leaves a state in the pool, the state is parked in
    # 8 bits and resumed in another slot, and decoding continues there token by token; the same
    # tokens in one plain scan from the parked (rounded) state give the same outputs
    b, L, T, D, N, width = 3, 50, 6, 40, 16, 4
    t = scan_inputs(180, b, L + T, D, N, BF16, initial=False)
    g = gen(181)
    cw, cb = normal(g, 1, D, width) * 0.5, normal(g, 1, D) * 0.1
    d = dict(zip(t, cuda(*t.values())))
    cwd, cbd = cuda(cw, cb)
    part = lambda v: v[:, :, :L].contiguous()  # noqa: E731
    _, last = scan.selective_scan_fwd(d["u"][:, :L].contiguous(), part(d["delta"]), d["A"],
                                      part(d["B"]), part(d["C"]), D=d["D"],
                                      z=d["z"][:, :L].contiguous(), delta_bias=d["bias"],
                                      return_last_state=True, conv_weight=cwd, conv_bias=cbd)
    pool = torch.zeros(8, D, N, device="cuda")
    window = torch.zeros(8, width - 1, D, dtype=BF16, device="cuda")
    live = torch.tensor([6, 1, 4], dtype=torch.int32, device="cuda")
    pool[live.long()] = last[0]
    codes = torch.zeros(4, D, N, dtype=torch.int8, device="cuda")
    scales = torch.zeros(4, D, device="cuda")
    spare = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    ops.selective_state_store(pool, codes, scales, src_slots=live, dst_slots=spare)
    pool.fill_(float("nan"))
    slots = torch.tensor([0, 7, 5], dtype=torch.int32, device="cuda")
    ops.selective_state_load(codes, scales, pool, src_slots=spare, dst_slots=slots)
    window[slots.long()] = d["u"][:, L - width + 1:L]
    resumed = pool[slots.long()].clone()
    outs = []
    for i in range(L, L + T):
        outs.append(ops.selective_scan_step(
            *(v[:, i].contiguous() for v in (d["u"], d["delta"][0])), d["A"],
            *(v[0, :, i].contiguous() for v in (d["B"], d["C"])), pool, D=d["D"],
            z=d["z"][:, i].contiguous(), delta_bias=d["bias"], slots=slots, conv_weight=cwd[0],
            conv_bias=cbd[0], conv_state=window))
    u = ref.f64(t["u"])
    conv = sum(u[:, L - width + 1 + j:L - width + 1 + j + T] * ref.f64(cw)[0, :, j]
               for j in range(width)) + ref.f64(cb)[0]
    tail = lambda v: ref.f64(v)[:, :, L:]  # noqa: E731
    want, wlast = ref.scan(conv * torch.sigmoid(conv), tail(t["delta"]), ref.f64(t["A"]),
                           tail(t["B"]), tail(t["C"]), ref.f64(t["D"]), ref.f64(t["z"])[:, L:],
                           ref.f64(t["bias"]), h0=ref.f64(resumed)[None])
    ref.close(torch.stack(outs, 1), want)
    ref.close(pool[slots.long()], wlast[0])
    assert torch.equal(window[slots.long()], d["u"][:, L + T - width + 1:])
    q = last[0].abs().amax(-1, keepdim=True) / 127
    assert ((resumed - last[0]).abs() <= q * 0.5001).all()


def test_two_layers_train_together(cuda_device):
    # a recurrence layer under a scan layer, one loss, gradients of every leaf
    g = gen(182)
    b, L, D, N = 2, 48, 16, 8
    t = scan_inputs(183, b, L, D, N, F32, initial=False)
    leaves = {n: t[n].cuda().requires_grad_() for n in ("delta", "A", "B", "C", "D", "z", "bias")}
    x, gate, gb = (v.cuda().requires_grad_() for v in (normal(g, b, L, D), normal(g, b, L, D),
                                                       normal(g, D)))
    h, _ = ops.gated_recurrence(x, gate, gb, complement=True)
    out, _ = ops.selective_scan(h, leaves["delta"], leaves["A"], leaves["B"], leaves["C"],
                                leaves["D"], leaves["z"], leaves["bias"])
    out.square().mean().backward()
    plain = {n: ref.f64(v).requires_grad_() for n, v in leaves.items()}
    px, pg, pb = (ref.f64(v).requires_grad_() for v in (x, gate, gb))
    hh, _ = ref.recurrence(px, pg, pb, complement=True)
    oo, _ = ref.scan(hh, plain["delta"], plain["A"], plain["B"], plain["C"], plain["D"], plain["z"],
                     plain["bias"])
    oo.square().mean().backward()
    # three operators in a row, each within its bound of the ones before it
    for n in leaves:
        ref.close(leaves[n].grad, plain[n].grad, tol=2e-4, what=n)
    for a, w in ((x, px), (gate, pg), (gb, pb)):
        ref.close(a.grad, w.grad, tol=2e-4)


def operators():
    """One call of each operator: (its tensors' seeded inputs, call -> outputs)."""
    t = scan_inputs(190, 2, 100, 40, 16, BF16, dirs=(0, 1))
    d = dict(zip(t, cuda(*t.values())))
    r = rec_inputs(191, 2, 300, 40, BF16, "sigmoid")
    e = dict(zip(r, cuda(*r.values())))
    s = step_inputs(192, 3, 40, 16, BF16, width=4)
    f = dict(zip(s, cuda(*s.values())))
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    codes = torch.zeros(8, 40, 8, dtype=torch.int8, device="cuda")
    scales, back = torch.zeros(8, 40, device="cuda"), torch.zeros(8, 40, 16, device="cuda")
    kept = ops.gated_recurrence_fwd(e["x"], e["gate"], gate_bias=e["gate_bias"])

    def bwd():
        g = ops.selective_scan_bwd(d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"], D=d["D"],
                                   z=d["z"], delta_bias=d["bias"], dirs=(0, 1),
                                   initial_state=d["h0"], dlast_state=d["dlast"], segments=3)
        return [v for v in g.values() if v is not None]

    def step():
        state, cs = f["state"].clone(), f["cs"].clone()
        out = ops.selective_scan_step(f["u"], f["delta"], f["A"], f["B"], f["C"], state, D=f["D"],
                                      z=f["z"], delta_bias=f["bias"], slots=slots,
                                      conv_weight=f["cw"], conv_bias=f["cb"], conv_state=cs)
        return [out, state, cs]

    def park():
        ops.selective_state_store(f["state"], codes, scales, bits=4)
        ops.selective_state_load(codes, scales, back, bits=4)
        return [codes.clone(), scales.clone(), back.clone()]

    return {"recurrence": lambda: list(ops.gated_recurrence_fwd(
                e["x"], e["gate"], gate_bias=e["gate_bias"], return_last_state=True)),
            "recurrence_bwd": lambda: [v for v in ops.gated_recurrence_bwd(
                e["dout"], e["x"], e["gate"], kept, gate_bias=e["gate_bias"]) if v is not None],
            "scan_bwd": bwd, "step": step, "park": park}


@pytest.mark.parametrize("name", ["recurrence", "recurrence_bwd", "scan_bwd", "step", "park"])
def test_captured_and_on_another_stream(cuda_device, name):
    call = operators()[name]
    want = [v.clone() for v in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # two graphs of one call, replayed in turn: neither uses what the other holds
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    for _ in range(2):
        for graph, out in zip(graphs, outs):
            for v in out:
                v.zero_()
            graph.replay()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_two_calls_at_once(cuda_device):
    # every operator on two streams, again and again without waiting: no call sees another's scratch
    calls = operators()
    want = {n: [v.clone() for v in c()] for n, c in calls.items() if n != "park"}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got += [(n, calls[n]()) for n in want]
    torch.cuda.synchronize()
    for n, vs in got:
        for a, b in zip(vs, want[n]):
            assert torch.equal(a, b), n


def guarded(like, fill=float("nan")):
    """A tensor like `like` inside a larger buffer whose margins hold a canary: (view, buffer)."""
    pad, n = 64, like.numel()
    buf = torch.full((n + 2 * pad,), 93, dtype=like.dtype, device="cuda")
    view = buf[pad:pad + n].view(like.shape)
    view.fill_(fill if like.is_floating_point() else 0)
    return view, buf


def check_guards(bufs, whole=()):
    for name, (view, buf) in bufs.items():
        assert (buf[:64] == 93).all() and (buf[-64:] == 93).all(), name
        if name in whole:
            assert torch.isfinite(view.float()).all(), name


@pytest.mark.parametrize("io", [F32, BF16])
def test_outputs_stay_in_their_bounds(cuda_device, io):
    # ragged sizes through the C entry points; every output element written, nothing beside them
    lib, code = ops.load(), scan._io_code(io)
    ref_, st = ops.ctypes.byref, torch.cuda.current_stream().cuda_stream
    for b, L, D, reverse in ((2, 333, 136, 0), (1, 4201, 72, 1)):
        r = rec_inputs(200 + L, b, L, D, io, "sigmoid")
        e = dict(zip(r, cuda(*r.values())))
        opts = ops.SsRecurrenceOpts(0, 1, reverse, 0)
        sh = scan.make_shape(b, L, D, 1, code)
        n = [ops.gated_recurrence_workspace_size(sh, opts, k) for k in (False, True)]
        o = {"out": guarded(e["x"]), "last": guarded(e["initial_state"]), "dx": guarded(e["x"]),
             "dgate": guarded(e["x"]), "dbias": guarded(e["gate_bias"]),
             "dinit": guarded(e["initial_state"]),
             "ws0": guarded(torch.zeros(n[0], dtype=torch.uint8)),
             "ws1": guarded(torch.zeros(n[1], dtype=torch.uint8))}
        p = {k: v[0].data_ptr() for k, v in o.items()}
        x, gate, gb, h0, dout, dlast = (e[k].data_ptr() for k in ("x", "gate", "gate_bias",
                                                                  "initial_state", "dout", "dlast"))
        assert lib.gated_recurrence_fwd(ref_(sh), ref_(opts), x, gate, gb, h0, p["out"], p["last"],
                                        p["ws0"], n[0], st) == 0
        assert lib.gated_recurrence_bwd(ref_(sh), ref_(opts), x, gate, gb, h0, p["out"], dout, dlast,
                                        p["dx"], p["dgate"], p["dbias"], p["dinit"], p["ws1"], n[1],
                                        st) == 0
        torch.cuda.synchronize()
        check_guards(o, ("out", "last", "dx", "dgate", "dbias", "dinit"))
    for dirs, H, W, L, segs in (((0,), 0, 0, 77, 3), ((0, 2, 1, 3), 7, 9, 63, 2)):
        t = scan_inputs(210 + L, 2, L, 136, 11, io, dirs=dirs)
        d = dict(zip(t, cuda(*t.values())))
        sh, dm = scan.make_shape(2, L, 136, 11, code), scan.make_dirmap(dirs, H, W)
        op = scan.make_opts(segs, 0, None, d["h0"].data_ptr())
        n = ops.selective_scan_bwd_workspace_size(sh, dm, op)
        names = ("u", "delta", "A", "B", "C", "D", "z", "bias", "h0")
        o = {k: guarded(d[k]) for k in names}
        o["ws"] = guarded(torch.zeros(n, dtype=torch.uint8))
        g = ops.SsScanGrads(*(o[k][0].data_ptr() for k in names))
        q = {k: v.data_ptr() for k, v in d.items()}
        assert lib.selective_scan_bwd(
            ref_(sh), q["u"], q["delta"], q["A"], q["B"], q["C"], q["D"], q["z"], q["bias"], 1,
            ref_(dm), q["dout"], q["dlast"], ref_(g), o["ws"][0].data_ptr(), n, st, ref_(op)) == 0
        torch.cuda.synchronize()
        check_guards(o, names)
    for N in (16, 12, 5):
        s = step_inputs(220 + N, 3, 136, N, io, width=4, slots=4)
        f = dict(zip(s, cuda(*s.values())))
        o = {"out": guarded(f["u"]), "state": guarded(f["state"]), "cs": guarded(f["cs"])}
        o["state"][0].copy_(f["state"])
        o["cs"][0].copy_(f["cs"])
        slots = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
        ops.selective_scan_step(f["u"], f["delta"], f["A"], f["B"], f["C"], o["state"][0], D=f["D"],
                                z=f["z"], delta_bias=f["bias"], slots=slots, conv_weight=f["cw"],
                                conv_bias=f["cb"], conv_state=o["cs"][0], out=o["out"][0])
        for bits in (8, 4):
            width = N if bits == 8 else (N + 1) // 2
            o["codes%d" % bits] = guarded(torch.zeros(4, 136, width, dtype=torch.int8))
            o["scales%d" % bits] = guarded(torch.zeros(4, 136))
            o["back%d" % bits] = guarded(f["state"])
            args = (o["codes%d" % bits][0], o["scales%d" % bits][0])
            ops.selective_state_store(o["state"][0], *args, bits=bits)
            ops.selective_state_load(*args, o["back%d" % bits][0], bits=bits)
        torch.cuda.synchronize()
        check_guards(o, ("out", "state", "cs", "scales8", "back8", "scales4", "back4"))


def test_far_rows_and_slots(cuda_device):
    # element offsets beyond 2^31: what lies there equals the same rows and slots in small tensors
    g = torch.Generator(device="cuda").manual_seed(230)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF16)  # noqa: E731
    b, L, D = 3, 131072, 6144
    assert (b - 1) * L * D > 2 ** 30 and b * L * D > 2 ** 31
    x, gate = rand(b, L, D), rand(b, L, D)
    gb = torch.full((D,), 3.0, device="cuda")
    out, last = ops.gated_recurrence_fwd(x, gate, gate_bias=gb, complement=True,
                                         return_last_state=True)
    x, gate = x[2:].clone(), gate[2:].clone()
    o, la = ops.gated_recurrence_fwd(x, gate, gate_bias=gb, complement=True, return_last_state=True)
    ref.close(out[2, -100:], o[0, -100:], tol=2.0 ** -7)  # (two roundings: the cluster may differ)
    ref.close(last[2], la[0])
    del x, gate, out, o
    torch.cuda.empty_cache()
    slots, D, N = 28000, 5120, 16
    assert slots * D * N > 2 ** 31
    s = step_inputs(231, 2, D, N, BF16, width=4, slots=2)
    f = dict(zip(s, cuda(*s.values())))
    far = torch.tensor([slots - 1, 7], dtype=torch.int32, device="cuda")
    pool = torch.empty(slots, D, N, device="cuda")
    window = torch.empty(slots, 3, D, dtype=BF16, device="cuda")
    pool[far.long()], window[far.long()] = f["state"], f["cs"]
    args = (f["u"], f["delta"], f["A"], f["B"], f["C"])
    kw = dict(D=f["D"], z=f["z"], delta_bias=f["bias"], conv_weight=f["cw"], conv_bias=f["cb"])
    out = ops.selective_scan_step(*args, pool, slots=far, conv_state=window, **kw)
    near = ops.selective_scan_step(*args, f["state"], conv_state=f["cs"], **kw)
    assert torch.equal(out, near) and torch.equal(pool[far.long()], f["state"])
    assert torch.equal(window[far.long()], f["cs"])
    for bits in (8, 4):
        codes = torch.empty(slots, D, N * bits // 8, dtype=torch.int8, device="cuda")
        scales = torch.empty(slots, D, device="cuda")
        c2, s2 = (torch.empty(2, *v.shape[1:], dtype=v.dtype, device="cuda") for v in (codes, scales))
        ops.selective_state_store(pool, codes, scales, bits=bits, src_slots=far, dst_slots=far)
        ops.selective_state_store(f["state"], c2, s2, bits=bits)
        assert torch.equal(codes[far.long()], c2) and torch.equal(scales[far.long()], s2)
        back = f["state"].clone()
        ops.selective_state_load(codes, scales, pool, bits=bits, src_slots=far, dst_slots=far)
        ops.selective_state_load(c2, s2, back, bits=bits)
        assert torch.equal(pool[far.long()], back)
        pool[far.long()] = f["state"]


def test_scan_bwd_far_rows(cuda_device):
    # a batch of more than 2^31 elements: its last row's gradients equal the row's own (the segments
    # of the two calls may differ, so two roundings to bf16 lie between them)
    g = torch.Generator(device="cuda").manual_seed(240)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF16)  # noqa: E731
    b, L, D, N = 3, 131072, 6144, 4
    assert b * L * D > 2 ** 31
    dout, u, delta, z = (rand(b, L, D) for _ in range(4))
    B, C = rand(b, L, N), rand(b, L, N)
    A = -torch.rand(D, N, generator=g, device="cuda") - 0.5
    o = ops.selective_scan_bwd(dout, u, delta, A, B, C, z=z)
    far = {k: o[k][2:, -64:].clone() for k in ("du", "ddelta", "dz")}
    far |= {k: o[k].reshape(b, L, N)[2:, -64:].clone() for k in ("dB", "dC")}
    del o
    dout, u, delta, z, B, C = (v[2:].clone() for v in (dout, u, delta, z, B, C))
    torch.cuda.empty_cache()
    o = ops.selective_scan_bwd(dout, u, delta, A, B, C, z=z)
    for k, v in far.items():
        ref.close(v, o[k].reshape(1, L, -1)[:, -64:], tol=2.0 ** -7)


def test_forward_scan_and_training_step_captured(cuda_device):
    # the forward scan under capture, alone and with its gradient as a whole training step
    t = scan_inputs(194, 2, 200, 40, 16, BF16, dirs=(0, 1))
    d = dict(zip(t, cuda(*t.values())))

    def fwd():
        return scan.selective_scan_fwd(d["u"], d["delta"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                                       delta_bias=d["bias"], dirs=(0, 1), segments=3)

    leaves = [d[n].clone().requires_grad_() for n in SCAN_NAMES]

    def train():
        out, last = ops.selective_scan(*leaves[:8], dirs=(0, 1), initial_state=leaves[8])
        return list(torch.autograd.grad(out.float().square().sum() + last.sum(), leaves))

    for call in (lambda: [fwd()], train):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = [v.clone() for v in call()]
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for v in got:
            v.zero_()
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_binding_refusals(cuda_device):
    x = torch.zeros(2, 4, 8, device="cuda")
    with pytest.raises(ValueError):
        ops.gated_recurrence_fwd(x, x[:, :3].contiguous())
    with pytest.raises(ValueError):
        ops.gated_recurrence_fwd(x.transpose(0, 1), x.transpose(0, 1))
    with pytest.raises(ValueError):
        ops.gated_recurrence_fwd(x, x, form="tanh")
    with pytest.raises(ValueError):
        ops.gated_recurrence_fwd(x, x, gate_bias=x[0, 0], form="exp")
    with pytest.raises(TypeError):
        ops.gated_recurrence_fwd(x.half(), x.half())
    with pytest.raises(TypeError):
        ops.gated_recurrence_fwd(x, x.bfloat16())
    y = torch.zeros(2, 4, 6, device="cuda")
    with pytest.raises(scan.ScanError) as e:
        ops.gated_recurrence_fwd(y, y)  # 24-byte rows
    assert e.value.status == 4
    s = step_inputs(193, 2, 8, 4, F32)
    f = dict(zip(s, cuda(*s.values())))
    args = (f["u"], f["delta"], f["A"], f["B"], f["C"])
    with pytest.raises(TypeError):
        ops.selective_scan_step(*args, f["state"], slots=torch.zeros(2, dtype=torch.int64,
                                                                     device="cuda"))
    with pytest.raises(ValueError):
        ops.selective_scan_step(*args, f["state"][:, :, :3].contiguous())
    with pytest.raises(ValueError):
        ops.selective_scan_step(*args, f["state"], conv_weight=torch.zeros(8, 5, device="cuda"))
    with pytest.raises(scan.ScanError):
        ops.selective_scan_step(*args, f["state"][:1])  # two rows, one slot
    codes = torch.zeros(8, 8, 4, dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError):
        ops.selective_state_store(f["state"], codes, torch.zeros(8, 8, device="cuda"), bits=4)
    with pytest.raises(ValueError):
        ops.selective_state_store(f["state"], codes, torch.zeros(8, 8, device="cuda"), bits=2)
    u = torch.zeros(2, 4, 8, device="cuda")
    A, B = torch.zeros(8, 4, device="cuda"), torch.zeros(2, 4, 4, device="cuda")
    with pytest.raises(ValueError):
        ops.selective_scan_bwd(u, u, u, A, B, B, dirs=(0, 1))
    with pytest.raises(scan.ScanError):
        ops.selective_scan_bwd(u, u, u, A, B, B, flags=scan.SS_FLAG_ZOH_EXACT)
