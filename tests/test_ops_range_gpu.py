"""GPU parity of the recurrent operators where decays close, stay next to one for long, or meet an
infinite state: bounds relative to every single element (terms of one sign, so that nothing
cancels), against the plain 64-bit implementations of tests/ops_util.py."""

import pytest
import torch

from selective_state_space_13_b200 import ops
from tests import ops_util as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def positive(g, *shape, dtype=F32, scale=1.0):
    return (scale * (torch.randn(*shape, generator=g).abs() + 0.1)).to(dtype)


def each(got, want, tol, what):
    """Every element within tol of its own value (and one rounding to a 16-bit type)."""
    tol += 2.0 ** -8 if got.dtype is BF16 else 0
    got, want = got.double().cpu(), want.double()
    assert torch.isfinite(got).all(), what
    err = ((got - want).abs() / want.abs()).max().item()
    assert err <= tol, "%s: %.3g > %.3g" % (what, err, tol)


def same_where_infinite(got, want, what):
    """Infinities and NaN where the definition has them; the rest within the usual bound."""
    got, want = got.double().cpu(), want.double()
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)]), what
    ref.close(got[finite], want[finite], tol=ref.TOL[F32], what=what)


# ----------------------------------------------------------------------------- closed gates

# few columns of many steps are cut into segments; the other sizes are not
SIZES = [(2, 70, 40), (1, 9000, 8)]


@pytest.mark.parametrize("level", [-3, -5, -8, -12, -16, -20, -30])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("b,L,D", SIZES)
def test_gradient_of_closed_gates(cuda_device, b, L, D, io, form, complement, level):
    # The decay is e^s (1 - ...) with s down to -33, 48 in base 2: the sum of gate and bias and its
    # product with log2(e) round that by at most half a step of [32, 64), 2^-19, each: 2.6e-6 of the
    # decay; the exponential and the reciprocal add 3.6e-7 and each of ten products 2^-24.  dbias
    # adds up to 9000 positive terms, whose rounding errors of both signs stay within 1e-6.
    g = gen(1)
    gate = (level + torch.randn(b, L, D, generator=g)).to(io)
    out, dout = positive(g, b, L, D, dtype=io), positive(g, b, L, D, dtype=io)
    x = -positive(g, b, L, D, dtype=io)  # h - x is a sum, too
    h0, dlast = positive(g, b, D), positive(g, b, D)
    bias = torch.zeros(D) if form == "sigmoid" else None
    on = [None if v is None else v.cuda() for v in (dout, x, gate, out, bias, h0, dlast)]
    r = [ref.f64(v) for v in (dout, x, gate, out, bias, h0, dlast)]
    for reverse in (False, True):
        got = ops.gated_recurrence_bwd(on[0], on[1], on[2], on[3], gate_bias=on[4],
                                       initial_state=on[5], dlast_state=on[6], form=form,
                                       complement=complement, reverse=reverse)
        want = ref.recurrence_grads(*r, form=form, complement=complement, reverse=reverse)
        for name, a, w in zip(("dx", "dgate", "dbias", "dh0"), got, want):
            if a is not None:
                each(a, w, 5e-6, "%s of gates at %d" % (name, level))


@pytest.mark.parametrize("closed", [-25.0, -200.0, -float("inf")])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("b,L,D", SIZES)
def test_a_closed_gate_leaves_nothing_of_the_state(cuda_device, b, L, D, form, complement, closed):
    # Blocks of 8 steps with inputs near 100 and near 1e-4 in turn, a closed gate at every border:
    # what a block holds is a positive sum or average of its own inputs (e^-25 of 1000 is 1e-8, 1e-4
    # of the small block's values and part of the definition).  At most 8 steps of an exponential
    # (2^-22) and three roundings: 8 (2^-22 + 3 2^-24) = 3.3e-6.
    g = gen(2)
    step = torch.arange(L) % 16
    x = positive(g, b, L, D) * torch.where(step < 8, 100.0, 1e-4)[None, :, None]
    gate = torch.full((b, L, D), 2.0 if form == "sigmoid" else -0.1)
    gate[:, ::8] = closed
    out, last = ops.gated_recurrence_fwd(x.cuda(), gate.cuda(), form=form, complement=complement,
                                         initial_state=torch.full((b, D), 300.0, device="cuda"),
                                         return_last_state=True)
    want, wlast = ref.recurrence(ref.f64(x), ref.f64(gate), h0=torch.full((b, D), 300.0).double(),
                                 form=form, complement=complement)
    each(out, want, 5e-6, "out")
    each(last, wlast, 5e-6, "last")
    if closed < -100:  # nothing but the input itself
        assert torch.equal(out[:, ::8].cpu(), x[:, ::8])


# ----------------------------------------------------------------------------- infinite states

@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("b,L,D", [(2, 300, 40), (1, 9000, 8)])
def test_infinite_states_stay(cuda_device, b, L, D, form, complement):
    g = gen(3)
    x = torch.randn(b, L, D, generator=g)
    s = torch.randn(b, L, D, generator=g)
    gate = s if form == "sigmoid" else torch.nn.functional.logsigmoid(s)
    h0 = torch.randn(b, D, generator=g)
    x[0, 40, 3] = float("inf")
    x[-1, L - 1, 2] = -float("inf")
    x[-1, L // 2, 5] = -float("inf")
    h0[0, 7] = float("inf")
    out, last = ops.gated_recurrence_fwd(x.cuda(), gate.cuda(), initial_state=h0.cuda(), form=form,
                                         complement=complement, return_last_state=True)
    want, wlast = ref.recurrence(ref.f64(x), ref.f64(gate), h0=ref.f64(h0), form=form,
                                 complement=complement)
    same_where_infinite(out, want, "out")
    same_where_infinite(last, wlast, "last")
    # ... and infinite gradients, towards the first step
    dout, dlast = torch.randn(b, L, D, generator=g), torch.randn(b, D, generator=g)
    x, h0 = torch.randn(b, L, D, generator=g), torch.randn(b, D, generator=g)
    kept = ref.recurrence(ref.f64(x), ref.f64(gate), h0=ref.f64(h0), form=form,
                          complement=complement)[0].float()
    dout[0, L - 20, 4] = float("inf")
    dlast[-1, 6] = -float("inf")
    got = ops.gated_recurrence_bwd(dout.cuda(), x.cuda(), gate.cuda(), kept.cuda(),
                                   initial_state=h0.cuda(), dlast_state=dlast.cuda(), form=form,
                                   complement=complement)
    want = ref.recurrence_grads(ref.f64(dout), ref.f64(x), ref.f64(gate), ref.f64(kept),
                                h0=ref.f64(h0), dlast=ref.f64(dlast), form=form,
                                complement=complement)
    for name, a, w in zip(("dx", "dgate", "dbias", "dh0"), got, want):
        if a is not None:
            same_where_infinite(a, w, name)


@pytest.mark.parametrize("complement", [False, True])
def test_states_next_to_overflow(cuda_device, complement):
    # a h + c x is finite although h - x is not: three products and a sum, 2^-22 for the gate
    h0 = torch.full((1, 8), 3e38)
    x, gate = torch.full((1, 3, 8), -3e38), torch.full((1, 3, 8), 1.5)
    out = ops.gated_recurrence_fwd(x.cuda(), gate.cuda(), initial_state=h0.cuda(),
                                   complement=complement)
    want, _ = ref.recurrence(ref.f64(x), ref.f64(gate), h0=ref.f64(h0), complement=complement)
    want = want[:, :1] if not complement else want  # (the sum of the second step leaves fp32)
    each(out[:, :want.shape[1]], want, 5e-6, "out")


# ----------------------------------------------------------------------------- gates and biases

def test_gates_and_biases_that_cancel(cuda_device):
    # gate + bias is exact in fp32 (multiples of 2^-10 below 2^12), so 1 - a has the accuracy that
    # it has for the sum itself
    g = gen(4)
    b, L, D = 2, 70, 40
    bias = 1000 + torch.randint(0, 1024, (D,), generator=g) / 1024
    gate = -998 + torch.randint(-2048, 2048, (b, L, D), generator=g) / 1024
    out, dout, x = positive(g, b, L, D), positive(g, b, L, D), -positive(g, b, L, D)
    got = ops.gated_recurrence_bwd(dout.cuda(), x.cuda(), gate.cuda(), out.cuda(),
                                   gate_bias=bias.cuda(), complement=True)
    want = ref.recurrence_grads(ref.f64(dout), ref.f64(x), ref.f64(gate), ref.f64(out),
                                ref.f64(bias), complement=True)
    # a step's gradient gathers the errors of at most some 1/(1 - a) < 150 decays a to come, each
    # 2^-22 (1 - a) on top of three roundings of both signs: below 3e-6
    for name, a, w in zip(("dx", "dgate", "dbias"), got, want):
        each(a, w, 6e-6, name)


# ----------------------------------------------------------------------------- long memories

@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("form,complement", [("exp", False), ("exp", True), ("sigmoid", False)])
def test_constant_gates_of_long_memory(cuda_device, io, form, complement):
    # One gate a channel at every step, memories of 500 to 2000 steps: an error of the decay itself
    # comes back multiplied by the memory.  1 - a has a relative error of 2^-22, which is that of the
    # state; rounding the state twice a step with random inputs adds sqrt(1000) 2 2^-25 = 1.9e-6 (rms),
    # six times that at most.  A product of the decays of some steps is rounded by at most half a step
    # of [1/2, 1), 2^-25, at every factor, each time in the same way: 2000 2^-25 = 6e-5.
    g = gen(5)
    b, L, D = 1, 8000, 256
    memory = torch.exp(torch.empty(D).uniform_(6.2, 7.6, generator=g))
    s = torch.log(memory - 1) if form == "sigmoid" else -1 / memory
    gate = s.expand(b, L, D).to(io).contiguous()
    x = positive(g, b, L, D, dtype=io)
    _, last = ops.gated_recurrence_fwd(x.cuda(), gate.cuda(), form=form, complement=complement,
                                       return_last_state=True)
    _, want = ref.recurrence(ref.f64(x), ref.f64(gate), form=form, complement=complement)
    each(last, want, 7.5e-5, "last")
