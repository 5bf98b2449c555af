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
    # six times that at most.  The product of the decays of 8 or 16 steps is rounded once, by at most half
    # a step of [1/2, 1), 2^-25, each time in the same way: 2000 / 8 2^-25 = 7.5e-6.
    g = gen(5)
    b, L, D = 1, 8000, 256
    memory = torch.exp(torch.empty(D).uniform_(6.2, 7.6, generator=g))
    s = torch.log(memory - 1) if form == "sigmoid" else -1 / memory
    gate = s.expand(b, L, D).to(io).contiguous()
    x = positive(g, b, L, D, dtype=io)
    _, last = ops.gated_recurrence_fwd(x.cuda(), gate.cuda(), form=form, complement=complement,
                                       return_last_state=True)
    _, want = ref.recurrence(ref.f64(x), ref.f64(gate), form=form, complement=complement)
    each(last, want, 2.5e-5, "last")


@pytest.mark.parametrize("chunk", [1, 3])
@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("form", ["sigmoid", "exp"])
def test_recurrence_token_after_token(cuda_device, form, io, chunk):
    # the same in calls of one or three steps, the state handed on: 3000 roundings of a decay, 2^-25,
    # all in the same way, would be 6e-5 of a memory of 2000
    g = gen(13)
    b, L, D = 2, 3000, 64
    memory = torch.exp(torch.empty(D).uniform_(5.7, 7.6, generator=g))
    s = torch.log(memory - 1) if form == "sigmoid" else -1 / memory
    gate = s.expand(b, chunk, D).to(io).contiguous()
    x = positive(g, L // chunk, b, chunk, D, dtype=io)
    on, h = (x.cuda(), gate.cuda()), torch.zeros(b, D, device="cuda")
    for i in range(L // chunk):
        _, h = ops.gated_recurrence_fwd(on[0][i], on[1], initial_state=h, form=form,
                                        return_last_state=True)
    whole = ref.f64(x).permute(1, 0, 2, 3).reshape(b, L, D)
    _, want = ref.recurrence(whole, ref.f64(gate[:, :1]).expand(b, L, D), form=form)
    each(h, want, 1.5e-5, "state")


@pytest.mark.parametrize("N", [1, 4, 16, 5])
@pytest.mark.parametrize("io", [F32, BF16])
def test_step_of_many_tokens(cuda_device, io, N):
    # 4000 tokens in place with one Delta a channel, memories of 300 to 2000 tokens: as above, an error
    # of the decay itself would be multiplied by the memory.  Relative errors of Delta (2^-22), of
    # Delta A and of 1 - a (2^-22) reach the state as they are, twice: 1e-6; the state's roundings 1.2e-5.
    g = gen(6 + N)
    b, D, T = 1, 64, 4000
    memory = torch.exp(torch.empty(D, N).uniform_(5.7, 7.6, generator=g))
    delta = torch.empty(D).uniform_(0.01, 0.1, generator=g).to(io)
    A = -1 / (memory * delta.float()[:, None])
    u, B = positive(g, T, b, D, dtype=io), positive(g, T, b, N, dtype=io)
    C = torch.ones(b, N, dtype=io)
    state = torch.zeros(b, D, N, device="cuda")
    on = [v.cuda() for v in (u, B, C, A, delta.expand(b, D).contiguous())]
    for t in range(T):
        ops.selective_scan_step(on[0][t].clone(), on[4], on[3], on[1][t].clone(), on[2], state,
                                softplus=False)
    h = torch.zeros(b, D, N, dtype=torch.float64)
    d64 = ref.f64(delta)[:, None]
    a = torch.exp(d64 * ref.f64(A))
    for t in range(T):
        h = a * h + d64 * ref.f64(u[t])[..., None] * ref.f64(B[t])[:, None]
    each(state, h, 1.5e-5, "state")


@pytest.mark.parametrize("N", [1, 3, 5, 8, 16])
def test_step_keeps_infinite_states(cuda_device, N):
    g = gen(7)
    b, D = 2, 40
    state = torch.randn(b, D, N, generator=g)
    state[0, 3, N - 1], state[1, 7, 0] = float("inf"), -float("inf")
    u, delta = torch.randn(b, D, generator=g), torch.rand(b, D, generator=g) * 0.1
    u[1, 9] = float("inf")
    A = -torch.rand(D, N, generator=g) - 0.1
    A[3, N - 1] = -30.0
    B, C = positive(g, b, N), positive(g, b, N)
    on = [v.cuda() for v in (u, delta, A, B, C, state)]
    out = ops.selective_scan_step(*on, softplus=False)
    r = [ref.f64(v) for v in (u, delta, A, B, state, C)]
    want = torch.exp(r[1][..., None] * r[2]) * r[4] + (r[1] * r[0])[..., None] * r[3][:, None]
    same_where_infinite(on[5], want, "state")
    same_where_infinite(out, (want * r[5][:, None]).sum(-1), "out")


# ----------------------------------------------------------------------------- strong decays

@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("N", [5, 16])
@pytest.mark.parametrize("io", [F32, BF16])
def test_scan_gradient_of_strong_decays(cuda_device, io, N, segments):
    # Delta |A| from 0.01 to 33 over the states of one channel, every factor positive.  Delta A is
    # rounded twice (33 2^-24 (1 + log2(e)) = 5e-6), the exponential adds 2^-22; the sums over 120
    # terms of one sign and their factors at most 20 2^-24 more.
    g = gen(8)
    b, L, D = 2, 60, 40
    u, delta = positive(g, b, L, D, dtype=io), (1 + 0.1 * torch.rand(b, L, D, generator=g)).to(io)
    A = -torch.exp(torch.linspace(-4.6, 3.4, N)).expand(D, N).contiguous()
    B, C = positive(g, b, L, N, dtype=io), positive(g, b, L, N, dtype=io)
    dout = positive(g, b, L, D, dtype=io)
    h0, dlast = positive(g, 1, b, D, N), positive(g, 1, b, D, N)
    got = ops.selective_scan_bwd(*(v.cuda() for v in (dout, u, delta, A, B, C)), softplus=False,
                                 initial_state=h0.cuda(), dlast_state=dlast.cuda(),
                                 segments=segments)
    leaves = [ref.f64(v).requires_grad_() for v in (A, h0)]
    out, last = ref.scan(ref.f64(u), ref.f64(delta)[None], leaves[0], ref.f64(B)[None],
                         ref.f64(C)[None], softplus=False, h0=leaves[1])
    wA, w0 = torch.autograd.grad((out * ref.f64(dout)).sum() + (last * ref.f64(dlast)).sum(), leaves)
    each(got["dA"], wA, 1e-5, "dA")
    each(got["dinitial_state"], w0, 1e-5, "dinitial_state")


@pytest.mark.parametrize("segments", [1, 4])
@pytest.mark.parametrize("N", [4, 16])
def test_scan_gradient_of_long_memories(cuda_device, N, segments):
    # One Delta a channel at every step, memories of 300 to 2000 steps, every factor positive: an error
    # of the decay would be multiplied by the memory (2^-24 by 2000: 1.2e-4).  The product of four decays
    # is known to 2^-22 of its distance from one, which is what the state gets of it, and the rounding
    # errors of a step, 2^-24 with both signs, add sqrt(1000) 2^-24 = 1.9e-6 (rms) to state and gradient.
    g = gen(9)
    b, L, D = 1, 3000, 32
    memory = torch.exp(torch.empty(D, N).uniform_(5.7, 7.6, generator=g))
    step = torch.empty(D).uniform_(0.01, 0.1, generator=g)
    A = -1 / (memory * step[:, None])
    u, delta = positive(g, b, L, D), step.expand(b, L, D).contiguous()
    B, C, dout = positive(g, b, L, N), positive(g, b, L, N), positive(g, b, L, D)
    h0 = positive(g, 1, b, D, N)
    got = ops.selective_scan_bwd(*(v.cuda() for v in (dout, u, delta, A, B, C)), softplus=False,
                                 initial_state=h0.cuda(), segments=segments)
    names = ("du", "ddelta", "dA", "dB", "dC", "dinitial_state")
    leaves = [ref.f64(v).requires_grad_() for v in (u, delta[None], A, B[None], C[None], h0)]
    out, _ = ref.scan(*leaves[:5], softplus=False, h0=leaves[5])
    want = torch.autograd.grad((out * ref.f64(dout)).sum(), leaves)
    for n, w in zip(names, want):
        if n == "ddelta":  # a difference of two large sums
            ref.close(got[n], w[0], what=n)
        else:
            each(got[n], w.reshape(got[n].shape), 1.5e-5, n)


def test_scan_gradient_of_steps_of_both_signs(cuda_device):
    # decays of e^-6 to e^6 whose products lie near one: 60 steps, each off by at most 2^-21
    g = gen(10)
    b, L, D, N = 2, 60, 16, 8
    delta = 3 * torch.where(torch.arange(L) % 2 == 0, 1.0, -1.0)[None, :, None] + \
        0.01 * torch.rand(b, L, D, generator=g)
    A = -torch.linspace(0.1, 2, N).expand(D, N).contiguous()
    u, B, C, dout = (torch.randn(b, L, n, generator=g) for n in (D, N, N, D))
    got = ops.selective_scan_bwd(*(v.cuda() for v in (dout, u, delta, A, B, C)), softplus=False,
                                 segments=2)
    names = ("du", "ddelta", "dA", "dB", "dC")
    leaves = [ref.f64(v).requires_grad_() for v in (u, delta[None], A, B[None], C[None])]
    out, _ = ref.scan(*leaves, softplus=False)
    for n, w in zip(names, torch.autograd.grad((out * ref.f64(dout)).sum(), leaves)):
        ref.close(got[n], w.reshape(got[n].shape), what=n)


# ----------------------------------------------------------------------------- growth

@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("io", [F32, BF16])
def test_gates_that_grow(cuda_device, io, complement):
    # "normally <= 0": a > 1 is the same recurrence; 200 steps of up to e^0.3, about e^20 in all.  Each
    # factor is off by at most 2^-22 and four roundings, over 200 steps 1e-4 of a state at the most, a
    # tenth of that with errors of both signs: within the usual bound.
    g = gen(11)
    b, L, D = 2, 200, 24
    gate = (0.1 + 0.1 * torch.randn(b, L, D, generator=g)).to(io)
    x, dout = torch.randn(b, L, D, generator=g).to(io), torch.randn(b, L, D, generator=g).to(io)
    h0, dlast = torch.randn(b, D, generator=g), torch.randn(b, D, generator=g)
    on = [v.cuda() for v in (x, gate, h0, dout, dlast)]
    out, last = ops.gated_recurrence_fwd(on[0], on[1], initial_state=on[2], form="exp",
                                         complement=complement, return_last_state=True)
    r = [ref.f64(v) for v in (x, gate, h0, dout, dlast)]
    want, wlast = ref.recurrence(r[0], r[1], h0=r[2], form="exp", complement=complement)
    ref.close(out, want, what="out")
    ref.close(last, wlast, what="last")
    got = ops.gated_recurrence_bwd(on[3], on[0], on[1], out, initial_state=on[2], dlast_state=on[4],
                                   form="exp", complement=complement)
    wants = ref.recurrence_grads(r[3], r[0], r[1], ref.f64(out), h0=r[2], dlast=r[4], form="exp",
                                 complement=complement)
    for name, a, w in zip(("dx", "dgate", "dbias", "dh0"), got, wants):
        if a is not None:
            ref.close(a, w, what=name)


@pytest.mark.parametrize("io", [F32, BF16])
def test_scan_gradient_of_growth(cuda_device, io):
    # A of both signs: decays of e^-0.5 to e^0.15 a step, 60 steps, as above
    g = gen(12)
    b, L, D, N = 2, 60, 16, 8
    delta = (0.5 + 0.5 * torch.rand(b, L, D, generator=g)).to(io)
    A = torch.linspace(-0.5, 0.15, N).expand(D, N).contiguous()
    u, B, C, dout = (torch.randn(b, L, n, generator=g).to(io) for n in (D, N, N, D))
    h0 = torch.randn(1, b, D, N, generator=g)
    for segments in (1, 3):
        got = ops.selective_scan_bwd(*(v.cuda() for v in (dout, u, delta, A, B, C)),
                                     softplus=False, initial_state=h0.cuda(), segments=segments)
        names = ("du", "ddelta", "dA", "dB", "dC", "dinitial_state")
        leaves = [ref.f64(v).requires_grad_() for v in (u, delta[None], A, B[None], C[None], h0)]
        out, _ = ref.scan(*leaves[:5], softplus=False, h0=leaves[5])
        for n, w in zip(names, torch.autograd.grad((out * ref.f64(dout)).sum(), leaves)):
            ref.close(got[n], w.reshape(got[n].shape), what=n)
