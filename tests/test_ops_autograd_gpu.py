"""The operators under torch.autograd where the incoming gradients are not what a sum leaves:
views that start between 16-byte borders, broadcast values, and none at all."""

import pytest
import torch

from selective_state_space_13_b200 import ops
from tests import ops_util as ref

pytestmark = pytest.mark.gpu


def leaf(g, *shape):
    return torch.randn(*shape, generator=g).cuda().requires_grad_()


def losses():
    """Ways from (out, last) to a scalar, by what they make of the incoming gradients."""
    def behind_one_value(out, last):
        # the gradient of out is a slice of a flat tensor, four bytes behind its start
        flat = torch.cat([out.new_ones(1), out.flatten(), last.flatten().to(out.dtype)])
        return (flat * torch.linspace(-1, 1, flat.numel(), device=flat.device)).sum()

    return {"behind one value": behind_one_value,
            "broadcast": lambda out, last: 3 * out.sum() - last.sum(),
            "transposed": lambda out, last: (out.transpose(1, 2).contiguous().square().sum()
                                             + last.transpose(-1, -2).contiguous().sin().sum()),
            "out alone": lambda out, last: out.square().sum(),
            "last alone": lambda out, last: last.square().sum()}


def check(call, plain, leaves, loss):
    grads = torch.autograd.grad(loss(*call(*leaves)), leaves)
    exact = [ref.f64(v).requires_grad_() for v in leaves]
    value = loss(*plain(*exact))
    want = torch.autograd.grad(value, exact, allow_unused=True, materialize_grads=True)
    for a, w in zip(grads, want):
        ref.close(a, w, tol=2e-4)  # the incoming gradients are fp32 outputs themselves


@pytest.mark.parametrize("name", sorted(losses()))
def test_recurrence_incoming_gradients(cuda_device, name):
    g = torch.Generator().manual_seed(1)
    b, L, D = 2, 37, 24
    leaves = [leaf(g, b, L, D), leaf(g, b, L, D), leaf(g, D), leaf(g, b, D)]
    check(lambda *v: ops.gated_recurrence(*v, complement=True),
          lambda *v: ref.recurrence(*v, complement=True), leaves, losses()[name])


@pytest.mark.parametrize("name", sorted(losses()))
def test_scan_incoming_gradients(cuda_device, name):
    g = torch.Generator().manual_seed(2)
    b, L, D, N = 2, 37, 24, 4
    leaves = [leaf(g, b, L, D), leaf(g, 1, b, L, D), leaf(g, D, N), leaf(g, 1, b, L, N),
              leaf(g, 1, b, L, N), leaf(g, D), leaf(g, b, L, D), leaf(g, D), leaf(g, 1, b, D, N)]
    with torch.no_grad():
        leaves[2].abs_().neg_()
    check(lambda *v: ops.selective_scan(*v[:8], initial_state=v[8]),
          lambda *v: ref.scan(*v[:8], h0=v[8]), leaves, losses()[name])
