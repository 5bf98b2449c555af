"""Plain 64-bit implementations of the operators around the scan (torch, CPU, one step after the
other; gradients by autograd of the plain forward), and the error bounds of the GPU tests.

Bounds: |got - ref| <= tol (|ref| + rms(ref)) + 2^-126 (a result below fp32's normal range may
become zero: its distance from zero is then below 2^-126).
  fp32 outputs  5e-5: a step rounds its state three times (2^-24 each) on top of the 2^-22 of its
                ex2, so about 5e-7 relative, and the tests' sequences add at most 1000 such errors
                of independent sign: sqrt(1000) 5e-7 = 1.6e-5; sums over channels or steps add
                rounding errors of 2^-24 per partial sum, which stay below that.
  bf16 outputs  the same, plus one rounding to bf16: half a step, 2^-8 relative.
"""

import torch

TOL = {torch.float32: 5e-5, torch.bfloat16: 2.0 ** -8 + 1e-4}


def close(got, ref, tol=None, what=""):
    tol = TOL[got.dtype] if tol is None else tol
    assert tuple(got.shape) == tuple(ref.shape), (what, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert torch.isfinite(got).all(), what
    rms = ref.square().mean().sqrt()
    err = (((got - ref).abs() - 2.0 ** -126).clamp(min=0) / (ref.abs() + rms + 1e-300)).max().item()
    assert err <= tol, "%s: %.3g > %.3g" % (what, err, tol)


def f64(t):
    return None if t is None else t.detach().double().cpu()


def order(d, L, H, W):
    """Positions visited by direction code d (0 forward, 1 reverse, 2 columns, 3 columns reversed)."""
    if d >= 2:
        p = [i * W + j for j in range(W) for i in range(H)]
    else:
        p = list(range(L))
    return p[::-1] if d in (1, 3) else p


def recurrence(x, gate, bias=None, h0=None, form="sigmoid", complement=False, reverse=False):
    if form == "sigmoid":
        s = gate if bias is None else gate + bias
        a, rest = torch.sigmoid(s), torch.sigmoid(-s)
    else:
        a, rest = torch.exp(gate), -torch.expm1(gate)
    b = rest * x if complement else x
    L = x.shape[1]
    h = torch.zeros_like(x[:, 0]) if L and h0 is None else h0
    if L == 0:
        h = torch.zeros(x.shape[0], x.shape[2], dtype=x.dtype) if h0 is None else h0
    outs = [None] * L
    for t in order(1 if reverse else 0, L, 0, 0):
        h = a[:, t] * h + b[:, t]
        outs[t] = h
    return (torch.stack(outs, 1) if L else x), h


def recurrence_grads(dout, x, gate, out, bias=None, h0=None, dlast=None, form="sigmoid",
                     complement=False, reverse=False):
    """The gradient's formulas with the states as they were kept (`out`)."""
    if form == "sigmoid":
        s = gate if bias is None else gate + bias
        a, rest = torch.sigmoid(s), torch.sigmoid(-s)
    else:
        a, rest = torch.exp(gate), -torch.expm1(gate)
    L = x.shape[1]
    steps = order(1 if reverse else 0, L, 0, 0)
    G = torch.zeros_like(x[:, 0]) if dlast is None else dlast
    dx, ds = torch.zeros_like(x), torch.zeros_like(x)
    for i in range(L - 1, -1, -1):
        t = steps[i]
        G = G + dout[:, t]
        before = out[:, steps[i - 1]] if i else (torch.zeros_like(G) if h0 is None else h0)
        if complement:
            before = before - x[:, t]
        dx[:, t] = (rest[:, t] if complement else 1) * G
        G = a[:, t] * G
        ds[:, t] = G * before * (rest[:, t] if form == "sigmoid" else 1)
    return dx, ds, ds.sum((0, 1)), G


def scan(u, delta, A, B, C, D=None, z=None, bias=None, softplus=True, dirs=(0,), H=0, W=0, h0=None):
    """(out, last_state) of the selective scan; delta, B, C: [K, ...]; u may be [K, b, L, D]."""
    K, b, L, Dm = delta.shape
    N = A.shape[-1]
    y_at = [[] for _ in range(L)]
    last = []
    for k, d in enumerate(dirs):
        uk = u[k] if u.dim() == 4 else u
        Ak, Dk, bk = (t if t is None or t.dim() == n else t[k]
                      for t, n in ((A, 2), (D, 1), (bias, 1)))
        h = torch.zeros(b, Dm, N, dtype=delta.dtype) if h0 is None else h0[k]
        for t, p in enumerate(order(d, L, H, W)):
            step = delta[k, :, t] if bk is None else delta[k, :, t] + bk
            if softplus:
                step = torch.nn.functional.softplus(step, threshold=700)
            h = torch.exp(step[..., None] * Ak) * h + \
                (step * uk[:, p])[..., None] * B[k, :, t, None]
            y = (h * C[k, :, t, None]).sum(-1)
            y_at[p].append(y if Dk is None else y + Dk * uk[:, p])
        last.append(h)
    out = torch.stack([sum(v) for v in y_at], 1) if L else torch.zeros(b, 0, Dm).double()
    if z is not None and L:
        out = out * z * torch.sigmoid(z)
    return out, torch.stack(last)


def park(h, bits):
    """Codes, scales and read-back values of states h (fp64 copies of fp32 values)."""
    q = 127 if bits == 8 else 7
    amax = h.abs().amax(-1)
    codes = torch.round(h * q / torch.where(amax > 0, amax, torch.ones_like(amax))[..., None])
    scale = (amax / q).float()
    return codes.to(torch.int8), scale


def pack4(codes):
    """Two codes a byte, the even state in the low half."""
    if codes.shape[-1] % 2:
        codes = torch.nn.functional.pad(codes, (0, 1))
    return (codes[..., 0::2] & 15) | (codes[..., 1::2] << 4)
