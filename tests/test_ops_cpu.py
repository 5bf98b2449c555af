"""The operators' C ABI on the host, without a GPU: exported symbols, and every refusal comes with
its status before any device is touched (the addresses given are never dereferenced, and no call
here is one that would be accepted)."""

import ctypes
import os
import re

import pytest

from selective_state_space_13_b200 import ops, scan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # 16-byte aligned, never dereferenced: validation fails first


def test_exports_are_the_header():
    text = open(os.path.join(ROOT, "include", "selective_scan_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*ss_status\s+([a-z_]+)\s*\(", text, flags=re.M))
    assert names == set(ops.EXPORTED)
    lib = ops.load()
    for name in names:
        assert hasattr(lib, name)


def shape(**kw):
    base = dict(batch=2, seqlen=64, dim=32, dstate=16, io_dtype=scan.SS_BF16)
    base.update(kw)
    return scan.make_shape(**base)


BAD_SHAPES = [(dict(batch=-1), 2), (dict(seqlen=1 << 31), 2), (dict(io_dtype=7), 3),
              (dict(dim=12), 4), (dict(dstate=0), 2), (dict(dstate=17), 6),
              (dict(seqlen=1 << 20, dim=1 << 12), 2), (dict(batch=1 << 20, seqlen=1 << 10), 2)]


@pytest.mark.parametrize("kw,expect", BAD_SHAPES)
def test_bwd_shapes(kw, expect):
    with pytest.raises(scan.ScanError) as e:
        ops.selective_scan_bwd_workspace_size(shape(**kw))
    assert e.value.status == expect


def bwd(sh=None, dmap=None, opts=None, ws=None, **kw):
    """The status of selective_scan_bwd with valid fake arguments, some replaced."""
    a = dict(u=FAKE, delta=FAKE, A=FAKE, B=FAKE, C=FAKE, D=FAKE, z=FAKE, bias=FAKE, dout=FAKE,
             dlast=None)
    g = dict(du=FAKE, ddelta=FAKE, dA=FAKE, dB=FAKE, dC=FAKE, dDskip=FAKE, dz=FAKE,
             ddelta_bias=FAKE, dinitial_state=None)
    for k, v in kw.items():
        (g if k in g else a)[k] = v
    sh = sh or shape()
    grads = ops.SsScanGrads(**g)
    need = ops.selective_scan_bwd_workspace_size(sh, dmap, opts) if ws is None else ws
    ref = ctypes.byref
    return ops.load().selective_scan_bwd(
        ref(sh), a["u"], a["delta"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], 1,
        ref(dmap) if dmap else None, a["dout"], a["dlast"], ref(grads), FAKE, need, None,
        ref(opts) if opts else None)


def test_bwd_arguments():
    for name in ("u", "delta", "A", "B", "C", "dout", "du", "ddelta", "dA", "dB", "dC", "dz"):
        assert bwd(**{name: None}) == 1, name
    for name in ("u", "delta", "B", "C", "z", "dout", "du", "ddelta", "dB", "dC", "dz"):
        assert bwd(**{name: FAKE + 8}) == 4, name
    for name in ("A", "D", "bias", "dlast", "dA", "dDskip", "ddelta_bias", "dinitial_state"):
        assert bwd(**{name: FAKE + 2}) == 4, name
    # a gradient of something that the call does not have
    assert bwd(z=None) == 6 and bwd(D=None) == 6 and bwd(bias=None) == 6
    need = ops.selective_scan_bwd_workspace_size(shape())
    assert bwd(ws=need - 1) == 8


def test_bwd_options():
    for flags in (scan.SS_FLAG_ZOH_EXACT, scan.SS_FLAG_TEST_WAIT_TIMEOUT, scan.SS_FLAG_DELTA_INT8,
                  1 << 20):
        assert bwd(opts=scan.make_opts(flags=flags), ws=1 << 40) == 6
    assert bwd(opts=scan.make_opts(conv_weight=FAKE, conv_width=4), ws=1 << 40) == 6
    assert bwd(opts=scan.make_opts(segments=-1), ws=1 << 40) == 6
    assert bwd(opts=scan.make_opts(segments=1025), ws=1 << 40) == 6
    for dirs, H, W in (((4,), 0, 0), ((2,), 8, 7), ((2,), 0, 64)):
        assert bwd(dmap=scan.make_dirmap(dirs, H, W), ws=1 << 40) == 5
    # what is supported has a workspace size
    for flags in (scan.SS_FLAG_GENERIC_A, scan.SS_FLAG_U_PER_DIRECTION,
                  scan.SS_FLAG_PARAMS_PER_DIRECTION):
        assert ops.selective_scan_bwd_workspace_size(
            shape(), scan.make_dirmap((0, 2, 1, 3), 8, 8), scan.make_opts(flags=flags)) > 0


def rec(backward=False, sh=None, form=0, dir=0, reserved=0, ws=1 << 40, **kw):
    a = dict(x=FAKE, gate=FAKE, bias=None, init=None, out=FAKE, last=None, dout=FAKE, dlast=None,
             dx=FAKE, dgate=FAKE, dbias=None, dinit=None, w=FAKE)
    a.update(kw)
    sh = sh or shape(dstate=1)
    o = ops.SsRecurrenceOpts(form, 0, dir, reserved)
    ref = ctypes.byref
    if backward:
        return ops.load().gated_recurrence_bwd(
            ref(sh), ref(o), a["x"], a["gate"], a["bias"], a["init"], a["out"], a["dout"],
            a["dlast"], a["dx"], a["dgate"], a["dbias"], a["dinit"], a["w"], ws, None)
    return ops.load().gated_recurrence_fwd(ref(sh), ref(o), a["x"], a["gate"], a["bias"], a["init"],
                                           a["out"], a["last"], a["w"], ws, None)


@pytest.mark.parametrize("backward", [False, True])
def test_recurrence_refusals(backward):
    for kw, expect in BAD_SHAPES:
        if "dstate" not in kw:
            assert rec(backward, sh=shape(**dict(dict(dstate=1), **kw))) == expect
    assert rec(backward, sh=shape(dstate=2)) == 2
    assert rec(backward, form=2) == 6 and rec(backward, reserved=1) == 6
    assert rec(backward, dir=2) == 5 and rec(backward, dir=-1) == 5
    assert rec(backward, form=1, bias=FAKE) == 6
    names = ("x", "gate", "out") + (("dout", "dx", "dgate") if backward else ())
    for name in names:
        assert rec(backward, **{name: None}) == 1
        assert rec(backward, **{name: FAKE + 8}) == 4
    assert rec(backward, bias=FAKE + 2) == 4
    n = ops.gated_recurrence_workspace_size(shape(dstate=1), ops.SsRecurrenceOpts(0, 0, 0, 0),
                                            backward)
    assert (n > 0) == backward
    if backward:
        assert rec(True, form=1, dbias=FAKE) == 6
        assert rec(True, ws=n - 1) == 8 and rec(True, w=None) == 8


def step(sh=None, slots=FAKE, num_slots=4, width=0, ws=None, **kw):
    a = dict(u=FAKE, delta=FAKE, A=FAKE, B=FAKE, C=FAKE, D=None, z=None, bias=None, state=FAKE,
             cw=None, cb=None, cs=None, out=FAKE)
    a.update(kw)
    return ops.load().selective_scan_step(
        ctypes.byref(sh or shape(seqlen=1)), num_slots, a["u"], a["delta"], a["A"], a["B"], a["C"],
        a["D"], a["z"], a["bias"], 1, a["state"], slots, a["cw"], a["cb"], width, a["cs"], a["out"],
        None)


def test_step_refusals():
    for kw, expect in BAD_SHAPES:
        if "seqlen" not in kw:
            assert step(sh=shape(**dict(dict(seqlen=1), **kw))) == expect
    assert step(sh=shape(seqlen=2)) == 2 and step(num_slots=0) == 2
    assert step(slots=None, num_slots=1) == 2  # two rows, one slot
    for name in ("u", "delta", "A", "B", "C", "state", "out"):
        assert step(**{name: None}) == 1, name
    for name in ("u", "delta", "B", "C", "state", "out", "z"):
        assert step(**{name: FAKE + 8}) == 4, name
    assert step(slots=FAKE + 2) == 4 and step(A=FAKE + 1) == 4
    assert step(cw=FAKE, width=4) == 1
    assert step(cw=FAKE, width=5, cs=FAKE) == 6 and step(cw=FAKE, width=0) == 6
    assert step(width=4) == 6 and step(cb=FAKE) == 6 and step(cs=FAKE) == 6


@pytest.mark.parametrize("load", [False, True])
def test_state_cache_refusals(load):
    lib = ops.load()

    def call(rows=2, D=8, N=16, bits=8, state=FAKE, nstate=4, src=FAKE, codes=FAKE, scales=FAKE,
             ncache=4, dst=FAKE):
        if load:
            return lib.selective_state_load(rows, D, N, bits, codes, scales, ncache, src, state,
                                            nstate, dst, None)
        return lib.selective_state_store(rows, D, N, bits, state, nstate, src, codes, scales, ncache,
                                         dst, None)

    assert call(rows=0) == 0 and call(D=0) == 0
    assert call(rows=-1) == 2 and call(D=-1) == 2 and call(N=0) == 2
    assert call(N=17) == 6 and call(bits=3) == 6
    assert call(nstate=0) == 2 and call(ncache=0) == 2
    assert call(rows=5, src=None) == 2 and call(rows=5, dst=None) == 2
    for name in ("state", "codes", "scales"):
        assert call(**{name: None}) == 1
    assert call(state=FAKE + 4) == 4 and call(codes=FAKE + 1) == 4 and call(src=FAKE + 2) == 4


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError):
        ops.gated_recurrence_fwd(x, x)
    with pytest.raises(ValueError):
        ops.selective_scan_step(x[:, 0], x[:, 0], torch.zeros(8, 4), x[:, 0], x[:, 0],
                                torch.zeros(2, 8, 4))
    with pytest.raises(ValueError):
        ops.selective_state_store(torch.zeros(2, 8, 4), torch.zeros(2, 8, 4, dtype=torch.int8),
                                  torch.zeros(2, 8))
    with pytest.raises(ValueError):
        ops.selective_scan_bwd(x, x, x, torch.zeros(8, 4), x, x)


def test_long_slot_lists_are_refused():
    # every row looks through the list before it: 2^20 rows are the most
    most = 1 << 20
    assert step(sh=shape(batch=most + 1, seqlen=1, dim=8, dstate=1), num_slots=4) == 2
    lib = ops.load()
    for src, dst in ((None, FAKE), (FAKE, FAKE)):
        assert lib.selective_state_store(most + 1, 8, 1, 8, FAKE, most + 1, src, FAKE, FAKE,
                                         most + 1, dst, None) == 2
        assert lib.selective_state_load(most + 1, 8, 1, 8, FAKE, FAKE, most + 1, src, FAKE,
                                        most + 1, dst, None) == 2
    # ... and what is refused for another reason keeps it
    assert step(sh=shape(batch=most + 1, seqlen=1, dim=8, dstate=1), slots=None,
                num_slots=most + 1, u=None) == 1
