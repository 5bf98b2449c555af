"""Flags that speak of shapes are the shapes': a call that names them against its tensors would read
behind them, and is refused before any device is asked for."""

import pytest
import torch

from selective_state_space_13_b200 import ops, scan

u, A, B = torch.zeros(2, 4, 8), torch.zeros(8, 4), torch.zeros(2, 2, 4, 4)
delta = torch.zeros(2, 2, 4, 8)
CALLS = {
    "fwd": lambda **kw: scan.selective_scan_fwd(u, delta, A, B, B, dirs=(0, 1), **kw),
    "host": lambda **kw: scan.selective_scan_fwd_host(u, delta, A, B, B, dirs=(0, 1),
                                                      device=torch.device("cuda", 0), **kw),
    "bwd": lambda **kw: ops.selective_scan_bwd(u, u, delta, A, B, B, dirs=(0, 1), **kw),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("flag", [scan.SS_FLAG_U_PER_DIRECTION, scan.SS_FLAG_PARAMS_PER_DIRECTION])
def test_flags_against_shapes(name, flag):
    with pytest.raises(ValueError, match="flags"):
        CALLS[name](flags=flag)


@pytest.mark.parametrize("name", ["fwd", "host"])
def test_int8_flag_without_codes(name):
    with pytest.raises(ValueError, match="flags"):
        CALLS[name](flags=scan.SS_FLAG_DELTA_INT8, delta_scale=torch.ones(8))
