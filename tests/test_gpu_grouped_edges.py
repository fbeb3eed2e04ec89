"""The products over ragged groups where values or calls are out of the
ordinary: ranges, non-finite weights, streams and captures, both sides of the
borders between kernels.  Tolerances as in test_gpu_grouped.py."""
import pytest
import torch

from calibration_free_channel_b200 import moe_reader as M
from tests.test_gpu_grouped import HALF, SLACK, close, dev, plan_of, swiglu_ref, sum_err, ws_for

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ SwiGLU
@pytest.mark.parametrize("u", [1.0, -2.0 ** 60, 2.0 ** 120])
def test_swiglu_keeps_small_gates(u):
    """silu(g) ~ g e^g for g far below zero, where exp(-g) leaves fp32 but the
    result does not.  g and u are single products, so exact."""
    gates = [-20.0, -80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -91.0, -95.0, -100.0, -103.0, -120.0, -150.0, 0.0,
             60.0, 90.0, 200.0]
    n = len(gates)
    x = torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = torch.tensor(gates), u
    wg, wu = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    wg[:, :, 0], wu[:, :, 1] = 1.0, 1.0
    off, _, _ = plan_of([n])
    a = torch.empty((n, 16), dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_grouped_workspace_bytes(1, n))
    M.moe_reader_grouped_swiglu(1, n, n, 16, 64, x, None, 1, off, wg, wu, a, ws, ws.numel())
    M.moe_reader_check_error(ws)
    ref, _ = swiglu_ref(x, wg[0], wu[0])
    # the exponential, the quotient and the products: 2^-20 together; below the
    # smallest normal bf16 a step of 2^-133
    close(a, ref, HALF * ref.abs() + 2.0 ** -20 * ref.abs() + 2.0 ** -133)
