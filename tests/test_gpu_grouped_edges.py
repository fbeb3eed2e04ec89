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


# ------------------------------------------------------------------ adapters
def adapter_call(T, A, K, N, r, seed=0, use_w=True, use_base=True, ids=None, inplace=False, **put):
    """One call over random ids (none among them); put: tensors to use in place of the drawn ones."""
    if ids is None:
        ids = torch.randint(-1, A, (T,), generator=torch.Generator("cuda").manual_seed(seed), device="cuda",
                            dtype=torch.int32)
    t = dict(x=dev(T, K, seed=seed + 1), w=dev(N, K, seed=seed + 2, scale=K ** -0.5) if use_w else None,
             base=dev(T, N, seed=seed + 3) if use_base else None, a=dev(A, r, K, seed=seed + 4, scale=K ** -0.5),
             b=dev(A, N, r, seed=seed + 5), scale=torch.linspace(-1.5, 2.0, A, device="cuda"))
    t.update(put)
    off, rows = torch.empty(A + 1, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    ws = ws_for(M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))
    M.moe_reader_group_rows(T, A, ids, off, rows, ws, ws.numel())
    y = t["base"].clone() if inplace else torch.full((T, N), 9.0, dtype=torch.bfloat16, device="cuda")
    M.moe_reader_adapter_product(T, A, N, K, r, t["x"], t["w"], y if inplace else t["base"], off, rows, t["a"], t["b"],
                                 t["scale"], y, ws, ws.numel())
    M.moe_reader_check_error(ws)
    return y, ids, t


@pytest.mark.parametrize("T,A", [(3, 2), (90, 5), (700, 40), (2100, 5), (2300, 60)])
@pytest.mark.parametrize("bad", ["a nan", "a inf", "scale"])
def test_adapters_down_side_nonfinite_stays_apart(T, A, bad):
    """Weights of A or a scale that are not finite reach the adapter's own tokens only."""
    K, N, r = 256, 264, 24
    y, ids, t = adapter_call(T, A, K, N, r)
    a, scale = t["a"].clone(), t["scale"].clone()
    if bad == "scale":
        scale[1] = float("inf")
    else:
        a[1, 5, 100:103] = float("nan" if bad == "a nan" else "inf")
    z, _, _ = adapter_call(T, A, K, N, r, a=a, scale=scale)
    mine = ids == 1
    assert torch.equal(z[~mine], y[~mine])
    assert not bool(torch.isfinite(z[mine]).any()) or bad != "a nan"
