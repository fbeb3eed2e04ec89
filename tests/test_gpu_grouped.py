"""The products over ragged groups against their definitions in 64 bits.

Tolerances.  A bf16 output is off by half a step, 2^-8 of its value, for the
one rounding at the end.  A sum of K exact products in fp32 is off by at most
K 2^-23 times the sum of the terms' sizes, whatever the order (2^-24 a step
if every step rounds to nearest, 2^-23 if it truncates).  An intermediate held
in bf16 is off by 2^-8 of its value, one held in two bf16 terms by 2^-16.
The errors of a chain are carried through it linearly; `SLACK` covers the
products of two such errors."""
import numpy as np
import pytest
import torch

from calibration_free_channel_b200 import moe_reader as M
from calibration_free_channel_b200 import synth
from oracle import oracle as O

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
SLACK = 1.05


def sum_err(K):
    return K * 2.0 ** -23


def dev(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def ws_for(nb):
    return torch.zeros(max(nb, 16), dtype=torch.uint8, device="cuda")


def plan_of(sizes, seed=0, extra=0):
    """offsets and a random row order for groups of the given sizes, `extra` rows of no group behind them."""
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n = int(off[-1]) + extra
    rows = np.random.default_rng(seed).permutation(n).astype(np.int32)
    return torch.from_numpy(off).cuda(), torch.from_numpy(rows).cuda(), n


def close(y, ref, tol):
    y = y.double()
    bad = ~((y - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float(((y - ref).abs() - tol).max()), tuple(bad.nonzero()[0].tolist()))


# ------------------------------------------------------------------ grouping
@pytest.mark.parametrize("n,G", [(1, 1), (1, 1024), (2, 1), (31, 3), (33, 128), (1023, 7), (1024, 1024), (1025, 5),
                                 (4097, 128), (20000, 1000), (65536, 128), (70001, 13), (1 << 20, 64)])
@pytest.mark.parametrize("kind", ["even", "one", "none", "mixed"])
def test_group_rows(n, G, kind):
    rng = np.random.default_rng(n * 7 + G)
    ids = {"even": rng.integers(0, G, n), "one": np.full(n, G - 1), "none": np.full(n, -1),
           "mixed": rng.integers(-2, G + 3, n)}[kind].astype(np.int32)
    if kind == "mixed":
        ids[:2] = [2 ** 31 - 1, -2 ** 31][:min(n, 2)]
    key = np.where((ids >= 0) & (ids < G), ids, G)
    offsets = torch.full((G + 1,), -7, dtype=torch.int32, device="cuda")
    rows = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    ws = ws_for(M.moe_reader_group_workspace_bytes(n, G))
    M.moe_reader_group_rows(n, G, torch.from_numpy(ids).cuda(), offsets, rows, ws, ws.numel())
    assert np.array_equal(rows.cpu().numpy(), np.argsort(key, kind="stable"))
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(key, minlength=G + 1)[:G])]))
    M.moe_reader_check_error(ws)


# ------------------------------------------------------------------ products
RAGGED = [0, 1, 2, 0, 15, 16, 17, 33, 64, 0, 127, 129, 255, 256, 257, 300, 0]


def run_product(x, w, sizes, layout, gather, scatter, extra=0, x_div=1, seed=0):
    """y from the library, and the 64-bit product with its sizes sum, for a plan of these sizes."""
    off, rows, P = plan_of(sizes, seed, extra)
    G = len(sizes)
    K, N = (w.shape[1], w.shape[2]) if layout else (w.shape[2], w.shape[1])
    y = torch.full((P, N), 7.25, dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_grouped_workspace_bytes(G, P))
    M.moe_reader_grouped_product(G, P, x.shape[0], P, N, K, layout, x, rows if gather else None, x_div, off, w, y,
                                 rows if scatter else None, ws, ws.numel())
    M.moe_reader_check_error(ws)
    ref = torch.full((P, N), 7.25, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    o = off.tolist()
    for g in range(G):
        p = torch.arange(o[g], o[g + 1], device="cuda")
        if p.numel() == 0:
            continue
        xr = x[rows[p].long() // x_div if gather else p].double()
        wg = w[g].double() if layout else w[g].double().T
        q = rows[p].long() if scatter else p
        ref[q], mag[q] = xr @ wg, xr.abs() @ wg.abs()
    return y, ref, HALF * ref.abs() + SLACK * sum_err(K) * mag


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (72, 136), (200, 120), (256, 16), (768, 2048), (1096, 520)])
def test_grouped_product(layout, K, N):
    G, n = len(RAGGED), sum(RAGGED)
    w = dev(G, K, N, seed=1) if layout else dev(G, N, K, seed=1)
    x = dev(n, K, seed=2)
    for gather, scatter in ((False, False), (True, False), (False, True), (True, True)):
        close(*run_product(x, w, RAGGED, layout, gather, scatter))


@pytest.mark.parametrize("sizes", [[1], [0, 1, 0], [5], [16], [1, 1, 1, 1], [0, 0, 700], [2000], [37] * 40, [3] * 300])
@pytest.mark.parametrize("layout", [0, 1])
def test_grouped_product_sizes(layout, sizes):
    K, N, G = 512, 384, len(sizes)
    w = dev(G, K, N, seed=3) if layout else dev(G, N, K, seed=3)
    close(*run_product(dev(sum(sizes), K, seed=4), w, sizes, layout, False, True))


@pytest.mark.parametrize("sizes", [[257, 0, 900, 3, 512], [2000, 512, 511, 513, 290, 1, 300], [640] * 9 + [7, 33, 256]])
@pytest.mark.parametrize("kind", ["layout 0", "layout 1", "gathered"])
def test_grouped_product_large_groups(sizes, kind):
    # groups of hundreds of rows, several tiles each, between small ones
    K, N, G = 392, 1032, len(sizes)
    layout = int(kind == "layout 1")
    w = dev(G, K, N, seed=18) if layout else dev(G, N, K, seed=18)
    close(*run_product(dev(sum(sizes), K, seed=19), w, sizes, layout, kind == "gathered", True))


@pytest.mark.parametrize("gather", [True, False])
def test_grouped_swiglu_large_groups(gather):
    sizes, I, d = [700, 2, 0, 290, 1500, 256], 200, 264
    off, rows, P = plan_of(sizes, 4)
    x, wg, wu = dev(P, d, seed=24), dev(6, I, d, seed=25, scale=2 * d ** -0.5), dev(6, I, d, seed=26)
    a = torch.empty((P, I), dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_grouped_workspace_bytes(6, P))
    M.moe_reader_grouped_swiglu(6, P, P, I, d, x, rows if gather else None, 1, off, wg, wu, a, ws, ws.numel())
    M.moe_reader_check_error(ws)
    o = off.tolist()
    for g in range(6):
        p = torch.arange(o[g], o[g + 1], device="cuda")
        if p.numel():
            ref, e = swiglu_ref(x[rows[p].long() if gather else p], wg[g], wu[g])
            close(a[p], ref, HALF * ref.abs() + SLACK * e)


def test_grouped_product_no_rows():
    # every group empty: nothing is written
    y, ref, tol = run_product(dev(64, 64, seed=5), dev(3, 64, 64, seed=6), [0, 0, 0], 0, False, False, extra=40)
    assert torch.equal(y.double(), ref)


def test_grouped_product_rows_of_no_group_stay():
    x, w = dev(100 + 60, 128, seed=7), dev(2, 256, 128, seed=8)
    y, ref, tol = run_product(x, w, [70, 30], 0, False, False, extra=60)
    close(y, ref, tol)
    assert torch.equal(y[100:], torch.full_like(y[100:], 7.25))


def test_grouped_product_division_and_repeats():
    # rows / x_div: the pairs of a token share its row of x
    close(*run_product(dev(50, 320, seed=9), dev(4, 128, 320, seed=10), [100, 0, 37, 13], 0, True, False, x_div=3))


def test_grouped_product_nonfinite_rows_stay_apart():
    # a row of infinities or NaN spoils no other row, in its group or the next, also inside one tile
    sizes = [20, 30, 5]
    x, w = dev(55, 256, seed=11), dev(3, 128, 256, seed=12)
    clean, ref, tol = run_product(x, w, sizes, 0, False, False)
    x2 = x.clone()
    x2[7], x2[20], x2[54] = float("nan"), float("inf"), -float("inf")
    y, _, _ = run_product(x2, w, sizes, 0, False, False)
    keep = [i for i in range(55) if i not in (7, 20, 54)]
    assert torch.equal(y[keep], clean[keep])
    assert not bool(torch.isfinite(y[[7, 20, 54]]).any())


def test_grouped_product_large_offsets():
    # the last weight element lies past 2^31 elements: 65 experts of 4096 x 8192
    G, K, N = 65, 4096, 8192
    sizes = [0] * G
    sizes[0], sizes[64] = 3, 20
    for layout in (0, 1):
        w = torch.empty((G, K, N) if layout else (G, N, K), dtype=torch.bfloat16, device="cuda")
        w[0], w[64] = dev(*w.shape[1:], seed=13), dev(*w.shape[1:], seed=14)
        close(*run_product(dev(23, K, seed=15), w, sizes, layout, False, False))
        del w


def swiglu_ref(x, wg, wu):
    """Definition in 64 bits and the tolerance of one group."""
    K = x.shape[1]
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.T, x @ wu.T
    eg, eu = sum_err(K) * (x.abs() @ wg.abs().T), sum_err(K) * (x.abs() @ wu.abs().T)
    s = g * torch.sigmoid(g)
    a = s * u
    # |silu'| <= 1.1; the exponential, the sum and the quotient in fp32 cost a few 2^-22 of the value
    ea = 1.1 * eg * u.abs() + s.abs() * eu + 1.1 * eg * eu + 2.0 ** -20 * a.abs()
    return a, ea


@pytest.mark.parametrize("I,d", [(8, 8), (16, 64), (100, 256), (77, 136), (768, 2048), (1, 64)])
@pytest.mark.parametrize("gather", [True, False])
def test_grouped_swiglu(I, d, gather):
    sizes, top = RAGGED, 3
    off, rows, P = plan_of(sizes, 3, extra=5)
    G = len(sizes)
    n_x = (P + top - 1) // top if gather else P
    x, wg, wu = dev(n_x, d, seed=21), dev(G, I, d, seed=22, scale=2 * d ** -0.5), dev(G, I, d, seed=23)
    a = torch.full((P, I), 3.5, dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_grouped_workspace_bytes(G, P))
    M.moe_reader_grouped_swiglu(G, P, n_x, I, d, x, rows if gather else None, top if gather else 1, off, wg, wu, a,
                                ws, ws.numel())
    M.moe_reader_check_error(ws)
    o = off.tolist()
    for g in range(G):
        p = torch.arange(o[g], o[g + 1], device="cuda")
        if p.numel() == 0:
            continue
        ref, e = swiglu_ref(x[rows[p].long() // top if gather else p], wg[g], wu[g])
        close(a[p], ref, HALF * ref.abs() + SLACK * e)
    assert torch.equal(a[o[-1]:], torch.full_like(a[o[-1]:], 3.5))


def test_grouped_swiglu_extremes():
    # gates far out: silu(-big) u -> 0 or -0, silu(big) u = big u, no NaN from exp overflow
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([300.0, -300.0, 3e18, -3e18])
    wg = torch.zeros((1, 16, 64), dtype=torch.bfloat16, device="cuda")
    wg[:, :, 0] = 1.0
    off, rows, P = plan_of([4])
    a = torch.empty((4, 16), dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_grouped_workspace_bytes(1, 4))
    M.moe_reader_grouped_swiglu(1, 4, 4, 16, 64, x, None, 1, off, wg, wg, a, ws, ws.numel())
    ref = torch.tensor([300.0 ** 2, 0.0, float(x[2, 0]) ** 2, 0.0], dtype=torch.float64)
    got = a[:, 0].double().cpu()
    assert torch.isfinite(a).all()
    assert ((got - ref).abs() <= HALF * ref.abs() + 1e-30).all(), got


# ------------------------------------------------------------------ adapters
def run_adapter(T, A, K, N, r, ids, use_w, use_base, use_scale=True, seed=0, inplace=False):
    x = dev(T, K, seed=seed + 31)
    w = dev(N, K, seed=seed + 32, scale=K ** -0.5) if use_w else None
    base = dev(T, N, seed=seed + 33) if use_base else None
    a, b = dev(A, r, K, seed=seed + 34, scale=K ** -0.5), dev(A, N, r, seed=seed + 35)
    scale = torch.linspace(-1.5, 2.0, A, device="cuda") if use_scale else None
    off = torch.empty(A + 1, dtype=torch.int32, device="cuda")
    rows = torch.empty(T, dtype=torch.int32, device="cuda")
    ws = ws_for(M.moe_reader_group_workspace_bytes(T, A))
    M.moe_reader_group_rows(T, A, ids, off, rows, ws, ws.numel())
    ws = ws_for(M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))
    ref = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    err = torch.zeros_like(ref)
    if use_base:
        ref += base.double()
        err += 2.0 ** -24 * base.double().abs()
    xd = x.double()
    if use_w:
        ref += xd @ w.double().T
        err += sum_err(K) * (xd.abs() @ w.double().abs().T)
    for g in range(A):
        t = (ids == g).nonzero().flatten()
        if t.numel() == 0:
            continue
        s = float(scale[g]) if use_scale else 1.0
        z, bd = s * (xd[t] @ a[g].double().T), b[g].double()
        ez = abs(s) * sum_err(K) * (xd[t].abs() @ a[g].double().abs().T) + (2.0 ** -16 + 2.0 ** -22) * z.abs()
        ref[t] += z @ bd.T
        err[t] += ez @ bd.abs().T + sum_err(2 * r + 8) * (z.abs() @ bd.abs().T)
    # the terms meet in one fp32 accumulator: a few roundings of the running value
    err += 2.0 ** -20 * ref.abs()
    y = base.clone() if inplace else torch.full((T, N), 9.0, dtype=torch.bfloat16, device="cuda")
    M.moe_reader_adapter_product(T, A, N, K, r, x, w, y if inplace else base, off, rows, a, b, scale, y, ws,
                                 ws.numel())
    M.moe_reader_check_error(ws)
    close(y, ref, HALF * ref.abs() + SLACK * err + 1e-30)
    return y


def ids_of(T, A, kind, seed=0):
    rng = np.random.default_rng(seed)
    v = {"all": np.zeros(T), "none": np.full(T, -1), "random": rng.integers(-1, A, T),
         "runs": np.repeat(rng.integers(-1, A, T), 37)[:T], "distinct": np.arange(T) % A}[kind]
    return torch.from_numpy(v.astype(np.int32)).cuda()


@pytest.mark.parametrize("T,A,kind", [(1, 1, "all"), (1, 4, "none"), (2, 5, "distinct"), (17, 3, "random"),
                                      (64, 64, "distinct"), (255, 9, "random"), (257, 1, "all"), (300, 300, "distinct"),
                                      (700, 6, "runs"), (1500, 40, "random"), (513, 4, "none")])
@pytest.mark.parametrize("use_w,use_base", [(True, False), (False, True), (True, True), (False, False)])
def test_adapter_product(T, A, kind, use_w, use_base):
    run_adapter(T, A, 320, 264, 24, ids_of(T, A, kind), use_w, use_base)


@pytest.mark.parametrize("r", [8, 16, 40, 64, 72, 128])
@pytest.mark.parametrize("K,N", [(8, 8), (200, 136), (2048, 2048)])
def test_adapter_product_ranks(r, K, N):
    run_adapter(70, 5, K, N, r, ids_of(70, 5, "random"), True, False)
    run_adapter(333, 3, K, N, r, ids_of(333, 3, "runs"), False, True, use_scale=False)


@pytest.mark.parametrize("use_w,use_base", [(True, True), (False, True)])
@pytest.mark.parametrize("kind", ["runs", "random", "all"])
def test_adapter_product_many_tiles(kind, use_w, use_base):
    # several tiles to a CTA pair, the ring going round many times between the adapters' stages
    T = 3001
    run_adapter(T, 5, 1096, 4096, 64, ids_of(T, 5, kind), use_w, use_base)


def test_adapter_product_in_place():
    ids = ids_of(90, 7, "random")
    y = run_adapter(90, 7, 256, 512, 16, ids, False, True, inplace=True)
    assert torch.equal(y, run_adapter(90, 7, 256, 512, 16, ids, False, True))


def test_adapter_product_nonfinite_tokens_stay_apart():
    T, A, K, N, r = 40, 3, 128, 256, 16
    ids = ids_of(T, A, "random", 5)
    clean = run_adapter(T, A, K, N, r, ids, True, True)
    off = torch.empty(A + 1, dtype=torch.int32, device="cuda")
    rows = torch.empty(T, dtype=torch.int32, device="cuda")
    ws = ws_for(M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))
    M.moe_reader_group_rows(T, A, ids, off, rows, ws, ws.numel())
    x = dev(T, K, seed=31)
    x[11], x[12] = float("nan"), float("inf")
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    M.moe_reader_adapter_product(T, A, N, K, r, x, dev(N, K, seed=32, scale=K ** -0.5), dev(T, N, seed=33), off, rows,
                                 dev(A, r, K, seed=34, scale=K ** -0.5), dev(A, N, r, seed=35),
                                 torch.linspace(-1.5, 2.0, A, device="cuda"), y, ws, ws.numel())
    keep = [i for i in range(T) if i not in (11, 12)]
    assert torch.equal(y[keep], clean[keep])
    assert not bool(torch.isfinite(y[11]).any())


# ------------------------------------------------------------------ the block
def block_ref(x, w, top, residual=None):
    """The block in 64 bits, the chosen experts, and the elementwise tolerance."""
    x = x.double()
    logits = x @ w["w_router"].double().T
    if w["router_bias"] is not None:
        logits = logits + w["router_bias"].double()
    vals, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, share = ids[:, :top], torch.softmax(vals[:, :top], 1)
    y, err = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(logits.shape[1]):
        t, k = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        a, ea = swiglu_ref(x[t], w["w_gate"][e], w["w_up"][e])
        wd, s = w["w_down"][e].double(), share[t, k][:, None]
        y[t] += s * (a @ wd)
        err[t] += s * ((ea + HALF * a.abs() + sum_err(a.shape[1] + 16) * a.abs()) @ wd.abs())
    if residual is not None:
        y = y + residual.double()
    return y, ids, HALF * y.abs() + SLACK * err


@pytest.mark.parametrize("B", [1, 2, 5, 17, 64, 300, 1000])
@pytest.mark.parametrize("bias,res", [(False, True), (True, False)])
def test_block_tiny(B, bias, res):
    W = {k: v.cuda() if v is not None else None for k, v in synth.layer_weights(synth.TINY, seed=3, bias=bias).items()}
    L = M.Layer(W, top_e=2)
    x = synth.tokens(256, B, seed=5).cuda()
    residual = dev(B, 256, seed=6) if res else None
    ids = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    y = L.forward_grouped(x, residual, ids)
    L.check()
    ref, rid, tol = block_ref(x, W, 2, residual)
    assert torch.equal(ids.long(), rid)
    close(y, ref, tol)


@pytest.mark.parametrize("E,I,d,top,B", [(5, 77, 512, 5, 40), (64, 100, 256, 1, 777), (33, 2048, 1024, 16, 50),
                                         (1024, 24, 256, 4, 200), (1, 16, 4096, 1, 130), (128, 768, 2048, 8, 300)])
def test_block_shapes(E, I, d, top, B):
    W = synth.layer_weights(synth.BlockShape(E, I, d, top), seed=4, bias=True, device="cuda")
    L = M.Layer(W, top_e=top)
    x = synth.tokens(d, B, seed=7).cuda()
    ids = torch.full((B, top), -1, dtype=torch.int32, device="cuda")
    y = L.forward_grouped(x, ids=ids)
    L.check()
    ref, rid, tol = block_ref(x, W, top)
    assert torch.equal(ids.long(), rid)
    close(y, ref, tol)


def test_block_agrees_with_the_dense_block():
    # up to 256 tokens the dense block computes the same thing without rounding the SwiGLU values
    W = synth.layer_weights(synth.TINY, seed=8)
    L = M.Layer(W, top_e=2)
    x = synth.tokens(256, 200, seed=9).cuda()
    yd, yg = L.forward_dense(x), L.forward_grouped(x)
    L.check()
    _, _, tol = block_ref(x, L.w, 2)
    assert ((yd.double() - yg.double()).abs() <= tol + HALF * yd.double().abs()).all()
    yo, y64 = O.forward_dense(x.cpu(), W, 2)[:2]
    assert np.abs(yg.double().cpu().numpy() - y64).max() <= float(tol.max())


def test_block_ties_go_to_the_lower_expert():
    # equal router rows: equal logits; zero tokens: every logit zero
    W = synth.layer_weights(synth.TINY, seed=10)
    W["w_router"][5] = W["w_router"][2]
    W["w_router"][7] = W["w_router"][2]
    L = M.Layer(W, top_e=2)
    x = synth.tokens(256, 100, seed=11).cuda()
    x[3] = 0
    ids = torch.empty((100, 2), dtype=torch.int32, device="cuda")
    y = L.forward_grouped(x, ids=ids)
    ref, rid, tol = block_ref(x, L.w, 2)
    assert ids[3].tolist() == [0, 1]
    assert torch.equal(ids.long(), rid)
    close(y, ref, tol)


def test_block_near_ties_are_decided_in_64_bits():
    # two router rows that differ in one bf16 step of one weight: logits closer than fp32 sums resolve
    W = synth.layer_weights(synth.BlockShape(16, 16, 2048, 3), seed=12, device="cuda")
    r = W["w_router"]
    r[9], r[1] = r[4], r[4]
    r[9, 100] = r[4, 100] + 2.0 ** -14
    r[1, 900] = r[4, 900] - 2.0 ** -14
    L = M.Layer(W, top_e=3)
    x = synth.tokens(2048, 2000, seed=13).cuda()
    x[:, 100] = (torch.randn(2000, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 1e-3).bfloat16()
    x[:, 900] = (torch.randn(2000, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) * 1e-3).bfloat16()
    ids = torch.empty((2000, 3), dtype=torch.int32, device="cuda")
    L.forward_grouped(x, ids=ids)
    L.check()
    _, rid, _ = block_ref(x, W, 3)
    assert torch.equal(ids.long(), rid)


def test_block_residual_in_place_and_repeatable():
    W = synth.layer_weights(synth.TINY, seed=14)
    L = M.Layer(W, top_e=2)
    x, res = synth.tokens(256, 333, seed=15).cuda(), dev(333, 256, seed=16)
    y = L.forward_grouped(x, res)
    z = res.clone()
    L.forward_grouped(x, z, out=z)
    assert torch.equal(y, z)
    assert torch.equal(y, L.forward_grouped(x, res))


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -20, 1.0, 2.0 ** 40, 2.0 ** 100])
def test_block_outputs_of_any_size(scale):
    # the pairs' outputs are held in 16 bits under a common exponent of 32 channels: no value over-
    # or underflows, and a channel far below its neighbours keeps its bits
    W = synth.layer_weights(synth.TINY, seed=26)
    W["w_down"] = (W["w_down"].float() * scale).bfloat16()
    W["w_down"][:, :, 5::32] *= 2.0 ** -20
    L = M.Layer(W, top_e=2)
    for B in (9, 700):
        x = synth.tokens(256, B, seed=27).cuda()
        y = L.forward_grouped(x)
        L.check()
        ref, _, tol = block_ref(x, L.w, 2)
        close(y, ref, tol)


def test_block_nan_token_stays_apart():
    W = synth.layer_weights(synth.TINY, seed=17)
    L = M.Layer(W, top_e=2)
    x = synth.tokens(256, 50, seed=18).cuda()
    y = L.forward_grouped(x)
    x2 = x.clone()
    x2[9] = float("nan")
    z = L.forward_grouped(x2)
    L.check()
    keep = [i for i in range(50) if i != 9]
    assert torch.equal(y[keep], z[keep])
    assert not bool(torch.isfinite(z[9]).any())
    # the experts of such a token are still experts, each once (few tokens and many)
    for B in (20, 50):
        x2[3] = float("inf")
        ids = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
        L.forward_grouped(x2[:B], ids=ids)
        L.check()
        assert ((ids >= 0) & (ids < 8)).all() and (ids[:, 0] != ids[:, 1]).all()


# ------------------------------------------------------------- bad plans
def product_call(off, P=64, x_rows=None, y_rows=None, n_x=64, n_y=64, G=3):
    x, w = dev(n_x, 64, seed=40), dev(G, 128, 64, seed=41)
    y = torch.full((n_y, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_grouped_workspace_bytes(G, P))
    t = [None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda") for v in (off, x_rows, y_rows)]
    M.moe_reader_grouped_product(G, P, n_x, n_y, 128, 64, 0, x, t[1], 1, t[0], w, y, t[2], ws, ws.numel())
    return y, ws


@pytest.mark.parametrize("off", [[0, 10, 5, 64], [0, 10, 20, 65], [-1, 10, 20, 64], [0, 10, 20, 2 ** 31 - 1],
                                 [0, -2 ** 31, 2 ** 31 - 1, 64]])
def test_bad_offsets_are_reported(off):
    y, ws = product_call(off)
    with pytest.raises(M.MoeError, match="MOE_EDEVICE"):
        M.moe_reader_check_error(ws)
    M.moe_reader_check_error(ws)  # cleared


@pytest.mark.parametrize("bad", [-1, 64, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("which", ["x_rows", "y_rows"])
def test_bad_rows_are_reported(bad, which):
    good = list(range(64))
    good[17] = bad
    y, ws = product_call([0, 10, 30, 64], **{which: good})
    with pytest.raises(M.MoeError, match="MOE_EDEVICE"):
        M.moe_reader_check_error(ws)
    ok, ws2 = product_call([0, 10, 30, 64])
    M.moe_reader_check_error(ws2)
    keep = [i for i in range(64) if i != 17]
    assert torch.equal(y[keep], ok[keep])
    if which == "y_rows":
        assert (y[17] == 5.0).all()


def test_bad_adapter_rows_are_reported():
    T, A, K, N, r = 20, 2, 64, 64, 8
    off = torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda")
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    rows[3] = T
    ws = ws_for(M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))
    y = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    M.moe_reader_adapter_product(T, A, N, K, r, dev(T, K, seed=1), None, None, off, rows, dev(A, r, K, seed=2),
                                 dev(A, N, r, seed=3), None, y, ws, ws.numel())
    with pytest.raises(M.MoeError, match="MOE_EDEVICE"):
        M.moe_reader_check_error(ws)


def test_strided_tensors_are_refused_by_the_binding():
    ids = torch.zeros(128, dtype=torch.int32, device="cuda")
    off, rows = torch.zeros(9, dtype=torch.int32, device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda")
    ws = ws_for(M.moe_reader_group_workspace_bytes(64, 8))
    for bad in (ids[::2], ids[:1].expand(64)):
        with pytest.raises(M.MoeError, match="MOE_EINVAL.*contiguous"):
            M.moe_reader_group_rows(64, 8, bad, off, rows, ws, ws.numel())


# ------------------------------------------- streams, graphs, used together
def test_captured_block_replays_on_new_inputs():
    W = synth.layer_weights(synth.TINY, seed=20)
    L = M.Layer(W, top_e=2)
    x = synth.tokens(256, 120, seed=21).cuda()
    y = torch.empty_like(x)
    L.forward_grouped(x, out=y)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        L.forward_grouped(x, out=y)
    for seed in (22, 23):
        x.copy_(synth.tokens(256, 120, seed=seed))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, L.forward_grouped(x))
        ref, _, tol = block_ref(x, L.w, 2)
        close(got, ref, tol)
    L.check()


@pytest.mark.parametrize("T", [3, 90, 900])
def test_captured_plan_and_adapters_replay_on_new_inputs(T):
    """Ids, plan and adapters in one graph: each replay uses the ids and tokens
    that the graph's own first kernels put there."""
    A, K, N, r = 6, 256, 520, 24
    x, w, base = dev(T, K, seed=80), dev(N, K, seed=81, scale=K ** -0.5), dev(T, N, seed=82)
    a, b = dev(A, r, K, seed=83, scale=K ** -0.5), dev(A, N, r, seed=84)
    new_x, new_ids = x.clone(), ids_of(T, A, "random")
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    off, rows = torch.zeros(A + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))

    def step():
        ids.copy_(new_ids)
        x.copy_(new_x)
        M.moe_reader_group_rows(T, A, ids, off, rows, ws, ws.numel())
        M.moe_reader_adapter_product(T, A, N, K, r, x, w, base, off, rows, a, b, None, y, ws, ws.numel())

    step()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for k in range(4):
        new_ids.copy_(ids_of(T, A, ("random", "none", "runs", "all")[k], seed=k))
        new_x.copy_(dev(T, K, seed=90 + k))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y)
        xd, idc = new_x.double(), new_ids
        ref = xd @ w.double().T + base.double()
        err = sum_err(K) * (xd.abs() @ w.double().abs().T)
        for q in range(A):
            t = (idc == q).nonzero().flatten()
            z = xd[t] @ a[q].double().T
            mag = xd[t].abs() @ a[q].double().abs().T
            ref[t] += z @ b[q].double().T
            err[t] += (sum_err(K) * mag + 2.0 ** -15 * z.abs()) @ b[q].double().abs().T
        close(got, ref, HALF * ref.abs() + SLACK * err + 2.0 ** -20 * (ref.abs() + base.double().abs()))
    M.moe_reader_check_error(ws)


def test_one_workspace_serves_every_entry_point_in_turn():
    """The counters that split sums use sit at one place for all: a workspace
    goes from one entry point and size to the next."""
    T, A, K, N, r, E = 70, 4, 2048, 512, 16, 4
    big = max(M.moe_reader_block_workspace_bytes(300, 8, 2, 128, 256), M.moe_reader_grouped_workspace_bytes(E, 600),
              M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))
    shared = ws_for(big)
    W = {k: v.cuda() if v is not None else None for k, v in synth.layer_weights(synth.TINY, seed=28).items()}
    st = M.Layer(W, top_e=2).struct(0)
    x, w, xb = dev(600, K, seed=85), dev(E, N, K, seed=86), synth.tokens(256, 300, seed=29).cuda()
    a, b = dev(A, r, K, seed=87, scale=K ** -0.5), dev(A, N, r, seed=88)
    off1, rows1, _ = plan_of([3, 0, 40, 27], 1)

    def run(ws_of):
        outs = []
        for n in (5, 300, 40):  # few tokens and many, so that sums are split and not
            y = torch.empty((n, 256), dtype=torch.bfloat16, device="cuda")
            M.moe_reader_forward_grouped(st, n, xb, None, y, None, ws_of(), big)
            outs.append(y)
            p = torch.empty((70, N), dtype=torch.bfloat16, device="cuda")
            M.moe_reader_grouped_product(E, 70, 600, 70, N, K, 0, x, None, 1, off1, w, p, None, ws_of(), big)
            outs.append(p)
            z = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
            M.moe_reader_adapter_product(T, A, N, K, r, x, w[0], None, off1, rows1, a, b, None, z, ws_of(), big)
            outs.append(z)
        return outs

    for u, v in zip(run(lambda: shared), run(lambda: ws_for(big))):
        assert torch.equal(u, v)
    M.moe_reader_check_error(shared)


def test_two_streams_with_their_own_workspaces():
    W = synth.layer_weights(synth.BlockShape(16, 256, 1024, 4), seed=24, device="cuda")
    layers = [M.Layer(W, top_e=4) for _ in range(2)]
    xs = [synth.tokens(1024, 500 + 33 * i, seed=25 + i).cuda() for i in range(2)]
    want = [layers[i].forward_grouped(xs[i]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(x) for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            layers[i].forward_grouped(xs[i], out=outs[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i])
        layers[i].check()


def test_a_model_step_prompt_then_decode():
    """Prompts of four requests through two layers (norm, adapted projection,
    grouped block), then one decode token each through the reader with the
    same adapters beside the block; against the same chain in 64 bits from
    each stage's own inputs."""
    d, E, I, top, r, A = 256, 8, 128, 2, 16, 3
    lens, owner = [40, 1, 130, 75], [2, -1, 0, 2]
    T = sum(lens)
    ids = torch.tensor(np.repeat(owner, lens).astype(np.int32)).cuda()
    layers = [M.Layer(synth.layer_weights(synth.TINY, seed=30 + i), top_e=top) for i in range(2)]
    for i, L in enumerate(layers):
        L.build_sketch(synth.rot_seed(i)).build_lowrank(8)
    proj = [dev(d, d, seed=50 + i, scale=d ** -0.5) for i in range(2)]
    a, b = dev(A, r, d, seed=60, scale=d ** -0.5), dev(A, d, r, seed=61, scale=0.3)
    scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")

    def plan(ids):
        n = ids.numel()
        off, rows = torch.empty(A + 1, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
        ws = ws_for(M.moe_reader_group_workspace_bytes(n, A))
        M.moe_reader_group_rows(n, A, ids, off, rows, ws, ws.numel())
        return off, rows

    def adapted(x, w, base, off, rows):
        n = x.shape[0]
        ws = ws_for(M.moe_reader_adapter_workspace_bytes(n, A, d, d, r))
        y = torch.empty_like(x)
        M.moe_reader_adapter_product(n, A, d, d, r, x, w, base, off, rows, a, b, scale, y, ws, ws.numel())
        M.moe_reader_check_error(ws)
        return y

    def adapted_ref(x, w, base, ids):
        x = x.double()
        y = torch.zeros_like(x) if w is None else x @ w.double().T
        e = torch.zeros_like(x) if w is None else sum_err(d) * (x.abs() @ w.double().abs().T)
        if base is not None:
            y = y + base.double()
        for g in range(A):
            t = (ids == g).nonzero().flatten()
            z = float(scale[g]) * (x[t] @ a[g].double().T)
            mag = float(scale[g]) * (x[t].abs() @ a[g].double().abs().T)
            y[t] += z @ b[g].double().T
            e[t] += (sum_err(d) * mag + 2.0 ** -15 * z.abs()) @ b[g].double().abs().T
        return y, HALF * y.abs() + SLACK * e + 2.0 ** -20 * y.abs()

    off, rows = plan(ids)
    h = synth.tokens(d, T, seed=70).cuda()
    n = torch.empty_like(h)
    for i, L in enumerate(layers):
        M.moe_reader_rmsnorm(T, d, 1e-6, h, n)
        p = adapted(n, proj[i], h, off, rows)
        close(p, *adapted_ref(n, proj[i], h, ids))
        M.moe_reader_rmsnorm(T, d, 1e-6, p, n)
        h = L.forward_grouped(n, p)
        ref, _, tol = block_ref(n, L.w, top, p)
        close(h, ref, tol)
        L.check()
    # decode: the last token of each request, its adapter beside the reader's block
    last = h[torch.tensor(np.cumsum(lens) - 1).cuda()].contiguous()
    did = torch.tensor(owner, dtype=torch.int32).cuda()
    off, rows = plan(did)
    m = torch.empty_like(last)
    M.moe_reader_rmsnorm(4, d, 1e-6, last, m)
    y = layers[0].forward(m, k=24, c=48, residual=last)
    layers[0].check()
    z = adapted(m, None, y, off, rows)
    close(z, *adapted_ref(m, None, y, did))
