"""The products over ragged groups where values or calls are out of the
ordinary: ranges, non-finite weights, streams and captures, both sides of the
borders between kernels.  Tolerances as in test_gpu_grouped.py."""
import threading

import pytest
import torch

from calibration_free_channel_b200 import moe_reader as M
from calibration_free_channel_b200 import synth
from tests.test_gpu_grouped import HALF, SLACK, block_ref, close, dev, plan_of, swiglu_ref, sum_err, ws_for

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
@pytest.mark.parametrize("r", [24, 64])
@pytest.mark.parametrize("bad", ["a nan", "a inf", "scale"])
def test_adapters_down_side_nonfinite_stays_apart(T, A, r, bad):
    """Weights of A or a scale that are not finite reach the adapter's own tokens only."""
    K, N = 256, 264
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


def adapter_ref(t, ids, N):
    """The definition in 64 bits and what fp32 sums and two bf16 terms of z may differ by."""
    x = t["x"].double()
    K, r = t["a"].shape[2], t["a"].shape[1]
    ref = torch.zeros((x.shape[0], N), dtype=torch.float64, device="cuda")
    err = torch.zeros_like(ref)
    if t["base"] is not None:
        ref += t["base"].double()
        err += 2.0 ** -24 * t["base"].double().abs()
    if t["w"] is not None:
        ref += x @ t["w"].double().T
        err += sum_err(K) * (x.abs() @ t["w"].double().abs().T)
    for g in range(t["a"].shape[0]):
        q = (ids == g).nonzero().flatten()
        if q.numel() == 0:
            continue
        s = 1.0 if t["scale"] is None else float(t["scale"][g])
        z, b = s * (x[q] @ t["a"][g].double().T), t["b"][g].double()
        ez = abs(s) * sum_err(K) * (x[q].abs() @ t["a"][g].double().abs().T) + (2.0 ** -16 + 2.0 ** -22) * z.abs()
        ref[q] += z @ b.T
        err[q] += ez @ b.abs().T + sum_err(2 * r + 8) * (z.abs() @ b.abs().T)
    # the terms meet in one fp32 accumulator: a few roundings of the running value
    return ref, HALF * ref.abs() + SLACK * (err + 2.0 ** -20 * ref.abs()) + 1e-30


@pytest.mark.parametrize("T,A", [(2, 2), (3, 2), (64, 32), (90, 5), (700, 40), (2100, 5), (2300, 60)])
@pytest.mark.parametrize("r", [24, 64])
@pytest.mark.parametrize("use_w,use_base,inplace", [(True, False, False), (False, True, True), (True, True, False)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_adapters_up_side_nonfinite_stays_apart(T, A, r, use_w, use_base, inplace, bad):
    """Weights of B that are not finite reach the adapter's own tokens only, in the channels that have them."""
    K, N = 264, 520
    y, ids, t = adapter_call(T, A, K, N, r, use_w=use_w, use_base=use_base)
    b = t["b"].clone()
    b[1, 0, 3] = b[1, 77, 0] = b[1, 78, 23] = b[1, 519, 8] = bad
    b[1, 256:300] = -bad
    z, _, _ = adapter_call(T, A, K, N, r, use_w=use_w, use_base=use_base, inplace=inplace, b=b)
    mine = ids == 1
    spoilt = ~torch.isfinite(b[1].float()).all(1)
    close(z[~mine], *(v[~mine] for v in adapter_ref(t, ids, N)))
    assert torch.equal(z[:, ~spoilt], y[:, ~spoilt])
    assert not bool(torch.isfinite(z[mine][:, spoilt]).any())
    # and the same bits again
    again, _, _ = adapter_call(T, A, K, N, r, use_w=use_w, use_base=use_base, inplace=inplace, b=b)
    assert torch.equal(z.view(torch.int16), again.view(torch.int16))


def test_adapters_of_one_batch_all_but_one_nonfinite():
    """Every block of 32 positions is met by adapters that are not finite in any weight, and a token by NaN of its own."""
    T, A, K, N, r = 400, 7, 136, 264, 16
    y, ids, t = adapter_call(T, A, K, N, r)
    b, x = t["b"].clone(), t["x"].clone()
    b[[0, 1, 3, 4, 5, 6]] = float("nan")
    free = (ids == 2) | (ids == -1)
    own = int(free.nonzero()[0])
    x[own, 130] = float("nan")
    z, _, _ = adapter_call(T, A, K, N, r, b=b, x=x)
    free[own] = False
    close(z[free], *(v[free] for v in adapter_ref(t, ids, N)))
    assert not bool(torch.isfinite(z[~free]).any())


@pytest.mark.parametrize("T,use_w", [(3, True), (64, True), (64, False)])
def test_adapters_nonfinite_where_sums_are_split(T, use_w):
    # few tiles over a long K: the parts of a sum, and of the adapters, meet
    A, K, N, r = 3, 2048, 512, 72
    y, ids, t = adapter_call(T, A, K, N, r, use_w=use_w, seed=7)
    b = t["b"].clone()
    b[1] = float("inf")
    z, _, _ = adapter_call(T, A, K, N, r, use_w=use_w, seed=7, b=b)
    mine = ids == 1
    close(z[~mine], *(v[~mine] for v in adapter_ref(t, ids, N)))
    assert not bool(torch.isfinite(z[mine]).any())


def test_adapters_infinite_results_stay():
    """Infinities that the definition has: a token's, a projection's, and both meeting."""
    T, A, K, N, r = 50, 3, 64, 64, 8
    y, ids, t = adapter_call(T, A, K, N, r)
    w, b = t["w"].clone(), t["b"].clone()
    w[5] = 0
    w[5, 3] = float("inf")
    b[0, 5] = 0
    b[0, 5, 2] = float("inf")
    b[1] = float("nan")
    z, _, _ = adapter_call(T, A, K, N, r, b=b, w=w)
    x, a, s = t["x"].double(), t["a"].double(), t["scale"]
    for q in range(T):
        g = int(ids[q])
        if g == 1:
            assert torch.isnan(z[q]).all()
            continue
        want = x[q, 3] * float("inf")
        if g == 0:
            want = want + (float(s[0]) * (a[0, 2] @ x[q])) * float("inf")
        got = z[q, 5].double()
        assert bool(torch.isnan(got)) if bool(torch.isnan(want)) else bool(got == want), (q, g, got, want)


# ------------------------------------------------ values held in two bf16 terms
# Between the largest bf16 and 2^128 a value rounds to infinity, but its two
# terms hold it.
@pytest.mark.parametrize("T", [5, 100, 2100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_adapters_two_terms_below_overflow(T, sign):
    K, N, r = 64, 64, 64
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    a = torch.zeros((1, r, K), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = sign * 255 * 2.0 ** 57, sign * 1.5 * 2.0 ** 60
    a[0, :, 0], a[0, :, 1] = 2.0 ** 63, 2.0 ** 59  # z = 0x1.ffp127 and half a step of 2^119 more
    b = torch.zeros((1, N, r), dtype=torch.bfloat16, device="cuda")
    b[0, :, 3] = 2.0 ** -100
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    y, _, t = adapter_call(T, 1, K, N, r, use_w=False, use_base=False, ids=ids, x=x, a=a, b=b, scale=None)
    close(y, *adapter_ref(t, ids, N))


def one_expert(d=256, I=16, E=1):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    return dict(w_router=z(E, d), router_bias=None, w_gate=z(E, I, d), w_up=z(E, I, d), w_down=z(E, I, d))


@pytest.mark.parametrize("B", [1, 40, 64])
def test_block_two_terms_below_overflow(B):
    W = one_expert()
    x = torch.zeros((B, 256), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = 1.96875 * 2.0 ** 63, 2.0 ** 64, 1.875 * 2.0 ** 57
    W["w_gate"][0, 3, 0] = W["w_up"][0, 3, 1] = W["w_up"][0, 3, 2] = 1.0  # silu(g) u = 1.9976 2^127
    W["w_down"][0, 3] = 2.0 ** -110
    L = M.Layer(W, top_e=1)
    y = L.forward_grouped(x)
    L.check()
    a = 1.96875 * 2.0 ** 63 * (2.0 ** 64 + 1.875 * 2.0 ** 57)
    ref = torch.full((B, 256), a * 2.0 ** -110, dtype=torch.float64, device="cuda")
    close(y, ref, (HALF + 2.0 ** -15) * ref)


@pytest.mark.parametrize("B", [3, 60, 200])
def test_block_infinite_down_weights_keep_their_sign(B):
    # two terms (few tokens an expert) or one: a x inf is an infinity of a's sign
    E, I, d = 2, 16, 256
    W = dict(one_expert(E=E), w_gate=dev(E, I, d, seed=3), w_up=dev(E, I, d, seed=4), w_down=dev(E, I, d, seed=5))
    W["w_down"][:, 7, 9] = float("inf")
    W["w_down"][:, 2, 11] = -float("inf")
    x = dev(B, d, seed=6, scale=0.1)
    L = M.Layer(W, top_e=1)
    y = L.forward_grouped(x).double()
    L.check()
    # zero router rows: expert 0 for every token
    g, u = x.double() @ W["w_gate"][0].double().T, x.double() @ W["w_up"][0].double().T
    s = torch.sign(g) * torch.sign(u)
    inf = torch.full((B,), float("inf"), dtype=torch.float64, device="cuda")
    assert torch.equal(y[:, 9], s[:, 7] * inf) and torch.equal(y[:, 11], -s[:, 2] * inf)
    assert torch.isfinite(y[:, 12:]).all()


# ---------------------------------------------------------- calls and shapes
def test_block_refuses_other_shapes_and_types():
    L = M.Layer(one_expert(E=3), top_e=2)
    x = dev(40, 256, seed=1)
    ids = torch.zeros((40, 2), dtype=torch.int32, device="cuda")
    y = L.forward_grouped(x, x, ids)
    wrong = [dict(x=x[:, :128].contiguous()), dict(x=x.view(80, 128)), dict(x=x.view(1, 40, 256)), dict(x=x.float()),
             dict(x=x.half()), dict(x=x.t()), dict(residual=x[:39]), dict(residual=x.float()), dict(out=y[:39]),
             dict(out=torch.empty(40, 256, device="cuda")), dict(ids=ids.long()), dict(ids=ids[:39]),
             dict(ids=ids[:, :1].contiguous()), dict(x=x.cpu())]
    for kw in wrong:
        with pytest.raises(M.MoeError, match="MOE_EINVAL"):
            L.forward_grouped(**dict(dict(x=x), **kw))
    L.check()
    assert torch.equal(y, L.forward_grouped(x.view(torch.int16), x.view(torch.int16)).view(torch.bfloat16))


def test_plan_refuses_64_bit_ids():
    ids = torch.randint(0, 8, (64,), device="cuda")
    off, rows = torch.zeros(9, dtype=torch.int32, device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda")
    ws = ws_for(M.moe_reader_group_workspace_bytes(64, 8))
    with pytest.raises(M.MoeError, match="MOE_EINVAL.*int64"):
        M.moe_reader_group_rows(64, 8, ids, off, rows, ws, ws.numel())
    M.moe_reader_group_rows(64, 8, ids.int(), off, rows, ws, ws.numel())
    assert torch.equal(rows.long(), torch.sort(ids, stable=True).indices)


# ------------------------------------------------- streams, growth, captures
SHAPE = synth.BlockShape(16, 256, 1024, 4)


def small_layer(seed=24):
    return M.Layer(synth.layer_weights(SHAPE, seed=seed, device="cuda"), top_e=4)


def tokens_of(*lengths):
    return [synth.tokens(1024, n, seed=40 + i).cuda() for i, n in enumerate(lengths)]


def leave_bytes(nb, *streams):
    """Memory that the allocator hands out next on these streams (and the current one) is full of ones."""
    for s in (torch.cuda.current_stream(), *streams):
        with torch.cuda.stream(s):
            junk = [torch.full((nb,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
            del junk
    torch.cuda.synchronize()


def keep_busy():
    torch.cuda._sleep(20_000_000)  # about 10 ms on the current stream


def test_block_on_a_side_stream_first_and_longer():
    """Workspace and output are made in the order of the stream that the call runs on, whatever the current one does."""
    xs = tokens_of(40, 33, 300, 900)
    L = small_layer()
    want = [L.forward_grouped(x) for x in xs]
    L.check()
    side = small_layer()
    s = torch.cuda.Stream()
    leave_bytes(M.moe_reader_block_workspace_bytes(900, SHAPE.E, 4, SHAPE.I, SHAPE.d), s)
    for x, w in zip(xs, want):
        torch.cuda.synchronize()
        keep_busy()
        y = side.forward_grouped(x, stream=s)
        s.synchronize()
        assert torch.equal(y, w)
        y = side.forward_grouped(x, stream=s.cuda_stream)  # a raw handle
        s.synchronize()
        assert torch.equal(y, w)
    side.check()


def test_block_of_one_layer_on_two_streams():
    xs = tokens_of(500, 37, 260)
    L = small_layer()
    want = [L.forward_grouped(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        outs = [L.forward_grouped(x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for y, w in zip(outs, want):
            assert torch.equal(y, w)
    L.check()


def test_block_inputs_may_be_dropped_behind_a_side_stream_call():
    x, = tokens_of(700)
    L = small_layer()
    want = L.forward_grouped(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        t = x.clone()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            keep_busy()
        outs.append(L.forward_grouped(t, stream=s))
        del t
        torch.full((700, 1024), float("nan"), dtype=torch.bfloat16, device="cuda")  # where t was, if it may be
    torch.cuda.synchronize()
    for y in outs:
        assert torch.equal(y, want)


def test_captured_block_outlives_longer_prompts():
    """A graph keeps its workspace: longer calls, other calls at the same time and freed memory leave it alone."""
    x, longer = tokens_of(120, 1500)
    L = small_layer()
    want, want2 = L.forward_grouped(x), None
    y = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward_grouped(x, out=y)
    want2 = L.forward_grouped(longer)
    torch.cuda.synchronize()
    leave_bytes(M.moe_reader_block_workspace_bytes(120, SHAPE.E, 4, SHAPE.I, SHAPE.d))
    s = torch.cuda.Stream()
    for _ in range(3):
        y.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        z = L.forward_grouped(x)  # beside the replay
        z2 = L.forward_grouped(longer)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want) and torch.equal(z2, want2)
    L.check()


def test_captured_block_without_a_call_before():
    x, = tokens_of(50)
    L = small_layer()
    leave_bytes(M.moe_reader_block_workspace_bytes(50, SHAPE.E, 4, SHAPE.I, SHAPE.d))
    ys = [torch.empty_like(x) for _ in range(3)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        L.forward_grouped(x, out=ys[0])
        L.forward_grouped(x, out=ys[1])
    with torch.cuda.graph(graphs[1]):  # while the first has never run
        L.forward_grouped(x, out=ys[2])
    want = L.forward_grouped(x)  # and an eager call before either
    torch.cuda.synchronize()
    ref, _, tol = block_ref(x, L.w, 4)
    close(want, ref, tol)
    for g in (graphs[1], graphs[0], graphs[1]):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)
    L.check()


def test_layers_share_a_workspace_that_is_passed():
    xs = tokens_of(40, 800)
    layers = [small_layer(seed) for seed in (24, 25)]
    want = [[L.forward_grouped(x) for x in xs] for L in layers]
    fresh = [small_layer(seed) for seed in (24, 25)]
    ws = fresh[0].block_workspace(800)
    for _ in range(2):
        for i, x in enumerate(xs):
            for L, w in zip(fresh, want):
                assert torch.equal(L.forward_grouped(x, workspace=ws), w[i])
    M.moe_reader_check_error(ws)
    assert not fresh[0]._wsg and not fresh[1]._wsg
    with pytest.raises(M.MoeError, match="MOE_EINVAL.*workspace"):
        fresh[0].forward_grouped(xs[1], workspace=fresh[0].block_workspace(40))
    with pytest.raises(M.MoeError, match="MOE_EINVAL"):
        fresh[0].block_workspace(32769)


def test_block_errors_survive_a_longer_call():
    xs = tokens_of(40, 800)
    L = small_layer()
    L.forward_grouped(xs[0])
    (ws,) = L._wsg.values()
    ws[:4].view(torch.int32)[0] = 8  # as a bad plan records it
    L.forward_grouped(xs[1])
    with pytest.raises(M.MoeError, match="MOE_EDEVICE"):
        L.check()
    L.check()


def test_decode_on_a_side_stream_first_and_longer():
    L = M.Layer(synth.layer_weights(synth.TINY, seed=31), top_e=2)
    L.build_sketch(synth.rot_seed(0)).build_lowrank(8)
    xs = [synth.tokens(256, n, seed=n).cuda() for n in (1, 2, 5, 40)]
    want = [(L.forward(x, k=24, c=48), L.forward_dense(x)) for x in xs]
    L.check()
    L._ws = None
    s = torch.cuda.Stream()
    leave_bytes(M.moe_reader_workspace_bytes(40, 8, 2, 128, 256, 1, 1, 8), s)
    for x, (w, wd) in zip(xs, want):
        torch.cuda.synchronize()
        keep_busy()
        y, yd = L.forward(x, k=24, c=48, stream=s), L.forward_dense(x, stream=s)
        s.synchronize()
        assert torch.equal(y, w) and torch.equal(yd, wd)
    L.check()


# ------------------------------------------------------------------- routing
def chosen(L, x, top, **kw):
    ids = torch.full((x.shape[0], top), -1, dtype=torch.int32, device="cuda")
    L.forward_grouped(x, ids=ids)
    L.check()
    logits = x.double() @ L.w["w_router"].double().T
    if L.w["router_bias"] is not None:
        logits = logits + L.w["router_bias"].double()
    return ids.long(), torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top]


@pytest.mark.parametrize("E", [16, 40])
@pytest.mark.parametrize("scale", [2.0 ** -125, 2.0 ** -100, 2.0 ** -70, 2.0 ** -20, 2.0 ** 30, 2.0 ** 90, 2.0 ** 121])
def test_block_near_ties_of_tokens_of_any_size(scale, E):
    """Router rows a bf16 step of one weight apart, and tokens whose squares
    (or products) leave the range of fp32: the order is still that of 64 bits."""
    W = synth.layer_weights(synth.BlockShape(E, 16, 2048, 3), seed=12, device="cuda")
    r = W["w_router"]
    r[9], r[1] = r[4], r[4]
    r[9, 100] = r[4, 100] + 2.0 ** -14
    r[1, 900] = r[4, 900] - 2.0 ** -14
    L = M.Layer(W, top_e=3)
    x = synth.tokens(2048, 1500, seed=13).cuda()
    x[:, 100] = dev(1500, seed=1, scale=1e-3)
    x[:, 900] = dev(1500, seed=2, scale=1e-3)
    x[7] = 0
    got, want = chosen(L, (x.float() * scale).bfloat16(), 3)
    assert torch.equal(got, want)


@pytest.mark.parametrize("B", [10, 100])
def test_block_products_below_fp32_decide(B):
    W = one_expert(E=8)
    W["w_router"][:, 5] = torch.arange(1, 9).cuda() * 2.0 ** -78
    L = M.Layer(W, top_e=2)
    x = torch.zeros((B, 256), dtype=torch.bfloat16, device="cuda")
    x[:, 5] = 2.0 ** -80
    x[3::5, 5] = -2.0 ** -80
    got, want = chosen(L, x, 2)
    assert torch.equal(got, want)


@pytest.mark.parametrize("E", [16, 40])
@pytest.mark.parametrize("mask", [float("-inf"), -3.38e38])
def test_block_masked_experts(E, mask):
    """A bias that takes experts out: none of them is chosen while others are left, and the rest keeps its order."""
    W = synth.layer_weights(synth.BlockShape(E, 16, 256, 3), seed=14, bias=True, device="cuda")
    W["router_bias"][::2] = mask
    L = M.Layer(W, top_e=3)
    x = synth.tokens(256, 200, seed=15).cuda()
    got, want = chosen(L, x, 3)
    assert torch.equal(got, want) and bool((got % 2 == 1).all())
    W["router_bias"][3:] = mask  # one expert left
    got, want = chosen(M.Layer(W, top_e=3), x, 3)
    assert torch.equal(got, want) and bool((got[:, 0] == 1).all())


# ------------------------------------------------------------------- threads
def test_plans_of_several_threads():
    """Calls of very different table sizes at once, a stream each: a launch never finds its shared memory taken back."""
    sizes = [(65536, 1024), (20000, 400), (3000, 1000), (40000, 700)]
    found = []

    def run(n, G, seed):
        try:
            ids = torch.randint(-1, G, (n,), generator=torch.Generator("cuda").manual_seed(seed), device="cuda",
                                dtype=torch.int32)
            key = torch.where(ids < 0, G, ids)
            want = torch.sort(key, stable=True).indices.int()
            off, rows = torch.empty(G + 1, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
            ws = ws_for(M.moe_reader_group_workspace_bytes(n, G))
            s = torch.cuda.Stream()
            torch.cuda.synchronize()
            for _ in range(400):
                M.moe_reader_group_rows(n, G, ids, off, rows, ws, ws.numel(), stream=s)
            s.synchronize()
            if not torch.equal(rows, want):
                found.append((n, G, "rows"))
        except Exception as e:  # noqa: BLE001 (shown below)
            found.append((n, G, e))

    threads = [threading.Thread(target=run, args=(n, G, i)) for i, (n, G) in enumerate(sizes)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not found, found


# ------------------------------------------- SwiGLU values between the products
def held_ref(x, w, top, held):
    """The block in 64 bits, and its tolerance with SwiGLU values that are off by `held` of themselves."""
    y, ids, _ = block_ref(x, w, top)
    xd, err = x.double(), torch.zeros_like(y)
    logits = xd @ w["w_router"].double().T
    if w["router_bias"] is not None:
        logits = logits + w["router_bias"].double()
    share = torch.softmax(torch.sort(logits, dim=1, descending=True, stable=True).values[:, :top], 1)
    for e in range(logits.shape[1]):
        t, k = (ids == e).nonzero(as_tuple=True)
        a, ea = swiglu_ref(xd[t], w["w_gate"][e], w["w_up"][e])
        wd = w["w_down"][e].double().abs()
        err[t] += share[t, k][:, None] * ((ea + (held + sum_err(2 * a.shape[1] + 16)) * a.abs()) @ wd)
    # the routing weights: logits in fp32 (d 2^-23 of the terms' sizes) and their exponentials
    err += (2 * sum_err(x.shape[1]) * xd.norm(dim=1) * w["w_router"].double().norm(dim=1).max())[:, None] * y.abs()
    return y, ids, HALF * y.abs() + SLACK * (err + 2.0 ** -20 * y.abs())


@pytest.mark.parametrize("E,top,B", [(8, 2, 1), (8, 2, 64), (8, 2, 65), (8, 2, 256), (1, 1, 64), (4, 4, 64), (16, 1, 1024),
                                     (8, 2, 257), (1, 1, 65), (16, 1, 1025)])
def test_block_holds_swiglu_in_two_terms_up_to_its_border(E, top, B):
    """Up to B top_e = 64 E the values keep 16 bits, above that 8."""
    d, I = 256, 128
    W = synth.layer_weights(synth.BlockShape(E, I, d, top), seed=50, device="cuda")
    L = M.Layer(W, top_e=top)
    x = synth.tokens(d, B, seed=51).cuda()
    y = L.forward_grouped(x)
    L.check()
    ref, _, tol = held_ref(x, L.w, top, 2.0 ** -16 if B * top <= 64 * E else HALF)
    close(y, ref, tol)


@pytest.mark.parametrize("E,B", [(1, 1), (1, 40), (1, 64), (4, 65), (4, 200), (4, 256), (40, 2000)])
def test_block_second_term_decides_where_the_first_cancels(E, B):
    """Pairs of channels that differ by 2^-10 of themselves and are subtracted:
    one bf16 term would leave nothing, or four times as much."""
    d, I = 256, 64
    W = one_expert(d, I, E)
    x = torch.zeros((B, d), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0 + torch.arange(B, device="cuda").bfloat16() / 64  # gates
    x[:, 1] = 1.0 + dev(B, seed=52).abs()
    x[:, 2] = x[:, 1] * 2.0 ** -10
    x[:, 3 + torch.arange(E, device="cuda")] = 0.0
    x[torch.arange(B, device="cuda"), 3 + torch.arange(B, device="cuda") % E] = 8.0  # the token's expert
    for e in range(E):
        W["w_router"][e, 3 + e] = 1.0
    W["w_gate"][:, :, 0] = 1.0
    W["w_up"][:, :, 1] = 1.0
    W["w_up"][:, 1::2, 2] = 1.0
    for c in range(I // 2):
        W["w_down"][:, 2 * c, c::32] = -1.0
        W["w_down"][:, 2 * c + 1, c::32] = 1.0
    L = M.Layer(W, top_e=1)
    y = L.forward_grouped(x)
    L.check()
    xd = x.double()
    silu = xd[:, 0] * torch.sigmoid(xd[:, 0])
    ref = (silu * xd[:, 2])[:, None].expand(B, d)
    # two values of 16 bits each, their fp32 arithmetic a few 2^-24
    tol = HALF * ref + 2 * (2.0 ** -16 + 2.0 ** -20) * (silu * xd[:, 1])[:, None]
    close(y, ref, tol)
    assert bool((tol < ref / 4).all())


# ------------------------ adapters on both sides of z's border (2048 tokens, more of rank below 64)
def border(r):
    """Tokens up to, and from, which z of rank r comes from another kernel."""
    most = max(2048, 2048 * 64 // r)
    return [most, most + 1, most + 450]


SIDES = [0, 1, 2]


def adapter_ids(T, A, kind, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda: torch.randint(-1, A, (T,), generator=g, device="cuda", dtype=torch.int32)
    if kind == "runs":
        return rnd().repeat_interleave(37)[:T].contiguous()
    return {"random": rnd, "all": lambda: torch.zeros(T, dtype=torch.int32, device="cuda"),
            "none": lambda: torch.full((T,), -1, dtype=torch.int32, device="cuda"),
            "distinct": lambda: torch.arange(T, device="cuda", dtype=torch.int32) % A,
            "one of many": lambda: torch.where(torch.arange(T, device="cuda") == T // 2, A - 1, -1).int()}[kind]()


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("r", [8, 72, 128])
@pytest.mark.parametrize("K", [8, 200])
def test_adapters_at_the_border_ranks(side, r, K):
    T = border(r)[side]
    for A, kind, w, base, scale in ((3, "random", True, False, {}), (4, "runs", False, True, dict(scale=None))):
        y, ids, t = adapter_call(T, A, K, 136, r, use_w=w, use_base=base, ids=adapter_ids(T, A, kind), **scale)
        close(y, *adapter_ref(t, ids, 136))


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("A,kind", [(1, "all"), (1, "none"), (300, "distinct"), (300, "random"), (1024, "distinct"),
                                    (1024, "one of many"), (40, "runs")])
def test_adapters_at_the_border_counts(side, A, kind):
    T = border(64)[side]
    for w, base in ((True, True), (False, False)):
        y, ids, t = adapter_call(T, A, 136, 264, 64, use_w=w, use_base=base, ids=adapter_ids(T, A, kind))
        close(y, *adapter_ref(t, ids, 264))


@pytest.mark.parametrize("side", SIDES)
def test_adapters_at_the_border_in_place(side):
    T = border(64)[side]
    a, ids, t = adapter_call(T, 7, 256, 520, 64, use_w=False)
    b, _, _ = adapter_call(T, 7, 256, 520, 64, use_w=False, inplace=True)
    assert torch.equal(a, b)
    close(a, *adapter_ref(t, ids, 520))


@pytest.mark.parametrize("side", SIDES)
def test_adapters_at_the_border_nonfinite_tokens(side):
    T = border(72)[side]
    y, ids, t = adapter_call(T, 6, 128, 264, 72)
    x = t["x"].clone()
    x[11], x[T - 1], x[700, 5] = float("nan"), float("inf"), float("nan")
    z, _, _ = adapter_call(T, 6, 128, 264, 72, x=x)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[11, T - 1, 700]] = False
    assert torch.equal(z[keep], y[keep])
    assert not bool(torch.isfinite(z[[11, 700]]).any())


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("where", [0, 700, -1])
@pytest.mark.parametrize("bad", [-1, "T", 2 ** 31 - 1, -2 ** 31])
def test_adapters_at_the_border_bad_rows(side, where, bad):
    A, K, N, r = 4, 64, 72, 64
    T = border(r)[side]
    y, ids, t = adapter_call(T, A, K, N, r)
    off, rows = torch.empty(A + 1, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    ws = ws_for(M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))
    M.moe_reader_group_rows(T, A, ids, off, rows, ws, ws.numel())
    lost = int(rows[where])
    rows[where] = T if bad == "T" else bad
    z = torch.full((T, N), 9.0, dtype=torch.bfloat16, device="cuda")
    M.moe_reader_adapter_product(T, A, N, K, r, t["x"], t["w"], t["base"], off, rows, t["a"], t["b"], t["scale"], z, ws,
                                 ws.numel())
    with pytest.raises(M.MoeError, match="MOE_EDEVICE"):
        M.moe_reader_check_error(ws)
    keep = torch.arange(T, device="cuda") != lost
    assert torch.equal(z[keep], y[keep]) and bool((z[lost] == 9.0).all())


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("off", [[0, 5, 4, 20], [-1, 5, 10, 20], [0, 5, 10, 5000], [0, 2 ** 31 - 1, -2 ** 31, 20]])
def test_adapters_at_the_border_bad_offsets(side, off):
    A, K, N, r = 3, 64, 72, 64
    T = border(r)[side]
    off = torch.tensor(off, dtype=torch.int32, device="cuda")
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    ws = ws_for(M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))
    y = torch.full((T + 1, N), 9.0, dtype=torch.bfloat16, device="cuda")
    M.moe_reader_adapter_product(T, A, N, K, r, dev(T, K, seed=1), dev(N, K, seed=2), None, off, rows,
                                 dev(A, r, K, seed=3), dev(A, N, r, seed=4), None, y, ws, ws.numel())
    with pytest.raises(M.MoeError, match="MOE_EDEVICE"):
        M.moe_reader_check_error(ws)
    M.moe_reader_check_error(ws)
    assert bool((y[T] == 9.0).all())


@pytest.mark.parametrize("side", SIDES)
def test_adapters_at_the_border_captured(side):
    A, K, N, r = 6, 264, 520, 64
    T = border(r)[side]
    x, w, base = dev(T, K, seed=80), dev(N, K, seed=81, scale=K ** -0.5), dev(T, N, seed=82)
    a, b = dev(A, r, K, seed=83, scale=K ** -0.5), dev(A, N, r, seed=84)
    ids = adapter_ids(T, A, "random")
    off, rows = torch.zeros(A + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_adapter_workspace_bytes(T, A, K, N, r))

    def step():
        M.moe_reader_group_rows(T, A, ids, off, rows, ws, ws.numel())
        M.moe_reader_adapter_product(T, A, N, K, r, x, w, base, off, rows, a, b, None, y, ws, ws.numel())

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k, kind in enumerate(("random", "none", "runs", "all")):
        ids.copy_(adapter_ids(T, A, kind, seed=k))
        x.copy_(dev(T, K, seed=90 + k))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        assert torch.equal(got, y)
        close(got, *adapter_ref(dict(x=x, w=w, base=base, a=a, b=b, scale=None), ids, N))
    M.moe_reader_check_error(ws)


# ---------------------------------------------------------- the largest sizes
def test_block_of_the_most_tokens():
    """32768 tokens, 16 of 16 experts each: the pairs' fp32 outputs pass 2^31 elements."""
    E, I, d, top, B = 16, 16, 4096, 16, 32768
    W = synth.layer_weights(synth.BlockShape(E, I, d, top), seed=60, device="cuda")
    L = M.Layer(W, top_e=top)
    x = synth.tokens(d, B, seed=61).cuda()
    ids = torch.full((B, top), -1, dtype=torch.int32, device="cuda")
    y = L.forward_grouped(x, ids=ids)
    L.check()
    for part in (slice(0, 40), slice(B // 2, B // 2 + 40), slice(B - 40, B)):
        ref, rid, tol = block_ref(x[part], L.w, top)
        assert torch.equal(ids[part].long(), rid)
        close(y[part], ref, tol)


@pytest.mark.parametrize("E,I,B,top", [(1024, 16, 3, 16), (1024, 16, 64, 4), (300, 24, 64, 1), (129, 16, 40, 2)])
def test_block_of_few_tokens_and_many_experts(E, I, B, top):
    W = synth.layer_weights(synth.BlockShape(E, I, 256, top), seed=62, bias=True, device="cuda")
    L = M.Layer(W, top_e=top)
    x = synth.tokens(256, B, seed=63).cuda()
    ids = torch.full((B, top), -1, dtype=torch.int32, device="cuda")
    y = L.forward_grouped(x, ids=ids)
    L.check()
    ref, rid, tol = block_ref(x, L.w, top)
    assert torch.equal(ids.long(), rid)
    close(y, ref, tol)


@pytest.mark.parametrize("layout", [0, 1])
def test_product_outputs_past_32_bits(layout):
    P, K, N, G = 70000, 16, 32768, 3
    off = torch.tensor([0, 30000, 30001, P], dtype=torch.int32, device="cuda")
    rows = torch.randperm(P, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).int()
    x, w = dev(P, K, seed=64), dev(G, K, N, seed=65) if layout else dev(G, N, K, seed=65)
    y = torch.empty((P, N), dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_grouped_workspace_bytes(G, P))
    M.moe_reader_grouped_product(G, P, P, P, N, K, layout, x, None, 1, off, w, y, rows, ws, ws.numel())
    M.moe_reader_check_error(ws)
    for p in (0, 29999, 30000, 30001, P - 1, int((rows == P - 1).nonzero())):
        wg = w[0 if p < 30000 else 1 if p == 30000 else 2].double()
        wg = wg if layout else wg.T
        ref, mag = x[p].double() @ wg, x[p].double().abs() @ wg.abs()
        close(y[int(rows[p])], ref, HALF * ref.abs() + SLACK * sum_err(K) * mag)


def test_swiglu_outputs_past_32_bits():
    P, d, I = 140000, 8, 16392
    off = torch.tensor([0, 70001, P], dtype=torch.int32, device="cuda")
    x, wg, wu = dev(P, d, seed=66), dev(2, I, d, seed=67), dev(2, I, d, seed=68)
    a = torch.empty((P, I), dtype=torch.bfloat16, device="cuda")
    ws = ws_for(M.moe_reader_grouped_workspace_bytes(2, P))
    M.moe_reader_grouped_swiglu(2, P, P, I, d, x, None, 1, off, wg, wu, a, ws, ws.numel())
    M.moe_reader_check_error(ws)
    for part, g in ((slice(0, 3), 0), (slice(70000, 70001), 0), (slice(70001, 70003), 1), (slice(P - 3, P), 1)):
        ref, e = swiglu_ref(x[part], wg[g], wu[g])
        close(a[part], ref, HALF * ref.abs() + SLACK * e)


def test_adapters_outputs_past_32_bits():
    T, A, K, N, r = 70000, 3, 16, 32768, 8
    y, ids, t = adapter_call(T, A, K, N, r, use_base=False)
    for part in (slice(0, 50), slice(T - 50, T)):
        close(y[part], *adapter_ref(dict(t, x=t["x"][part]), ids[part], N))


def test_graphs_without_a_call_before_share_their_memory():
    """Any number of graphs captured without a call before them: one workspace, and each replay is right."""
    xs = tokens_of(50, 20, 50, 33)
    L = small_layer()
    ys = [torch.empty_like(x) for x in xs]
    graphs = []
    for x, y in zip(xs, ys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            L.forward_grouped(x, out=y)
            L.forward_grouped(x, residual=x, out=y)
            L.forward_grouped(x, out=y)
    assert len(L._captured) == 1
    for g in (graphs[2], graphs[0], graphs[1], graphs[3], graphs[2]):
        g.replay()
    torch.cuda.synchronize()
    other = small_layer()
    for x, y in zip(xs, ys):
        assert torch.equal(y, other.forward_grouped(x))
    L.check()


def test_check_before_a_graph_has_run():
    """A graph's own workspace holds no error before its first replay, whatever its memory held."""
    x, = tokens_of(50)
    nb = M.moe_reader_block_workspace_bytes(50, SHAPE.E, 4, SHAPE.I, SHAPE.d)
    first, g = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        junk = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
        del junk  # the next graph's workspace gets its memory
    first.replay()
    torch.cuda.synchronize()
    L, y = small_layer(), torch.empty_like(x)
    with torch.cuda.graph(g, pool=first.pool()):
        L.forward_grouped(x, out=y)
    L.check()
    g.replay()
    torch.cuda.synchronize()
    L.check()
    assert torch.equal(y, L.forward_grouped(x))
