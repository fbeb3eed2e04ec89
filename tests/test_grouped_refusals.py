"""The grouped entry points reject bad arguments on the host, before anything
is enqueued (no GPU needed)."""
import ctypes as C

import pytest
import torch

from calibration_free_channel_b200 import build as Bld
from calibration_free_channel_b200 import moe_reader as M

F = 0x10000  # 16-byte aligned, never dereferenced: validation runs first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    Bld.build()
    return M.lib()


def call(lib, name, order, defaults, **kw):
    args = dict(defaults, **kw)
    return getattr(lib, name)(*[args[n] for n in order])


GROUP = ("n n_groups ids offsets rows ws nb stream".split(),
         dict(n=64, n_groups=8, ids=F, offsets=F, rows=F, ws=F, nb=BIG, stream=None))
SWIGLU = ("G P n_x I d x x_rows x_div offsets wg wu a ws nb stream".split(),
          dict(G=8, P=64, n_x=32, I=128, d=256, x=F, x_rows=F, x_div=2, offsets=F, wg=F, wu=F, a=0x20000, ws=F, nb=BIG,
               stream=None))
PRODUCT = ("G P n_x n_y N K layout x x_rows x_div offsets w y y_rows ws nb stream".split(),
           dict(G=8, P=64, n_x=64, n_y=64, N=128, K=256, layout=0, x=F, x_rows=None, x_div=1, offsets=F, w=F, y=0x20000,
                y_rows=None, ws=F, nb=BIG, stream=None))
ADAPTER = ("T A N K r x w base offsets rows a b scale y ws nb stream".split(),
           dict(T=64, A=8, N=128, K=256, r=16, x=F, w=F, base=None, offsets=F, rows=F, a=F, b=F, scale=None,
                y=0x20000, ws=F, nb=BIG, stream=None))


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=(1 << 20) + 1), dict(n_groups=0), dict(n_groups=1025), dict(ids=None), dict(ids=F + 4),
    dict(offsets=None), dict(rows=None), dict(rows=F + 8), dict(ws=None), dict(ws=F + 2), dict(nb=16)])
def test_group_rows_refuses(lib, kw):
    assert call(lib, "moe_reader_group_rows", *GROUP, **kw) == M.MOE_EINVAL
    assert lib.moe_reader_last_error()


@pytest.mark.parametrize("kw", [
    dict(G=0), dict(G=2000), dict(P=0), dict(P=-1), dict(P=(1 << 20) + 1), dict(n_x=0), dict(n_x=(1 << 20) + 1),
    dict(I=0), dict(I=32769), dict(d=0), dict(d=252), dict(d=32776), dict(x=None), dict(x=F + 2),
    dict(x_rows=None), dict(x_rows=None, x_div=1), dict(x_rows=F + 4), dict(x_div=0), dict(offsets=None),
    dict(wg=None), dict(wu=None), dict(wu=F + 8), dict(a=None), dict(a=F + 2), dict(a=F), dict(ws=None), dict(nb=16)])
def test_grouped_swiglu_refuses(lib, kw):
    assert call(lib, "moe_reader_grouped_swiglu", *SWIGLU, **kw) == M.MOE_EINVAL
    assert lib.moe_reader_last_error()


@pytest.mark.parametrize("kw", [
    dict(G=0), dict(P=0), dict(n_x=63), dict(n_y=63), dict(n_y=0), dict(n_y=(1 << 20) + 1), dict(N=0), dict(N=12),
    dict(N=32776), dict(K=4), dict(K=260), dict(layout=2), dict(layout=-1), dict(x=None), dict(x_div=2),
    dict(offsets=F + 4), dict(w=None), dict(w=F + 8), dict(y=None), dict(y=F), dict(y_rows=F + 4), dict(ws=None), dict(nb=0)])
def test_grouped_product_refuses(lib, kw):
    assert call(lib, "moe_reader_grouped_product", *PRODUCT, **kw) == M.MOE_EINVAL
    assert lib.moe_reader_last_error()


@pytest.mark.parametrize("kw", [
    dict(T=0), dict(T=(1 << 20) + 1), dict(A=0), dict(A=1025), dict(N=4), dict(N=100), dict(K=100), dict(r=0),
    dict(r=4), dict(r=12), dict(r=136), dict(x=None), dict(w=F + 8), dict(base=F + 8), dict(offsets=None),
    dict(rows=None), dict(a=None), dict(b=None), dict(scale=F + 4), dict(y=None), dict(y=F), dict(ws=None),
    dict(nb=8)])
def test_adapter_product_refuses(lib, kw):
    assert call(lib, "moe_reader_adapter_product", *ADAPTER, **kw) == M.MOE_EINVAL
    assert lib.moe_reader_last_error()


def _layer(**kw):
    base = dict(E=8, I=128, d=256, top_e=2, w_router=F, w_gate=F, w_up=F, w_down=F)
    base.update(kw)
    return M.MoeReaderLayer(**base)


def _block(lib, layer, B=300, x=F, residual=None, y=0x20000, ids=None, ws=F, nb=BIG):
    return lib.moe_reader_forward_grouped(C.byref(layer), B, x, residual, y, ids, ws, nb, None)


@pytest.mark.parametrize("kw,args", [
    (dict(d=200), {}), (dict(I=8), {}), (dict(top_e=9), {}), (dict(E=2000), {}), (dict(w_gate=None), {}),
    (dict(w_down=F + 8), {}), ({}, dict(B=0)), ({}, dict(B=32769)), ({}, dict(x=None)), ({}, dict(y=F)),
    ({}, dict(y=None)), ({}, dict(ids=F + 4)), ({}, dict(residual=F + 2)), ({}, dict(ws=None)), ({}, dict(nb=1024))])
def test_forward_grouped_refuses(lib, kw, args):
    assert _block(lib, _layer(**kw), **args) == M.MOE_EINVAL
    assert lib.moe_reader_last_error()


def test_forward_grouped_refuses_compacted_shards(lib):
    assert _block(lib, _layer(expert_slot=F)) == M.MOE_EUNSUPPORTED
    assert b"expert_slot" in lib.moe_reader_last_error()


def test_host_tensors_are_refused_by_the_binding():
    t = torch.zeros(64, dtype=torch.int32)
    with pytest.raises(M.MoeError, match="MOE_EINVAL.*cpu"):
        M.moe_reader_group_rows(64, 8, t, F, F, F, BIG)
    with pytest.raises(M.MoeError, match="MOE_EINVAL.*cpu"):
        M.moe_reader_forward_grouped(_layer(), 300, t, None, F, None, F, BIG)


def test_workspace_queries(lib):
    assert M.moe_reader_group_workspace_bytes(1, 1) >= 16
    assert M.moe_reader_grouped_workspace_bytes(128, 65536) >= 16
    assert M.moe_reader_adapter_workspace_bytes(1, 1, 2048, 2048, 16) >= 16
    # the pairs' fp32 outputs and SwiGLU values pass 32 bits at the largest block
    assert M.moe_reader_block_workspace_bytes(32768, 128, 16, 2048, 4096) > 1 << 33
    assert M.moe_reader_group_workspace_bytes(0, 1) == 0
    assert M.moe_reader_grouped_workspace_bytes(1025, 1) == 0
    assert M.moe_reader_adapter_workspace_bytes(1, 1, 2048, 2048, 136) == 0
    assert M.moe_reader_block_workspace_bytes(40000, 128, 8, 768, 2048) == 0


# ------------------------------------------------- what the binding refuses
class Fake:
    """What the binding asks of a tensor, on the device it takes for the current one before CUDA is set up."""

    def __init__(self, n, dtype, contiguous=True):
        self.shape, self.dtype, self.contiguous = (n,), dtype, contiguous
        self.nbytes = n * dtype.itemsize

    def get_device(self):
        return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else None

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.shape[0]

    def data_ptr(self):
        raise AssertionError("a refused tensor's address was taken")


BF, I32, F32, I64 = torch.bfloat16, torch.int32, torch.float32, torch.int64
WRONG = {"type": "use torch", "elements": "elements of", "contiguous": "not contiguous"}


def _wrong(how, n, dtype):
    if how == "type":
        return Fake(n, {BF: torch.float16, I32: I64, F32: torch.float64}[dtype])
    return Fake(n - 1, dtype) if how == "elements" else Fake(n, dtype, contiguous=False)


BINDING = {
    "moe_reader_group_rows": (dict(n=64, n_groups=8, ids=F, offsets=F, rows=F, workspace=F, ws_bytes=BIG),
                              dict(ids=(64, I32), offsets=(9, I32), rows=(64, I32))),
    "moe_reader_grouped_swiglu": (dict(n_groups=8, n_rows=64, n_x=32, I=128, d=256, x=F, x_rows=F, x_div=2, offsets=F,
                                       w_gate=F, w_up=F, a=F, workspace=F, ws_bytes=BIG),
                                  dict(x=(32 * 256, BF), x_rows=(64, I32), offsets=(9, I32), w_gate=(8 * 128 * 256, BF),
                                       w_up=(8 * 128 * 256, BF), a=(64 * 128, BF))),
    "moe_reader_grouped_product": (dict(n_groups=8, n_rows=64, n_x=32, n_y=70, N=128, K=256, w_layout=0, x=F, x_rows=F,
                                        x_div=2, offsets=F, w=F, y=F, y_rows=F, workspace=F, ws_bytes=BIG),
                                   dict(x=(32 * 256, BF), x_rows=(64, I32), offsets=(9, I32), w=(8 * 128 * 256, BF),
                                        y=(70 * 128, BF), y_rows=(64, I32))),
    "moe_reader_adapter_product": (dict(T=64, n_adapters=8, N=128, K=256, r=16, x=F, w=F, base=F, offsets=F, rows=F,
                                        a=F, b=F, scale=F, y=F, workspace=F, ws_bytes=BIG),
                                   dict(x=(64 * 256, BF), w=(128 * 256, BF), base=(64 * 128, BF), offsets=(9, I32),
                                        rows=(64, I32), a=(8 * 16 * 256, BF), b=(8 * 128 * 16, BF), scale=(8, F32),
                                        y=(64 * 128, BF))),
    "moe_reader_forward_grouped": (dict(layer=_layer(), B=300, x=F, residual=F, y=F, ids=F, workspace=F, ws_bytes=BIG),
                                   dict(x=(300 * 256, BF), residual=(300 * 256, BF), y=(300 * 256, BF),
                                        ids=(600, I32))),
}


@pytest.mark.parametrize("how", list(WRONG))
@pytest.mark.parametrize("name,arg", [(f, a) for f in BINDING for a in BINDING[f][1]])
def test_the_binding_refuses_what_is_not_the_array(name, arg, how):
    args, arrays = BINDING[name]
    with pytest.raises(M.MoeError, match="MOE_EINVAL.*" + WRONG[how]):
        getattr(M, name)(**dict(args, **{arg: _wrong(how, *arrays[arg])}))


@pytest.mark.parametrize("name", list(BINDING))
def test_the_binding_refuses_a_workspace_that_is_smaller_than_said(name):
    with pytest.raises(M.MoeError, match="MOE_EINVAL.*workspace"):
        getattr(M, name)(**dict(BINDING[name][0], workspace=Fake(1 << 20, torch.uint8), ws_bytes=(1 << 20) + 1))
