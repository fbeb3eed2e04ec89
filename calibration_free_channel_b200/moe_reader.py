"""Python binding of the C ABI in include/moe_reader.h.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch provides device memory and streams.  If the library is not
built, importing the functions raises; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_reader.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_ECUDA, MOE_ETIMEOUT, MOE_EDEVICE = range(6)
_STATUS = {0: "MOE_OK", 1: "MOE_EINVAL", 2: "MOE_EUNSUPPORTED", 3: "MOE_ECUDA", 4: "MOE_ETIMEOUT",
           5: "MOE_EDEVICE"}

EXPORTS = ["moe_reader_workspace_bytes", "moe_reader_build_sketch", "moe_reader_lowrank_workspace_bytes",
           "moe_reader_build_lowrank", "moe_reader_forward", "moe_reader_forward_dense",
           "moe_reader_forward_host", "moe_reader_rmsnorm", "moe_reader_check_error", "moe_reader_launch_plan",
           "moe_reader_forward_noalloc", "moe_reader_forward_ep", "moe_reader_ep_finish", "moe_reader_last_error",
           "moe_reader_sketch_row_bytes", "moe_reader_sketch_to_base3", "moe_reader_group_workspace_bytes",
           "moe_reader_group_rows", "moe_reader_grouped_workspace_bytes", "moe_reader_grouped_swiglu",
           "moe_reader_grouped_product", "moe_reader_adapter_workspace_bytes", "moe_reader_adapter_product",
           "moe_reader_block_workspace_bytes", "moe_reader_forward_grouped"]

# size queries return a byte count, moe_reader_last_error a string; every other function a status
_NO_STATUS = {"moe_reader_workspace_bytes", "moe_reader_lowrank_workspace_bytes", "moe_reader_last_error",
              "moe_reader_sketch_row_bytes", "moe_reader_group_workspace_bytes", "moe_reader_grouped_workspace_bytes",
              "moe_reader_adapter_workspace_bytes", "moe_reader_block_workspace_bytes"}


class MoeReaderLayer(C.Structure):
    _fields_ = [("E", C.c_int32), ("I", C.c_int32), ("d", C.c_int32), ("top_e", C.c_int32), ("r", C.c_int32),
                ("w_router", C.c_void_p), ("router_bias", C.c_void_p), ("w_gate", C.c_void_p),
                ("w_up", C.c_void_p), ("w_down", C.c_void_p), ("rot_sign", C.c_void_p),
                ("sk_gate", C.c_void_p), ("sk_up", C.c_void_p), ("alpha_gate", C.c_void_p),
                ("alpha_up", C.c_void_p), ("u_sigma", C.c_void_p), ("v", C.c_void_p),
                ("recovery_input", C.c_int32), ("path", C.c_int32), ("cluster_size", C.c_int32),
                ("sketch_format", C.c_int32), ("expert_slot", C.c_void_p)]


class MoeReaderDebug(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("ids", "weights", "dot_gate", "dot_up", "score", "cand", "kept",
                                          "a_kept", "y_expert", "phase_ns", "ev_before", "ev_after")] + \
               [("wait_limit_us", C.c_uint32), ("withhold_copy", C.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with calibration_free_channel_b200.build.build()")
        L = C.CDLL(LIB_PATH)
        P, i32, sz = C.c_void_p, C.c_int, C.c_size_t
        L.moe_reader_workspace_bytes.restype = sz
        L.moe_reader_workspace_bytes.argtypes = [i32] * 8
        L.moe_reader_build_sketch.argtypes = [i32, i32, i32, P, P, C.c_uint64, P, P, P, P, P, P]
        L.moe_reader_lowrank_workspace_bytes.restype = sz
        L.moe_reader_lowrank_workspace_bytes.argtypes = [i32] * 4
        L.moe_reader_build_lowrank.argtypes = [i32, i32, i32, i32, P, P, P, P, sz, P]
        L.moe_reader_forward.argtypes = [C.POINTER(MoeReaderLayer), i32, i32, i32, P, P, P,
                                         C.POINTER(MoeReaderDebug), P, sz, P]
        L.moe_reader_forward_dense.argtypes = [C.POINTER(MoeReaderLayer), i32, P, P, P, P, sz, P]
        L.moe_reader_forward_ep.argtypes = [C.POINTER(MoeReaderLayer), i32, i32, i32, P, i32, i32, P,
                                            C.POINTER(MoeReaderDebug), P, sz, P]
        L.moe_reader_ep_finish.argtypes = [i32, i32, P, P, P, P]
        L.moe_reader_forward_host.argtypes = [C.POINTER(MoeReaderLayer), i32, i32, i32, P, P, P, P, P, sz, P]
        L.moe_reader_rmsnorm.argtypes = [i32, i32, C.c_float, P, P, P]
        L.moe_reader_check_error.argtypes = [P, P]
        L.moe_reader_launch_plan.argtypes = [i32] * 7 + [P]
        L.moe_reader_forward_noalloc.argtypes = [C.POINTER(MoeReaderLayer), i32, i32, i32, P, P, P, P]
        L.moe_reader_last_error.restype = C.c_char_p
        L.moe_reader_last_error.argtypes = []
        L.moe_reader_sketch_row_bytes.restype = sz
        L.moe_reader_sketch_row_bytes.argtypes = [i32, i32]
        L.moe_reader_sketch_to_base3.argtypes = [i32, i32, i32, P, P, P]
        L.moe_reader_group_workspace_bytes.restype = sz
        L.moe_reader_group_workspace_bytes.argtypes = [i32] * 2
        L.moe_reader_group_rows.argtypes = [i32, i32, P, P, P, P, sz, P]
        L.moe_reader_grouped_workspace_bytes.restype = sz
        L.moe_reader_grouped_workspace_bytes.argtypes = [i32] * 2
        L.moe_reader_grouped_swiglu.argtypes = [i32] * 5 + [P, P, i32, P, P, P, P, P, sz, P]
        L.moe_reader_grouped_product.argtypes = [i32] * 7 + [P, P, i32, P, P, P, P, P, sz, P]
        L.moe_reader_adapter_workspace_bytes.restype = sz
        L.moe_reader_adapter_workspace_bytes.argtypes = [i32] * 5
        L.moe_reader_adapter_product.argtypes = [i32] * 5 + [P] * 10 + [sz, P]
        L.moe_reader_block_workspace_bytes.restype = sz
        L.moe_reader_block_workspace_bytes.argtypes = [i32] * 5
        L.moe_reader_forward_grouped.argtypes = [C.POINTER(MoeReaderLayer), i32, P, P, P, P, P, sz, P]
        for f in EXPORTS:
            if f not in _NO_STATUS:
                getattr(L, f).restype = C.c_int
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != MOE_OK:
        raise MoeError(status, lib().moe_reader_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_cuda_set_up = False


def _device():
    """The current device's index, None before torch has set CUDA up."""
    global _cuda_set_up
    if not _cuda_set_up:
        if not torch.cuda.is_initialized():
            return None
        _cuda_set_up = True
    return torch._C._cuda_getDevice()


# what the grouped entry points' arrays may hold (bf16 also as bit patterns)
_BF16 = frozenset((torch.bfloat16, torch.uint16, torch.int16))
_I32 = frozenset((torch.int32, torch.uint32))
_F32 = frozenset((torch.float32,))


def _ptrs(*args):
    """Pointers of the grouped entry points' arrays, each given as (tensor or
    address, its types, the elements it must have) or, for a workspace, as
    (tensor or address, None, bytes).  Tensors have to be contiguous, on the
    current device, of such a type and large enough: the kernels would read or
    write memory that is not their values otherwise."""
    dev = _device()
    out = []
    for t, types, n in args:
        if t is None or type(t) is int:
            out.append(t)
        elif (t.get_device() == dev and t.is_contiguous() and
              (t.nbytes >= n if types is None else t.dtype in types and t.numel() >= n)):
            out.append(t.data_ptr())
        elif t.get_device() != dev:
            raise MoeError(MOE_EINVAL, f"a tensor is on {t.device}, not on the current CUDA device")
        elif not t.is_contiguous():
            raise MoeError(MOE_EINVAL, f"a tensor of shape {tuple(t.shape)} is not contiguous")
        elif types is None:
            raise MoeError(MOE_EINVAL, f"a workspace has {t.nbytes} bytes, less than the {n} it is said to have")
        elif t.dtype not in types:
            raise MoeError(MOE_EINVAL, f"a tensor of shape {tuple(t.shape)} is {t.dtype}: use " +
                           " or ".join(sorted(str(d) for d in types)))
        else:
            raise MoeError(MOE_EINVAL, f"a tensor of shape {tuple(t.shape)} has {t.numel()} elements of {n}")
    return out


def _stream(stream):
    if stream is None:
        # the current stream's handle without building a Stream object (which costs more than a launch);
        # before torch has set CUDA up, that is the default stream
        dev = _device()
        return torch._C._cuda_getCurrentRawStream(dev) if dev is not None else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


# ------------------------------------------------------ the C ABI, by name
def moe_reader_workspace_bytes(B, E, top_e, I, d, k, c, r) -> int:
    return int(lib().moe_reader_workspace_bytes(B, E, top_e, I, d, k, c, r))


def moe_reader_lowrank_workspace_bytes(E, I, d, r) -> int:
    return int(lib().moe_reader_lowrank_workspace_bytes(E, I, d, r))


def moe_reader_build_sketch(E, I, d, w_gate, w_up, rot_seed, rot_sign, sk_gate, sk_up, alpha_gate, alpha_up,
                            stream=None):
    _check(lib().moe_reader_build_sketch(E, I, d, _ptr(w_gate), _ptr(w_up), rot_seed & ((1 << 64) - 1),
                                         _ptr(rot_sign), _ptr(sk_gate), _ptr(sk_up), _ptr(alpha_gate),
                                         _ptr(alpha_up), _stream(stream)))


def moe_reader_sketch_row_bytes(d, fmt) -> int:
    return int(lib().moe_reader_sketch_row_bytes(d, fmt))


def moe_reader_sketch_to_base3(E, I, d, sk_codes, sk_base3, stream=None):
    _check(lib().moe_reader_sketch_to_base3(E, I, d, _ptr(sk_codes), _ptr(sk_base3), _stream(stream)))


def moe_reader_build_lowrank(E, I, d, r, w_down, u_sigma, v, workspace, ws_bytes, stream=None):
    _check(lib().moe_reader_build_lowrank(E, I, d, r, _ptr(w_down), _ptr(u_sigma), _ptr(v), _ptr(workspace),
                                          ws_bytes, _stream(stream)))


def moe_reader_forward_ep(layer: MoeReaderLayer, B, k, c, x, ep_rank, ep_size, y_partial, dbg, workspace, ws_bytes,
                          stream=None):
    _check(lib().moe_reader_forward_ep(C.byref(layer), B, k, c, _ptr(x), ep_rank, ep_size, _ptr(y_partial),
                                       C.byref(dbg) if dbg is not None else None, _ptr(workspace), ws_bytes,
                                       _stream(stream)))


def moe_reader_ep_finish(B, d, y_sum, residual, y, stream=None):
    _check(lib().moe_reader_ep_finish(B, d, _ptr(y_sum), _ptr(residual), _ptr(y), _stream(stream)))


def moe_reader_forward(layer: MoeReaderLayer, B, k, c, x, residual, y, dbg, workspace, ws_bytes, stream=None):
    _check(lib().moe_reader_forward(C.byref(layer), B, k, c, _ptr(x), _ptr(residual), _ptr(y),
                                    C.byref(dbg) if dbg is not None else None, _ptr(workspace), ws_bytes,
                                    _stream(stream)))


def moe_reader_forward_dense(layer: MoeReaderLayer, B, x, residual, y, workspace, ws_bytes, stream=None):
    _check(lib().moe_reader_forward_dense(C.byref(layer), B, _ptr(x), _ptr(residual), _ptr(y), _ptr(workspace),
                                          ws_bytes, _stream(stream)))


def moe_reader_forward_noalloc(layer: MoeReaderLayer, B, k, c, x, residual, y, stream=None):
    """The step with the library's fixed device scratch (no workspace
    argument): for callers that cannot allocate device memory."""
    _check(lib().moe_reader_forward_noalloc(C.byref(layer), B, k, c, _ptr(x), _ptr(residual), _ptr(y),
                                            _stream(stream)))


def moe_reader_forward_host(layer: MoeReaderLayer, B, k, c, x_host, x_dev, y_dev, y_host, workspace, ws_bytes,
                            stream=None):
    _check(lib().moe_reader_forward_host(C.byref(layer), B, k, c, _ptr(x_host), _ptr(x_dev), _ptr(y_dev),
                                         _ptr(y_host), _ptr(workspace), ws_bytes, _stream(stream)))


def moe_reader_group_workspace_bytes(n, n_groups) -> int:
    return int(lib().moe_reader_group_workspace_bytes(n, n_groups))


def moe_reader_group_rows(n, n_groups, ids, offsets, rows, workspace, ws_bytes, stream=None):
    p = _ptrs((ids, _I32, n), (offsets, _I32, n_groups + 1), (rows, _I32, n), (workspace, None, ws_bytes))
    _check(lib().moe_reader_group_rows(n, n_groups, *p, ws_bytes, _stream(stream)))


def moe_reader_grouped_workspace_bytes(n_groups, n_rows) -> int:
    return int(lib().moe_reader_grouped_workspace_bytes(n_groups, n_rows))


def moe_reader_grouped_swiglu(n_groups, n_rows, n_x, I, d, x, x_rows, x_div, offsets, w_gate, w_up, a, workspace,
                              ws_bytes, stream=None):
    x, x_rows, *rest = _ptrs((x, _BF16, n_x * d), (x_rows, _I32, n_rows), (offsets, _I32, n_groups + 1),
                             (w_gate, _BF16, n_groups * I * d), (w_up, _BF16, n_groups * I * d),
                             (a, _BF16, n_rows * I), (workspace, None, ws_bytes))
    _check(lib().moe_reader_grouped_swiglu(n_groups, n_rows, n_x, I, d, x, x_rows, x_div, *rest, ws_bytes,
                                           _stream(stream)))


def moe_reader_grouped_product(n_groups, n_rows, n_x, n_y, N, K, w_layout, x, x_rows, x_div, offsets, w, y, y_rows,
                               workspace, ws_bytes, stream=None):
    x, x_rows, *rest = _ptrs((x, _BF16, n_x * K), (x_rows, _I32, n_rows), (offsets, _I32, n_groups + 1),
                             (w, _BF16, n_groups * N * K), (y, _BF16, n_y * N), (y_rows, _I32, n_rows),
                             (workspace, None, ws_bytes))
    _check(lib().moe_reader_grouped_product(n_groups, n_rows, n_x, n_y, N, K, w_layout, x, x_rows, x_div, *rest,
                                            ws_bytes, _stream(stream)))


def moe_reader_adapter_workspace_bytes(T, n_adapters, K, N, r) -> int:
    return int(lib().moe_reader_adapter_workspace_bytes(T, n_adapters, K, N, r))


def moe_reader_adapter_product(T, n_adapters, N, K, r, x, w, base, offsets, rows, a, b, scale, y, workspace, ws_bytes,
                               stream=None):
    p = _ptrs((x, _BF16, T * K), (w, _BF16, N * K), (base, _BF16, T * N), (offsets, _I32, n_adapters + 1),
              (rows, _I32, T), (a, _BF16, n_adapters * r * K), (b, _BF16, n_adapters * N * r),
              (scale, _F32, n_adapters), (y, _BF16, T * N), (workspace, None, ws_bytes))
    _check(lib().moe_reader_adapter_product(T, n_adapters, N, K, r, *p, ws_bytes, _stream(stream)))


def moe_reader_block_workspace_bytes(B, E, top_e, I, d) -> int:
    return int(lib().moe_reader_block_workspace_bytes(B, E, top_e, I, d))


def moe_reader_forward_grouped(layer: MoeReaderLayer, B, x, residual, y, ids, workspace, ws_bytes, stream=None):
    n = B * layer.d
    p = _ptrs((x, _BF16, n), (residual, _BF16, n), (y, _BF16, n), (ids, _I32, B * layer.top_e),
              (workspace, None, ws_bytes))
    _check(lib().moe_reader_forward_grouped(C.byref(layer), B, *p, ws_bytes, _stream(stream)))


def moe_reader_rmsnorm(B, d, eps, x, h, stream=None):
    _check(lib().moe_reader_rmsnorm(B, d, eps, _ptr(x), _ptr(h), _stream(stream)))


def moe_reader_check_error(workspace, stream=None):
    """workspace None: the error word of moe_reader_forward_noalloc's scratch."""
    _check(lib().moe_reader_check_error(_ptr(workspace), _stream(stream)))


def timing_debug(ev_before, ev_after) -> MoeReaderDebug:
    """A debug block that only records two torch.cuda.Event around the expert
    kernels of one call (no per-stage outputs)."""
    d = MoeReaderDebug()
    d.ev_before = ev_before.cuda_event
    d.ev_after = ev_after.cuda_event
    return d


def moe_reader_launch_plan(dense: bool, B, E, top_e, I, d, r) -> dict:
    out = (C.c_int32 * 4)()
    _check(lib().moe_reader_launch_plan(int(dense), B, E, top_e, I, d, r, C.cast(out, C.c_void_p)))
    return dict(cluster_size=out[0], ring_rows=out[1], smem_bytes=out[2], max_active_clusters=out[3])


# ----------------------------------------------------------- convenience
class Layer:
    """A resident MoE layer on the GPU: bf16 weights, the sketch and the
    low-rank map, with the C struct that describes them."""

    def __init__(self, weights: dict, top_e: int, device="cuda", expert_slot=None):
        """weights: w_router [E, d] (and router_bias [E]) for every expert;
        w_gate, w_up, w_down for all E experts, or (with expert_slot, [E]
        int32: the index of each expert in those arrays, -1 if not held) for
        the held experts only, compacted."""
        dev = torch.device(device)
        self.w = {k: (v.to(dev).contiguous() if v is not None else None) for k, v in weights.items()}
        Eh, I, d = self.w["w_gate"].shape
        E = self.w["w_router"].shape[0]
        if expert_slot is None and Eh != E:
            raise ValueError(f"{Eh} experts of weights for a router of {E}: pass expert_slot")
        self.E, self.E_held, self.I, self.d, self.top_e, self.r = E, Eh, I, d, top_e, 0
        self.rot_sign = torch.empty(d, dtype=torch.int8, device=dev)
        self.sk_gate = torch.empty((Eh, I, d // 16), dtype=torch.int32, device=dev)
        self.sk_up = torch.empty_like(self.sk_gate)
        self.alpha_gate = torch.empty((Eh, I), dtype=torch.float32, device=dev)
        self.alpha_up = torch.empty_like(self.alpha_gate)
        self.u_sigma = None
        self.v = None
        self._ws = None        # workspaces of the reader and of forward_grouped (see _scratch)
        self._wsg = None
        self._captured = []
        self.path = 0          # which reader runs a sparse step (see struct)
        self.sketch_format = 0  # 0: 2-bit codes, 1: base 3 (build_sketch(packing=...))
        # [E] int32 weight slot of each expert (held experts only, compacted), or None
        self.expert_slot = None if expert_slot is None else \
            torch.as_tensor(expert_slot, dtype=torch.int32).to(dev).contiguous()
        self.cluster_size = 0  # CTAs per cluster of the cluster kernels (0: automatic)

    def build_sketch(self, rot_seed: int, stream=None, packing: str = "2bit"):
        """packing "2bit": [E, I, d/16] words of 2-bit codes; "base3": [E, I,
        sketch_row_bytes] bytes, five trits per byte (the codes are built,
        repacked and dropped)."""
        if packing not in ("2bit", "base3"):
            raise ValueError(f"packing {packing!r}: use '2bit' or 'base3'")
        dev = self.w["w_gate"].device
        Eh = self.E_held
        if self.sk_gate.dtype != torch.int32:  # rebuilt after a base-3 packing
            self.sk_gate = torch.empty((Eh, self.I, self.d // 16), dtype=torch.int32, device=dev)
            self.sk_up = torch.empty_like(self.sk_gate)
        moe_reader_build_sketch(Eh, self.I, self.d, self.w["w_gate"], self.w["w_up"], rot_seed,
                                self.rot_sign, self.sk_gate, self.sk_up, self.alpha_gate, self.alpha_up, stream)
        self.sketch_format = 0
        if packing == "base3":
            rb = moe_reader_sketch_row_bytes(self.d, 1)
            g3 = torch.empty((Eh, self.I, rb), dtype=torch.uint8, device=dev)
            u3 = torch.empty_like(g3)
            moe_reader_sketch_to_base3(Eh, self.I, self.d, self.sk_gate, g3, stream)
            moe_reader_sketch_to_base3(Eh, self.I, self.d, self.sk_up, u3, stream)
            torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()
            self.sk_gate, self.sk_up, self.sketch_format = g3, u3, 1
        return self

    def build_lowrank(self, r: int, stream=None):
        dev = self.w["w_down"].device
        Eh = self.E_held
        self.u_sigma = torch.empty((Eh, self.I, r), dtype=torch.bfloat16, device=dev)
        self.v = torch.empty((Eh, self.d, r), dtype=torch.bfloat16, device=dev)
        nb = moe_reader_lowrank_workspace_bytes(Eh, self.I, self.d, r)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        moe_reader_build_lowrank(Eh, self.I, self.d, r, self.w["w_down"], self.u_sigma, self.v, ws, nb, stream)
        torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()
        del ws
        self.r = r
        return self

    def set_lowrank(self, u_sigma, v):
        """Use given factors ([E, I, r], [E, d, r] bf16) or none (None)."""
        if u_sigma is None:
            self.u_sigma = self.v = None
            self.r = 0
        else:
            dev = self.w["w_down"].device
            self.u_sigma = u_sigma.to(dev).contiguous()
            self.v = v.to(dev).contiguous()
            self.r = int(u_sigma.shape[-1])
        return self

    def struct(self, r: int | None = None, recovery_input: int = 0, path: int | None = None,
               cluster_size: int | None = None) -> MoeReaderLayer:
        """The C description of the layer.  path: 0 automatic, 1 one-cluster
        reader, 2 streamed reader (default: this layer's `path`);
        cluster_size: 0 automatic (default: this layer's `cluster_size`)."""
        rr = self.r if r is None else r
        return MoeReaderLayer(self.E, self.I, self.d, self.top_e, rr, _ptr(self.w["w_router"]),
                              _ptr(self.w.get("router_bias")), _ptr(self.w["w_gate"]), _ptr(self.w["w_up"]),
                              _ptr(self.w["w_down"]), _ptr(self.rot_sign), _ptr(self.sk_gate), _ptr(self.sk_up),
                              _ptr(self.alpha_gate), _ptr(self.alpha_up),
                              _ptr(self.u_sigma) if rr else None, _ptr(self.v) if rr else None, recovery_input,
                              self.path if path is None else path,
                              self.cluster_size if cluster_size is None else cluster_size, self.sketch_format,
                              _ptr(self.expert_slot))

    def shard(self, rank: int, world: int) -> "Layer":
        """What rank `rank` of a `world`-way expert-parallel step holds: the
        experts e % world == rank of this layer (weights, sketch, low-rank
        map) copied into new compacted arrays, the router whole, and
        expert_slot[e] = e // world for them, -1 elsewhere."""
        import copy
        dev = self.w["w_gate"].device
        own = torch.arange(rank, self.E, world, device=dev)
        S = copy.copy(self)
        S.w = {n: (v if v is None or n in ("w_router", "router_bias") else v.index_select(0, own).contiguous())
               for n, v in self.w.items()}
        for n in ("sk_gate", "sk_up", "alpha_gate", "alpha_up", "u_sigma", "v"):
            t = getattr(self, n)
            setattr(S, n, t.index_select(0, own).contiguous() if t is not None else None)
        slot = torch.full((self.E,), -1, dtype=torch.int32)
        slot[rank::world] = torch.arange(own.numel(), dtype=torch.int32)
        S.expert_slot = slot.to(dev)
        S.E_held = int(own.numel())
        S._ws = S._wsg = None
        S._captured = []
        return S

    def _scratch(self, pool: str, nb: int, handle):
        """The layer's workspace of at least nb bytes for calls on the stream
        `handle`, which has to be the current one: it is allocated, zeroed and,
        once a longer call replaces it, freed in that stream's order.  Calls on
        two streams never share one.

        A captured call gets one that eager calls no longer use and that lives
        as long as the layer: of an earlier capture, or an eager one of before
        the capture; without any, memory of a graph, which every captured call
        that uses it zeroes first."""
        held = getattr(self, pool)
        if held is None:
            held = {}
            setattr(self, pool, held)
        if torch.cuda.is_current_stream_capturing():
            for p, zeroed, ws in self._captured:
                if p == pool and zeroed and ws.numel() >= nb:
                    return ws
            for h, ws in held.items():
                if ws.numel() >= nb:
                    del held[h]
                    self._captured.append((pool, True, ws))
                    return ws
            for p, _, ws in self._captured:
                if p == pool and ws.numel() >= nb:
                    return ws.zero_()
            ws = torch.zeros(nb, dtype=torch.uint8, device=self.w["w_gate"].device)
            with torch.cuda.stream(torch.cuda.Stream(ws.device)):
                ws[:4].zero_()  # at once: check() may come before the first replay
            self._captured.append((pool, False, ws))
            return ws
        ws = held.get(handle)
        if ws is None or ws.numel() < nb:
            new = torch.zeros(nb, dtype=torch.uint8, device=self.w["w_gate"].device)
            if ws is not None:
                new[:4].copy_(ws[:4])  # the error word
            held[handle] = ws = new
        return ws

    @contextlib.contextmanager
    def _elsewhere(self, side, tensors):
        """Makes `side` the current stream, so that what a call allocates is in
        that stream's order; the caching allocator then learns of its use of
        tensors from elsewhere, and of the caller's use of what it returns."""
        back = torch.cuda.current_stream(side.device)
        made = []
        with torch.cuda.stream(side):
            yield made
        for t in tensors:
            if t is not None:
                t.record_stream(side)
        for t in made:
            t.record_stream(back)

    def _on(self, stream, *tensors):
        """(handle, context) of a call on `stream` (None: the current one) that
        uses `tensors`; the context takes the list of tensors it returns."""
        handle = _stream(stream) or 0
        if stream is None or handle == _stream(None):
            return handle, contextlib.nullcontext([])
        if not isinstance(stream, torch.cuda.Stream):
            dev = self.w["w_gate"].device
            stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
        return handle, self._elsewhere(stream, tensors)

    def _reader_bytes(self, B):
        return moe_reader_workspace_bytes(B, self.E, self.top_e, self.I, self.d, 1, 1, self.r)

    def workspace(self, B: int, stream=None):
        """The reader's workspace for steps of up to B tokens on `stream`."""
        handle, on = self._on(stream)
        with on:
            return self._scratch("_ws", self._reader_bytes(B), handle)

    def block_workspace(self, B: int):
        """A new workspace for forward_grouped of up to B tokens.  Layers of one
        shape may use one in turn; calls that may overlap need one each."""
        nb = moe_reader_block_workspace_bytes(B, self.E, self.top_e, self.I, self.d)
        if nb == 0:
            raise MoeError(MOE_EINVAL, f"no block of {B} tokens")
        return torch.zeros(nb, dtype=torch.uint8, device=self.w["w_gate"].device)

    def _debug(self, B, k, c, dev):
        P = (B, self.top_e)
        dbg_t = dict(ids=torch.empty(P, dtype=torch.int32, device=dev),
                     weights=torch.empty(P, dtype=torch.float32, device=dev),
                     dot_gate=torch.empty(P + (self.I,), dtype=torch.int32, device=dev),
                     dot_up=torch.empty(P + (self.I,), dtype=torch.int32, device=dev),
                     score=torch.empty(P + (self.I,), dtype=torch.float32, device=dev),
                     cand=torch.empty(P + (c,), dtype=torch.int32, device=dev),
                     kept=torch.empty(P + (k,), dtype=torch.int32, device=dev),
                     a_kept=torch.empty(P + (k,), dtype=torch.float32, device=dev),
                     y_expert=torch.empty(P + (self.d,), dtype=torch.float32, device=dev),
                     phase_ns=torch.zeros((B * self.top_e, 16), dtype=torch.int64, device=dev))
        dbg = MoeReaderDebug()
        for n, v in dbg_t.items():
            setattr(dbg, n, _ptr(v))
        return dbg_t, dbg

    def forward_ep(self, x, k: int, c: int, ep_rank: int, ep_size: int, debug: bool = False, r: int | None = None,
                   stream=None, out=None, recovery_input: int = 0):
        """This rank's fp32 partial of the block ([B, d]) over the experts
        e % ep_size == ep_rank; sum it over the ranks, then ep_finish."""
        B = x.shape[0]
        handle, on = self._on(stream, x, out)
        with on as made:
            ws = self._scratch("_ws", self._reader_bytes(B), handle)
            yp = out if out is not None else torch.empty((B, self.d), dtype=torch.float32, device=x.device)
            dbg_t, dbg = self._debug(B, k, c, x.device) if debug else (None, None)
            moe_reader_forward_ep(self.struct(r, recovery_input), B, k, c, x, ep_rank, ep_size, yp, dbg, ws,
                                  ws.numel(), handle)
            made += [yp, *(dbg_t or {}).values()]
        return (yp, dbg_t) if debug else yp

    def forward(self, x, k: int, c: int, residual=None, debug: bool = False, r: int | None = None, stream=None,
                out=None, recovery_input: int = 0, path: int | None = None, events=None):
        """events: (ev_before, ev_after) torch.cuda.Event recorded around the
        expert kernels (timing only; not with debug)."""
        B = x.shape[0]
        handle, on = self._on(stream, x, residual, out)
        with on as made:
            ws = self._scratch("_ws", self._reader_bytes(B), handle)
            y = out if out is not None else torch.empty_like(x)
            dbg_t, dbg = self._debug(B, k, c, x.device) if debug else (None, None)
            if events is not None:
                dbg = timing_debug(*events)
            moe_reader_forward(self.struct(r, recovery_input, path), B, k, c, x, residual, y, dbg, ws, ws.numel(),
                               handle)
            made += [y, *(dbg_t or {}).values()]
        return (y, dbg_t) if debug else y

    def forward_dense(self, x, residual=None, stream=None, out=None):
        B = x.shape[0]
        handle, on = self._on(stream, x, residual, out)
        with on as made:
            ws = self._scratch("_ws", self._reader_bytes(B), handle)
            y = out if out is not None else torch.empty_like(x)
            moe_reader_forward_dense(self.struct(0), B, x, residual, y, ws, ws.numel(), handle)
            made.append(y)
        return y

    def forward_grouped(self, x, residual=None, ids=None, stream=None, out=None, workspace=None):
        """The all-channel block over any number of tokens (prompts): x,
        residual and out [B, d] bf16; ids, if given, receives the chosen
        experts ([B, top_e] int32).

        workspace: of block_workspace, or the layer's own (None), of which it
        keeps one for each stream it is called on.  Pass one to let the layers
        of a model share it, or where captured graphs of this layer (or
        branches of one) may run at the same time; it has to outlive the graphs, and its errors are read
        by moe_reader_check_error."""
        B = x.shape[0]
        for name, t, shape in (("x", x, (B, self.d)), ("residual", residual, (B, self.d)), ("out", out, (B, self.d)),
                               ("ids", ids, (B, self.top_e))):
            if t is not None and tuple(t.shape) != shape:
                raise MoeError(MOE_EINVAL, f"{name} has shape {tuple(t.shape)}, not {shape}")
        if x.device != self.w["w_gate"].device:
            raise MoeError(MOE_EINVAL, f"x is on {x.device}, the layer on {self.w['w_gate'].device}")
        nb = moe_reader_block_workspace_bytes(B, self.E, self.top_e, self.I, self.d)
        with torch.cuda.device(x.device):
            handle, on = self._on(stream, x, residual, out, ids, workspace)
            with on as made:
                ws = workspace if workspace is not None else self._scratch("_wsg", max(nb, 16), handle)
                y = out if out is not None else torch.empty_like(x)
                moe_reader_forward_grouped(self.struct(0), B, x, residual, y, ids, ws, ws.nbytes, handle)
                made.append(y)
        return y

    def check(self, stream=None):
        """Raises what the layer's calls recorded on the device since the last
        check; waits for `stream` and for the streams that they ran on."""
        found = None
        if not all(zeroed for _, zeroed, _ in self._captured):
            torch.cuda.synchronize(self.w["w_gate"].device)
        held = [(h, ws) for pool in (self._ws, self._wsg) for h, ws in (pool or {}).items()]
        for h, ws in held + [(None, ws) for _, _, ws in self._captured]:
            for s in (stream,) if h is None or h == _stream(stream) else (stream, h):
                try:
                    moe_reader_check_error(ws, s)
                except MoeError as e:
                    found = found or e
        if found is not None:
            raise found
