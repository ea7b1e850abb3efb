"""Thin ctypes binding of libmoe_int4.so (include/moe_int4.h).

Argument marshalling only: every step of the layer runs in the HIP library.
torch supplies device memory and the current stream; it is imported before
the library is loaded so that the library binds to the HIP runtime torch
already loaded (both carry the same soname).
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MOE_INT4_LIB", os.path.join(HERE, "libmoe_int4.so"))
HEADER = os.path.join(os.path.dirname(HERE), "include", "moe_int4.h")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP, MOE_EBUFFER, MOE_EFORMAT = (
    0, -1, -2, -3, -4, -5, -6)
MOE_ESCRATCH = -7
NOALLOC_SCRATCH_BYTES = 320 * 1024
MODE_PREFILL, MODE_DECODE, MODE_ROUTE = 0, 1, 2
GEMM_AUTO, GEMM_EXACT, GEMM_WIDE = 0, 1, 2
BF16, F16, F32 = 0, 1, 2
OUT8_NONE, OUT8_INT8, OUT8_E4M3 = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3
GATE_NONE, GATE_SILU, GATE_SIGMOID = 0, 1, 2
HEADER_BYTES = 256

_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_f64 = ctypes.c_double


class MoeDims(ctypes.Structure):
    _fields_ = [("H", _i32), ("I", _i32), ("E", _i32), ("top_k", _i32), ("block_m", _i32),
                ("gemm", _i32)]


class MoeLayerWeights(ctypes.Structure):
    _fields_ = [("router_w3", _vp), ("router_w", _vp), ("router_bias", _vp),
                ("experts_gate_up", _vp), ("experts_down", _vp),
                ("shared_gate_up", _vp), ("shared_down", _vp)]


class MoeRouteOut(ctypes.Structure):
    _fields_ = [("topk_idx", _vp), ("topk_w", _vp), ("hist", _vp), ("offsets", _vp),
                ("perm", _vp), ("inv_perm", _vp), ("block_map", _vp), ("num_blocks", _vp)]


class MoeNorm(ctypes.Structure):
    _fields_ = [("H", _i32), ("dtype", _i32), ("weight_dtype", _i32), ("out8", _i32), ("group", _i32),
                ("eps", _f32), ("weight_offset", _f32)]


class MoeGate(ctypes.Structure):
    _fields_ = [("E", _i32), ("top_k", _i32), ("block_m", _i32), ("score", _i32), ("n_groups", _i32),
                ("topk_groups", _i32), ("group_score", _i32), ("renorm", _i32), ("scale", _f32),
                ("balance_bias", _vp)]


class MoeAdapters(ctypes.Structure):
    _fields_ = [("n", _i32), ("R", _i32), ("A", _vp), ("B", _vp), ("ranks", _vp), ("scales", _vp)]


class MoeRopeScaling(ctypes.Structure):
    _fields_ = [("kind", _i32), ("base", _f64), ("factor", _f64), ("context", _f64), ("slow", _f64), ("fast", _f64)]


class MoeRotary(ctypes.Structure):
    _fields_ = [("head_dim", _i32), ("rot_dim", _i32), ("dtype", _i32), ("interleaved", _i32), ("inverse", _i32),
                ("magnitude", _f32), ("turns", _vp)]


class MoeLinear(ctypes.Structure):
    _fields_ = [("qk_heads", _i32), ("v_heads", _i32), ("qk_dim", _i32), ("v_dim", _i32), ("scale", _f32)]


class MoeBlockNorm(ctypes.Structure):
    _fields_ = [("H", _i32), ("dtype", _i32), ("weight_dtype", _i32), ("normalize", _i32), ("group", _i32),
                ("gate", _i32), ("gate_per_row", _i32), ("next", _i32), ("out8", _i32), ("out8_group", _i32),
                ("eps", _f32), ("weight_offset", _f32), ("scale", _f32), ("next_eps", _f32), ("next_offset", _f32)]


class MoeError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


_lib = None


def header_functions():
    """Names of the functions declared in include/moe_int4.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[A-Za-z_][\w]*\s*\**\s*([a-z_][\w]*)\s*\(", text, flags=re.M)


def lib():
    """Load libmoe_int4.so (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is None:
        import torch  # noqa: F401  (binds the library to torch's HIP runtime)
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        L.moe_max_blocks.argtypes = [P(MoeDims), _i32]
        L.moe_max_blocks.restype = _i64
        L.moe_packed_bytes.argtypes = [_i32, _i32, _i32, _i32]
        L.moe_packed_bytes.restype = _sz
        L.pack_int4_g64.argtypes = [_vp] * 6 + [_i32, _i32, _i32, _vp, _sz]
        L.moe_router_packed_bytes.argtypes = [_i32, _i32]
        L.moe_router_packed_bytes.restype = _sz
        L.pack_router_bf16x3.argtypes = [_vp, _i32, _i32, _vp, _sz]
        L.moe_workspace_bytes.argtypes = [P(MoeDims), _i32, _i32, P(_sz)]
        L.moe_route.argtypes = [P(MoeDims), _vp, _i32, P(MoeRouteOut), _vp, _sz, _vp]
        L.moe_prefill_layer.argtypes = [P(MoeDims), P(MoeLayerWeights), _vp, _vp, _i32, _i32,
                                        _vp, P(MoeRouteOut), _vp, _sz, _vp]
        L.moe_decode_layer.argtypes = [P(MoeDims), P(MoeLayerWeights), _vp, _vp, _i32, _vp,
                                       P(MoeRouteOut), _vp, _sz, _vp]
        L.moe_prefill_layer_profiled.argtypes = L.moe_prefill_layer.argtypes + [_vp, _i32]
        L.moe_prefill_layer_host_routed.argtypes = [P(MoeDims), P(MoeLayerWeights), _vp, _vp, _i32,
                                                    _i32, _vp, _sz, _vp]
        L.moe_unfused_weight_bytes.argtypes = [P(MoeDims), P(_sz)]
        L.moe_prefill_layer_unfused.argtypes = [P(MoeDims), P(MoeLayerWeights), _vp, _vp, _i32, _i32,
                                                _vp, _sz, _vp, _sz, _vp]
        L.moe_decode_layer_profiled.argtypes = L.moe_decode_layer.argtypes + [_vp, _i32]
        L.moe_decode_layer_noalloc.argtypes = [P(MoeDims), P(MoeLayerWeights), _vp, _vp, _i32, _vp,
                                               P(MoeRouteOut), _vp]
        L.moe_ceiling_read.argtypes = [_vp, _sz, _vp, _vp]
        L.moe_ceiling_mfma.argtypes = [_i32, _i32, _vp, _vp, P(ctypes.c_double), _vp]
        L.moe_add_rmsnorm.argtypes = [P(MoeNorm), _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp,
                                      _i64, _vp, _i32, _vp]
        L.moe_gate_max_blocks.argtypes = [P(MoeGate), _i32]
        L.moe_gate_max_blocks.restype = _i64
        L.moe_gate_workspace_bytes.argtypes = [P(MoeGate), _i32, P(_sz)]
        L.moe_route_gated.argtypes = [P(MoeGate), _vp, _i32, P(MoeRouteOut), _vp, _sz, _vp]
        L.moe_prefill_layer_gated.argtypes = [P(MoeDims), P(MoeGate)] + L.moe_prefill_layer.argtypes[1:]
        L.moe_decode_layer_gated.argtypes = [P(MoeDims), P(MoeGate)] + L.moe_decode_layer.argtypes[1:]
        L.moe_project_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, P(_sz)]
        L.moe_project.argtypes = [_vp, _i32, _i32, _vp, _i64, _vp, _i64, _i32, P(MoeAdapters), _vp, _i32,
                                  _vp, _sz, _vp]
        L.moe_project_int8_workspace_bytes.argtypes = [_i32, _i32, _i32, P(_sz)]
        L.moe_project_int8.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _i32, _i32, _vp, _sz, _vp]
        L.moe_rope_radians.argtypes = [P(MoeRopeScaling), _i32, _vp, P(_f32)]
        L.moe_rope_turns.argtypes = [_vp, _i32, _vp]
        L.moe_rope.argtypes = [P(MoeRotary)] + [_vp, _i64, _vp, _i64, _i32] * 2 + [_vp, _i32, _vp]
        L.moe_linear_workspace_bytes.argtypes = [P(MoeLinear), _i32, _i32, P(_sz)]
        states = [_vp, _vp, _i32] * 2
        L.moe_linear_attention.argtypes = ([P(MoeLinear)] + [_vp, _i64] * 4 + [_vp, _i32] + states +
                                           [_vp, _i64, _i32, _vp, _sz, _vp])
        L.moe_linear_attention_step.argtypes = [P(MoeLinear)] + [_vp, _i64] * 4 + states + [_vp, _i64, _i32, _vp]
        L.moe_gated_norm.argtypes = [P(MoeBlockNorm), _vp, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp,
                                     _i64, _vp, _i64, _vp, _i32, _vp]
        L.moe_strerror.argtypes = [ctypes.c_int]
        L.moe_strerror.restype = ctypes.c_char_p
        L.moe_test_dequant.argtypes = [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp]
        for name in ("pack_int4_g64", "pack_router_bf16x3", "moe_workspace_bytes", "moe_route",
                     "moe_prefill_layer", "moe_decode_layer", "moe_test_dequant",
                     "moe_prefill_layer_profiled", "moe_decode_layer_profiled",
                     "moe_prefill_layer_host_routed", "moe_unfused_weight_bytes",
                     "moe_prefill_layer_unfused", "moe_ceiling_read", "moe_ceiling_mfma",
                     "moe_decode_layer_noalloc", "moe_add_rmsnorm", "moe_gate_workspace_bytes",
                     "moe_route_gated", "moe_prefill_layer_gated", "moe_decode_layer_gated",
                     "moe_project_workspace_bytes", "moe_project", "moe_project_int8_workspace_bytes",
                     "moe_project_int8", "moe_rope_radians", "moe_rope_turns", "moe_rope",
                     "moe_linear_workspace_bytes", "moe_linear_attention", "moe_linear_attention_step",
                     "moe_gated_norm"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().moe_strerror(code).decode()


def _check(code, what):
    if code != MOE_OK:
        raise MoeError(code, what)


def dims(H, I, E=256, top_k=8, block_m=32, gemm=GEMM_AUTO) -> MoeDims:
    return MoeDims(H, I, E, top_k, block_m, gemm)


def _ptr(t):
    """Device or host address of a torch tensor / numpy array (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        assert t.flags["C_CONTIGUOUS"]
        return t.ctypes.data
    assert t.is_contiguous(), "tensors passed to the library must be contiguous"
    return t.data_ptr()


def _stream(stream, device=None):
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream(device).cuda_stream


# ------------------------------------------------------------------ packing (host)

def moe_max_blocks(d: MoeDims | MoeGate, T: int) -> int:
    if isinstance(d, MoeGate):
        return moe_gate_max_blocks(d, T)
    v = lib().moe_max_blocks(ctypes.byref(d), T)
    if v < 0:
        raise MoeError(int(v), "moe_max_blocks")
    return int(v)


def moe_packed_bytes(count, N, K, paired) -> int:
    return int(lib().moe_packed_bytes(count, N, K, int(paired)))


def pack_int4_g64(q0, s0, b0, q1=None, s1=None, b1=None) -> np.ndarray:
    """Pack [count][N][K] codes with [count][N][K/64] bf16 scales/biases (host)."""
    q0 = np.ascontiguousarray(q0, np.uint8)
    count, N, K = q0.shape
    arrs = [q0, np.ascontiguousarray(s0, np.uint16), np.ascontiguousarray(b0, np.uint16)]
    paired = q1 is not None
    if paired:
        arrs += [np.ascontiguousarray(q1, np.uint8), np.ascontiguousarray(s1, np.uint16),
                 np.ascontiguousarray(b1, np.uint16)]
    else:
        arrs += [None, None, None]
    nbytes = moe_packed_bytes(count, N, K, paired)
    if nbytes == 0:
        raise MoeError(MOE_EUNSUPPORTED, "moe_packed_bytes")
    out = np.empty(nbytes, np.uint8)
    _check(lib().pack_int4_g64(*[_ptr(a) for a in arrs], count, N, K, _ptr(out), nbytes),
           "pack_int4_g64")
    return out


def pack_router_bf16x3(wr) -> np.ndarray:
    wr = np.ascontiguousarray(wr, np.float32)
    E, H = wr.shape
    nbytes = int(lib().moe_router_packed_bytes(E, H))
    if nbytes == 0:
        raise MoeError(MOE_EUNSUPPORTED, "moe_router_packed_bytes")
    out = np.empty(nbytes, np.uint8)
    _check(lib().pack_router_bf16x3(_ptr(wr), E, H, _ptr(out), nbytes), "pack_router_bf16x3")
    return out


def moe_workspace_bytes(d: MoeDims, T_chunk: int, mode: int) -> int:
    n = _sz(0)
    _check(lib().moe_workspace_bytes(ctypes.byref(d), T_chunk, mode, ctypes.byref(n)),
           "moe_workspace_bytes")
    return int(n.value)


# ------------------------------------------------------------------ device buffers

class DeviceWeights:
    """Packed layer weights resident on the GPU (torch uint8 tensors)."""

    def __init__(self, d: MoeDims, tensors: dict):
        self.dims = d
        self.t = tensors
        self.struct = MoeLayerWeights(
            _ptr(tensors["router_w3"]), _ptr(tensors["router_w"]), _ptr(tensors.get("router_bias")),
            _ptr(tensors["experts_gate_up"]), _ptr(tensors["experts_down"]),
            _ptr(tensors["shared_gate_up"]), _ptr(tensors["shared_down"]))

    @staticmethod
    def pack_host(w):
        """Host blobs of a logical layer (anything with the synth.LayerWeights fields)."""
        E = w.E
        blobs = {
            "router_w3": pack_router_bf16x3(w.router_w),
            "router_w": np.ascontiguousarray(w.router_w, np.float32),
            "experts_gate_up": pack_int4_g64(w.q["gate"][:E], w.scale["gate"][:E], w.bias["gate"][:E],
                                             w.q["up"][:E], w.scale["up"][:E], w.bias["up"][:E]),
            "experts_down": pack_int4_g64(w.q["down"][:E], w.scale["down"][:E], w.bias["down"][:E]),
            "shared_gate_up": pack_int4_g64(w.q["gate"][E:], w.scale["gate"][E:], w.bias["gate"][E:],
                                            w.q["up"][E:], w.scale["up"][E:], w.bias["up"][E:]),
            "shared_down": pack_int4_g64(w.q["down"][E:], w.scale["down"][E:], w.bias["down"][E:]),
        }
        if w.router_bias is not None:
            blobs["router_bias"] = np.ascontiguousarray(w.router_bias, np.float32)
        return blobs

    @classmethod
    def upload(cls, d: MoeDims, host_blobs: dict, device="cuda"):
        import torch
        t = {k: torch.from_numpy(v).to(device) for k, v in host_blobs.items()}
        return cls(d, t)

    @classmethod
    def from_logical(cls, w, device="cuda"):
        d = dims(w.H, w.I, w.E)
        return cls.upload(d, cls.pack_host(w), device)

    def clone(self):
        """A second copy at new device addresses (same contents)."""
        return DeviceWeights(self.dims, {k: v.clone() for k, v in self.t.items()})

    @property
    def expert_bytes_read(self):
        return sum(v.numel() * v.element_size() for v in self.t.values())


class RouteBuffers:
    """Device buffers for moe_route_out sized for T tokens (of a layer's dims or a gate)."""

    def __init__(self, d: MoeDims | MoeGate, T: int, device="cuda"):
        import torch
        k = d.top_k
        mb = moe_max_blocks(d, T)
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_idx = torch.full((T, k), -1, **i32)
        self.topk_w = torch.zeros((T, k), dtype=torch.float32, device=device)
        self.hist = torch.full((d.E,), -1, **i32)
        self.offsets = torch.full((d.E + 1,), -1, **i32)
        self.perm = torch.full((T * k,), -1, **i32)
        self.inv_perm = torch.full((T * k,), -1, **i32)
        self.block_map = torch.full((mb, 3), -1, **i32)
        self.num_blocks = torch.full((1,), -1, **i32)
        self.struct = MoeRouteOut(*[_ptr(getattr(self, f)) for f, _ in MoeRouteOut._fields_])

    def to_numpy(self):
        out = {f: getattr(self, f).cpu().numpy() for f, _ in MoeRouteOut._fields_}
        nb = int(out["num_blocks"][0])
        out["num_blocks"] = nb
        out["block_map"] = out["block_map"][:nb]
        return out


def workspace(d: MoeDims, T_chunk: int, mode: int, device="cuda"):
    import torch
    return torch.zeros(moe_workspace_bytes(d, T_chunk, mode), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ entry points

def moe_route(d: MoeDims, logits, T: int, out: RouteBuffers, ws, stream=None):
    _check(lib().moe_route(ctypes.byref(d), _ptr(logits), T, ctypes.byref(out.struct), _ptr(ws),
                           ws.numel(), _stream(stream)), "moe_route")


def moe_prefill_layer(d: MoeDims, w: DeviceWeights, x, y, T: int, chunk_T: int = 0,
                      logits_out=None, route_out: RouteBuffers | None = None, ws=None,
                      stream=None):
    ro = ctypes.byref(route_out.struct) if route_out is not None else None
    _check(lib().moe_prefill_layer(ctypes.byref(d), ctypes.byref(w.struct), _ptr(x), _ptr(y), T,
                                   chunk_T, _ptr(logits_out), ro, _ptr(ws),
                                   0 if ws is None else ws.numel(), _stream(stream)),
           "moe_prefill_layer")


def moe_prefill_layer_host_routed(d: MoeDims, w: DeviceWeights, x, y, T: int, chunk_T: int = 0,
                                  ws=None, stream=None):
    _check(lib().moe_prefill_layer_host_routed(ctypes.byref(d), ctypes.byref(w.struct), _ptr(x),
                                               _ptr(y), T, chunk_T, _ptr(ws),
                                               0 if ws is None else ws.numel(), _stream(stream)),
           "moe_prefill_layer_host_routed")


def unfused_weights(d: MoeDims, device="cuda"):
    """Device buffer for moe_prefill_layer_unfused's bf16 weights."""
    import torch
    n = _sz(0)
    _check(lib().moe_unfused_weight_bytes(ctypes.byref(d), ctypes.byref(n)), "moe_unfused_weight_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def moe_prefill_layer_unfused(d: MoeDims, w: DeviceWeights, x, y, T: int, wbuf, chunk_T: int = 0,
                              ws=None, stream=None):
    _check(lib().moe_prefill_layer_unfused(ctypes.byref(d), ctypes.byref(w.struct), _ptr(x), _ptr(y), T,
                                           chunk_T, _ptr(wbuf), wbuf.numel(), _ptr(ws),
                                           0 if ws is None else ws.numel(), _stream(stream)),
           "moe_prefill_layer_unfused")


def moe_decode_layer(d: MoeDims, w: DeviceWeights, x, y, T: int, logits_out=None,
                     route_out: RouteBuffers | None = None, ws=None, stream=None):
    ro = ctypes.byref(route_out.struct) if route_out is not None else None
    _check(lib().moe_decode_layer(ctypes.byref(d), ctypes.byref(w.struct), _ptr(x), _ptr(y), T,
                                  _ptr(logits_out), ro, _ptr(ws),
                                  0 if ws is None else ws.numel(), _stream(stream)),
           "moe_decode_layer")


def moe_decode_layer_noalloc(d: MoeDims, w: DeviceWeights, x, y, T: int, logits_out=None,
                             route_out: RouteBuffers | None = None, stream=None):
    """moe_decode_layer on the library's static scratch (no workspace argument)."""
    ro = ctypes.byref(route_out.struct) if route_out is not None else None
    _check(lib().moe_decode_layer_noalloc(ctypes.byref(d), ctypes.byref(w.struct), _ptr(x), _ptr(y), T,
                                          _ptr(logits_out), ro, _stream(stream)),
           "moe_decode_layer_noalloc")


def _event_array(events):
    """ctypes array of raw hipEvent_t handles from torch.cuda.Event objects."""
    handles = []
    for e in events:
        if not e.cuda_event:
            e.record()          # torch creates the underlying event lazily
        handles.append(e.cuda_event)
    return (ctypes.c_void_p * len(handles))(*handles)


def moe_prefill_layer_profiled(d: MoeDims, w: DeviceWeights, x, y, T: int, chunk_T: int, events,
                               logits_out=None, route_out: RouteBuffers | None = None, ws=None,
                               stream=None):
    ro = ctypes.byref(route_out.struct) if route_out is not None else None
    arr = events if isinstance(events, ctypes.Array) else _event_array(events)
    _check(lib().moe_prefill_layer_profiled(ctypes.byref(d), ctypes.byref(w.struct), _ptr(x),
                                            _ptr(y), T, chunk_T, _ptr(logits_out), ro, _ptr(ws),
                                            0 if ws is None else ws.numel(), _stream(stream),
                                            ctypes.cast(arr, _vp), len(arr)),
           "moe_prefill_layer_profiled")


def moe_decode_layer_profiled(d: MoeDims, w: DeviceWeights, x, y, T: int, events,
                              logits_out=None, route_out: RouteBuffers | None = None, ws=None,
                              stream=None):
    ro = ctypes.byref(route_out.struct) if route_out is not None else None
    arr = events if isinstance(events, ctypes.Array) else _event_array(events)
    _check(lib().moe_decode_layer_profiled(ctypes.byref(d), ctypes.byref(w.struct), _ptr(x),
                                           _ptr(y), T, _ptr(logits_out), ro, _ptr(ws),
                                           0 if ws is None else ws.numel(), _stream(stream),
                                           ctypes.cast(arr, _vp), len(arr)),
           "moe_decode_layer_profiled")


def moe_ceiling_read(buf, sink, stream=None):
    """Enqueue one streaming read of the device buffer `buf` (measurement helper)."""
    _check(lib().moe_ceiling_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                  _stream(stream)), "moe_ceiling_read")


CEILING_MFMA_BLOCKS = 1024  # blocks of the matrix-core loop (two clock values each)


def moe_ceiling_mfma(iters: int, sink, random: bool = True, clocks=None, stream=None) -> float:
    """Enqueue the bf16 matrix-core loop (random or nearly constant operands);
    `clocks`, if given, is an int64 device tensor of 2 * CEILING_MFMA_BLOCKS
    values that receives each block's real-time and shader-clock ticks.
    Returns the launch's flop count."""
    if clocks is not None and clocks.numel() * clocks.element_size() < 16 * CEILING_MFMA_BLOCKS:
        raise ValueError("moe_ceiling_mfma: clocks needs 2 * CEILING_MFMA_BLOCKS int64 values")
    flops = ctypes.c_double(0.0)
    _check(lib().moe_ceiling_mfma(iters, int(random), _ptr(sink), _ptr(clocks), ctypes.byref(flops),
                                  _stream(stream)), "moe_ceiling_mfma")
    return flops.value


def ceiling_clock_mhz(clocks) -> float:
    """Mean shader clock of the last moe_ceiling_mfma launch that wrote `clocks`
    (shader-clock ticks over 100 MHz real-time ticks, summed over the blocks)."""
    c = clocks.view(-1, 2).cpu().double()
    return float(c[:, 1].sum() / c[:, 0].sum() * 100.0)


def moe_test_dequant(blob, count, N, K, paired, expert, out, stream=None):
    _check(lib().moe_test_dequant(_ptr(blob), count, N, K, int(paired), expert, _ptr(out),
                                  _stream(stream)), "moe_test_dequant")


# ------------------------------------------------------------------ around the layer
#
# These wrappers also check what the C entry points cannot see: the tensors'
# sizes, types and devices (ValueError). The work goes to the current stream
# of the tensors' device unless `stream` says otherwise.

def _type_code(dtype):
    import torch
    codes = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
    if isinstance(dtype, int) and dtype in codes.values():
        return dtype
    if dtype not in codes:
        raise ValueError(f"rows of {dtype} are not supported (bfloat16, float16 or float32)")
    return codes[dtype]


_types = None  # per type code the torch types whose bits a tensor of it may hold; at BITS8 + out8 those of 8 bits
BITS8 = 3


def _types_of(code):
    global _types
    if _types is None:
        import torch
        _types = ((torch.bfloat16,), (torch.float16,), (torch.float32,), (), (torch.int8, torch.uint8),
                  (torch.float8_e4m3fn, torch.uint8), (torch.bfloat16, torch.int16, torch.uint16))
    if not 0 <= code < len(_types) or not _types[code]:
        raise ValueError(f"element type {code} is not known")
    return _types[code]


_BF16_BITS = BITS8 + 3


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _rows(t, T, width, dtypes, dev, name):
    """Address and row stride of a [>= T, width] tensor whose rows are contiguous, on GPU `dev`."""
    shape, stride = t.shape, t.stride()
    if t.dtype not in dtypes or len(shape) != 2 or shape[0] < T or shape[1] != width:
        raise ValueError(f"{name}: [{T}, {width}] of {dtypes[0]} is needed, got {list(shape)} of {t.dtype}")
    if stride[1] != 1 and width > 1:
        raise ValueError(f"{name}: the values of a row have to be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, other tensors on device {dev}: one GPU is needed")
    # the stride of a single row says nothing (it may be any)
    return t.data_ptr(), (stride[0] if T > 1 else width)


def _flat(t, n, dtype, name, dev=None):
    """Address of at least n contiguous values."""
    if t.dtype != dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name}: {n} contiguous values of {dtype} are needed, got {list(t.shape)} of {t.dtype}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, other tensors on device {dev}: one GPU is needed")
    return t.data_ptr()


def _bits(t, n, dtypes, name, dev):
    """Address of at least n contiguous values of one of `dtypes`, on GPU `dev`."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {n} contiguous values of {dtypes[0]} are needed, got {list(t.shape)} of {t.dtype}")
    return _flat(t, n, t.dtype, name, dev)


def _gpu(t):
    """Index of the GPU that t is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"tensors on a GPU are needed, got {t.device}")
    return dev


_entry = {}  # C entry points by name, as `_call` finds them


def _call(name, dev, stream, *args):
    """The C entry point with a stream as its last argument, GPU `dev` being current."""
    import torch
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(lib(), name)
    if dev == torch.cuda.current_device():
        code = f(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream)
    else:
        with torch.cuda.device(dev):
            code = f(*args, _stream(stream))
    if code != MOE_OK:
        raise MoeError(code, name)


def norm(H, dtype=BF16, weight_dtype=None, eps=1e-6, weight_offset=0.0, out8=OUT8_NONE, group=0) -> MoeNorm:
    """What moe_add_rmsnorm does to rows of H values (dtype: a torch type or BF16 / F16 / F32)."""
    code = _type_code(dtype)
    return MoeNorm(H, code, code if weight_dtype is None else _type_code(weight_dtype), out8, group, eps,
                   weight_offset)


def moe_add_rmsnorm(n: MoeNorm, x, weight, T: int, residual=None, h_out=None, y=None, q=None, scales=None,
                    stream=None):
    """h = x + residual, y = h / rms(h) * weight for T rows, and q, scales: y in 8 bits."""
    H, types, dev = n.H, _types_of(n.dtype), x.get_device()
    xp, ldx = _rows(x, T, H, types, dev, "x")
    rp = hp = yp = qp = sp = None
    ldr = ldh = ldy = ldq = 0
    if residual is not None:
        rp, ldr = _rows(residual, T, H, types, dev, "residual")
    if h_out is not None:
        hp, ldh = _rows(h_out, T, H, types, dev, "h_out")
    if y is not None:
        yp, ldy = _rows(y, T, H, types, dev, "y")
    if q is not None:
        qp, ldq = _rows(q, T, H, _types_of(BITS8 + (n.out8 or OUT8_INT8)), dev, "q")
    if scales is not None:
        sp = _flat(scales, T * (H // n.group if n.group else 1), _types_of(F32)[0], "scales", dev)
    wp = _flat(weight, H, _types_of(n.weight_dtype)[0], "weight", dev)
    _call("moe_add_rmsnorm", _gpu(x), stream, ctypes.byref(n), xp, ldx, rp, ldr, wp, hp, ldh, yp, ldy, qp, ldq, sp, T)


def gate(E=256, top_k=8, block_m=32, score=SCORE_SOFTMAX, n_groups=1, topk_groups=1, group_score=GROUP_MAX,
         renorm=True, scale=1.0, balance_bias=None) -> MoeGate:
    """A routing rule (balance_bias: an fp32 device tensor [E] that the gate keeps alive)."""
    bias = None if balance_bias is None else _flat(balance_bias, E, _types_of(F32)[0], "balance_bias")
    g = MoeGate(E, top_k, block_m, score, n_groups, topk_groups, group_score, int(renorm), scale, bias)
    g.bias_tensor = balance_bias
    return g


def _bias_on(g, dev):
    bias = getattr(g, "bias_tensor", None)
    if bias is not None and bias.get_device() != dev:
        raise ValueError(f"balance_bias: on {bias.device}, other tensors on device {dev}: one GPU is needed")


def moe_gate_max_blocks(g: MoeGate, T: int) -> int:
    v = lib().moe_gate_max_blocks(ctypes.byref(g), T)
    if v < 0:
        raise MoeError(int(v), "moe_gate_max_blocks")
    return int(v)


def gate_workspace(g: MoeGate, T: int, device="cuda"):
    """Workspace of moe_route_gated for up to T tokens."""
    import torch
    n = _sz(0)
    _check(lib().moe_gate_workspace_bytes(ctypes.byref(g), T, ctypes.byref(n)), "moe_gate_workspace_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def moe_route_gated(g: MoeGate, logits, T: int, out: RouteBuffers, ws, stream=None):
    """moe_route with a gate: the routing metadata of T tokens from fp32 logits."""
    dev = _gpu(logits)
    lp = _flat(logits, T * g.E, _types_of(F32)[0], "logits", dev)
    if (out.topk_idx.numel() < T * g.top_k or out.hist.numel() < g.E or
            out.block_map.shape[0] < (T * g.top_k + g.block_m - 1) // g.block_m + g.E):
        raise ValueError("route_out: buffers of this gate and T are needed")
    if out.topk_idx.get_device() != dev:
        raise ValueError("logits and route_out: one GPU is needed")
    _bias_on(g, dev)
    wp = _flat(ws, 0, _types_of(BITS8 + OUT8_INT8)[1], "ws", dev)
    _call("moe_route_gated", dev, stream, ctypes.byref(g), lp, T, ctypes.byref(out.struct), wp, ws.numel())


def _layer_args(d, g, w, x, y, T, last, logits_out, route_out, ws):
    """The gated layer's pointer arguments after their checks; last: tokens that route_out describes."""
    dev, bits = x.get_device(), _types_of(_BF16_BITS)
    xp, yp = _bits(x, T * d.H, bits, "x", dev), _bits(y, T * d.H, bits, "y", dev)
    lp = None if logits_out is None else _flat(logits_out, T * d.E, _types_of(F32)[0], "logits_out", dev)
    ro = wp = None
    wn = 0
    if route_out is not None:
        if (route_out.topk_idx.numel() < last * d.top_k or route_out.hist.numel() < d.E or
                route_out.block_map.shape[0] < (last * d.top_k + d.block_m - 1) // d.block_m + d.E):
            raise ValueError(f"route_out: buffers of {last} tokens of this layer are needed")
        if route_out.topk_idx.get_device() != dev:
            raise ValueError("route_out: on another device than x")
        ro = ctypes.byref(route_out.struct)
    if ws is not None:
        wn, wp = ws.numel(), _flat(ws, 0, _types_of(BITS8 + OUT8_INT8)[1], "ws", dev)
    for name, t in w.t.items():
        if t.get_device() != dev:
            raise ValueError(f"weights: {name} on {t.device}, other tensors on device {dev}: one GPU is needed")
    _bias_on(g, dev)
    return ctypes.byref(d), ctypes.byref(g), ctypes.byref(w.struct), xp, yp, lp, ro, wp, wn


def moe_prefill_layer_gated(d: MoeDims, g: MoeGate, w: DeviceWeights, x, y, T: int, chunk_T: int = 0,
                            logits_out=None, route_out: RouteBuffers | None = None, ws=None, stream=None):
    """moe_prefill_layer routed by a gate."""
    chunk = chunk_T if 0 < chunk_T < T else T
    last = T - (T - 1) // chunk * chunk if T > 0 else 0
    dp, gp, sp, xp, yp, lp, ro, wp, wn = _layer_args(d, g, w, x, y, T, last, logits_out, route_out, ws)
    _call("moe_prefill_layer_gated", _gpu(x), stream, dp, gp, sp, xp, yp, T, chunk_T, lp, ro, wp, wn)


def moe_decode_layer_gated(d: MoeDims, g: MoeGate, w: DeviceWeights, x, y, T: int, logits_out=None,
                           route_out: RouteBuffers | None = None, ws=None, stream=None):
    """moe_decode_layer routed by a gate."""
    dp, gp, sp, xp, yp, lp, ro, wp, wn = _layer_args(d, g, w, x, y, T, T, logits_out, route_out, ws)
    _call("moe_decode_layer_gated", _gpu(x), stream, dp, gp, sp, xp, yp, T, lp, ro, wp, wn)


class Adapters:
    """Low-rank adapters of one projection: A [n, R, K] and B [n, N, R] bf16, ranks [n] int32 (None: R
    each), scales [n] fp32 (None: 1 each), all on one device."""

    def __init__(self, A, B, ranks=None, scales=None):
        import torch
        bf16 = _types_of(_BF16_BITS)
        _need(A.dim() == 3 and B.dim() == 3 and A.shape[0] == B.shape[0] and A.shape[1] == B.shape[2] and
              A.dtype in bf16 and B.dtype in bf16 and A.is_contiguous() and B.is_contiguous(),
              "adapters: contiguous A [n, R, K] and B [n, N, R] of bfloat16 are needed")
        _need(all(t is None or t.device == A.device for t in (B, ranks, scales)), "adapters: one device is needed")
        self.n, self.R, self.K = A.shape
        self.N = B.shape[1]
        self.t = (A, B, ranks, scales)
        self.device = A.device
        self.struct = MoeAdapters(self.n, self.R, A.data_ptr(), B.data_ptr(),
                                  None if ranks is None else _flat(ranks, self.n, torch.int32, "ranks"),
                                  None if scales is None else _flat(scales, self.n, torch.float32, "scales"))


def project_workspace(N, K, T, adapters: Adapters | None = None, device=None):
    """Workspace of moe_project for up to T tokens."""
    import torch
    n = _sz(0)
    _check(lib().moe_project_workspace_bytes(N, K, adapters.R if adapters else 0, T, ctypes.byref(n)),
           "moe_project_workspace_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=device or (adapters.device if adapters else "cuda"))


def moe_project(blob, N: int, K: int, x, y, T: int, adapters: Adapters | None = None, adapter_of=None,
                gemm: int = GEMM_AUTO, ws=None, stream=None):
    """y[t] = W x[t] + scale B_a (A_a x[t]) for a packed int4 matrix [N, K] (pack_int4_g64 of one unpaired
    matrix) and the adapter a = adapter_of[t] of each token (-1: none)."""
    import torch
    dev, types = x.get_device(), _types_of(_BF16_BITS)
    # (the bytes moe_packed_bytes gives: a header, the codes, scales and biases, to 256 bytes)
    if N % 64 == 0 and K % 64 == 0:
        _flat(blob, HEADER_BYTES + (N * K // 2 + N * K // 16 + 255) // 256 * 256, torch.uint8, "blob", dev)
    xp, ldx = _rows(x, T, K, types, dev, "x")
    yp, ldy = _rows(y, T, N, types, dev, "y")
    ap = op = wp = None
    wn = 0
    if adapters is not None:
        if adapters.N != N or adapters.K != K or adapters.t[0].get_device() != dev:
            raise ValueError("adapters: another projection's, or on another device")
        ap = ctypes.byref(adapters.struct)
    if adapter_of is not None:
        op = _flat(adapter_of, T, torch.int32, "adapter_of", dev)
    if ws is not None:
        wn = ws.numel()
        wp = _flat(ws, 0, torch.uint8, "ws", dev)
    _call("moe_project", _gpu(x), stream, blob.data_ptr(), N, K, xp, ldx, yp, ldy, T, ap, op, gemm, wp, wn)


# ------------------------------------------------------------------ the mixer half of a block
#
# Checks and streams as above.

def project_int8_workspace(N, K, T, device="cuda"):
    """Workspace of moe_project_int8 for up to T tokens: None, as it needs none at any size."""
    import torch
    n = _sz(0)
    _check(lib().moe_project_int8_workspace_bytes(N, K, T, ctypes.byref(n)), "moe_project_int8_workspace_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None


def moe_project_int8(w, w_scales, x, x_scales, y, T: int, bias=None, ws=None, stream=None):
    """y[t] = x_scales[t] w_scales (w x[t]) + bias for int8 rows x [T, K] (moe_add_rmsnorm's q and scales) and
    int8 weights w [N, K]; y bfloat16, float16 or float32."""
    import torch
    dev = x.get_device()
    if w.dim() != 2:
        raise ValueError(f"w: [N, K] is needed, got {list(w.shape)}")
    N, K = w.shape
    code = _type_code(y.dtype)
    wp = _flat(w, N * K, torch.int8, "w", dev)
    sp = _flat(w_scales, N, torch.float32, "w_scales", dev)
    xp, ldx = _rows(x, T, K, _types_of(BITS8 + OUT8_INT8), dev, "x")
    xs = _flat(x_scales, T, torch.float32, "x_scales", dev)
    yp, ldy = _rows(y, T, N, _types_of(code), dev, "y")
    bp = None if bias is None else _flat(bias, N, torch.float32, "bias", dev)
    kp, kn = (None, 0) if ws is None else (_flat(ws, 0, torch.uint8, "ws", dev), ws.numel())
    _call("moe_project_int8", _gpu(x), stream, wp, sp, bp, N, K, xp, ldx, xs, yp, ldy, code, T, kp, kn)


def rope_radians(rot_dim, base=10000.0, scaling=ROPE_PLAIN, factor=1.0, context=0.0, slow=1.0, fast=32.0):
    """(radians per position of each pair, float64; the factor on cosine and sine) of scaled rotary positions. ROPE_YARN's
    ramp is linear in a pair's turns over the context; models whose ramp runs over the pairs' index pass rope their own
    `radians`."""
    out, m = np.empty(max(rot_dim, 0) // 2, np.float64), _f32(0)
    s = MoeRopeScaling(scaling, base, factor, context, slow, fast)
    _check(lib().moe_rope_radians(ctypes.byref(s), rot_dim, _ptr(out), ctypes.byref(m)), "moe_rope_radians")
    return out, m.value


def rope(head_dim, rot_dim=None, dtype=BF16, interleaved=False, inverse=False, base=10000.0, scaling=ROPE_PLAIN,
         factor=1.0, context=0.0, slow=1.0, fast=32.0, radians=None, magnitude=None, device="cuda") -> MoeRotary:
    """How moe_rope turns heads of head_dim values, the first rot_dim (None: all) of them. The frequencies are those of
    rope_radians, or `radians` [rot_dim / 2] of a model's own (then magnitude is 1 unless given)."""
    import torch
    rot = head_dim if rot_dim is None else rot_dim
    if radians is None:
        radians, m = rope_radians(rot, base, scaling, factor, context, slow, fast)
    else:
        radians, m = np.ascontiguousarray(radians, np.float64), 1.0
        if radians.shape != (rot // 2,):
            raise ValueError(f"radians: {rot // 2} values are needed, got {list(radians.shape)}")
    turns = np.empty(len(radians), np.uint64)
    _check(lib().moe_rope_turns(_ptr(radians), len(radians), _ptr(turns)), "moe_rope_turns")
    table = torch.from_numpy(turns.view(np.int64)).to(device)
    r = MoeRotary(head_dim, rot, _type_code(dtype), int(interleaved), int(inverse), m if magnitude is None else magnitude,
                  table.data_ptr())
    r.table = table  # kept alive with the plan
    return r


def _heads(t, T, heads, dim, dtypes, dev, name):
    """Address and row stride of a [>= T, heads, dim] (or [>= T, heads * dim]) tensor whose rows are contiguous, on GPU
    `dev`."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        return _rows(t, T, heads * dim, dtypes, dev, name)
    if t.dtype not in dtypes or shape[0] < T or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name}: [{T}, {heads}, {dim}] of {dtypes[0]} is needed, got {list(shape)} of {t.dtype}")
    if (stride[2] != 1 and dim > 1) or (stride[1] != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a row have to be contiguous, got strides {list(stride)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, other tensors on device {dev}: one GPU is needed")
    return t.data_ptr(), (stride[0] if T > 1 else heads * dim)


def moe_rope(r: MoeRotary, positions, T: int, q, k=None, q_out=None, k_out=None, stream=None):
    """Turns q [T, q_heads, head_dim] and k [T, k_heads, head_dim] by their tokens' positions (int32), into q_out and
    k_out or in place."""
    import torch
    dev, types, D = q.get_device(), _types_of(r.dtype), r.head_dim

    def heads_of(t, out, name):
        shape = t.shape
        heads = shape[1] if len(shape) == 3 else shape[-1] // max(D, 1)
        p, ld = _heads(t, T, heads, D, types, dev, name)
        if out is None or out is t:
            return p, ld, p, ld, heads
        return (p, ld) + _heads(out, T, heads, D, types, dev, name + "_out") + (heads,)
    args = heads_of(q, q_out, "q")
    if k is not None:
        args += heads_of(k, k_out, "k")
    else:
        _need(k_out is None, "k_out without k")
        args += (None, 0, None, 0, 0)
    pp = _flat(positions, T, torch.int32, "positions", dev)
    table = getattr(r, "table", None)
    if table is not None and table.get_device() != dev:
        raise ValueError(f"rope: its frequencies are on {table.device}, the tensors on device {dev}: one GPU is needed")
    _call("moe_rope", _gpu(q), stream, ctypes.byref(r), *args, pp, T)


def linear_attention(qk_heads, v_heads, qk_dim, v_dim, scale=None) -> MoeLinear:
    """Heads of moe_linear_attention (scale None: qk_dim ** -0.5)."""
    return MoeLinear(qk_heads, v_heads, qk_dim, v_dim, qk_dim ** -0.5 if scale is None else scale)


def linear_attention_workspace(l: MoeLinear, n_seqs: int, T: int, device="cuda"):
    """Workspace of moe_linear_attention for up to n_seqs sequences of T tokens together, or None where none is needed."""
    import torch
    n = _sz(0)
    _check(lib().moe_linear_workspace_bytes(ctypes.byref(l), n_seqs, T, ctypes.byref(n)), "moe_linear_workspace_bytes")
    return torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None


def _state(s, slots, l, heads, n_seqs, dev, name):
    """Addresses of a state and its slots, and how many states it has."""
    if s is None:
        _need(slots is None, f"slots_{name} without state_{name}")
        return None, None, 0
    shape, (f32,) = s.shape, _types_of(F32)
    if len(shape) != 4 or shape[1] != heads or shape[2] != l.qk_dim or shape[3] != l.v_dim or s.dtype != f32 or not s.is_contiguous():
        raise ValueError(f"state_{name}: contiguous [slots, {heads}, {l.qk_dim}, {l.v_dim}] of float32 is needed, got {list(shape)} "
                         f"of {s.dtype}")
    if s.get_device() != dev:
        raise ValueError(f"state_{name}: on {s.device}, other tensors on device {dev}: one GPU is needed")
    if slots is None:  # (the sequence's index: states past the pool's end would be lost without a word)
        if shape[0] < n_seqs:
            raise ValueError(f"state_{name}: {n_seqs} states are needed without slots, got {shape[0]}")
        return s.data_ptr(), None, shape[0]
    return s.data_ptr(), _flat(slots, n_seqs, _i32_type(), f"slots_{name}", dev), shape[0]


_int32 = None


def _i32_type():
    global _int32
    if _int32 is None:
        import torch
        _int32 = torch.int32
    return _int32


def _decay(g, T, heads, dev):
    """Address and row stride of the logarithms of the decay."""
    if g.dim() != 1:
        return _rows(g, T, heads, _types_of(F32), dev, "log_decay")
    _need(g.numel() == heads, "log_decay: [v_heads] or [T, v_heads] is needed")
    return _flat(g, heads, _types_of(F32)[0], "log_decay", dev), 0


def moe_linear_attention(l: MoeLinear, q, k, v, log_decay, o, cu_seqlens, T: int, state_in=None, slots_in=None,
                         state_out=None, slots_out=None, ws=None, stream=None):
    """o = linear attention of the sequences that cu_seqlens [n + 1] (int32) cuts T tokens into; log_decay
    [T, v_heads] or [v_heads]. Their states start as state_in[slots_in] and end as state_out[slots_out]; without slots
    sequence i has state i."""
    import torch
    n = cu_seqlens.numel() - 1
    _need(n >= 0, "cu_seqlens: n + 1 values are needed")
    dev, bits, hk, hv, dk, dv = q.get_device(), _types_of(_BF16_BITS), l.qk_heads, l.v_heads, l.qk_dim, l.v_dim
    qp, ldq = _heads(q, T, hk, dk, bits, dev, "q")
    kp, ldk = _heads(k, T, hk, dk, bits, dev, "k")
    vp, ldv = _heads(v, T, hv, dv, bits, dev, "v")
    op, ldo = _heads(o, T, hv, dv, bits, dev, "o")
    gp, ldg = _decay(log_decay, T, hv, dev)
    si, sli, ni = _state(state_in, slots_in, l, hv, n, dev, "in")
    so, slo, no = _state(state_out, slots_out, l, hv, n, dev, "out")
    cp = _flat(cu_seqlens, n + 1, torch.int32, "cu_seqlens", dev)
    wp, wn = (None, 0) if ws is None else (_flat(ws, 0, torch.uint8, "ws", dev), ws.numel())
    _call("moe_linear_attention", _gpu(q), stream, ctypes.byref(l), qp, ldq, kp, ldk, vp, ldv, gp, ldg, cp, n, si, sli, ni, so,
          slo, no, op, ldo, T, wp, wn)


def moe_linear_attention_step(l: MoeLinear, q, k, v, log_decay, o, T: int, state_in=None, slots_in=None, state_out=None,
                              slots_out=None, stream=None):
    """One token of each of T sequences (decode): moe_linear_attention with a token a sequence."""
    dev, bits, hk, hv, dk, dv = q.get_device(), _types_of(_BF16_BITS), l.qk_heads, l.v_heads, l.qk_dim, l.v_dim
    qp, ldq = _heads(q, T, hk, dk, bits, dev, "q")
    kp, ldk = _heads(k, T, hk, dk, bits, dev, "k")
    vp, ldv = _heads(v, T, hv, dv, bits, dev, "v")
    op, ldo = _heads(o, T, hv, dv, bits, dev, "o")
    gp, ldg = _decay(log_decay, T, hv, dev)
    si, sli, ni = _state(state_in, slots_in, l, hv, T, dev, "in")
    so, slo, no = _state(state_out, slots_out, l, hv, T, dev, "out")
    _call("moe_linear_attention_step", dev if dev >= 0 else _gpu(q), stream, ctypes.byref(l), qp, ldq, kp, ldk, vp, ldv, gp, ldg,
          si, sli, ni, so, slo, no, op, ldo, T)


def gated_norm(H, dtype=BF16, weight_dtype=None, normalize=True, group=0, eps=1e-6, weight_offset=0.0, gate=GATE_NONE,
               gate_per_row=False, scale=1.0, next_norm=False, next_eps=1e-6, next_offset=0.0, out8=OUT8_NONE,
               out8_group=0) -> MoeBlockNorm:
    """What moe_gated_norm does to rows of H values (dtype: a torch type or BF16 / F16 / F32)."""
    code = _type_code(dtype)
    return MoeBlockNorm(H, code, code if weight_dtype is None else _type_code(weight_dtype), int(normalize), group, gate,
                        int(gate_per_row), int(next_norm), out8, out8_group, eps, weight_offset, scale, next_eps,
                        next_offset)


def moe_gated_norm(n: MoeBlockNorm, x, T: int, weight=None, gate=None, channel_scale=None, residual=None,
                   next_weight=None, h_out=None, y=None, q=None, scales=None, stream=None):
    """h = residual + scale channel_scale act(gate) norm(x), y = norm(h) of T rows, and q, scales: that in 8 bits."""
    H, types, wtypes, dev = n.H, _types_of(n.dtype), _types_of(n.weight_dtype), x.get_device()
    xp, ldx = _rows(x, T, H, types, dev, "x")
    gp = rp = hp = yp = qp = sp = None
    ldg = ldr = ldh = ldy = ldq = 0
    if gate is not None:
        if n.gate_per_row and gate.dim() == 1:
            gate = gate[:, None]
        gp, ldg = _rows(gate, T, 1 if n.gate_per_row else H, types, dev, "gate")
    if residual is not None:
        rp, ldr = _rows(residual, T, H, types, dev, "residual")
    if h_out is not None:
        hp, ldh = _rows(h_out, T, H, types, dev, "h_out")
    if y is not None:
        yp, ldy = _rows(y, T, H, types, dev, "y")
    if q is not None:
        qp, ldq = _rows(q, T, H, _types_of(BITS8 + (n.out8 or OUT8_INT8)), dev, "q")
    if scales is not None:
        sp = _flat(scales, T * (H // n.out8_group if n.out8_group else 1), _types_of(F32)[0], "scales", dev)
    wp = None if weight is None else _flat(weight, n.group or H, wtypes[0], "weight", dev)
    cp = None if channel_scale is None else _flat(channel_scale, H, wtypes[0], "channel_scale", dev)
    np_ = None if next_weight is None else _flat(next_weight, H, wtypes[0], "next_weight", dev)
    _call("moe_gated_norm", _gpu(x), stream, ctypes.byref(n), xp, ldx, wp, gp, ldg, cp, rp, ldr, np_, hp, ldh, yp, ldy, qp,
          ldq, sp, T)
