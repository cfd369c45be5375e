"""GB300-native Gated DeltaNet (GDN) layer hot path.

A thin ctypes binding over ``libgdn.so`` (the C ABI of ``include/gdn.h``):
the functions below carry the C entry points' names and only marshal
arguments -- torch tensors in, device pointers and sizes out. Every step of
the layer runs in the library's CUDA kernels; there is no Python or CPU
fallback. If the library is missing or fails to load, every call raises.

torch is used only for device memory, streams and dtypes.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import sysconfig
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")
# (build.binding_path; its name says which torch and which Python it links)
BINDING_PATH = os.path.join(_PKG, f"_binding.{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA = 0, 1, 2, 3
GDN_ERR_SCRATCH_LIMIT = 4
GDN_NOALLOC_SCRATCH_BYTES = 64 << 20
GDN_BF16, GDN_F32 = 0, 1
GDN_CONV_DIM_FIRST, GDN_CONV_TAP_FIRST = 0, 1
GDN_GATE_FUSED, GDN_GATE_DIRECT = 0, 1
GDN_DEVERR_SLOT_RANGE, GDN_DEVERR_SEQLENS, GDN_DEVERR_TIMEOUT = 1, 2, 4
GDN_DEVERR_BLOCKS, GDN_DEVERR_BLOCK_RANGE = 8, 16
GDN_TEST_FAULT_NONE, GDN_TEST_FAULT_DECODE_CONSUMER, GDN_TEST_FAULT_PREFILL_PASS = 0, 1, 2
GDN_TEST_FAULT_ATTENTION = 4
GDN_ACT_SILU, GDN_ACT_SIGMOID = 0, 1
GDN_ROPE_HALVES, GDN_ROPE_INTERLEAVED = 0, 1
GDN_ROPE_PLAIN, GDN_ROPE_LINEAR, GDN_ROPE_NTK, GDN_ROPE_YARN = 0, 1, 2, 3


class GDNError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class gdn_dims(ctypes.Structure):
    _fields_ = [("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
                ("conv_width", ctypes.c_int32), ("state_bf16", ctypes.c_int32)]


@dataclass(frozen=True)
class Dims:
    Hk: int
    Hv: int
    dk: int
    dv: int
    W: int = 4

    @property
    def D(self) -> int:
        return 2 * self.Hk * self.dk + self.Hv * self.dv

    def c(self, state_bf16: bool = False) -> gdn_dims:
        return gdn_dims(self.Hk, self.Hv, self.dk, self.dv, self.W, int(bool(state_bf16)))


class gdn_cache_dims(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32)]


class gdn_output_gate(ctypes.Structure):
    _fields_ = [("z", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("weight_offset", ctypes.c_float), ("eps", ctypes.c_float),
                ("act", ctypes.c_int32)]


class OutputGate:
    """The GDN block's output gate (include/gdn.h, gdn_output_gate): out = o / rms(o) *
    (weight + weight_offset) * act(z) per value head. z: bf16 [tokens, Hv, dv] on the device;
    weight: f32 [dv] on the device; act "silu" or "sigmoid"."""

    def __init__(self, z, weight, *, weight_offset=0.0, eps=1e-6, act="silu"):
        if z.dtype != torch.bfloat16 or weight.dtype != torch.float32:
            raise ValueError("z must be bfloat16 and weight float32")
        self.z, self.weight = z, weight
        self._c = gdn_output_gate(_ptr(z), _ptr(weight), float(weight_offset), float(eps),
                                  {"silu": GDN_ACT_SILU, "sigmoid": GDN_ACT_SIGMOID}[act])

    def ref(self):
        return ctypes.byref(self._c)


def _gate(gate):
    return None if gate is None else gate.ref()


def _sdims(dims: "Dims", ssm_state) -> gdn_dims:
    """dims for a call: the state storage type follows the pool tensor's dtype."""
    if ssm_state.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("the recurrent state pool must be float32 or bfloat16")
    return dims.c(ssm_state.dtype == torch.bfloat16)


_lib = None


def lib():
    """Load libgdn.so (raises if it is absent: build it with build.build_library())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: the CUDA library must be built "
                               "(gated_deltanet_linear_gdn_gb300.build.build_library())")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        L.gdn_conv_update.restype = I32
        L.gdn_conv_update.argtypes = [P, P, I32, I32, P, P, I32, P, I32, I32, I32, I32, P, P, P]
        L.gdn_decode_step.restype = I32
        L.gdn_decode_step.argtypes = [P, P, P, I32, P, P, P, P, I32, P, I32, I32, P, P, I32, I32,
                                      gdn_dims, F, I32, P, P, I32, P, P]
        L.gdn_chunked_prefill_workspace_size.restype = ctypes.c_size_t
        L.gdn_chunked_prefill_workspace_size.argtypes = [I32, I32, gdn_dims, I32]
        L.gdn_chunked_prefill.restype = I32
        L.gdn_chunked_prefill.argtypes = [P, P, P, I32, P, P, P, P, I32, P, I32, I32, P, P, P, P,
                                          I32, I32, I32, gdn_dims, F, I32, I32, P, P, I32, P,
                                          ctypes.c_size_t, P, P]
        L.gdn_chunked_prefill_noalloc.restype = I32
        L.gdn_chunked_prefill_noalloc.argtypes = [P, P, P, I32, P, P, P, P, I32, P, I32, I32, P,
                                                  P, P, P, I32, I32, I32, gdn_dims, F, I32, I32,
                                                  P, P, I32, P, P]
        L.gdn_mixed_step.restype = I32
        L.gdn_mixed_step.argtypes = [P, P, P, I32, P, P, P, P, I32, P, I32, I32, P, P, I32, P, P,
                                     I32, I32, I32, gdn_dims, F, I32, I32, P, P, I32, P,
                                     ctypes.c_size_t, P, P]
        L.gdn_decode_graph_create.restype = I32
        L.gdn_decode_graph_create.argtypes = [P, P, P, I32, P, P, P, P, I32, P, I32, I32, P, P,
                                              I32, I32, gdn_dims, F, I32, P, P, I32, P,
                                              ctypes.POINTER(ctypes.c_void_p)]
        L.gdn_graph_launch.restype = I32
        L.gdn_graph_launch.argtypes = [P, P]
        L.gdn_graph_destroy.restype = None
        L.gdn_graph_destroy.argtypes = [P]
        I64, SZ = ctypes.c_int64, ctypes.c_size_t
        L.gdn_cache_tables.restype = I32
        L.gdn_cache_tables.argtypes = [P, P, I32, P, I32, P, I32, P, P, I32, I32, P, P, P, P, P, P]
        L.gdn_cache_append.restype = I32
        L.gdn_cache_append.argtypes = [P, I64, P, I64, P, I32, P, P, P, P, I32, gdn_cache_dims, P,
                                       P]
        L.gdn_attn_decode_workspace_size.restype = SZ
        L.gdn_attn_decode_workspace_size.argtypes = [I32, I32, gdn_cache_dims]
        L.gdn_attn_decode.restype = I32
        L.gdn_attn_decode.argtypes = [P, I64, P, P, P, P, I32, P, I32, P, I32, gdn_cache_dims, F, P,
                                      P, SZ, P, P]
        L.gdn_attn_prefill_workspace_size.restype = SZ
        L.gdn_attn_prefill_workspace_size.argtypes = [I32, I32, I32, gdn_cache_dims]
        L.gdn_attn_prefill.restype = I32
        L.gdn_attn_prefill.argtypes = [P, I64, P, P, P, P, P, I32, P, I32, P, I32, I32,
                                       gdn_cache_dims, F, P, P, SZ, P, P]
        L.gdn_rope.restype = I32
        L.gdn_rope.argtypes = [P, I64, P, I64, P, I32, I32, I32, I32, I32, I32, P, F, P, I64, P, I64, P]
        L.gdn_rope_frequencies.restype = I32
        L.gdn_rope_frequencies.argtypes = [I32, ctypes.c_double, I32, ctypes.c_double, I32, P, P]
        L.gdn_rope_turns.restype = I32
        L.gdn_rope_turns.argtypes = [P, I32, P]
        L.gdn_cache4_append.restype = I32
        L.gdn_cache4_append.argtypes = [P, I64, P, I64, P, I32, P, P, P, P, I32, gdn_cache_dims, P, P]
        L.gdn_cache4_read.restype = I32
        L.gdn_cache4_read.argtypes = [P, P, P, P, I32, P, I32, gdn_cache_dims, P, I64, P, I64, P, P]
        L.gdn_attn4_decode_workspace_size.restype = SZ
        L.gdn_attn4_decode_workspace_size.argtypes = [I32, I32, gdn_cache_dims]
        L.gdn_attn4_decode.restype = I32
        L.gdn_attn4_decode.argtypes = L.gdn_attn_decode.argtypes
        L.gdn_attn4_prefill_workspace_size.restype = SZ
        L.gdn_attn4_prefill_workspace_size.argtypes = [I32, I32, I32, I32, gdn_cache_dims]
        L.gdn_attn4_prefill.restype = I32
        L.gdn_attn4_prefill.argtypes = [P, I64, P, P, P, P, P, I32, P, I32, P, I32, I32, I32,
                                        gdn_cache_dims, F, P, P, SZ, P, P]
        L.gdn_validate_slots.restype = I32
        L.gdn_validate_slots.argtypes = [P, I32, I32]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_status_string.argtypes = [I32]
        L.gdn_testing_set_fault.restype = I32
        L.gdn_testing_set_fault.argtypes = [I32]
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if t.numel() and not t.is_cuda:
            raise ValueError("device tensors expected")
        if t.numel() and not t.is_contiguous():
            raise ValueError("contiguous tensors expected")
        return ctypes.c_void_p(t.data_ptr()) if t.numel() else None
    return ctypes.c_void_p(int(t))


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(torch._C._cuda_getDevice())  # current_stream() without its object
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dt(t) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _check(status: int):
    if status != GDN_OK:
        raise GDNError(status, lib().gdn_status_string(status).decode())


def status_string(status: int) -> str:
    return lib().gdn_status_string(int(status)).decode()


# --------------------------------------------------------------------------- entry points

def gdn_conv_update(x, conv_state, weight, bias, slot, out, *, silu=True,
                    conv_layout=GDN_CONV_DIM_FIRST, err=None, stream=None):
    """Decode conv update (in place on conv_state). x, out: [B, D] bf16."""
    B, D = x.shape
    _check(lib().gdn_conv_update(_ptr(x), _ptr(conv_state), _dt(conv_state), int(conv_layout),
                                 _ptr(weight), _ptr(bias), int(bool(silu)), _ptr(slot), B, D,
                                 weight.shape[1], conv_state.shape[0], _ptr(out), _ptr(err),
                                 _stream(stream)))


def _gate_mode(a):
    return GDN_GATE_DIRECT if a.dtype == torch.float32 else GDN_GATE_FUSED


def gdn_decode_step(mixed_qkv, a, b, A_log, dt_bias, conv_weight, conv_bias, conv_state,
                    ssm_state, slot, out, dims: Dims, *, silu=True,
                    conv_layout=GDN_CONV_DIM_FIRST, scale=None, qk_l2norm=True, gate=None,
                    err=None, stream=None):
    """One fused decode step (conv state and ssm_state updated in place).

    a, b: bf16 [B, Hv] (fused gates with A_log, dt_bias) or f32 g, beta (direct).
    gate: an OutputGate, or None for the plain core output."""
    B = mixed_qkv.shape[0]
    scale = dims.dk ** -0.5 if scale is None else scale
    conv_dt = _dt(conv_state) if conv_state is not None else GDN_BF16
    _check(lib().gdn_decode_step(
        _ptr(mixed_qkv), _ptr(a), _ptr(b), _gate_mode(a), _ptr(A_log), _ptr(dt_bias),
        _ptr(conv_weight), _ptr(conv_bias), int(bool(silu)), _ptr(conv_state), conv_dt,
        int(conv_layout), _ptr(ssm_state), _ptr(slot), B, ssm_state.shape[0],
        _sdims(dims, ssm_state), float(scale), int(bool(qk_l2norm)), _gate(gate), _ptr(out),
        _dt(out), _ptr(err), _stream(stream)))


def gdn_chunked_prefill_workspace_size(total_tokens, num_seqs, dims: Dims, chunk=64) -> int:
    return int(lib().gdn_chunked_prefill_workspace_size(int(total_tokens), int(num_seqs),
                                                        dims.c(), int(chunk)))


def gdn_chunked_prefill(mixed_qkv, a, b, A_log, dt_bias, conv_weight, conv_bias, conv_state,
                        ssm_state, cu_seqlens, slot, has_initial_state, out, workspace,
                        dims: Dims, *, chunk=64, silu=True, conv_layout=GDN_CONV_DIM_FIRST,
                        scale=None, qk_l2norm=True, gate=None, err=None, stream=None):
    """Chunked prefill over packed sequences (states updated in place by slot)."""
    T = mixed_qkv.shape[0]
    N = slot.shape[0]
    scale = dims.dk ** -0.5 if scale is None else scale
    conv_dt = _dt(conv_state) if conv_state is not None else GDN_BF16
    _check(lib().gdn_chunked_prefill(
        _ptr(mixed_qkv), _ptr(a), _ptr(b), _gate_mode(a), _ptr(A_log), _ptr(dt_bias),
        _ptr(conv_weight), _ptr(conv_bias), int(bool(silu)), _ptr(conv_state), conv_dt,
        int(conv_layout), _ptr(ssm_state), _ptr(cu_seqlens), _ptr(slot),
        _ptr(has_initial_state), N, T, ssm_state.shape[0], _sdims(dims, ssm_state),
        float(scale), int(bool(qk_l2norm)), int(chunk), _gate(gate), _ptr(out), _dt(out),
        _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream)))


def gdn_chunked_prefill_noalloc(mixed_qkv, a, b, A_log, dt_bias, conv_weight, conv_bias,
                                conv_state, ssm_state, cu_seqlens, slot, has_initial_state, out,
                                dims: Dims, *, chunk=64, silu=True,
                                conv_layout=GDN_CONV_DIM_FIRST, scale=None, qk_l2norm=True,
                                gate=None, err=None, stream=None):
    """gdn_chunked_prefill without a caller workspace, for callers that cannot allocate device
    memory: the library's fixed GDN_NOALLOC_SCRATCH_BYTES array serves as the workspace.
    Raises GDNError(GDN_ERR_SCRATCH_LIMIT) when the call needs more than that. Calls that may
    overlap on the GPU share the array and race; make the first call on a device before any
    stream capture."""
    T = mixed_qkv.shape[0]
    N = slot.shape[0]
    scale = dims.dk ** -0.5 if scale is None else scale
    conv_dt = _dt(conv_state) if conv_state is not None else GDN_BF16
    _check(lib().gdn_chunked_prefill_noalloc(
        _ptr(mixed_qkv), _ptr(a), _ptr(b), _gate_mode(a), _ptr(A_log), _ptr(dt_bias),
        _ptr(conv_weight), _ptr(conv_bias), int(bool(silu)), _ptr(conv_state), conv_dt,
        int(conv_layout), _ptr(ssm_state), _ptr(cu_seqlens), _ptr(slot),
        _ptr(has_initial_state), N, T, ssm_state.shape[0], _sdims(dims, ssm_state),
        float(scale), int(bool(qk_l2norm)), int(chunk), _gate(gate), _ptr(out), _dt(out),
        _ptr(err), _stream(stream)))


def gdn_mixed_step(mixed_qkv, a, b, A_log, dt_bias, conv_weight, conv_bias, conv_state,
                   ssm_state, slot, num_decode, cu_seqlens, has_initial_state, out, workspace,
                   dims: Dims, *, chunk=64, silu=True, conv_layout=GDN_CONV_DIM_FIRST,
                   scale=None, qk_l2norm=True, gate=None, err=None, stream=None):
    """A step of num_decode decode rows followed by prefill sequences, packed in one token
    array (include/gdn.h, gdn_mixed_step). slot: decode rows' slots then one per prefill
    sequence; cu_seqlens: offsets within the prefill part; workspace: the prefill part's."""
    nd = int(num_decode)
    N = slot.shape[0] - nd
    T = mixed_qkv.shape[0] - nd
    scale = dims.dk ** -0.5 if scale is None else scale
    conv_dt = _dt(conv_state) if conv_state is not None else GDN_BF16
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().gdn_mixed_step(
        _ptr(mixed_qkv), _ptr(a), _ptr(b), _gate_mode(a), _ptr(A_log), _ptr(dt_bias),
        _ptr(conv_weight), _ptr(conv_bias), int(bool(silu)), _ptr(conv_state), conv_dt,
        int(conv_layout), _ptr(ssm_state), _ptr(slot), nd, _ptr(cu_seqlens),
        _ptr(has_initial_state), N, T, ssm_state.shape[0], _sdims(dims, ssm_state),
        float(scale), int(bool(qk_l2norm)), int(chunk), _gate(gate), _ptr(out), _dt(out),
        _ptr(workspace), ws_bytes, _ptr(err), _stream(stream)))


# ------------------------------------------------- paged 8-bit cache and its attention
#
# A step makes these calls once per layer, and the smallest take a few microseconds on the GPU:
# pointers go to the library as plain integers and shapes are checked once.

_I32, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32
_E4M3 = (torch.float8_e4m3fn, torch.uint8)


def _dense(t, dtype, shape, name):
    """The address of a dense device tensor of this type and shape."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, not {t.dtype} "
                         f"{tuple(t.shape)}")
    if not (t.is_cuda and t.is_contiguous()) and t.numel():
        raise ValueError(f"{name} must be a contiguous device tensor")
    return t.data_ptr()


def _tokens(t, shape, name):
    """(address, elements from one token to the next) of a bf16 tensor [tokens, heads, d] whose
    heads are dense; the token stride is free (a slice of a wider projection)."""
    if t.dtype is not _BF16 or t.shape != shape:
        raise ValueError(f"{name} must be bfloat16 of shape {tuple(shape)}, not {t.dtype} "
                         f"{tuple(t.shape)}")
    n, heads, d = shape
    if n == 0:
        return 0, heads * d
    step, of_head, of_d = t.stride()
    if not t.is_cuda or (of_d != 1 and d > 1) or (of_head != d and heads > 1):
        raise ValueError(f"{name} must be a device tensor with dense heads")
    return t.data_ptr(), (step if n > 1 else heads * d)  # (one token: its stride means nothing)


@functools.lru_cache(maxsize=None)
def _cache_dims(q_heads, kv_heads, head_dim, block_size):
    return gdn_cache_dims(q_heads, kv_heads, head_dim, block_size)


def _cache(k_cache, v_cache, k_scale, v_scale):
    """The cache's addresses and shape [num_blocks, Hkv, block_size, head_dim]."""
    shape, dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or dtype not in _E4M3:
        raise ValueError("the caches must be float8_e4m3fn (or its bytes) [num_blocks, Hkv, "
                         "block_size, head_dim]")
    return (_dense(k_cache, dtype, shape, "k_cache"), _dense(v_cache, dtype, shape, "v_cache"),
            _dense(k_scale, _F32, shape[:2], "k_scale"),
            _dense(v_scale, _F32, shape[:2], "v_scale")), shape


def gdn_cache_tables(lens_old, lens_new, block_table, free_ring, pool, pool_out, cu_tokens,
                     slot_map, positions, lens, block_size, *, err=None, stream=None):
    """The step's block tables, slots and positions from its requests' lengths (include/gdn.h).
    block_table [B, max_blocks], free_ring [num_blocks], pool and pool_out [2] (head, free
    count): in place; writes cu_tokens [B + 1], slot_map and positions [capacity], lens [B]."""
    (B,), (T,), (N,), W = lens_old.shape, slot_map.shape, free_ring.shape, block_table.shape[-1]
    _check(lib().gdn_cache_tables(
        _dense(lens_old, _I32, (B,), "lens_old"), _dense(lens_new, _I32, (B,), "lens_new"), B,
        _dense(block_table, _I32, (B, W), "block_table"), W,
        _dense(free_ring, _I32, (N,), "free_ring"), N, _dense(pool, _I32, (2,), "pool"),
        _dense(pool_out, _I32, (2,), "pool_out"), block_size, T,
        _dense(cu_tokens, _I32, (B + 1,), "cu_tokens"), _dense(slot_map, _I32, (T,), "slot_map"),
        _dense(positions, _I32, (T,), "positions"), _dense(lens, _I32, (B,), "lens"),
        _ptr(err), _stream(stream)))


def gdn_cache_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, *, err=None,
                     stream=None):
    """Writes k, v [T, Hkv, d] (bf16, any token stride) into the 8-bit cache at slot_map [T]."""
    addresses, (NB, H, bs, d) = _cache(k_cache, v_cache, k_scale, v_scale)
    (T,) = slot_map.shape
    _check(lib().gdn_cache_append(*_tokens(k, (T, H, d), "k"), *_tokens(v, (T, H, d), "v"),
                                  _dense(slot_map, _I32, (T,), "slot_map"), T, *addresses, NB,
                                  _cache_dims(H, H, d, bs), _ptr(err), _stream(stream)))


def gdn_attn_decode_workspace_size(batch, max_blocks, num_q_heads, num_kv_heads, head_dim,
                                   block_size) -> int:
    return int(lib().gdn_attn_decode_workspace_size(
        int(batch), int(max_blocks),
        gdn_cache_dims(num_q_heads, num_kv_heads, head_dim, block_size)))


def gdn_attn_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, out, workspace, *,
                    scale=None, err=None, stream=None):
    """Attention of one token per request over the 8-bit cache. q, out: [B, Hq, d] bf16 (q with
    any token stride); scale: head_dim ** -0.5 if None."""
    addresses, (NB, H, bs, d) = _cache(k_cache, v_cache, k_scale, v_scale)
    B, Hq, W = q.shape[0], q.shape[1], block_table.shape[-1]
    _check(lib().gdn_attn_decode(
        *_tokens(q, (B, Hq, d), "q"), *addresses, NB,
        _dense(block_table, _I32, (B, W), "block_table"), W, _dense(lens, _I32, (B,), "lens"), B,
        _cache_dims(Hq, H, d, bs), d ** -0.5 if scale is None else scale,
        _dense(out, _BF16, (B, Hq, d), "out"), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream)))


def gdn_attn_prefill_workspace_size(total_tokens, num_seqs, max_blocks, num_q_heads,
                                    num_kv_heads, head_dim, block_size) -> int:
    return int(lib().gdn_attn_prefill_workspace_size(
        int(total_tokens), int(num_seqs), int(max_blocks),
        gdn_cache_dims(num_q_heads, num_kv_heads, head_dim, block_size)))


def gdn_attn_prefill(q, cu_tokens, k_cache, v_cache, k_scale, v_scale, block_table, lens, out,
                     workspace, *, scale=None, err=None, stream=None):
    """Causal attention of packed prompt tokens over the 8-bit cache, which holds them already.
    q, out: [T, Hq, d] bf16 (q with any token stride); cu_tokens [B + 1], lens [B] int32."""
    addresses, (NB, H, bs, d) = _cache(k_cache, v_cache, k_scale, v_scale)
    T, Hq, B, W = q.shape[0], q.shape[1], lens.shape[0], block_table.shape[-1]
    _check(lib().gdn_attn_prefill(
        *_tokens(q, (T, Hq, d), "q"), _dense(cu_tokens, _I32, (B + 1,), "cu_tokens"), *addresses,
        NB, _dense(block_table, _I32, (B, W), "block_table"), W,
        _dense(lens, _I32, (B,), "lens"), B, T, _cache_dims(Hq, H, d, bs),
        d ** -0.5 if scale is None else scale, _dense(out, _BF16, (T, Hq, d), "out"),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err),
        _stream(stream)))


# ---------------------------------------------- rotary positions, the cache in 4 bits

# These calls' arguments are marshalled in C++ (csrc/gdn_binding.cpp): the smallest take 2 us on the GPU.


class RopeTable:
    """The frequencies of a model's rotary positions, as gdn_rope reads them (include/gdn.h, gdn_rope_frequencies): scaling
    "none", "linear", "ntk" or "yarn" by `factor`, trained_len the positions that the model was trained on ("yarn" alone); or
    `freqs`, rot_dim / 2 frequencies of its own with the `factor` of the rotated values. Kept on `device`."""

    def __init__(self, rot_dim, *, base=10000.0, scaling="none", factor=1.0, trained_len=0, freqs=None, device="cuda"):
        if rot_dim <= 0 or rot_dim % 2:
            raise ValueError("rot_dim must be even and positive")
        half = rot_dim // 2
        w, f = (ctypes.c_double * half)(), ctypes.c_float(float(factor))
        if freqs is None:
            kinds = {"none": GDN_ROPE_PLAIN, "linear": GDN_ROPE_LINEAR, "ntk": GDN_ROPE_NTK, "yarn": GDN_ROPE_YARN}
            if scaling not in kinds:
                raise ValueError(f"scaling must be one of {', '.join(kinds)}, not {scaling!r}")
            kind = kinds[scaling]
            _check(lib().gdn_rope_frequencies(rot_dim, float(base), kind, float(factor), int(trained_len), w, ctypes.byref(f)))
        else:
            if len(freqs) != half:
                raise ValueError(f"freqs must have rot_dim / 2 = {half} frequencies")
            w[:] = [float(x) for x in freqs]
        turns = (ctypes.c_uint64 * half)()
        _check(lib().gdn_rope_turns(w, half, turns))
        self.rot_dim, self.factor, self.freqs = rot_dim, f.value, list(w)
        self.turns = torch.frombuffer(bytearray(turns), dtype=torch.int64).to(device)


_marshal = None


def _binding():
    """The marshalling functions of the binding in C++, bound to the library's entry points. Raises if it is absent, or there for
    another torch or Python alone."""
    global _marshal
    if _marshal is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is missing: it must be built, for this torch and this Python "
                               "(gated_deltanet_linear_gdn_gb300.build.build_library())")
        spec = importlib.util.spec_from_file_location(__name__ + "._binding", BINDING_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        L = lib()
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.gdn_rope, L.gdn_cache4_append, L.gdn_cache4_read, L.gdn_attn4_decode, L.gdn_attn4_prefill)))
        _marshal = m
    return _marshal


def _raw(stream):
    """A stream as an address; None for the current one."""
    return stream if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def gdn_rope(q, k, positions, q_out, k_out, rope: RopeTable, *, interleaved=False, stream=None):
    """Rotary positions of q [T, Hq, d] and k [T, Hkv, d] (bf16, any token stride) into q_out and k_out (which may be q and k
    themselves). positions [T] int32; k and k_out may be None."""
    status = (_marshal or _binding()).rope(q, k, positions, q_out, k_out, rope.turns, rope.rot_dim, rope.factor, bool(interleaved),
                                           _raw(stream))
    if status:
        _check(status)


def gdn_cache4_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, *, err=None, stream=None):
    """Writes k, v [T, Hkv, d] (bf16, any token stride) into the 4-bit cache at slot_map [T] (include/gdn.h). k_cache
    [num_blocks, Hkv, block_size, d / 2] and v_cache [num_blocks, Hkv, block_size / 2, d] uint8; the scales [num_blocks, Hkv,
    block_size, d / 32] float8_e8m0fnu or its bytes."""
    status = (_marshal or _binding()).cache4_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, err, _raw(stream))
    if status:
        _check(status)


def gdn_cache4_read(k_cache, v_cache, k_scale, v_scale, slot_map, k, v, *, err=None, stream=None):
    """The values of the 4-bit cache's tokens at slot_map [T], into k and v [T, Hkv, d] (bf16, any token stride)."""
    status = (_marshal or _binding()).cache4_read(k_cache, v_cache, k_scale, v_scale, slot_map, k, v, err, _raw(stream))
    if status:
        _check(status)


def gdn_attn4_decode_workspace_size(batch, max_blocks, num_q_heads, num_kv_heads, head_dim, block_size) -> int:
    return int(lib().gdn_attn4_decode_workspace_size(
        int(batch), int(max_blocks), gdn_cache_dims(num_q_heads, num_kv_heads, head_dim, block_size)))


def gdn_attn4_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, out, workspace, *, scale=None, err=None,
                     stream=None):
    """Attention of one token per request over the 4-bit cache. q, out: [B, Hq, d] bf16 (q with any token stride); scale:
    head_dim ** -0.5 if None."""
    status = (_marshal or _binding()).attn4_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, out, workspace, scale,
                                                   err, _raw(stream))
    if status:
        _check(status)


def gdn_attn4_prefill_workspace_size(total_tokens, num_seqs, max_blocks, num_q_heads, num_kv_heads, head_dim, block_size, *,
                                     held_blocks=None) -> int:
    """held_blocks: a bound on the blocks that the call's requests hold together; num_seqs * max_blocks if None."""
    return int(lib().gdn_attn4_prefill_workspace_size(
        int(total_tokens), int(num_seqs), int(max_blocks),
        min(num_seqs * max_blocks, 0x7fffffff) if held_blocks is None else int(held_blocks),
        gdn_cache_dims(num_q_heads, num_kv_heads, head_dim, block_size)))


def gdn_attn4_prefill(q, cu_tokens, k_cache, v_cache, k_scale, v_scale, block_table, lens, out, workspace, *,
                      held_blocks=None, scale=None, err=None, stream=None):
    """Causal attention of packed prompt tokens over the 4-bit cache, which holds them already. q, out: [T, Hq, d] bf16 (q
    with any token stride); cu_tokens [B + 1], lens [B] int32; held_blocks as for the workspace's size."""
    status = (_marshal or _binding()).attn4_prefill(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, out, workspace, scale,
                                                    err, _raw(stream), cu_tokens, held_blocks)
    if status:
        _check(status)


class DecodeGraph:
    """A captured decode step over fixed buffers (gdn_decode_graph_create). The tensors passed
    at creation are kept referenced here: write each step's inputs into them, then launch()."""

    def __init__(self, mixed_qkv, a, b, A_log, dt_bias, conv_weight, conv_bias, conv_state,
                 ssm_state, slot, out, dims: Dims, *, silu=True, conv_layout=GDN_CONV_DIM_FIRST,
                 scale=None, qk_l2norm=True, gate=None, err=None):
        self._keep = (mixed_qkv, a, b, A_log, dt_bias, conv_weight, conv_bias, conv_state,
                      ssm_state, slot, out, err, gate)
        B = mixed_qkv.shape[0]
        scale = dims.dk ** -0.5 if scale is None else scale
        conv_dt = _dt(conv_state) if conv_state is not None else GDN_BF16
        h = ctypes.c_void_p()
        _check(lib().gdn_decode_graph_create(
            _ptr(mixed_qkv), _ptr(a), _ptr(b), _gate_mode(a), _ptr(A_log), _ptr(dt_bias),
            _ptr(conv_weight), _ptr(conv_bias), int(bool(silu)), _ptr(conv_state), conv_dt,
            int(conv_layout), _ptr(ssm_state), _ptr(slot), B, ssm_state.shape[0],
            _sdims(dims, ssm_state), float(scale), int(bool(qk_l2norm)), _gate(gate), _ptr(out),
            _dt(out), _ptr(err), ctypes.byref(h)))
        self._h = h

    def launch(self, stream=None):
        _check(lib().gdn_graph_launch(self._h, _stream(stream)))

    def close(self):
        if getattr(self, "_h", None):
            lib().gdn_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gdn_testing_set_fault(mode: int) -> None:
    """Test hook (include/gdn_testing.h): make one bounded wait of the kernels run out."""
    _check(lib().gdn_testing_set_fault(int(mode)))


def gdn_validate_slots(host_slot, num_slots) -> int:
    """Host-side duplicate / range check of a host slot table (0 ok, 1 range, 2 repeat)."""
    import numpy as np
    s = np.ascontiguousarray(host_slot, dtype=np.int32)
    return int(lib().gdn_validate_slots(s.ctypes.data_as(ctypes.c_void_p), s.size,
                                        int(num_slots)))
