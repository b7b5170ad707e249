"""ctypes binding of libhsnf4.so (the C ABI in include/hsnf4.h).

Argument marshalling only: torch tensors provide device memory and streams,
every step of the path runs in the library's CUDA kernels.  There is no
fallback -- if the library or a CUDA device is missing, calls raise.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, Structure, c_char_p, c_float, c_int, c_int64, c_size_t, c_uint32, \
    c_uint64, c_void_p
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhsnf4.so")
MAX_PROJ = 8

OK, ERR_INVALID, ERR_OOM, ERR_CUDA, ERR_TIMEOUT, ERR_STATE, ERR_DEVICE = range(7)
BASE_NF4, BASE_BF16 = 0, 1  # formats of the frozen base weight


class Nf4WeightC(Structure):
    _fields_ = [("codes", c_void_p), ("absmax", c_void_p), ("n_out", c_int64), ("k_in", c_int64),
                ("format", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_DROPOUT_FIELDS = [("dropout_p", c_float), ("reserved", ctypes.c_uint32),
                   ("dropout_seed", c_uint64), ("dropout_offset", c_uint64)]


class FwdArgs(Structure):
    _fields_ = [("W", Nf4WeightC), ("X", c_void_p), ("A", c_void_p), ("B", c_void_p),
                ("Y", c_void_p), ("t_save", c_void_p)] + _DROPOUT_FIELDS


class BwdArgs(Structure):
    _fields_ = [("W", Nf4WeightC), ("X", c_void_p), ("t_save", c_void_p), ("A", c_void_p),
                ("B", c_void_p), ("dY", c_void_p), ("dX", c_void_p), ("dA", c_void_p),
                ("dB", c_void_p)] + _DROPOUT_FIELDS


class LayerDesc(Structure):
    _fields_ = [("n_proj", c_int), ("n_out", c_int64 * MAX_PROJ), ("k_in", c_int64 * MAX_PROJ),
                ("base_format", c_int)]


# int gather(void *slot, size_t shard_bytes, int world, int block, void *copy_stream, void *user)
GATHER_FN = ctypes.CFUNCTYPE(c_int, c_void_p, c_size_t, c_int, c_int, c_void_p, c_void_p)


class StreamConfig(Structure):
    _fields_ = [("block_size", c_int), ("enable_prefetch", c_int), ("reuse_resident", c_int),
                ("poison_on_release", c_int), ("n_slots", c_int), ("shard_world", c_int),
                ("shard_rank", c_int), ("gather", GATHER_FN), ("gather_user", c_void_p),
                ("shard_slab", c_int)]


class StreamStats(Structure):
    _fields_ = [("h2d_bytes", c_uint64), ("copies", c_uint64), ("reuses", c_uint64),
                ("acquires", c_uint64), ("releases", c_uint64), ("gathers", c_uint64)]


class KernelTime(Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", c_uint64), ("total_ms", ctypes.c_double),
                ("work", ctypes.c_double)]


class GemmPlanInfo(Structure):
    _fields_ = [("stream_k", ctypes.c_int32), ("pairs", ctypes.c_int32),
                ("units", ctypes.c_int32), ("split_tiles", ctypes.c_int32),
                ("total_steps", c_int64), ("max_pair_steps", c_int64),
                ("min_pair_steps", c_int64), ("covered", ctypes.c_int32),
                ("fixup_tiles", ctypes.c_int32)]


ROPE_HALF, ROPE_ADJACENT = 0, 1
ROPE_MAX_PAIRS = 128
GRAD_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class RopeC(Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("pairing", ctypes.c_int32), ("scale", c_float),
                ("inv_freq", c_float * ROPE_MAX_PAIRS), ("axis", ctypes.c_uint8 * ROPE_MAX_PAIRS)]


class PackedAttentionC(Structure):
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("q_stride", c_int64),
                ("k_stride", c_int64), ("v_stride", c_int64), ("cu_q", c_void_p),
                ("cu_k", c_void_p), ("Tq", c_int64), ("Tk", c_int64), ("n_seq", ctypes.c_int32),
                ("H", ctypes.c_int32), ("KV", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("scale", c_float)]


class GradC(Structure):
    _fields_ = [("g", c_void_p), ("out", c_void_p), ("n", c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class GradPlanC(Structure):
    _fields_ = [("table", c_void_p), ("chunks", c_int64), ("elements", c_int64),
                ("n", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class HsNf4Error(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"[{status}] {detail}")
        self.status = status
        self.detail = detail


_lib = None

_SIGS = {
    "hsnf4_status_string": ([c_int], c_char_p),
    "hsnf4_last_error": ([c_char_p, c_size_t], c_int),
    "hsnf4_device_status": ([c_void_p, POINTER(c_uint32)], c_int),
    "hsnf4_inject_fault": ([c_char_p], c_int),
    "hsnf4_selftest_stall": ([c_void_p], c_int),
    "hsnf4_profile": ([c_int], c_int),
    "hsnf4_profile_kinds": ([c_uint32], c_int),
    "hsnf4_kernel_launches": ([], c_uint64),
    "hsnf4_profile_read": ([POINTER(KernelTime), c_int], c_int),
    "nf4_codebook": ([POINTER(c_float)], c_int),
    "nf4_quantize_pack": ([c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p], c_int),
    "nf4_dequant": ([c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_void_p], c_int),
    "lora_merge": ([POINTER(Nf4WeightC), c_void_p, c_void_p, c_int, c_float, c_void_p, c_void_p],
                   c_int),
    "decoder_rmsnorm_fwd": ([c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int64,
                             c_float, c_void_p], c_int),
    "decoder_rmsnorm_bwd": ([c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_int64, c_int64, c_float, c_void_p], c_int),
    "decoder_swiglu_fwd": ([c_void_p, c_void_p, c_void_p, c_int64, c_void_p], c_int),
    "decoder_swiglu_bwd": ([c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p],
                           c_int),
    "decoder_add": ([c_void_p, c_void_p, c_void_p, c_int64, c_void_p], c_int),
    "decoder_attention_fwd": ([c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int,
                               c_int, c_void_p], c_int),
    "decoder_attention_scratch_bytes": ([c_int64, c_int], c_size_t),
    "decoder_attention_bwd": ([c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                               c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int, c_int,
                               c_void_p], c_int),
    "decoder_rope_fwd": ([POINTER(RopeC), c_void_p, c_int64, c_int, c_int] +
                         [c_void_p, c_int64] * 4 + [c_void_p], c_int),
    "decoder_rope_bwd": ([POINTER(RopeC), c_void_p, c_int64, c_int, c_int] +
                         [c_void_p, c_int64] * 4 + [c_void_p], c_int),
    "decoder_attention_packed_fwd": ([POINTER(PackedAttentionC), c_void_p, c_int64, c_void_p,
                                      c_void_p], c_int),
    "decoder_attention_packed_workspace": ([c_int64, c_int64, c_int, c_int, c_int, c_int],
                                           c_size_t),
    "decoder_attention_packed_bwd": ([POINTER(PackedAttentionC), c_void_p, c_int64, c_void_p] +
                                     [c_void_p, c_int64] * 4 + [c_void_p, c_size_t, c_void_p],
                                     c_int),
    "lora_grad_table_bytes": ([c_int], c_size_t),
    "lora_grad_plan": ([POINTER(GradC), c_int, c_void_p, c_size_t, POINTER(GradPlanC), c_void_p],
                       c_int),
    "lora_grad_workspace": ([POINTER(GradPlanC)], c_size_t),
    "lora_grad_norm": ([POINTER(GradPlanC), c_void_p, c_void_p, c_size_t, c_void_p], c_int),
    "lora_grad_clip": ([POINTER(GradPlanC), c_float, c_void_p, c_void_p, c_size_t, c_void_p],
                       c_int),
    "lora_dropout_apply": ([c_void_p, c_int64, c_int64, c_float, c_uint64, c_uint64, c_void_p,
                            c_void_p], c_int),
    "lora_linear_fwd_workspace": ([c_int64, c_int64, c_int64, c_int], c_size_t),
    "lora_linear_bwd_workspace": ([c_int64, c_int64, c_int64, c_int], c_size_t),
    "lora_linear_fwd": ([POINTER(Nf4WeightC), c_void_p, c_int64, c_void_p, c_void_p, c_int, c_float,
                         c_void_p, c_void_p, c_void_p, c_size_t, c_void_p], c_int),
    "lora_linear_bwd": ([POINTER(Nf4WeightC), c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_int,
                         c_float, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                         c_void_p], c_int),
    "lora_linear_fwd_noalloc": ([POINTER(Nf4WeightC), c_void_p, c_int64, c_void_p, c_void_p, c_int,
                                 c_float, c_void_p, c_void_p, c_void_p], c_int),
    "hsnf4_gemm_plan": ([c_int, POINTER(c_int64), POINTER(c_int64), c_int, c_int64, c_int,
                         POINTER(GemmPlanInfo)], c_int),
    "lora_group_fwd_workspace": ([POINTER(FwdArgs), c_int, c_int64, c_int], c_size_t),
    "lora_group_bwd_workspace": ([POINTER(BwdArgs), c_int, c_int64, c_int], c_size_t),
    "lora_group_fwd": ([POINTER(FwdArgs), c_int, c_int64, c_int, c_float, c_void_p, c_size_t,
                        c_void_p], c_int),
    "lora_group_bwd": ([POINTER(BwdArgs), c_int, c_int64, c_int, c_float, c_void_p, c_size_t,
                        c_void_p], c_int),
    "stream_layer_bytes": ([POINTER(LayerDesc), POINTER(c_size_t)], c_int),
    "stream_layer_offsets": ([POINTER(LayerDesc), c_int, POINTER(c_size_t), POINTER(c_size_t)], c_int),
    "stream_slab_bytes": ([POINTER(LayerDesc), c_int, POINTER(c_size_t)], c_int),
    "stream_ring_bytes": ([POINTER(LayerDesc), c_int, c_int, POINTER(c_size_t)], c_int),
    "stream_slot_bytes": ([POINTER(LayerDesc), c_int, c_int, POINTER(c_size_t)], c_int),
    "stream_prefetch_ahead": ([c_void_p, POINTER(c_int), c_int, POINTER(c_int)], c_int),
    "stream_shard_range": ([c_size_t, c_int, c_int, POINTER(c_size_t), POINTER(c_size_t),
                            POINTER(c_size_t)], c_int),
    "stream_shard_slab_layout": ([POINTER(LayerDesc), c_int, c_int, c_int, c_int, c_int,
                                  POINTER(c_size_t), POINTER(c_size_t), POINTER(c_size_t)], c_int),
    "stream_slot_bytes_sharded": ([POINTER(LayerDesc), c_int, c_int, c_int, POINTER(c_size_t)],
                                  c_int),
    "stream_create": ([c_void_p, c_size_t, POINTER(LayerDesc), c_int, POINTER(StreamConfig), c_void_p,
                       c_size_t, c_void_p, POINTER(c_void_p)], c_int),
    "stream_num_blocks": ([c_void_p], c_int),
    "stream_block_prefetch": ([c_void_p, c_int], c_int),
    "stream_block_acquire": ([c_void_p, c_int, c_void_p, POINTER(Nf4WeightC), c_int], c_int),
    "stream_block_acquire_host": ([c_void_p, c_int, c_int], c_int),
    "stream_block_release": ([c_void_p, c_int, c_void_p], c_int),
    "stream_stats": ([c_void_p, POINTER(StreamStats)], c_int),
    "stream_destroy": ([c_void_p], c_int),
}

EXPORTS = tuple(_SIGS)


def lib():
    """Load libhsnf4.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m host_streamed_nf4_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def last_error() -> str:
    buf = ctypes.create_string_buffer(512)
    lib().hsnf4_last_error(buf, 512)
    return buf.value.decode(errors="replace")


def _check(rc: int):
    if rc != OK:
        raise HsNf4Error(rc, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, device=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# ------------------------------------------------------------------ diagnostics

def device_status(stream=None) -> int:
    flags = c_uint32(0)
    rc = lib().hsnf4_device_status(_stream(stream), ctypes.byref(flags))
    if rc not in (OK, ERR_DEVICE):
        _check(rc)
    return int(flags.value)


def kernel_launches() -> int:
    """Kernels this library has launched in this process so far."""
    return int(lib().hsnf4_kernel_launches())


PROFILE_KINDS = ("lora_gemm_fwd", "lora_gemm_dx", "nf4_dequant", "lora_merge", "lora_project",
                 "lora_grad")


def profile(enable: bool, kinds=None):
    """Start (clearing) or stop kernel timing; `kinds`, a subset of
    PROFILE_KINDS, times only those launches."""
    if enable and kinds is not None:
        mask = 0
        for k in kinds:
            mask |= 1 << PROFILE_KINDS.index(k)
        _check(lib().hsnf4_profile_kinds(mask))
    else:
        _check(lib().hsnf4_profile(int(bool(enable))))


def gemm_plan(mode: str, shapes, T: int, r: int) -> dict:
    """The fused GEMM's work plan for a group of (n_out, k_in) shapes (host
    only): mode "fwd" or "dx"."""
    n = len(shapes)
    n_out = (c_int64 * n)(*[s[0] for s in shapes])
    k_in = (c_int64 * n)(*[s[1] for s in shapes])
    info = GemmPlanInfo()
    _check(lib().hsnf4_gemm_plan({"fwd": 0, "dx": 1}[mode], n_out, k_in, n, T, r,
                                 ctypes.byref(info)))
    return {f[0]: getattr(info, f[0]) for f in GemmPlanInfo._fields_}


def profile_read() -> dict:
    """{kernel name: {"launches", "total_ms", "work"}} since profile(True)."""
    out = (KernelTime * 8)()
    n = lib().hsnf4_profile_read(out, 8)
    if n < 0:
        _check(-n)
    return {out[i].name.decode(): {"launches": int(out[i].launches), "total_ms": out[i].total_ms,
                                   "work": out[i].work} for i in range(n)}


def selftest_stall(stream=None):
    _check(lib().hsnf4_selftest_stall(_stream(stream)))


def inject_fault(site: str | None):
    _check(lib().hsnf4_inject_fault(site.encode() if site else None))


def codebook() -> list[float]:
    out = (c_float * 16)()
    _check(lib().nf4_codebook(out))
    return list(out)


# ------------------------------------------------------------------ NF4

@dataclass
class Nf4Weight:
    """An NF4 weight in device memory (codes uint8, absmax fp32)."""
    codes: torch.Tensor
    absmax: torch.Tensor
    n_out: int
    k_in: int

    def c(self) -> Nf4WeightC:
        return Nf4WeightC(self.codes.data_ptr(), self.absmax.data_ptr(), self.n_out, self.k_in,
                          BASE_NF4, 0)


@dataclass
class Bf16Weight:
    """A dense bf16 base weight [n_out, k_in] in device memory (the
    quantization="bf16_bitwise" base: streamed, never dequantized)."""
    w: torch.Tensor

    @property
    def n_out(self) -> int:
        return self.w.shape[0]

    @property
    def k_in(self) -> int:
        return self.w.shape[1]

    def c(self) -> Nf4WeightC:
        _need(self.w, "w", torch.bfloat16)
        return Nf4WeightC(self.w.data_ptr(), None, self.n_out, self.k_in, BASE_BF16, 0)


def nf4_quantize_pack(w: torch.Tensor, codes=None, absmax=None, stream=None) -> Nf4Weight:
    _need(w, "w", torch.bfloat16)
    n, k = w.shape
    if codes is None:
        codes = torch.empty(n * k // 2, dtype=torch.uint8, device=w.device)
    if absmax is None:
        absmax = torch.empty(n * k // 64, dtype=torch.float32, device=w.device)
    _check(lib().nf4_quantize_pack(_ptr(w), n, k, _ptr(codes), _ptr(absmax), _stream(stream)))
    return Nf4Weight(codes, absmax, n, k)


def nf4_dequant(W: Nf4Weight, out=None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty(W.n_out, W.k_in, dtype=torch.bfloat16, device=W.codes.device)
    _check(lib().nf4_dequant(_ptr(W.codes), _ptr(W.absmax), W.n_out, W.k_in, _ptr(out),
                             _stream(stream)))
    return out


def lora_merge(W, A: torch.Tensor, B: torch.Tensor, alpha: float, out=None, stream=None):
    """W' = deq(W) + (alpha/r) B A as a bf16 [n_out, k_in] tensor (merge_and_unload)."""
    r = A.shape[0]
    dev = A.device
    if out is None:
        out = torch.empty(W.n_out, W.k_in, dtype=torch.bfloat16, device=dev)
    _check(lib().lora_merge(_weight_arg(W), _ptr(A), _ptr(B), r, float(alpha), _ptr(out),
                            _stream(stream)))
    return out


# ------------------------------------------------------------------ decoder glue

def _pp(t):
    return None if t is None else _ptr(t)


def rmsnorm_fwd(x, g, eps, res=None, h_out=None, y=None, stream=None):
    """y = rmsnorm(x [+ res]) (bf16 [T, n]); with res, h_out receives x + res."""
    T, n = x.shape
    if y is None:
        y = torch.empty_like(x)
    if res is not None and h_out is None:
        h_out = torch.empty_like(x)
    _check(lib().decoder_rmsnorm_fwd(_ptr(x), _pp(res), _ptr(g), _pp(h_out), _ptr(y), T, n,
                                     float(eps), _stream(stream)))
    return (y, h_out) if res is not None else y


def rmsnorm_bwd(x, g, dys, eps, dres=None, dx=None, stream=None):
    """dx = dres + drmsnorm(x)/dx . sum(dys) (1..3 bf16 branch gradients)."""
    T, n = x.shape
    if dx is None:
        dx = torch.empty_like(x)
    d = list(dys) + [None] * (3 - len(dys))
    _check(lib().decoder_rmsnorm_bwd(_ptr(x), _ptr(g), _ptr(d[0]), _pp(d[1]), _pp(d[2]), _pp(dres),
                                     _ptr(dx), T, n, float(eps), _stream(stream)))
    return dx


def swiglu_fwd(a, b, m=None, stream=None):
    if m is None:
        m = torch.empty_like(a)
    _check(lib().decoder_swiglu_fwd(_ptr(a), _ptr(b), _ptr(m), a.numel(), _stream(stream)))
    return m


def swiglu_bwd(a, b, dm, da=None, db=None, stream=None):
    da = torch.empty_like(a) if da is None else da
    db = torch.empty_like(a) if db is None else db
    _check(lib().decoder_swiglu_bwd(_ptr(a), _ptr(b), _ptr(dm), _ptr(da), _ptr(db), a.numel(),
                                    _stream(stream)))
    return da, db


def add(x, y, out=None, stream=None):
    out = torch.empty_like(x) if out is None else out
    _check(lib().decoder_add(_ptr(x), _ptr(y), _ptr(out), x.numel(), _stream(stream)))
    return out


def attention_fwd(q, k, v, H, KV, o=None, lse=None, stream=None):
    T = q.shape[0]
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty(H, T, dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().decoder_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), T, H, KV,
                                       _stream(stream)))
    return o, lse


def attention_scratch_bytes(T: int, H: int) -> int:
    return int(lib().decoder_attention_scratch_bytes(T, H))


def attention_bwd(q, k, v, o, lse, dout, H, KV, dq=None, dk=None, dv=None, scratch=None,
                  stream=None):
    T = q.shape[0]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if scratch is None:
        scratch = torch.empty(attention_scratch_bytes(T, H), dtype=torch.uint8, device=q.device)
    _check(lib().decoder_attention_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                       _ptr(dq), _ptr(dk), _ptr(dv), _ptr(scratch), T, H, KV,
                                       _stream(stream)))
    return dq, dk, dv


# ------------------------------------------------------------------ rotary positions

_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32
# the current stream's handle without building a Stream object, and the
# current device's index
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_cur_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or \
    torch.cuda.is_current_stream_capturing


def _launch(index: int, stream, fn, *args):
    """fn(*args, stream) on device `index` (the library launches on the
    current device), on `stream` or that device's current one."""
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        st = _raw_stream(index)
    elif stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    else:
        st = stream.cuda_stream
    if index == _cur_device():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, st)
    if rc != OK:
        raise HsNf4Error(rc, last_error())


def _new(make, shape, dtype, device, stream):
    """A tensor that a call on `stream` will write, made and owned there: on
    the current stream its filling could come after the call, and its memory
    be handed on before it."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _bad(t, name, dtype, index, shape):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the others on cuda:{index}")
    raise ValueError(f"{name} must be {shape}, got {list(t.shape)}, strides {t.stride()}")


def _rows(t: torch.Tensor, name: str, index: int, shape) -> int:
    """Row stride of a bf16 tensor of that (rows, columns) with contiguous
    rows, on device `index`."""
    if t.dtype is not _bf16 or t.get_device() != index or t.shape != shape:
        _bad(t, name, _bf16, index, shape)
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] != 1:
        _bad(t, name, _bf16, index, f"{shape} with contiguous rows")
    if shape[0] <= 1:
        return shape[1]
    if s0 < shape[1]:  # an expanded tensor: stride 0 would mean contiguous rows
        _bad(t, name, _bf16, index, f"{shape} with rows that do not overlap")
    return s0


def _plain(t: torch.Tensor, name: str, index: int, dtype, numel: int) -> int:
    """Address of a contiguous tensor of that type and size on device `index`."""
    if t.dtype is not dtype or t.get_device() != index or t.numel() != numel or \
            not t.is_contiguous():
        _bad(t, name, dtype, index, f"contiguous, {numel} values")
    return t.data_ptr()


def rope_inv_freq(rot_dim: int, theta: float) -> torch.Tensor:
    """theta^(-2i / rot_dim) for i < rot_dim / 2, in 64 bits rounded to fp32."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    return (float(theta) ** (-2.0 * i / rot_dim)).to(torch.float32)


class Rope:
    """Rotary positions of a head: the frequencies, and the axis each follows.

    inv_freq: rot_dim / 2 frequencies (rope_inv_freq, or any other table);
    values of a head past rot_dim are not turned.  sections: how many
    frequencies each axis has (time, height, width), in order; interleaved
    deals them out in turn instead (0, 1, 2, 0, 1, 2, ... while an axis has
    some left).  pairing "half" turns (i, i + rot_dim / 2), "adjacent"
    (2i, 2i + 1).  scale multiplies the rotation."""

    def __init__(self, head_dim: int, inv_freq, sections=None, interleaved: bool = False,
                 pairing: str = "half", scale: float = 1.0):
        f = [float(x) for x in inv_freq]
        if len(f) > ROPE_MAX_PAIRS:
            raise ValueError(f"at most {ROPE_MAX_PAIRS} frequencies (got {len(f)})")
        if pairing not in ("half", "adjacent"):
            raise ValueError(f"pairing must be 'half' or 'adjacent' (got {pairing!r})")
        sections = [len(f)] if sections is None else [int(n) for n in sections]
        if sum(sections) != len(f) or min(sections) < 0:
            raise ValueError(f"sections {sections} do not add up to {len(f)} frequencies")
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
        if interleaved:
            axis = [a for i in range(max(sections)) for a, n in enumerate(sections) if i < n]
        self.n_axes, self.head_dim = len(sections), int(head_dim)
        self.c = RopeC(self.head_dim, 2 * len(f), self.n_axes,
                       ROPE_HALF if pairing == "half" else ROPE_ADJACENT, float(scale))
        self.c.inv_freq[:len(f)] = f
        self.c.axis[:len(f)] = axis
        self._ref = ctypes.byref(self.c)


def _rope(fn, rope, pos, q, k, q_out, k_out, stream):
    dev, d, shape = q.get_device(), rope.head_dim, q.shape
    T, wq = shape
    if wq % d:
        raise ValueError(f"q has {wq} columns, not a multiple of {d}")
    if pos.shape != (rope.n_axes, T) and (rope.n_axes > 1 or pos.shape != (T,)):
        _bad(pos, "pos", pos.dtype, pos.get_device(), f"[{rope.n_axes}, {T}]")
    p = _plain(pos, "pos", dev, _i32, rope.n_axes * T)
    if q_out is None:
        q_out = _new(torch.empty, shape, _bf16, q.device, stream)
    qs, qos = _rows(q, "q", dev, shape), _rows(q_out, "q_out", dev, shape)
    if k is None:
        _launch(dev, stream, fn, rope._ref, p, T, wq // d, 0, q.data_ptr(), qs, None, 0,
                q_out.data_ptr(), qos, None, 0)
        return q_out
    wk = k.shape[1]
    shape = (T, wk)
    if wk % d:
        raise ValueError(f"k has {wk} columns, not a multiple of {d}")
    if k_out is None:
        k_out = _new(torch.empty, shape, _bf16, q.device, stream)
    ks, kos = _rows(k, "k", dev, shape), _rows(k_out, "k_out", dev, shape)
    _launch(dev, stream, fn, rope._ref, p, T, wq // d, wk // d, q.data_ptr(), qs, k.data_ptr(), ks,
            q_out.data_ptr(), qos, k_out.data_ptr(), kos)
    return q_out, k_out


def rope_fwd(rope: Rope, pos, q, k=None, q_out=None, k_out=None, stream=None):
    """q [T, H * head_dim] and k [T, KV * head_dim] turned to their positions
    pos (int32 [n_axes, T], or [T] for one axis).  Rows may be strided
    (columns of a fused tensor); q_out / k_out may be q / k.  Returns
    (q_out, k_out), or q_out without k."""
    return _rope(lib().decoder_rope_fwd, rope, pos, q, k, q_out, k_out, stream)


def rope_bwd(rope: Rope, pos, dq, dk=None, dq_out=None, dk_out=None, stream=None):
    """Gradients of rope_fwd's inputs from those of its outputs."""
    return _rope(lib().decoder_rope_bwd, rope, pos, dq, dk, dq_out, dk_out, stream)


# ------------------------------------------------------------------ packed attention

def _packed(q, k, v, cu_q, cu_k, H, KV, causal, scale):
    dev, sq = q.get_device(), q.shape
    Tq, wq = sq
    Tk = k.shape[0]
    if H < 1 or KV < 1 or wq % H:
        raise ValueError(f"q has {wq} columns for {H} heads (KV heads: {KV})")
    d = wq // H
    sk = (Tk, KV * d)
    n = cu_q.numel()
    if n < 2:
        raise ValueError("cu_q must have n_seq + 1 values")
    pq = _plain(cu_q, "cu_q", dev, _i32, n)
    pk = pq if cu_k is None or cu_k is cu_q else _plain(cu_k, "cu_k", dev, _i32, n)
    return dev, sq, sk, d, PackedAttentionC(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _rows(q, "q", dev, sq), _rows(k, "k", dev, sk),
        _rows(v, "v", dev, sk), pq, pk, Tq, Tk, n - 1, H, KV, d, 1 if causal else 0,
        d ** -0.5 if scale is None else scale)


def attention_packed_fwd(q, k, v, cu_q, H, KV, causal=True, cu_k=None, scale=None, o=None,
                         lse=None, stream=None):
    """Attention over packed sequences: q [Tq, H * d], k, v [Tk, KV * d]
    (rows may be strided), sequence s the tokens cu_q[s]..cu_q[s + 1] (int32,
    on the device; cu_k: the keys', if they differ).  Rows outside every
    sequence are left as they are in o and lse.  Returns (o, lse [H, Tq])."""
    dev, sq, _, _, a = _packed(q, k, v, cu_q, cu_k, H, KV, causal, scale)
    Tq = sq[0]
    if o is None:
        o = _new(torch.zeros, sq, _bf16, q.device, stream)
    if lse is None:
        lse = _new(torch.zeros, (H, Tq), _f32, q.device, stream)
    elif lse.shape != (H, Tq):
        _bad(lse, "lse", lse.dtype, lse.get_device(), f"[{H}, {Tq}]")
    _launch(dev, stream, lib().decoder_attention_packed_fwd, ctypes.byref(a), o.data_ptr(),
            _rows(o, "o", dev, sq), _plain(lse, "lse", dev, _f32, H * Tq))
    return o, lse


def attention_packed_workspace_bytes(Tq, Tk, n_seq, H, KV, d) -> int:
    n = int(lib().decoder_attention_packed_workspace(Tq, Tk, n_seq, H, KV, d))
    if n == 0:
        raise HsNf4Error(ERR_INVALID, last_error())
    return n


def attention_packed_bwd(q, k, v, o, lse, dout, cu_q, H, KV, causal=True, cu_k=None, scale=None,
                         dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Its gradients from the forward's o and lse: (dq, dk, dv).  Rows outside
    every sequence are left as they are."""
    dev, sq, sk, d, a = _packed(q, k, v, cu_q, cu_k, H, KV, causal, scale)
    if lse.shape != (H, sq[0]):
        _bad(lse, "lse", lse.dtype, lse.get_device(), f"[{H}, {sq[0]}]")
    dq = _new(torch.zeros, sq, _bf16, q.device, stream) if dq is None else dq
    dk = _new(torch.zeros, sk, _bf16, q.device, stream) if dk is None else dk
    dv = _new(torch.zeros, sk, _bf16, q.device, stream) if dv is None else dv
    if workspace is None:
        with torch.cuda.device(dev):
            n = attention_packed_workspace_bytes(sq[0], sk[0], a.n_seq, H, KV, d)
        workspace = _new(torch.empty, n, torch.uint8, q.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    _launch(dev, stream, lib().decoder_attention_packed_bwd, ctypes.byref(a), o.data_ptr(),
            _rows(o, "o", dev, sq), _plain(lse, "lse", dev, _f32, H * sq[0]),
            dout.data_ptr(), _rows(dout, "dout", dev, sq), dq.data_ptr(), _rows(dq, "dq", dev, sq),
            dk.data_ptr(), _rows(dk, "dk", dev, sk), dv.data_ptr(), _rows(dv, "dv", dev, sk),
            workspace.data_ptr(), workspace.nbytes)
    return dq, dk, dv


# ------------------------------------------------------------------ gradient norm

class GradSet:
    """A fixed list of gradient tensors (fp32, bf16 or fp16, contiguous, any
    mix) for grad_norm and grad_clip.  outs: where clipped gradients go, each
    of its gradient's type and size (default: in place).  The set keeps the
    tensors' addresses, so their memory must not be replaced, and a graph that
    captured a call needs the set for as long as it is replayed.

    Make it once, for gradients that stay where they are: it fills a table on
    the device and waits for that, 0.04 to 0.1 ms for 14 tensors, 0.9 to 1.7 ms
    for 1120, as long as plain torch operations take to clip them."""

    def __init__(self, tensors, outs=None, stream=None):
        self.tensors = list(tensors)
        self.outs = self.tensors if outs is None else list(outs)
        if not self.tensors or len(self.outs) != len(self.tensors):
            raise ValueError("GradSet takes one tensor or more, and as many outs")
        dev = self.tensors[0].device
        index = self.tensors[0].get_device()
        arr = (GradC * len(self.tensors))()
        for i, (g, o, c) in enumerate(zip(self.tensors, self.outs, arr)):
            t = GRAD_DTYPES.get(g.dtype)
            if t is None or o.dtype is not g.dtype:
                raise TypeError(f"tensor {i}: fp32, bf16 or fp16 and its out the same "
                                f"(got {g.dtype}, {o.dtype})")
            n = g.numel()
            if index < 0 or g.get_device() != index or not g.is_contiguous():
                raise ValueError(f"tensor {i} is not a contiguous tensor on {dev}")
            if o is not g and (o.get_device() != index or not o.is_contiguous() or
                               o.numel() != n):
                raise ValueError(f"out {i} is not a contiguous tensor of {n} values on {dev}")
            c.g, c.out, c.n, c.dtype = g.data_ptr(), o.data_ptr(), n, t
        self.device, self.index, self.plan = dev, index, GradPlanC()
        n = len(self.tensors)
        self.table = _new(torch.empty, int(lib().lora_grad_table_bytes(n)) or 16, torch.uint8, dev,
                          stream)
        _launch(index, stream, lambda *a: lib().lora_grad_plan(arr, n, self.table.data_ptr(),
                                                               self.table.numel(),
                                                               ctypes.byref(self.plan), *a))
        self.workspace = self.new_workspace(stream)
        self._ref = ctypes.byref(self.plan)
        # a workspace per stream that calls were made on
        self._spaces = {_raw_stream(index) if stream is None else stream.cuda_stream:
                        self.workspace}

    def new_workspace(self, stream=None) -> torch.Tensor:
        """A workspace for calls on `stream`.  Without one, the calls on a
        stream share the set's for that stream, and a captured call has one of
        its graph, so that streams and graphs may run at the same time."""
        with torch.cuda.device(self.index):
            n = int(lib().lora_grad_workspace(ctypes.byref(self.plan)))
        return _new(torch.empty, n, torch.uint8, self.device, stream)

    def _first_call_on(self, stream, at):
        if stream is not None and stream.device.index != self.index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {self.device}")
        used = torch.cuda.current_stream(self.index) if stream is None else stream
        # else a set dropped after the call would give its table back too early
        self.table.record_stream(used)
        self.workspace.record_stream(used)
        if _capturing():  # the stream's memory is the graph's now; a later call makes the set's
            return None
        ws = self._spaces[at] = self.new_workspace(stream)
        return ws

    def _call(self, fn, args, norm, workspace, stream):
        if norm is None:
            norm = _new(torch.empty, (), _f32, self.device, stream)
        at = _raw_stream(self.index) if stream is None else stream.cuda_stream
        ws = self._spaces.get(at)
        if ws is None:
            ws = self._first_call_on(stream, at)
        if workspace is not None:
            ws = workspace
            if ws.get_device() != self.index or not ws.is_contiguous():
                raise ValueError(f"workspace must be a contiguous tensor on {self.device}")
        elif _capturing():
            ws = self.new_workspace(stream)
        _launch(self.index, stream, fn, self._ref, *args,
                _plain(norm, "norm", self.index, _f32, 1), ws.data_ptr(), ws.nbytes)
        return norm


def grad_norm(grads: GradSet, norm=None, workspace=None, stream=None) -> torch.Tensor:
    """The 2-norm of every gradient of the set together (fp32 scalar tensor)."""
    return grads._call(lib().lora_grad_norm, (), norm, workspace, stream)


def grad_clip(grads: GradSet, max_norm: float, norm=None, workspace=None,
              stream=None) -> torch.Tensor:
    """Scale every gradient of the set by min(1, max_norm / (norm + 1e-6));
    returns the norm before that."""
    return grads._call(lib().lora_grad_clip, (float(max_norm),), norm, workspace, stream)


# ------------------------------------------------------------------ LoRA linear

def fwd_workspace_bytes(T, n_out, k_in, r) -> int:
    return int(lib().lora_linear_fwd_workspace(T, n_out, k_in, r))


def bwd_workspace_bytes(T, n_out, k_in, r) -> int:
    return int(lib().lora_linear_bwd_workspace(T, n_out, k_in, r))


def _weight_arg(W):
    return ctypes.byref(_wc(W))


def lora_linear_fwd(W, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float,
                    Y=None, t_save=None, workspace=None, stream=None):
    """Y = X deq(W)^T + (alpha/r) (X A^T) B^T.  Returns (Y bf16 [T, n_out], t fp32 [T, r])."""
    n_out, k_in = W.n_out, W.k_in
    T, r = X.shape[0], A.shape[0]
    if Y is None:
        Y = torch.empty(T, n_out, dtype=torch.bfloat16, device=X.device)
    if t_save is None:
        t_save = torch.empty(T, r, dtype=torch.float32, device=X.device)
    ws = fwd_workspace_bytes(T, n_out, k_in, r)
    if workspace is None:
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=X.device)
    _check(lib().lora_linear_fwd(_weight_arg(W), _ptr(X), T, _ptr(A), _ptr(B), r, float(alpha),
                                 _ptr(Y), _ptr(t_save), _ptr(workspace), workspace.numel(),
                                 _stream(stream)))
    return Y, t_save


def lora_linear_fwd_noalloc(W, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float,
                            Y=None, t_save=None, stream=None):
    """The forward without a workspace argument, for callers that cannot
    allocate device memory: the library's built-in 64 MiB scratch is used.
    (The output buffers passed here may be preallocated by the caller.)"""
    n_out = W.n_out
    T, r = X.shape[0], A.shape[0]
    if Y is None:
        Y = torch.empty(T, n_out, dtype=torch.bfloat16, device=X.device)
    if t_save is None:
        t_save = torch.empty(T, r, dtype=torch.float32, device=X.device)
    _check(lib().lora_linear_fwd_noalloc(_weight_arg(W), _ptr(X), T, _ptr(A), _ptr(B), r,
                                         float(alpha), _ptr(Y), _ptr(t_save), _stream(stream)))
    return Y, t_save


def lora_linear_bwd(W, X, t_save, A, B, dY, alpha: float, dX=None, dA=None, dB=None,
                    workspace=None, stream=None):
    """Returns (dX bf16 [T, k_in], dA fp32 [r, k_in], dB fp32 [n_out, r])."""
    n_out, k_in = W.n_out, W.k_in
    T, r = X.shape[0], A.shape[0]
    dev = X.device
    if dX is None:
        dX = torch.empty(T, k_in, dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty(r, k_in, dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty(n_out, r, dtype=torch.float32, device=dev)
    ws = bwd_workspace_bytes(T, n_out, k_in, r)
    if workspace is None:
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
    _check(lib().lora_linear_bwd(_weight_arg(W), _ptr(X), _ptr(t_save), T, _ptr(A), _ptr(B), r,
                                 float(alpha), _ptr(dY), _ptr(dX), _ptr(dA), _ptr(dB),
                                 _ptr(workspace), workspace.numel(), _stream(stream)))
    return dX, dA, dB


def _wc(W):
    return W.c() if isinstance(W, (Nf4Weight, Bf16Weight)) else W


def _p(t):
    return None if t is None else t.data_ptr()


def fwd_args(W, X, A, B, Y, t_save=None, dropout=None) -> FwdArgs:
    """One problem of a grouped forward (tensors are kept alive by the caller).
    dropout: (p, seed, offset) for the adapter branch, or None."""
    p, seed, off = dropout or (0.0, 0, 0)
    return FwdArgs(_wc(W), _p(X), _p(A), _p(B), _p(Y), _p(t_save), p, 0, seed, off)


def bwd_args(W, X, t_save, A, B, dY, dX, dA, dB, dropout=None) -> BwdArgs:
    p, seed, off = dropout or (0.0, 0, 0)
    return BwdArgs(_wc(W), _p(X), _p(t_save), _p(A), _p(B), _p(dY), _p(dX), _p(dA), _p(dB),
                   p, 0, seed, off)


def lora_dropout_apply(X: torch.Tensor, p: float, seed: int, offset: int, out=None,
                       stream=None) -> torch.Tensor:
    """X_d = dropout(X) on the adapter branch's definition (bf16 [T, K])."""
    _need(X, "X", torch.bfloat16)
    T, K = X.shape
    if out is None:
        out = torch.empty_like(X)
    _check(lib().lora_dropout_apply(_ptr(X), T, K, float(p), seed, offset, _ptr(out),
                                    _stream(stream)))
    return out


def group_fwd_workspace_bytes(args, T, r) -> int:
    arr = (FwdArgs * len(args))(*args)
    return int(lib().lora_group_fwd_workspace(arr, len(args), T, r))


def group_bwd_workspace_bytes(args, T, r) -> int:
    arr = (BwdArgs * len(args))(*args)
    return int(lib().lora_group_bwd_workspace(arr, len(args), T, r))


def lora_group_fwd(args, T: int, r: int, alpha: float, workspace: torch.Tensor, stream=None):
    """Forward of len(args) independent LoRA linears in one grouped call."""
    arr = (FwdArgs * len(args))(*args)
    _check(lib().lora_group_fwd(arr, len(args), T, r, float(alpha), _ptr(workspace),
                                workspace.numel(), _stream(stream)))


def lora_group_bwd(args, T: int, r: int, alpha: float, workspace: torch.Tensor, stream=None):
    arr = (BwdArgs * len(args))(*args)
    _check(lib().lora_group_bwd(arr, len(args), T, r, float(alpha), _ptr(workspace),
                                workspace.numel(), _stream(stream)))


# ------------------------------------------------------------------ streamer

def layer_desc(shapes, base_format: int = 0) -> LayerDesc:
    """shapes: [(n_out, k_in), ...] of one layer's projections; base_format
    BASE_NF4 (codes + absmax) or BASE_BF16 (dense bf16 weights)."""
    d = LayerDesc()
    d.n_proj = len(shapes)
    d.base_format = base_format
    for i, (n, k) in enumerate(shapes):
        d.n_out[i] = n
        d.k_in[i] = k
    return d


def layer_bytes(desc: LayerDesc) -> int:
    out = c_size_t(0)
    _check(lib().stream_layer_bytes(ctypes.byref(desc), ctypes.byref(out)))
    return out.value


def layer_offsets(desc: LayerDesc, proj: int):
    co, ao = c_size_t(0), c_size_t(0)
    _check(lib().stream_layer_offsets(ctypes.byref(desc), proj, ctypes.byref(co), ctypes.byref(ao)))
    return co.value, ao.value


def _desc_array(descs):
    arr = (LayerDesc * len(descs))(*descs)
    return arr


def slab_bytes(descs) -> int:
    out = c_size_t(0)
    _check(lib().stream_slab_bytes(_desc_array(descs), len(descs), ctypes.byref(out)))
    return out.value


def ring_bytes(descs, block_size: int, n_slots: int = 2, shard_world: int = 0) -> int:
    """Device bytes of an n_slots ring; shard_world >= 1: of a sharded stream."""
    out = c_size_t(0)
    if shard_world >= 1:
        _check(lib().stream_slot_bytes_sharded(_desc_array(descs), len(descs), block_size,
                                               shard_world, ctypes.byref(out)))
    else:
        _check(lib().stream_slot_bytes(_desc_array(descs), len(descs), block_size,
                                       ctypes.byref(out)))
    return out.value * n_slots


def shard_range(block_bytes: int, world: int, rank: int):
    """(stride S, offset, length) of rank's shard of a block shared by world ranks."""
    S, off, n = c_size_t(0), c_size_t(0), c_size_t(0)
    _check(lib().stream_shard_range(block_bytes, world, rank, ctypes.byref(S), ctypes.byref(off),
                                    ctypes.byref(n)))
    return S.value, off.value, n.value


def shard_slab_layout(descs, block_size: int, world: int, rank: int):
    """Rank's shard slab: ([(offset in the shard slab, length) per block], total bytes)."""
    arr = _desc_array(descs)
    total = c_size_t(0)
    _check(lib().stream_shard_slab_layout(arr, len(descs), block_size, world, rank, -1, None,
                                          None, ctypes.byref(total)))
    n_blocks = (len(descs) + block_size - 1) // block_size
    out = []
    for b in range(n_blocks):
        off, n = c_size_t(0), c_size_t(0)
        _check(lib().stream_shard_slab_layout(arr, len(descs), block_size, world, rank, b,
                                              ctypes.byref(off), ctypes.byref(n), None))
        out.append((off.value, n.value))
    return out, total.value


class Streamer:
    """Pinned-host NF4 stack -> 2-slot VRAM ring, prefetched one block ahead.

    shard=(rank, world, gather): stream 1/world of every block over this
    rank's link; gather(slot_offset, shard_bytes, world, block) must enqueue,
    on the current CUDA stream (the copy stream), the in-place all-gather of
    the ring bytes [slot_offset, slot_offset + world * shard_bytes).
    shard_slab: the slab holds only this rank's shards (shard_slab_layout)."""

    def __init__(self, slab: torch.Tensor, descs, block_size: int, ring: torch.Tensor,
                 copy_stream: torch.cuda.Stream, enable_prefetch=True, reuse_resident=True,
                 poison_on_release=False, n_slots=2, shard=None, shard_slab=False):
        _need(slab, "slab", torch.uint8, device=False)
        if not slab.is_pinned():
            raise ValueError("slab must be page-locked (pin_memory)")
        _need(ring, "ring", torch.uint8)
        self.descs = list(descs)
        self._arr = _desc_array(self.descs)
        cfg = StreamConfig(block_size, int(bool(enable_prefetch)), int(bool(reuse_resident)),
                           int(bool(poison_on_release)), int(n_slots))
        self._gather_error = None
        self._gather_cb = None
        if shard is not None:
            rank, world, fn = shard
            base = ring.data_ptr()

            def _cb(slot, shard_bytes, world_, block, stream, user):
                try:
                    with torch.cuda.stream(copy_stream):
                        fn(slot - base, shard_bytes, world_, block)
                    return 0
                except Exception as e:  # reported through the library's status
                    self._gather_error = e
                    return 1

            self._gather_cb = GATHER_FN(_cb)
            cfg.shard_world, cfg.shard_rank = world, rank
            cfg.gather = self._gather_cb
            cfg.shard_slab = int(bool(shard_slab))
        self.n_slots = n_slots
        h = c_void_p()
        _check(lib().stream_create(_ptr(slab), slab.numel(), self._arr, len(self.descs),
                                   ctypes.byref(cfg), _ptr(ring), ring.numel(),
                                   ctypes.c_void_p(copy_stream.cuda_stream), ctypes.byref(h)))
        self._h = h
        self.slab, self.ring, self.copy_stream = slab, ring, copy_stream
        self.block_size = block_size
        self.n_blocks = lib().stream_num_blocks(h)

    def _check(self, rc: int):
        err, self._gather_error = self._gather_error, None
        if rc != 0 and err is not None:
            raise HsNf4Error(rc, f"{last_error()} ({type(err).__name__}: {err})") from err
        _check(rc)

    def prefetch(self, b: int):
        self._check(lib().stream_block_prefetch(self._h, b))

    def prefetch_ahead(self, upcoming) -> int:
        arr = (c_int * len(upcoming))(*upcoming)
        issued = c_int(0)
        self._check(lib().stream_prefetch_ahead(self._h, arr, len(upcoming), ctypes.byref(issued)))
        return issued.value

    def acquire(self, b: int, stream=None):
        first = b * self.block_size
        n = sum(d.n_proj for d in self.descs[first:first + self.block_size])
        out = (Nf4WeightC * n)()
        self._check(lib().stream_block_acquire(self._h, b, _stream(stream), out, n))
        return list(out)

    def acquire_host(self, b: int, timeout_ms: int):
        _check(lib().stream_block_acquire_host(self._h, b, timeout_ms))

    def release(self, b: int, stream=None):
        _check(lib().stream_block_release(self._h, b, _stream(stream)))

    def stats(self) -> dict:
        s = StreamStats()
        _check(lib().stream_stats(self._h, ctypes.byref(s)))
        return {f: int(getattr(s, f)) for f, _ in StreamStats._fields_}

    def close(self):
        if self._h:
            rc = lib().stream_destroy(self._h)
            self._h = None
            _check(rc)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
