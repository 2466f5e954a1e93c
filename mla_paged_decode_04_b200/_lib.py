"""ctypes binding of libmla_decode.so (argument marshalling only).

The functions carry the C ABI's names (include/mla_decode.h) and pass raw
device pointers and the current CUDA stream; every step of the decode runs
in the library's kernels. PyTorch is used only to own device memory and
streams. If the shared library is missing this module raises at import: there
is no fallback path. With MLA_DECODE_BOUNDS_CHECK=1 in the environment the
bounds-checking build, libmla_decode_check.so, is loaded instead (slower; its
kernels set MLA_DEV_BOUNDS instead of accessing memory outside a buffer).
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
NORMAL_LIB_PATH = os.path.join(_HERE, "libmla_decode.so")
CHECK_LIB_PATH = os.path.join(_HERE, "libmla_decode_check.so")
LIB_PATH = CHECK_LIB_PATH if os.environ.get("MLA_DECODE_BOUNDS_CHECK", "0") == "1" else NORMAL_LIB_PATH

MLA_BF16, MLA_FP16, MLA_FP8_E4M3 = 0, 1, 2
DTYPES = {"bf16": MLA_BF16, "fp16": MLA_FP16, "fp8": MLA_FP8_E4M3}
_TORCH_CODES = {torch.bfloat16: MLA_BF16, torch.float16: MLA_FP16, torch.float8_e4m3fn: MLA_FP8_E4M3}
MLA_KERNEL_AUTO, MLA_KERNEL_TCGEN05, MLA_KERNEL_SIMT, MLA_KERNEL_TCGEN05_SOLO = 0, 1, 2, 3
KERNELS = {"auto": MLA_KERNEL_AUTO, "tcgen05": MLA_KERNEL_TCGEN05, "simt": MLA_KERNEL_SIMT,
           "tcgen05_solo": MLA_KERNEL_TCGEN05_SOLO}

MLA_DEV_BAD_PAGE, MLA_DEV_SEQ_TOO_LONG, MLA_DEV_TIMEOUT, MLA_DEV_BAD_QLEN, MLA_DEV_BOUNDS = 0x1, 0x2, 0x4, 0x8, 0x10
(MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED_SHAPE, MLA_ERR_WORKSPACE_TOO_SMALL, MLA_ERR_ARCH, MLA_ERR_CUDA,
 MLA_ERR_PLAN_MISMATCH) = (-1, -2, -3, -4, -5, -6)

EXPORTED = ["mla_decode_plan", "mla_decode_plan_custom", "mla_decode", "mla_decode_partial",
            "mla_decode_combine", "mla_decode_status", "mla_status_string", "mla_version",
            "mla_decode_no_alloc", "mla_decode_no_alloc_status", "mla_last_cuda_error", "mla_kv_pack", "mla_kv_amax",
            "mla_decode_plan_window", "mla_prefill_plan", "mla_prefill_plan_custom", "mla_prefill",
            "mla_prefill_partial", "mla_prefill_combine", "mla_bounds_checked",
            "mla_decode_plan_sinks", "mla_key_weights", "mla_cache_evict"]
MLA_NO_ALLOC_SCRATCH_BYTES = 48 << 20


class MlaPlan(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("q_len", ctypes.c_int32), ("num_heads", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("fold", ctypes.c_int32), ("q_groups", ctypes.c_int32), ("rows_per_unit", ctypes.c_int32),
        ("split_kv", ctypes.c_int32), ("keys_per_split", ctypes.c_int32),
        ("kernel", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_uint64), ("partial_offset", ctypes.c_uint64),
        ("lse_offset", ctypes.c_uint64), ("magic", ctypes.c_uint32), ("schedule", ctypes.c_uint32),
        ("window", ctypes.c_int32), ("varlen", ctypes.c_int32), ("fault_test", ctypes.c_int32),
        ("sinks", ctypes.c_int32),
    ]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class MlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = f"{what} failed: {status_string(code)} ({code})"
        self.cuda_error = None
        if code == -5:  # MLA_ERR_CUDA: name the CUDA runtime error behind it
            self.cuda_error = last_cuda_error()
            msg += f" [{self.cuda_error[1]} ({self.cuda_error[0]})]"
        super().__init__(msg)
        self.code = code


def load_library(path):
    """The library at `path` (the normal or the bounds-checking build) with its argument types set."""
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python mla_paged_decode_04_b200/build.py"
            f"{' --check' if path == CHECK_LIB_PATH else ''}` (there is no non-CUDA fallback)")
    lib = ctypes.CDLL(path)
    i32, i64, u64, f32, vp = (ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float,
                              ctypes.c_void_p)
    P = ctypes.POINTER(MlaPlan)
    lib.mla_decode_plan.argtypes = [i32, i32, i32, i32, i32, P]
    lib.mla_decode_plan.restype = i32
    lib.mla_decode_plan_custom.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, P]
    lib.mla_decode_plan_custom.restype = i32
    for name in ("mla_decode", "mla_decode_partial", "mla_decode_combine"):
        fn = getattr(lib, name)
        fn.argtypes = [P, vp, vp, i64, i32, vp, i32, vp, f32, f32, f32, vp, vp, vp, u64, vp]
        fn.restype = i32
    lib.mla_decode_status.argtypes = [vp, vp, i32, ctypes.POINTER(ctypes.c_int32)]
    lib.mla_decode_status.restype = i32
    lib.mla_status_string.argtypes = [i32]
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_version.argtypes = []
    lib.mla_version.restype = ctypes.c_char_p
    lib.mla_last_cuda_error.argtypes = [ctypes.POINTER(ctypes.c_char_p)]
    lib.mla_last_cuda_error.restype = i32
    lib.mla_prefill_plan.argtypes = [i32, i32, i32, i32, i32, P]
    lib.mla_prefill_plan.restype = i32
    lib.mla_prefill_plan_custom.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, P]
    lib.mla_prefill_plan_custom.restype = i32
    for name in ("mla_prefill", "mla_prefill_partial", "mla_prefill_combine"):
        fn = getattr(lib, name)
        fn.argtypes = [P, vp, i64, vp, vp, i64, i32, vp, i32, vp, f32, f32, f32, vp, vp, vp, u64, vp]
        fn.restype = i32
    lib.mla_decode_plan_window.argtypes = [P, i32]
    lib.mla_decode_plan_window.restype = i32
    lib.mla_kv_pack.argtypes = [vp, vp, i64, vp, vp, i64, i32, i32, i32, f32, vp, vp]
    lib.mla_kv_pack.restype = i32
    lib.mla_kv_amax.argtypes = [vp, vp, i64, i32, vp, vp]
    lib.mla_kv_amax.restype = i32
    lib.mla_decode_plan_sinks.argtypes = [P, i32]
    lib.mla_decode_plan_sinks.restype = i32
    lib.mla_key_weights.argtypes = [P, vp, i64, vp, vp, i64, i32, vp, i32, vp, f32, f32, f32, vp, vp, i64, f32, vp,
                                    i64, i64, vp, vp]
    lib.mla_key_weights.restype = i32
    lib.mla_cache_evict.argtypes = [vp, i64, i64, vp, i32, i32, i32, i32, vp, i64, i32, vp, i32, vp, i64, vp, i32,
                                    i32, vp, vp, vp, i64, vp, vp]
    lib.mla_cache_evict.restype = i32
    lib.mla_bounds_checked.argtypes = []
    lib.mla_bounds_checked.restype = i32
    return lib


_lib = load_library(LIB_PATH)


def bounds_checked() -> bool:
    """True when the loaded library is the bounds-checking build."""
    return bool(_lib.mla_bounds_checked())


def lib():
    return _lib


def status_string(code: int) -> str:
    return _lib.mla_status_string(int(code)).decode()


def last_cuda_error():
    """(code, name) of the CUDA runtime error behind this thread's last MLA_ERR_CUDA."""
    name = ctypes.c_char_p()
    code = _lib.mla_last_cuda_error(ctypes.byref(name))
    return int(code), (name.value.decode() if name.value else "")


def mla_version() -> str:
    return _lib.mla_version().decode()


def _dtype_code(dtype) -> int:
    if isinstance(dtype, str):
        return DTYPES[dtype]
    code = _TORCH_CODES.get(dtype)
    return int(dtype) if code is None else code


def mla_decode_plan(batch, q_len, num_heads, max_seq_len, dtype) -> MlaPlan:
    p = MlaPlan()
    rc = _lib.mla_decode_plan(batch, q_len, num_heads, max_seq_len, _dtype_code(dtype), ctypes.byref(p))
    if rc != 0:
        raise MlaError(rc, "mla_decode_plan")
    return p


def mla_decode_plan_custom(batch, q_len, num_heads, max_seq_len, dtype, split_kv=0, fold=0,
                           kernel="auto") -> MlaPlan:
    p = MlaPlan()
    k = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    rc = _lib.mla_decode_plan_custom(batch, q_len, num_heads, max_seq_len, _dtype_code(dtype),
                                     split_kv, fold, k, ctypes.byref(p))
    if rc != 0:
        raise MlaError(rc, "mla_decode_plan_custom")
    return p


def mla_decode_plan_window(plan: MlaPlan, window: int) -> MlaPlan:
    """Set the plan's sliding window in place (0 = full attention) and return it."""
    rc = _lib.mla_decode_plan_window(ctypes.byref(plan), int(window))
    if rc != 0:
        raise MlaError(rc, "mla_decode_plan_window")
    return plan


def mla_decode_plan_sinks(plan: MlaPlan, sinks: int) -> MlaPlan:
    """Keep the first `sinks` keys visible beside the plan's window, in place (0 = none), and return it."""
    rc = _lib.mla_decode_plan_sinks(ctypes.byref(plan), int(sinks))
    if rc != 0:
        raise MlaError(rc, "mla_decode_plan_sinks")
    return plan


def mla_prefill_plan(batch, max_q_len, num_heads, max_seq_len, dtype, split_kv=0, fold=0,
                     kernel="auto") -> MlaPlan:
    """Plan of a ragged-query (prefill) shape: max_q_len = the most new tokens an entry may have."""
    p = MlaPlan()
    k = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    rc = _lib.mla_prefill_plan_custom(batch, max_q_len, num_heads, max_seq_len, _dtype_code(dtype),
                                      split_kv, fold, k, ctypes.byref(p))
    if rc != 0:
        raise MlaError(rc, "mla_prefill_plan")
    return p


# Small calls are bound by the host: the helpers below take the cheapest
# accessor of each property (device indexes instead of device objects, the raw
# stream instead of a Stream object, plain integers for pointers).
def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_tensors(q, /, **named):
    """Every tensor argument is a contiguous CUDA tensor on q's device."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda):
        raise ValueError("q must be a CUDA tensor")
    index = q.get_device()
    for k, t in named.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.get_device() != index:
            raise ValueError(f"{k} must be a CUDA tensor on {q.device} (got "
                             f"{t.device if isinstance(t, torch.Tensor) else type(t).__name__})")
        if not t.is_contiguous():
            raise ValueError(f"{k} must be contiguous")
    for k in ("block_tables", "seq_lens"):
        t = named.get(k)
        if t is not None and t.dtype != torch.int32:
            raise ValueError(f"{k} must be int32")


def _call(name, plan, q, kv_cache, block_tables, seq_lens, softmax_scale, out, lse, workspace,
          q_scale, kv_scale, stream):
    _check_tensors(q, kv_cache=kv_cache, block_tables=block_tables, seq_lens=seq_lens, out=out,
                   lse=lse, workspace=workspace)
    rc = getattr(_lib, name)(ctypes.byref(plan), _ptr(q), _ptr(kv_cache), kv_cache.size(0), kv_cache.size(1),
                             _ptr(block_tables), block_tables.size(1), _ptr(seq_lens),
                             float(softmax_scale), float(q_scale), float(kv_scale), _ptr(out),
                             _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream_of(q, stream))
    if rc != 0:
        raise MlaError(rc, name)


def mla_decode(plan: MlaPlan, q, kv_cache, block_tables, seq_lens, softmax_scale, out, lse,
               workspace, q_scale=1.0, kv_scale=1.0, stream=None) -> None:
    """Enqueue one decode step on `stream` (default: torch's current stream).

    Tensors are device tensors in the layouts of include/mla_decode.h; `out`
    (bf16 [B, q_len, H, 512]), `lse` (fp32 [B, q_len, H] or None) and
    `workspace` (uint8, >= plan.workspace_bytes, 256-byte aligned) are written.
    """
    _call("mla_decode", plan, q, kv_cache, block_tables, seq_lens, softmax_scale, out, lse,
          workspace, q_scale, kv_scale, stream)


def mla_decode_partial(plan: MlaPlan, q, kv_cache, block_tables, seq_lens, softmax_scale, out,
                       lse, workspace, q_scale=1.0, kv_scale=1.0, stream=None) -> None:
    """First kernel only (split-KV partials; writes out/lse itself when split_kv == 1)."""
    _call("mla_decode_partial", plan, q, kv_cache, block_tables, seq_lens, softmax_scale, out,
          lse, workspace, q_scale, kv_scale, stream)


def mla_decode_combine(plan: MlaPlan, q, kv_cache, block_tables, seq_lens, softmax_scale, out,
                       lse, workspace, q_scale=1.0, kv_scale=1.0, stream=None) -> None:
    """Second kernel only (LSE merge of the partials; no-op when split_kv == 1)."""
    _call("mla_decode_combine", plan, q, kv_cache, block_tables, seq_lens, softmax_scale, out,
          lse, workspace, q_scale, kv_scale, stream)


def _call_prefill(name, plan, q, cu_seqlens_q, kv_cache, block_tables, seq_lens, softmax_scale, out, lse,
                  workspace, q_scale, kv_scale, stream):
    _check_tensors(q, cu_seqlens_q=cu_seqlens_q, kv_cache=kv_cache, block_tables=block_tables,
                   seq_lens=seq_lens, out=out, lse=lse, workspace=workspace)
    if cu_seqlens_q is None or cu_seqlens_q.dtype != torch.int32:
        raise ValueError("cu_seqlens_q must be an int32 CUDA tensor")
    num_pages, page_size = int(kv_cache.shape[0]), int(kv_cache.shape[1])
    rc = getattr(_lib, name)(ctypes.byref(plan), _ptr(q), int(q.shape[0]), _ptr(cu_seqlens_q), _ptr(kv_cache),
                             num_pages, page_size, _ptr(block_tables), int(block_tables.shape[1]), _ptr(seq_lens),
                             float(softmax_scale), float(q_scale), float(kv_scale), _ptr(out), _ptr(lse),
                             _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                             _stream_of(q, stream))
    if rc != 0:
        raise MlaError(rc, name)


def mla_prefill(plan: MlaPlan, q, cu_seqlens_q, kv_cache, block_tables, seq_lens, softmax_scale, out, lse,
                workspace, q_scale=1.0, kv_scale=1.0, stream=None) -> None:
    """Enqueue one ragged prefill step: q [total_q, H, 576] packed, cu_seqlens_q int32 [B + 1],
    out bf16 [total_q, H, 512], lse fp32 [total_q, H] or None (include/mla_decode.h)."""
    _call_prefill("mla_prefill", plan, q, cu_seqlens_q, kv_cache, block_tables, seq_lens, softmax_scale, out,
                  lse, workspace, q_scale, kv_scale, stream)


def mla_prefill_partial(plan: MlaPlan, q, cu_seqlens_q, kv_cache, block_tables, seq_lens, softmax_scale, out,
                        lse, workspace, q_scale=1.0, kv_scale=1.0, stream=None) -> None:
    """First kernel of mla_prefill only."""
    _call_prefill("mla_prefill_partial", plan, q, cu_seqlens_q, kv_cache, block_tables, seq_lens, softmax_scale,
                  out, lse, workspace, q_scale, kv_scale, stream)


def mla_decode_status(workspace, clear=True, stream=None) -> int:
    """Synchronise and read the device status word (MLA_DEV_* bits)."""
    if stream is None:
        stream = torch.cuda.current_stream(workspace.device).cuda_stream
    v = ctypes.c_int32(0)
    rc = _lib.mla_decode_status(_ptr(workspace), ctypes.c_void_p(stream), int(bool(clear)),
                                ctypes.byref(v))
    if rc != 0:
        raise MlaError(rc, "mla_decode_status")
    return int(v.value)


def _stream_of(t, stream):
    """The raw cudaStream_t to launch on: torch's current stream of t's device unless `stream` is given."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def _allocating_on(t, stream):
    """Context in which torch allocates and fills for work that is launched on `stream`."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, t.device) if stream else torch.cuda.default_stream(t.device)
    return torch.cuda.stream(stream)


def kv_pack(latent, rope, slot_mapping, kv_cache, kv_scale=1.0, device_status=None, stream=None) -> None:
    """Write tokens into the paged cache, fused with FP8 quantisation when kv_cache is FP8.

    latent [n, 512] and rope [n, 64] (bf16 or fp16), slot_mapping [n] int64
    (page * 64 + offset; negative = skip), kv_cache [num_pages, 64, 576] of
    the inputs' dtype or float8_e4m3fn; see include/mla_decode.h.
    """
    _check_tensors(latent, rope=rope, slot_mapping=slot_mapping, kv_cache=kv_cache, device_status=device_status)
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if latent.dtype != rope.dtype:
        raise ValueError("latent and rope must have one dtype")
    in_dtype = _dtype_code(latent.dtype)
    cache_dtype = _dtype_code(kv_cache.dtype)
    rc = _lib.mla_kv_pack(_ptr(latent), _ptr(rope), int(latent.shape[0]), _ptr(slot_mapping), _ptr(kv_cache),
                          int(kv_cache.shape[0]), int(kv_cache.shape[1]), in_dtype, cache_dtype, float(kv_scale),
                          _ptr(device_status), _stream_of(latent, stream))
    if rc != 0:
        raise MlaError(rc, "mla_kv_pack")


def kv_amax(latent, rope, out=None, stream=None) -> torch.Tensor:
    """Device fp32 [1]: the largest |x| over latent and rope (NaN ignored)."""
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=latent.device)
    _check_tensors(latent, rope=rope, out=out)
    rc = _lib.mla_kv_amax(_ptr(latent), _ptr(rope), int(latent.shape[0]), _dtype_code(latent.dtype), _ptr(out),
                          _stream_of(latent, stream))
    if rc != 0:
        raise MlaError(rc, "mla_kv_amax")
    return out


def _weight_rows(name, t, index):
    """Checks an fp32 [B, columns] tensor on device `index` whose rows may lie apart; returns its row stride."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{index}")
    if t.dtype is not torch.float32 or t.dim() != 2 or (t.stride(1) != 1 and t.size(1) > 1):
        raise ValueError(f"{name} must be float32 [batch, columns] with adjacent columns")
    stride = t.stride(0)
    return stride if t.size(0) > 1 else max(stride, t.size(1))


def key_weights(plan: MlaPlan, q, kv_cache, block_tables, seq_lens, softmax_scale, lse, out, device_status,
                weights=None, decay=1.0, q_scale=1.0, kv_scale=1.0, cu_seqlens_q=None, stream=None) -> torch.Tensor:
    """The attention weight every cached key received in one step: out[b, j] = decay * weights[b, j] + the sum of
    exp(scaled score - lse) over the step's rows that see key j, for j < seq_lens[b] (the rest of `out` stays).

    Pass the plan, q, cache, tables and lse of the attention call it follows (cu_seqlens_q too for a prefill plan).
    `weights` and `out` are fp32 [B, columns] (rows may be strided) and may be the same tensor; weights = None counts
    as zeros. device_status: an int32 device word for MLA_DEV_* bits. See include/mla_decode.h.
    """
    _check_tensors(q, q=q, kv_cache=kv_cache, block_tables=block_tables, seq_lens=seq_lens, lse=lse,
                   cu_seqlens_q=cu_seqlens_q, device_status=device_status)
    index, batch = q.get_device(), plan.batch
    dtype, rows = q.dtype, q.numel() // 576
    if dtype is not kv_cache.dtype or _TORCH_CODES.get(dtype) != plan.dtype:
        raise ValueError("q and kv_cache must have the plan's dtype")
    if kv_cache.dim() != 3 or kv_cache.size(2) != 576 or q.size(-1) != 576:
        raise ValueError("q and kv_cache must have 576 dims")
    if plan.varlen:
        if q.dim() != 3 or q.size(1) != plan.num_heads:
            raise ValueError("q must be [total_q, num_heads, 576]")
        if cu_seqlens_q is not None and (cu_seqlens_q.dtype is not torch.int32 or cu_seqlens_q.numel() != batch + 1):
            raise ValueError("cu_seqlens_q must be int32 [batch + 1]")
    elif rows != batch * plan.q_len * plan.num_heads:
        raise ValueError("q must be [batch, q_len, num_heads, 576] of the plan")
    if lse is None or lse.dtype is not torch.float32 or lse.numel() != rows:
        raise ValueError("lse must be float32 with one value per query row")
    if device_status is None or device_status.dtype is not torch.int32:
        raise ValueError("device_status must be an int32 CUDA tensor")
    if block_tables.dim() != 2 or block_tables.size(0) != batch or seq_lens.numel() != batch:
        raise ValueError("block_tables and seq_lens must have one row per batch entry")
    out_stride, in_stride = _weight_rows("out", out, index), 0
    if out.size(0) != batch:
        raise ValueError("out must have one row per batch entry")
    if weights is not None:
        in_stride = _weight_rows("weights", weights, index)
        if weights.shape != out.shape:
            raise ValueError("weights and out must have one shape")
    rc = _lib.mla_key_weights(ctypes.byref(plan), _ptr(q), q.size(0), _ptr(cu_seqlens_q), _ptr(kv_cache),
                              kv_cache.size(0), kv_cache.size(1), _ptr(block_tables), block_tables.size(1),
                              _ptr(seq_lens), float(softmax_scale), float(q_scale), float(kv_scale), _ptr(lse),
                              _ptr(weights), in_stride, float(decay), _ptr(out), out_stride, out.size(1),
                              _ptr(device_status), _stream_of(q, stream))
    if rc != 0:
        raise MlaError(rc, "mla_key_weights")
    return out


def cache_evict(weights, seq_lens, kv_cache, block_tables, out_cache, out_block_tables, budget, sinks=0, recent=0,
                out_seq_lens=None, kept=None, out_weights=None, device_status=None, stream=None):
    """Cut every sequence to at most `budget` keys: the first `sinks`, the last `recent` and, between them, those
    with the largest `weights` (fp32 [B, columns]); the rows that stay move, in order, to the pages of
    out_block_tables in out_cache (which may be kv_cache, on pages block_tables does not name).

    Returns (out_seq_lens int32 [B], kept int32 [B, budget]: the positions that stay, then -1, out_weights fp32
    [B, budget]: their weights); each is allocated when not given. See include/mla_decode.h.
    """
    _check_tensors(seq_lens, seq_lens=seq_lens, kv_cache=kv_cache, block_tables=block_tables, out_cache=out_cache,
                   out_block_tables=out_block_tables, out_seq_lens=out_seq_lens, kept=kept,
                   device_status=device_status)
    B, budget, index, dtype = seq_lens.numel(), int(budget), seq_lens.get_device(), kv_cache.dtype
    if dtype is not out_cache.dtype or kv_cache.dim() != 3 or out_cache.dim() != 3 or kv_cache.size(2) != 576 or \
            out_cache.size(2) != 576 or out_cache.size(1) != kv_cache.size(1):
        raise ValueError("kv_cache and out_cache must be [pages, 64, 576] of one dtype")
    if out_block_tables.dtype is not torch.int32 or (device_status is not None and
                                                     device_status.dtype is not torch.int32):
        raise ValueError("out_block_tables and device_status must be int32")
    stride = _weight_rows("weights", weights, index)
    if block_tables.dim() != 2 or out_block_tables.dim() != 2 or block_tables.size(0) != B or \
            out_block_tables.size(0) != B or weights.size(0) != B:
        raise ValueError("weights and the block tables must have one row per batch entry")
    if budget < 1:
        raise MlaError(MLA_ERR_INVALID_ARG, "mla_cache_evict")
    with _allocating_on(seq_lens, stream):
        if out_seq_lens is None:
            out_seq_lens = torch.empty(B, dtype=torch.int32, device=seq_lens.device)
        if kept is None:
            kept = torch.empty((B, budget), dtype=torch.int32, device=seq_lens.device)
        if out_weights is None:
            out_weights = torch.zeros((B, budget), dtype=torch.float32, device=seq_lens.device)
    if out_seq_lens.dtype is not torch.int32 or out_seq_lens.numel() != B:
        raise ValueError("out_seq_lens must be int32 [batch]")
    if kept.dtype is not torch.int32 or kept.dim() != 2 or kept.size(0) != B or kept.size(1) != budget:
        raise ValueError("kept must be int32 [batch, budget]")
    out_stride = _weight_rows("out_weights", out_weights, index)
    if out_weights.size(0) != B or out_weights.size(1) < budget:
        raise ValueError("out_weights must be float32 [batch, >= budget]")
    rc = _lib.mla_cache_evict(_ptr(weights), stride, weights.size(1), _ptr(seq_lens), B, budget, int(sinks),
                              int(recent), _ptr(kv_cache), kv_cache.size(0), kv_cache.size(1), _ptr(block_tables),
                              block_tables.size(1), _ptr(out_cache), out_cache.size(0), _ptr(out_block_tables),
                              out_block_tables.size(1), _TORCH_CODES.get(dtype, -1), _ptr(out_seq_lens), _ptr(kept),
                              _ptr(out_weights), out_stride, _ptr(device_status), _stream_of(seq_lens, stream))
    if rc != 0:
        raise MlaError(rc, "mla_cache_evict")
    return out_seq_lens, kept, out_weights


def alloc_workspace(plan: MlaPlan, device) -> torch.Tensor:
    """A zeroed workspace tensor of plan.workspace_bytes (torch allocations are 256-byte aligned)."""
    return torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device=device)


class _WithWorkspace:
    """The workspace of a plan (it may be replaced by another of the plan's size) and its status word."""

    @property
    def workspace(self) -> torch.Tensor:
        return self._workspace

    @workspace.setter
    def workspace(self, workspace: torch.Tensor) -> None:
        self._workspace = workspace
        # the status word, where every kernel of this object reports
        self._status = None if workspace is None else workspace.view(-1).view(torch.uint8)[:4].view(torch.int32)

    def status(self, clear=True) -> int:
        return mla_decode_status(self.workspace, clear)


class MlaDecoder(_WithWorkspace):
    """Plan + workspace for one decode shape; call it once per decode step."""

    def __init__(self, batch, q_len, num_heads, max_seq_len, dtype, device, split_kv=0, fold=0,
                 kernel="auto", window=0, sinks=0):
        self.plan = mla_decode_plan_custom(batch, q_len, num_heads, max_seq_len, dtype,
                                           split_kv, fold, kernel)
        if window:
            mla_decode_plan_window(self.plan, window)
        if sinks:
            mla_decode_plan_sinks(self.plan, sinks)
        self.device = torch.device(device)
        self.workspace = alloc_workspace(self.plan, self.device)
        self.batch, self.q_len, self.num_heads = batch, q_len, num_heads

    def __call__(self, q, kv_cache, block_tables, seq_lens, softmax_scale, q_scale=1.0,
                 kv_scale=1.0, out=None, lse=None, want_lse=True, stream=None):
        B, T, H = self.batch, self.q_len, self.num_heads
        if out is None:
            out = torch.empty((B, T, H, 512), dtype=torch.bfloat16, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((B, T, H), dtype=torch.float32, device=self.device)
        mla_decode(self.plan, q, kv_cache, block_tables, seq_lens, softmax_scale, out, lse,
                   self.workspace, q_scale, kv_scale, stream)
        return out, lse

    def key_weights(self, q, kv_cache, block_tables, seq_lens, softmax_scale, lse, out, weights=None,
                    decay=1.0, q_scale=1.0, kv_scale=1.0, stream=None):
        """The weight every cached key received in the step that returned `lse` (see key_weights); device-side
        problems show in status()."""
        return key_weights(self.plan, q, kv_cache, block_tables, seq_lens, softmax_scale, lse, out, self._status,
                           weights, decay, q_scale, kv_scale, stream=stream)


class MlaPrefill(_WithWorkspace):
    """Plan + workspace for one ragged prefill shape (batch, longest entry, H, longest sequence)."""

    def __init__(self, batch, max_q_len, num_heads, max_seq_len, dtype, device, split_kv=0, fold=0,
                 kernel="auto", window=0, sinks=0):
        self.plan = mla_prefill_plan(batch, max_q_len, num_heads, max_seq_len, dtype, split_kv, fold, kernel)
        if window:
            mla_decode_plan_window(self.plan, window)
        if sinks:
            mla_decode_plan_sinks(self.plan, sinks)
        self.device = torch.device(device)
        self.workspace = alloc_workspace(self.plan, self.device)
        self.num_heads = num_heads

    def __call__(self, q, cu_seqlens_q, kv_cache, block_tables, seq_lens, softmax_scale, q_scale=1.0,
                 kv_scale=1.0, out=None, lse=None, want_lse=True, stream=None):
        total_q, H = int(q.shape[0]), self.num_heads
        if out is None:
            out = torch.empty((total_q, H, 512), dtype=torch.bfloat16, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((total_q, H), dtype=torch.float32, device=self.device)
        mla_prefill(self.plan, q, cu_seqlens_q, kv_cache, block_tables, seq_lens, softmax_scale, out, lse,
                    self.workspace, q_scale, kv_scale, stream)
        return out, lse

    def key_weights(self, q, cu_seqlens_q, kv_cache, block_tables, seq_lens, softmax_scale, lse, out, weights=None,
                    decay=1.0, q_scale=1.0, kv_scale=1.0, stream=None):
        """The weight every cached key received in the step that returned `lse` (see key_weights); device-side
        problems show in status()."""
        return key_weights(self.plan, q, kv_cache, block_tables, seq_lens, softmax_scale, lse, out, self._status,
                           weights, decay, q_scale, kv_scale, cu_seqlens_q, stream=stream)
