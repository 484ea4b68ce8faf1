"""GB300 (sm_103a) MLA latent decode: thin Python binding of libmla_decode.so.

Every function here only marshals arguments (torch tensors -> device
pointers, the current CUDA stream) into the C ABI declared in
include/mla_decode.h; all arithmetic runs in the library's CUDA kernels.
There is no CPU fallback: if the library is missing, loading it raises.

    import mla_latent_decode_gb300 as mla
    O_part, LSE_part = mla.decode_partial(q_nope, q_rope, kv, ..., num_splits)
    out, lse = mla.lse_combine(O_part, LSE_part)
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_decode.so")
ROW_DIM, NOPE_DIM, ROPE_DIM, VALUE_DIM, PAGE_SIZE = 576, 512, 64, 512, 64
KV_BF16, KV_FP8_E4M3, KV_FP4_E2M1 = 0, 1, 2
_KV_DTYPE = {"bf16": KV_BF16, "fp8_e4m3": KV_FP8_E4M3, "fp4_e2m1": KV_FP4_E2M1}
FP4_ROW_BYTES = 352  # 512 E2M1 codes, 32 E4M3 block scales, 64 E4M3 RoPE codes
FP4_FEW_ROWS = 96  # query rows a request up to which one CTA serves a part
PLAN_FEW_SPLITS = 160  # the default planners' largest split count for such requests
ROWS_PER_UNIT = 256  # query rows per work unit of the BF16 tensor-core kernel
STATUS_WAIT_TIMEOUT, STATUS_BAD_LENGTH, STATUS_BAD_SLOT, STATUS_BAD_WORK = 1, 2, 4, 8
STATUS_BAD_POSITION = 16
STATUS_NO_PAGES, STATUS_BAD_PARENT, STATUS_BAD_SCORE = 32, 64, 128
BEAM_MAX_W, BEAM_MAX_K, FORK_MAX_ROWS, PREFILL_MAX_PARTS = 32, 64, 4096, 32
_LOGITS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

_lib = None
_lock = threading.Lock()


class MlaError(RuntimeError):
    """A non-zero return code of the C library, with its message."""

    def __init__(self, code: int, msg: str):
        super().__init__(f"{msg} (code {code})")
        self.code = code


def library() -> ctypes.CDLL:
    """Load libmla_decode.so (built by ``build.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        p, i32, i64, f32, f64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                 ctypes.c_float, ctypes.c_double)
        sig = {
            "mla_last_error_string": (ctypes.c_char_p, []),
            "mla_num_sms": (i32, [i32]),
            "mla_cluster_slots": (i32, []),
            "mla_plan_heuristic": (i32, [i32, i32]),
            "mla_plan_ex": (i32, [i32, i32, i32, i32, p, i32, i32, f64, f64, p, p, p]),
            "mla_plan": (i32, [i32, i32, i32, i32, i32, p, i32, p, p]),
            "mla_plan_parts_ex": (i32, [i32, i32, i32, i32, p, i32, i32, i32, f64,
                                        f64, p, p, p, p]),
            "mla_plan_parts": (i32, [i32, i32, i32, i32, i32, p, i32, i32, p, p,
                                     p]),
            "mla_plan_sched_ex": (i32, [i32, i32, i32, i32, p, i32, i32, i32, f64,
                                        f64, p, p, p, i64, p, p, p]),
            "mla_plan_sched": (i32, [i32, i32, i32, i32, i32, p, i32, i32, p, p,
                                     p, i64, p, p]),
            "mla_check_page_table": (i32, [p, i64, p, p, i32, i32, i32, i64]),
            "mla_decode_partial": (i32, [p, p, p, p, i32, i64, p, i64, p, p, i32,
                                         i32, i32, i32, i32, f32, i32, p, p, i32,
                                         p, p, p, p]),
            "mla_decode_partial_bf16_parts": (i32, [p, p, p, p, i32, i64, p, i64, p,
                                                    p, i32, i32, i32, i32, i32, f32,
                                                    i32, p, p, i32, p, p, p, p]),
            "mla_decode_partial_simt": (i32, [p, p, p, p, i32, i64, p, i64, p, p,
                                              i32, i32, i32, i32, i32, f32, i32, p,
                                              p, p, p, p]),
            "mla_decode": (i32, [p, p, p, p, i32, i64, p, i64, p, p, i32, i32,
                                 i32, i32, i32, f32, i32, p, p, i32, p, p, p, p,
                                 p, p, p]),
            "mla_decode_scratch": (i32, [p, p, p, p, i32, i64, p, i64, p, p, i32,
                                         i32, i32, i32, i32, f32, i32, p, p, i32,
                                         p, p, p, p]),
            "mla_scratch_bytes": (i64, [i32, i32, i32, i32, i32]),
            "mla_kv_write": (i32, [p, i64, p, p, i32, p, i64, p, p]),
            "mla_kv_append": (i32, [p, i64, i64, p, f32, p, p, p, i64, i32, p, i32, p,
                                    i64, p, i64, i64, p, i64, i64, i32, p, p]),
            "mla_kv_read": (i32, [p, i32, p, i64, p, i64, p, i64, p, p]),
            "mla_add_rms_norm": (i32, [p, i64, p, i64, p, i64, p, f32, i64, i32, p, i64,
                                       p, i64, p, i64, i32, p]),
            "mla_plan_prefill": (i32, [p, p, p, i32, i32, i32, i32, i32, p, i64, p, p, p]),
            "mla_prefill": (i32, [p, i64, i64, p, i64, i64, i64, p, i64, i64, p, i64, p, i64, i64,
                                  i64, i32, p, p, p, i32, i32, f32, p, i32, i32, i32, p, p, p, p, p,
                                  p]),
            "mla_beam_select": (i32, [p, i32, i64, i64, p, p, i32, i32, i32, i32, i32, p, p, p, p,
                                      p]),
            "mla_pages_fork": (i32, [p, i64, p, p, p, p, i32, p, i64, p, p, i64, p, p, p, p]),
            "mla_pages_compact": (i32, [p, i64, p, i32, p, i64, p, i64, p, p, i32, p, p, p]),
            "mla_kv_copy": (i32, [p, i32, p, i64, p, p, p, p, i64, p, p]),
            "mla_absorb_q": (i32, [p, p, p, i32, i32, p, p]),
            "mla_project_out": (i32, [p, p, p, i32, i32, p, p]),
            "mla_lse_combine": (i32, [p, p, i32, i64, p, p, p]),
            "mla_lse_combine_bf16_parts": (i32, [p, p, i32, i64, p, p, p]),
            "mla_debug_gather": (i32, [p, i32, i64, p, i64, p, p, i32, i32, p, p]),
            "mla_debug_wait": (i32, [i32, i32, p, p, p]),
            "mla_debug_quotients": (i32, [p, p, p]),
            "mla_debug_beam_math": (i32, [p, p, i64, p, p, p]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(rc: int) -> int:
    if rc < 0:
        raise MlaError(rc, library().mla_last_error_string().decode())
    return rc


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_HERE_ALREADY = contextlib.nullcontext()
# torch.cuda.current_stream(), without the Stream object around the handle
# (2.9 us of a call's host time on a Grace core, against 0.1 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# torch.cuda.current_device() without its test for a first use of CUDA, which a
# CUDA tensor has behind it (0.3 us of host time against 0.1)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(t: torch.Tensor):
    """Make the tensor's device current for a call: the library launches
    on (and looks up per-device state for) the current device."""
    if t.is_cuda and t.device.index == torch.cuda.current_device():
        return _HERE_ALREADY
    return torch.cuda.device(t.device)


def _stream(stream: Optional[torch.cuda.Stream]):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _launch(t: torch.Tensor, stream: Optional[torch.cuda.Stream], fn, *args) -> None:
    """fn(*args, stream) on the tensor's device; raises what it returns."""
    if t.is_cuda and _raw_stream is not None and t.device.index == (dev := _current_device()):
        rc = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    else:
        with _on(t):
            rc = fn(*args, _stream(stream))
    if rc < 0:
        _check(rc)


def _host_i32(x) -> "ctypes.Array":
    vals = [int(v) for v in (x.tolist() if torch.is_tensor(x) else x)]
    return (ctypes.c_int32 * len(vals))(*vals)


# ------------------------------------------------------------------ planning
def num_sms(device: int = 0) -> int:
    return _check(library().mla_num_sms(device))


def cluster_slots() -> int:
    """Concurrently resident work units (4-CTA clusters) of the tensor-core
    decode kernel on this device."""
    return _check(library().mla_cluster_slots())


def _s_max(kv_dtype: str, q_len: int, H: int) -> int:
    """The default planners' largest split count."""
    return PLAN_FEW_SPLITS if kv_dtype == "fp4_e2m1" and q_len * H <= FP4_FEW_ROWS else 64


def plan_heuristic(B: int, q_len: int) -> int:
    """The pages' split rule max(1, min(148 // B // (2 q_len), 32))."""
    return _check(library().mla_plan_heuristic(B, q_len))


def plan_ex(seq_lens: Sequence[int], q_len: int, H: int, slots: int,
            s_max: int = 64, c0: float = 32.0, lam: float = 1.0,
            rows_per_unit: int = ROWS_PER_UNIT):
    """Wave-rounding planner: returns (num_splits, wave_eff, makespan)."""
    arr = _host_i32(seq_lens)
    S, eff, ms = ctypes.c_int(), ctypes.c_float(), ctypes.c_double()
    _check(library().mla_plan_ex(len(arr), q_len, H, rows_per_unit, arr,
                                 slots, s_max, float(c0), float(lam),
                                 ctypes.byref(S), ctypes.byref(eff),
                                 ctypes.byref(ms)))
    return S.value, eff.value, ms.value


def plan(B: int, q_len: int, H: int, seq_lens, num_shards: int = 1,
         num_sms: int = 0, kv_dtype: str = "bf16"):
    """Planner with the library defaults for the kernel that serves
    `kv_dtype`; num_sms=0 asks the device."""
    arr = _host_i32(seq_lens)
    assert len(arr) == B * num_shards
    S, eff = ctypes.c_int(), ctypes.c_float()
    _check(library().mla_plan(B, q_len, H, num_shards, _KV_DTYPE[kv_dtype],
                              arr, num_sms, ctypes.byref(S), ctypes.byref(eff)))
    return S.value, eff.value


def plan_parts_ex(seq_lens: Sequence[int], q_len: int, H: int, slots: int,
                  s_max: int = 64, max_parts: int = 8, c0: float = 32.0,
                  lam: float = 1.0, rows_per_unit: int = ROWS_PER_UNIT):
    """Per-request split planner: returns (S, boundaries np.int32 [V, S+1],
    wave_eff, makespan)."""
    import numpy as np
    arr = _host_i32(seq_lens)
    V = len(arr)
    out = (ctypes.c_int32 * (V * (s_max + 1)))()
    S, eff, ms = ctypes.c_int(), ctypes.c_float(), ctypes.c_double()
    _check(library().mla_plan_parts_ex(V, q_len, H, rows_per_unit, arr, slots,
                                       s_max, max_parts, float(c0), float(lam),
                                       out, ctypes.byref(S), ctypes.byref(eff),
                                       ctypes.byref(ms)))
    bnd = np.frombuffer(out, dtype=np.int32)[:V * (S.value + 1)]
    return S.value, bnd.reshape(V, S.value + 1).copy(), eff.value, ms.value


def plan_parts(B: int, q_len: int, H: int, seq_lens, num_shards: int = 1,
               num_sms: int = 0, kv_dtype: str = "bf16", max_parts: int = 8):
    """Per-request split planner with the library defaults for the kernel
    that serves `kv_dtype`: returns (S, boundaries np.int32 [V, S+1],
    wave_eff); num_sms=0 asks the device."""
    import numpy as np
    arr = _host_i32(seq_lens)
    V = len(arr)
    assert V == B * num_shards
    out = (ctypes.c_int32 * (V * (_s_max(kv_dtype, q_len, H) + 1)))()
    S, eff = ctypes.c_int(), ctypes.c_float()
    _check(library().mla_plan_parts(B, q_len, H, num_shards, _KV_DTYPE[kv_dtype],
                                    arr, num_sms, max_parts, out,
                                    ctypes.byref(S), ctypes.byref(eff)))
    bnd = np.frombuffer(out, dtype=np.int32)[:V * (S.value + 1)]
    return S.value, bnd.reshape(V, S.value + 1).copy(), eff.value


def plan_sched_ex(seq_lens: Sequence[int], q_len: int, H: int, slots: int,
                  s_max: int = 64, max_parts: int = 8, c0: float = 32.0,
                  lam: float = 1.0, rows_per_unit: int = ROWS_PER_UNIT):
    """Work-balanced scheduler: returns (S, boundaries np.int32 [V, S+1],
    work np.int32 [V*S*U] (unit ids, longest first), wave_eff, makespan)."""
    import numpy as np
    arr = _host_i32(seq_lens)
    V = len(arr)
    U = -(-q_len * H // rows_per_unit)
    cap = V * s_max * U
    bnd_out = (ctypes.c_int32 * (V * (s_max + 1)))()
    work_out = (ctypes.c_int32 * cap)()
    S, n = ctypes.c_int(), ctypes.c_int64()
    eff, ms = ctypes.c_float(), ctypes.c_double()
    _check(library().mla_plan_sched_ex(V, q_len, H, rows_per_unit, arr, slots,
                                       s_max, max_parts, float(c0), float(lam),
                                       bnd_out, ctypes.byref(S), work_out, cap,
                                       ctypes.byref(n), ctypes.byref(eff),
                                       ctypes.byref(ms)))
    bnd = np.frombuffer(bnd_out, dtype=np.int32)[:V * (S.value + 1)]
    work = np.frombuffer(work_out, dtype=np.int32)[:n.value].copy()
    return S.value, bnd.reshape(V, S.value + 1).copy(), work, eff.value, ms.value


def plan_sched(B: int, q_len: int, H: int, seq_lens, num_shards: int = 1,
               num_sms: int = 0, kv_dtype: str = "bf16", max_parts: int = 8):
    """Work-balanced scheduler with the library defaults for the kernel that
    serves `kv_dtype`: returns (S, boundaries np.int32 [V, S+1], work
    np.int32 [V*S*U] in launch order, wave_eff); num_sms=0 asks the device."""
    import numpy as np
    arr = _host_i32(seq_lens)
    V = len(arr)
    assert V == B * num_shards
    s_max = _s_max(kv_dtype, q_len, H)
    cap = V * s_max * (-(-q_len * H // (FP4_FEW_ROWS if kv_dtype == "fp4_e2m1" else 128)))
    bnd_out = (ctypes.c_int32 * (V * (s_max + 1)))()
    work_out = (ctypes.c_int32 * cap)()
    S, n, eff = ctypes.c_int(), ctypes.c_int64(), ctypes.c_float()
    _check(library().mla_plan_sched(B, q_len, H, num_shards, _KV_DTYPE[kv_dtype],
                                    arr, num_sms, max_parts, bnd_out,
                                    ctypes.byref(S), work_out, cap,
                                    ctypes.byref(n), ctypes.byref(eff)))
    bnd = np.frombuffer(bnd_out, dtype=np.int32)[:V * (S.value + 1)]
    work = np.frombuffer(work_out, dtype=np.int32)[:n.value].copy()
    return S.value, bnd.reshape(V, S.value + 1).copy(), work, eff.value


def check_page_table(req_to_token, seq_lens, kv_limit, q_len: int,
                     num_slots: int, page_size: int = PAGE_SIZE) -> None:
    """Host validation of a page table (raises MlaError on a bad entry)."""
    r2t = req_to_token.detach().to("cpu", torch.int32).contiguous()
    sl = seq_lens.detach().to("cpu", torch.int32).contiguous()
    kl = None if kv_limit is None else kv_limit.detach().to("cpu", torch.int32).contiguous()
    _check(library().mla_check_page_table(
        _ptr(r2t), r2t.shape[1], _ptr(sl), _ptr(kl), r2t.shape[0], q_len,
        page_size, num_slots))


# ------------------------------------------------------------------ kernels
_BF16, _F32, _I32, _BYTES = (torch.bfloat16, torch.float32, torch.int32,
                             (torch.uint8, torch.float8_e4m3fn))


def _kv_dtype(kv: torch.Tensor) -> int:
    dtype = kv.dtype
    if dtype is _BF16:
        return KV_BF16
    if dtype in _BYTES:
        # the two byte pools differ in their row: 576 E4M3 codes, or 352 bytes
        return KV_FP4_E2M1 if kv.shape[-1] == FP4_ROW_BYTES else KV_FP8_E4M3
    raise TypeError(f"kv dtype {kv.dtype}: expected bfloat16 or uint8 (E4M3, FP4)")


def _not_a_buffer(t: torch.Tensor, name: str, dtype, n: int) -> ValueError:
    return ValueError(f"{name}: expected {n} contiguous {dtype} values, got {t.dtype} "
                      f"{tuple(t.shape)} with strides {t.stride()}")


def _check_buffer(t: torch.Tensor, name: str, dtype, n: int) -> None:
    """An array that the library reads or writes by its address alone."""
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise _not_a_buffer(t, name, dtype, n)


def _check_fp4(shape, q_nope, q_rope, kv, kv_scale, req_to_token, seq_lens, kv_limit, num_shards,
               num_splits, split_pages, work, status) -> int:
    """The layouts the FP4 decode reads (its pool and its queries are told from
    the other formats' by shape, so a wrong one is refused here); returns the
    number of query rows.  shape: q_nope's.  (An attribute of a tensor costs 0.06
    to 0.2 us, a call 0.1, and a small decode takes 9: each is read once, in place.)"""
    B, q_len, H, width = shape
    rows, V = B * q_len * H, B * num_shards
    if q_nope.dtype is not _BF16 or width != NOPE_DIM or not q_nope.is_contiguous():
        raise ValueError("q_nope: expected contiguous bfloat16 [B, q_len, H, 512], got "
                         f"{q_nope.dtype} {tuple(q_nope.shape)} with strides {q_nope.stride()}")
    if q_rope.dtype is not _BF16 or q_rope.numel() != rows * ROPE_DIM or not q_rope.is_contiguous():
        raise ValueError("q_rope: expected contiguous bfloat16 [B, q_len, H, 64], got "
                         f"{q_rope.dtype} {tuple(q_rope.shape)} with strides {q_rope.stride()}")
    if not kv.is_contiguous() or kv.ndim != 2:
        raise ValueError(f"kv: expected a contiguous [num_slots, {FP4_ROW_BYTES}] pool")
    if kv_scale is None or kv_scale.dtype is not _F32 or kv_scale.numel() < 1:
        raise ValueError("kv_scale: expected one float32 value, the pool's factor")
    if req_to_token.dtype is not _I32 or req_to_token.ndim != 2 or \
            req_to_token.stride()[1] != 1 or req_to_token.shape[0] < V:
        raise ValueError(f"req_to_token: expected int32 [{V}, stride] with contiguous rows, got "
                         f"{req_to_token.dtype} {tuple(req_to_token.shape)}")
    if seq_lens.dtype is not _I32 or seq_lens.numel() < V or not seq_lens.is_contiguous():
        raise _not_a_buffer(seq_lens, "seq_lens", _I32, V)
    if kv_limit is not None:
        _check_buffer(kv_limit, "kv_limit", _I32, V * q_len)
    if split_pages is not None and (
            split_pages.dtype is not _I32 or split_pages.numel() < V * (num_splits + 1) or
            not split_pages.is_contiguous()):
        raise _not_a_buffer(split_pages, "split_pages", _I32, V * (num_splits + 1))
    # its length is checked by the library
    if work is not None and (work.dtype is not _I32 or not work.is_contiguous()):
        raise _not_a_buffer(work, "work", _I32, 0)
    if status is not None:
        _check_buffer(status, "status", _I32, 1)
    return rows


def decode_partial(q_nope, q_rope, kv, kv_scale, req_to_token, seq_lens,
                   kv_limit, num_splits: int, sm_scale: float,
                   num_shards: int = 1, O_part=None, LSE_part=None,
                   status=None, simt: bool = False, stream=None,
                   split_pages=None, work=None, part_dtype=None):
    """Partial (O, LSE) per split and shard; see mla_decode_partial.
    `kv`: bf16 [slots, 576], uint8 [slots, 576] (E4M3, kv_scale fp32 [slots]) or
    uint8 [slots, 352] (FP4, kv_scale fp32 [1]);
    `split_pages`: device int32 [num_shards*B, num_splits+1] or None;
    `work`: device int32 unit ids in launch order (plan_sched) or None
    (tensor-core path only).  A bf16 O_part (given, or part_dtype=
    torch.bfloat16) calls mla_decode_partial_bf16_parts.

    Returns (O_part [S, shards, B, q, H, 512], fp32 unless bf16 was asked
    for, LSE_part fp32 [S, shards, B, q, H]); outputs are allocated with
    torch unless given.
    """
    B, q_len, H, _ = shape = q_nope.shape
    kind = _kv_dtype(kv)
    if kind == KV_FP4_E2M1:
        parts = num_splits * num_shards * _check_fp4(
            shape, q_nope, q_rope, kv, kv_scale, req_to_token, seq_lens, kv_limit, num_shards,
            num_splits, split_pages, work, status)
        if O_part is not None and (
                O_part.dtype not in (_F32, _BF16) or O_part.numel() < parts * VALUE_DIM or
                not O_part.is_contiguous()):
            raise _not_a_buffer(O_part, "O_part", "float32 or bfloat16", parts * VALUE_DIM)
        if LSE_part is not None and (
                LSE_part.dtype is not _F32 or LSE_part.numel() < parts or
                not LSE_part.is_contiguous()):
            raise _not_a_buffer(LSE_part, "LSE_part", _F32, parts)
    if O_part is None:
        O_part = torch.empty((num_splits, num_shards, B, q_len, H, VALUE_DIM),
                             dtype=part_dtype or torch.float32, device=q_nope.device)
    bf16_parts = O_part.dtype is _BF16
    if LSE_part is None:
        LSE_part = torch.empty((num_splits, num_shards, B, q_len, H),
                               dtype=torch.float32, device=q_nope.device)
    args = (q_nope.data_ptr(), q_rope.data_ptr(), kv.data_ptr(),
            None if kv_scale is None else kv_scale.data_ptr(),
            kind, kv.shape[0], req_to_token.data_ptr(),
            req_to_token.stride()[0], seq_lens.data_ptr(),
            None if kv_limit is None else kv_limit.data_ptr(), B, q_len,
            H, num_shards, PAGE_SIZE, float(sm_scale), num_splits,
            None if split_pages is None else split_pages.data_ptr())
    tail = (O_part.data_ptr(), LSE_part.data_ptr(), None if status is None else status.data_ptr())
    if simt:
        if work is not None or bf16_parts:
            raise ValueError("the CUDA-core path takes no work list and "
                             "writes fp32 parts")
        _launch(q_nope, stream, library().mla_decode_partial_simt, *args, *tail)
    else:
        fn = (library().mla_decode_partial_bf16_parts if bf16_parts
              else library().mla_decode_partial)
        listed = (None, 0) if work is None else (work.data_ptr(), work.numel())
        _launch(q_nope, stream, fn, *args, *listed, *tail)
    return O_part, LSE_part


def fused_counters(B: int, q_len: int, H: int, device) -> torch.Tensor:
    """Zeroed arrival counters for decode_fused (int32 [B * ceil(q_len*H/128)]);
    every call leaves them zero again, so one tensor serves every call."""
    return torch.zeros((B * ((q_len * H + 127) // 128),), dtype=torch.int32,
                       device=device)


def decode_fused(q_nope, q_rope, kv, kv_scale, req_to_token, seq_lens,
                 kv_limit, num_splits: int, sm_scale: float,
                 num_shards: int = 1, O_part=None, LSE_part=None,
                 counters=None, out=None, lse_out=None, status=None,
                 stream=None, split_pages=None, work=None):
    """Partial decode and LSE combine in one launch; see mla_decode.

    Returns (out bf16 [B, q, H, 512], lse fp32 [B, q, H]); workspace and
    outputs are allocated with torch unless given."""
    B, q_len, H, _ = shape = q_nope.shape
    dev = q_nope.device
    kind = _kv_dtype(kv)
    if kind == KV_FP4_E2M1:
        rows = _check_fp4(shape, q_nope, q_rope, kv, kv_scale, req_to_token, seq_lens, kv_limit,
                          num_shards, num_splits, split_pages, work, status)
        parts = num_splits * num_shards * rows
        for t, name, dtype, n in ((O_part, "O_part", torch.float32, parts * VALUE_DIM),
                                  (LSE_part, "LSE_part", torch.float32, parts),
                                  (counters, "counters", torch.int32, B * ((q_len * H + 127) // 128)),
                                  (out, "out", torch.bfloat16, rows * VALUE_DIM),
                                  (lse_out, "lse_out", torch.float32, rows)):
            if t is not None:
                _check_buffer(t, name, dtype, n)
    if O_part is None:
        O_part = torch.empty((num_splits, num_shards, B, q_len, H, VALUE_DIM),
                             dtype=torch.float32, device=dev)
    if LSE_part is None:
        LSE_part = torch.empty((num_splits, num_shards, B, q_len, H),
                               dtype=torch.float32, device=dev)
    if counters is None:
        counters = fused_counters(B, q_len, H, dev)
    if out is None:
        out = torch.empty((B, q_len, H, VALUE_DIM), dtype=torch.bfloat16, device=dev)
    if lse_out is None:
        lse_out = torch.empty((B, q_len, H), dtype=torch.float32, device=dev)
    with _on(q_nope):
        _check(library().mla_decode(
            _ptr(q_nope), _ptr(q_rope), _ptr(kv), _ptr(kv_scale), kind,
            kv.shape[0], _ptr(req_to_token), req_to_token.stride(0),
            _ptr(seq_lens), _ptr(kv_limit), B, q_len, H, num_shards, PAGE_SIZE,
            float(sm_scale), num_splits, _ptr(split_pages), _ptr(work),
            0 if work is None else work.numel(), _ptr(O_part), _ptr(LSE_part),
            _ptr(counters), _ptr(out), _ptr(lse_out), _ptr(status),
            _stream(stream)))
    return out, lse_out


def scratch_bytes(B: int, q_len: int, H: int, num_shards: int,
                  num_splits: int) -> int:
    """Static scratch bytes decode_scratch needs (see mla_scratch_bytes)."""
    return _check(library().mla_scratch_bytes(B, q_len, H, num_shards, num_splits))


def decode_scratch(q_nope, q_rope, kv, kv_scale, req_to_token, seq_lens,
                   kv_limit, num_splits: int, sm_scale: float,
                   num_shards: int = 1, out=None, lse_out=None, status=None,
                   stream=None, split_pages=None, work=None):
    """decode_fused with its workspace in the library's static scratch; see
    mla_decode_scratch (calls that may overlap on a device race on it)."""
    B, q_len, H, _ = shape = q_nope.shape
    dev = q_nope.device
    kind = _kv_dtype(kv)
    if kind == KV_FP4_E2M1:
        rows = _check_fp4(shape, q_nope, q_rope, kv, kv_scale, req_to_token, seq_lens, kv_limit,
                          num_shards, num_splits, split_pages, work, status)
        if out is not None:
            _check_buffer(out, "out", torch.bfloat16, rows * VALUE_DIM)
        if lse_out is not None:
            _check_buffer(lse_out, "lse_out", torch.float32, rows)
    if out is None:
        out = torch.empty((B, q_len, H, VALUE_DIM), dtype=torch.bfloat16, device=dev)
    if lse_out is None:
        lse_out = torch.empty((B, q_len, H), dtype=torch.float32, device=dev)
    with _on(q_nope):  # the scratch array used is the current device's
        _check(library().mla_decode_scratch(
            _ptr(q_nope), _ptr(q_rope), _ptr(kv), _ptr(kv_scale), kind,
            kv.shape[0], _ptr(req_to_token), req_to_token.stride(0),
            _ptr(seq_lens), _ptr(kv_limit), B, q_len, H, num_shards, PAGE_SIZE,
            float(sm_scale), num_splits, _ptr(split_pages), _ptr(work),
            0 if work is None else work.numel(), _ptr(out), _ptr(lse_out),
            _ptr(status), _stream(stream)))
    return out, lse_out


def kv_write(rows, slots, kv, kv_scale=None, status=None, stream=None):
    """Store bf16 latent rows [n, 576] at `slots` of the pool `kv` (bf16, or
    uint8 E4M3 bytes with `kv_scale`); see mla_kv_write."""
    n = rows.shape[0]
    _launch(kv, stream, library().mla_kv_write, _ptr(rows), n, _ptr(slots), _ptr(kv),
            _kv_dtype(kv), _ptr(kv_scale), kv.shape[0], _ptr(status))


def _rows_arg(t: torch.Tensor, name: str, n: int, width: int, dtype=torch.bfloat16):
    """A 2-D argument of n rows of `width` contiguous values (any row stride):
    its address and row stride."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not dtype or shape != (n, width) or (stride[1] != 1 and width > 1):
        raise ValueError(f"{name}: expected {dtype} [{n}, {width}] with contiguous rows, "
                         f"got {t.dtype} {tuple(shape)} with strides {stride}")
    return t.data_ptr(), stride[0] if n > 1 else max(stride[0], width)


def _int32_arg(t: torch.Tensor, name: str, n: int):
    if t.dtype is not torch.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous int32 values, got {t.dtype} "
                         f"{tuple(t.shape)}")
    return t.data_ptr()


def _pool_args(kv: torch.Tensor, kv_scale: Optional[torch.Tensor]):
    kind = _kv_dtype(kv)
    slots, width = kv.shape if kv.dim() == 2 else (0, 0)
    if width != (FP4_ROW_BYTES if kind == KV_FP4_E2M1 else ROW_DIM) or not kv.is_contiguous():
        raise ValueError(f"kv: expected a contiguous [num_slots, {ROW_DIM}] (FP4: "
                         f"{FP4_ROW_BYTES}) pool, got {tuple(kv.shape)} with strides {kv.stride()}")
    if kv_scale is None:
        return kv.data_ptr(), kind, None, slots
    need = slots if kind == KV_FP8_E4M3 else 1
    if kv_scale.dtype != torch.float32 or kv_scale.numel() < need or not kv_scale.is_contiguous():
        raise ValueError(f"kv_scale: expected {need} contiguous float32 values")
    return kv.data_ptr(), kind, kv_scale.data_ptr(), slots


def kv_append(rows, slots, positions, cos_sin, kv, kv_scale=None, norm_weight=None,
              eps: float = 1e-6, q_rope=None, q_out=None, interleaved: bool = True,
              status=None, stream=None):
    """Append new tokens to the pool: RMS norm of the latent (norm_weight bf16
    [512] or None), rotation of the RoPE key and of the queries by position,
    and the write in the pool's format, in one launch; see mla_kv_append.

    rows bf16 [n, 576] (rows may be strided), slots / positions int32 [n],
    cos_sin fp32 [max_pos, 64]; kv: bf16 [slots, 576], uint8 [slots, 576]
    (E4M3, kv_scale fp32 [slots]) or uint8 [slots, 352] (FP4, kv_scale fp32
    [1]); q_rope bf16 [n, H, 64] (strided) or None.  Returns q_out (allocated
    unless given; q_out=q_rope rotates in place), None without queries."""
    n = rows.shape[0]
    row_ptr, row_stride = _rows_arg(rows, "rows", n, ROW_DIM)
    kv_ptr, kind, scale_ptr, num_slots = _pool_args(kv, kv_scale)
    max_pos, pairs = cos_sin.shape if cos_sin.dim() == 2 else (0, 0)
    if cos_sin.dtype != torch.float32 or pairs != ROPE_DIM or not cos_sin.is_contiguous():
        raise ValueError("cos_sin: expected contiguous float32 [max_pos, 64]")
    weight_ptr = None
    if norm_weight is not None:
        if norm_weight.dtype != torch.bfloat16 or norm_weight.numel() != NOPE_DIM \
                or not norm_weight.is_contiguous():
            raise ValueError("norm_weight: expected 512 contiguous bfloat16 values")
        weight_ptr = norm_weight.data_ptr()
    H, q_args = 0, (None, 0, 0, None, 0, 0)
    if q_rope is not None:
        if q_out is None:
            q_out = torch.empty(q_rope.shape, dtype=torch.bfloat16, device=q_rope.device)
        shape, qs, os_ = q_rope.shape, q_rope.stride(), q_out.stride()
        if len(shape) != 3 or shape[0] != n or shape[2] != ROPE_DIM or q_out.shape != shape or \
                q_rope.dtype != torch.bfloat16 or q_out.dtype != torch.bfloat16 or \
                qs[2] != 1 or os_[2] != 1:
            raise ValueError(f"q_rope, q_out: expected bfloat16 [{n}, H, 64] with contiguous head "
                             f"rows, got {q_rope.dtype} {tuple(shape)} {qs} and {q_out.dtype} "
                             f"{tuple(q_out.shape)} {os_}")
        H = shape[1]
        q_args = (q_rope.data_ptr(), qs[0], qs[1], q_out.data_ptr(), os_[0], os_[1])
    slots_ptr, pos_ptr = _int32_arg(slots, "slots", n), _int32_arg(positions, "positions", n)
    _launch(rows, stream, library().mla_kv_append,
            row_ptr, row_stride, n, weight_ptr, eps, slots_ptr, pos_ptr, cos_sin.data_ptr(),
            max_pos, 1 if interleaved else 0, kv_ptr, kind, scale_ptr, num_slots, *q_args, H,
            _ptr(status))
    return q_out if q_rope is not None else None


def kv_read(kv, slots, kv_scale=None, out=None, status=None, stream=None):
    """The rows at `slots` (int32 [n]) of any pool as bf16 [n, 576]; see
    mla_kv_read."""
    n = slots.numel()
    kv_ptr, kind, scale_ptr, num_slots = _pool_args(kv, kv_scale)
    if out is None:
        out = torch.empty((n, ROW_DIM), dtype=torch.bfloat16, device=kv.device)
    out_ptr, out_stride = _rows_arg(out, "out", n, ROW_DIM)
    _launch(kv, stream, library().mla_kv_read, kv_ptr, kind, scale_ptr, num_slots,
            _int32_arg(slots, "slots", n), n, out_ptr, out_stride, _ptr(status))
    return out


def add_rms_norm(x, weight, residual=None, eps: float = 1e-6, out=None, out8=None,
                 scales=None, group: int = 0, residual_out=None, e4m3: bool = False,
                 stream=None):
    """Residual addition and RMS norm over the rows of x bf16 [n, d]; see
    mla_add_rms_norm.  Writes `out` (bf16) and / or `out8` (E4M3) with `scales`
    (fp32 [n, 1], or [n, d // group] with group 32, 64 or 128), whichever are
    given; with neither, `out` is allocated, or with e4m3=True out8 and scales.
    The residual is updated in place unless residual_out is given.

    Returns (out, out8, scales, residual_out), None for what was not asked."""
    if x.dim() != 2:
        raise ValueError(f"x: expected [n, d], got {tuple(x.shape)}")
    n, d = x.shape
    if out is None and out8 is None and not e4m3:
        out = torch.empty((n, d), dtype=torch.bfloat16, device=x.device)
    if out8 is None and e4m3:
        out8 = torch.empty((n, d), dtype=torch.float8_e4m3fn, device=x.device)
    if out8 is not None and scales is None:
        scales = torch.empty((n, d // group if group else 1), dtype=torch.float32, device=x.device)
    if residual is not None and residual_out is None:
        residual_out = residual
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without a residual")
    if weight.dtype != torch.bfloat16 or weight.numel() != d or not weight.is_contiguous():
        raise ValueError(f"weight: expected {d} contiguous bfloat16 values")
    none = (None, 0)
    x_args = _rows_arg(x, "x", n, d)
    res_args = none if residual is None else _rows_arg(residual, "residual", n, d)
    ro_args = none if residual is None else _rows_arg(residual_out, "residual_out", n, d)
    out_args = none if out is None else _rows_arg(out, "out", n, d)
    out8_args = sc_args = none
    if out8 is not None:
        if out8.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise ValueError(f"out8: expected float8_e4m3fn or uint8, got {out8.dtype}")
        out8_args = _rows_arg(out8, "out8", n, d, out8.dtype)
        sc_args = _rows_arg(scales, "scales", n, d // group if group else 1, torch.float32)
    _launch(x, stream, library().mla_add_rms_norm,
            *x_args, *res_args, *ro_args, weight.data_ptr(), eps, n, d, *out_args, *out8_args,
            *sc_args, group)
    return out, out8, scales, residual_out


def absorb_q(q_nope, w_kc, out=None, status=None, stream=None):
    """q_nope bf16 [B, q, H, 128] . w_kc bf16 [H, 128, 512] -> bf16 [B, q, H,
    512] (the absorbed query); see mla_absorb_q."""
    B, q, H, _ = q_nope.shape
    if out is None:
        out = torch.empty((B, q, H, NOPE_DIM), dtype=torch.bfloat16, device=q_nope.device)
    _launch(q_nope, stream, library().mla_absorb_q, _ptr(q_nope), _ptr(w_kc), _ptr(out), B * q, H,
            _ptr(status))
    return out


def project_out(o_latent, w_vc, out=None, status=None, stream=None):
    """o_latent bf16 [B, q, H, 512] . w_vc bf16 [H, 512, 128] -> bf16 [B, q, H,
    128]; see mla_project_out."""
    B, q, H, _ = o_latent.shape
    if out is None:
        out = torch.empty((B, q, H, 128), dtype=torch.bfloat16, device=o_latent.device)
    _launch(o_latent, stream, library().mla_project_out, _ptr(o_latent), _ptr(w_vc), _ptr(out),
            B * q, H, _ptr(status))
    return out


def lse_combine(O_part, LSE_part, out=None, lse_out=None, stream=None):
    """LSE merge over the leading part dims -> (bf16 [rows, 512], fp32 [rows])."""
    shape = LSE_part.shape
    # leading dims (splits, shards) are parts; the rest are rows
    lead = 2 if len(shape) == 5 else 1
    parts = shape[0] * shape[1] if lead == 2 else shape[0]
    if out is None:
        out = torch.empty(tuple(shape[lead:]) + (VALUE_DIM,), dtype=torch.bfloat16,
                          device=O_part.device)
    if lse_out is None:
        lse_out = torch.empty(tuple(shape[lead:]), dtype=torch.float32, device=O_part.device)
    fn = (library().mla_lse_combine_bf16_parts if O_part.dtype == torch.bfloat16
          else library().mla_lse_combine)
    _launch(O_part, stream, fn, O_part.data_ptr(), LSE_part.data_ptr(), parts,
            LSE_part.numel() // parts, out.data_ptr(), lse_out.data_ptr())
    return out, lse_out


# ------------------------------------------------------- prompts and beams
def _check_device(first: torch.Tensor, names: str, *tensors) -> None:
    """All arrays (None: not given) are where the first one is: the kernels read them
    by address.  (A call of get_device takes 0.05 us, of device with a comparison 0.15.)"""
    at = first.get_device()
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != at:
            raise ValueError(f"{names.split()[i]}: expected on {first.device}, got {t.device}")


def plan_prefill(q_lens: Sequence[int], kv_lens: Sequence[int], H: int, prefix=None,
                 causal: bool = True, num_sms: int = 0, ctas: int = 0):
    """Plan of `prefill` for sequences of these query and key lengths (host
    numbers): (work np.int32 [n, 8], or [n, 2, 8] for blocks on pairs of CTAs,
    num_parts).  ctas = 1 or 2 asks for one form, 0 for the faster; see
    mla_plan_prefill."""
    import numpy as np
    lq, lk = _host_i32(q_lens), _host_i32(kv_lens)
    pre = None if prefix is None else _host_i32(prefix)
    if len(lk) != len(lq) or (pre is not None and len(pre) != len(lq)):
        raise ValueError("q_lens, kv_lens and prefix differ in length")
    cap = sum(-(-max(n, 0) // 256) for n in lq) * 16 * PREFILL_MAX_PARTS
    out = np.empty(cap, dtype=np.int32)
    n, c, parts = ctypes.c_int64(), ctypes.c_int(), ctypes.c_int()
    _check(library().mla_plan_prefill(lq, lk, pre, len(lq), H, 1 if causal else 0, ctas, num_sms,
                                      out.ctypes.data, cap, ctypes.byref(n), ctypes.byref(c),
                                      ctypes.byref(parts)))
    work = out[:n.value * c.value * 8].copy()
    return work.reshape((-1, 8) if c.value == 1 else (-1, 2, 8)), parts.value


def _heads_arg(t: torch.Tensor, name: str, T: int, H: int, width: int):
    """bf16 [T, H, width] with contiguous head rows: address, token and head stride."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not _BF16 or shape != (T, H, width) or stride[2] != 1:
        raise ValueError(f"{name}: expected bfloat16 [{T}, {H}, {width}] with contiguous head rows, "
                         f"got {t.dtype} {tuple(shape)} with strides {stride}")
    return t.data_ptr(), stride[0], stride[1]


def prefill(q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_kv, work, sm_scale: float, prefix=None,
            causal: bool = True, num_parts: int = 0, O_part=None, LSE_part=None, out=None,
            lse_out=None, status=None, stream=None):
    """Attention within packed prompts, before absorption; see mla_prefill.

    q_nope bf16 [Tq, H, 128], q_rope bf16 [Tq, H, 64], k_nope and v bf16 [Tk, H,
    128] (any of them may be views into wider rows), k_rope bf16 [Tk, 64] for all
    heads; cu_q, cu_kv int32 [N + 1] where the sequences start; work and num_parts
    from plan_prefill (work as a device int32 tensor).  A sequence's queries stand
    at the end of its keys; `prefix` int32 [N]: keys that all of them see.

    Returns (out bf16 [Tq, H, 128], lse fp32 [Tq, H]); rows past the last sequence
    are left as they were.  The workspace (O_part fp32 [num_parts, H, 256, 128],
    LSE_part fp32 [num_parts, H, 256]) is allocated unless given."""
    if q_nope.dim() != 3 or k_rope.dim() != 2:
        raise ValueError(f"q_nope, k_rope: expected [Tq, H, 128] and [Tk, 64], got "
                         f"{tuple(q_nope.shape)} and {tuple(k_rope.shape)}")
    Tq, H, _ = q_nope.shape
    Tk = k_rope.shape[0]
    N = cu_q.numel() - 1
    if N < 0:
        raise ValueError("cu_q: expected N + 1 values")
    if work.dtype is not _I32 or work.shape[1:] not in ((8,), (2, 8)) or not work.is_contiguous():
        raise ValueError(f"work: expected contiguous int32 [n, 8] or [n, 2, 8], got {work.dtype} "
                         f"{tuple(work.shape)}")
    qn = _heads_arg(q_nope, "q_nope", Tq, H, 128)
    qr = _heads_arg(q_rope, "q_rope", Tq, H, ROPE_DIM)
    kn = _heads_arg(k_nope, "k_nope", Tk, H, 128)
    vv = _heads_arg(v, "v", Tk, H, 128)
    kr = _rows_arg(k_rope, "k_rope", Tk, ROPE_DIM)
    cu_args = _int32_arg(cu_q, "cu_q", N + 1), _int32_arg(cu_kv, "cu_kv", N + 1), \
        None if prefix is None else _int32_arg(prefix, "prefix", N)
    _check_device(q_nope, "q_rope k_nope k_rope v cu_q cu_kv work prefix O_part LSE_part out lse_out status",
                  q_rope, k_nope, k_rope, v, cu_q, cu_kv, work, prefix, O_part, LSE_part, out, lse_out, status)
    dev = q_nope.device
    if out is None:
        out = torch.empty((Tq, H, 128), dtype=_BF16, device=dev)
    elif out.dtype is not _BF16 or out.shape != (Tq, H, 128) or not out.is_contiguous():
        raise _not_a_buffer(out, "out", _BF16, Tq * H * 128)
    if lse_out is None:
        lse_out = torch.empty((Tq, H), dtype=_F32, device=dev)
    elif lse_out.dtype is not _F32 or lse_out.shape != (Tq, H) or not lse_out.is_contiguous():
        raise _not_a_buffer(lse_out, "lse_out", _F32, Tq * H)
    ws = (None, None)
    if num_parts > 0:
        rows = num_parts * H * 256
        if O_part is None:
            O_part = torch.empty((num_parts, H, 256, 128), dtype=_F32, device=dev)
        if LSE_part is None:
            LSE_part = torch.empty((num_parts, H, 256), dtype=_F32, device=dev)
        _check_buffer(O_part, "O_part", _F32, rows * 128)
        _check_buffer(LSE_part, "LSE_part", _F32, rows)
        ws = O_part.data_ptr(), LSE_part.data_ptr()
    if status is not None:
        _check_buffer(status, "status", _I32, 1)
    _launch(q_nope, stream, library().mla_prefill, *qn, *qr, Tq, *kn, *kr, *vv, Tk, H, *cu_args, N,
            1 if causal else 0, sm_scale, work.data_ptr(), work.shape[0], work.dim() - 1, num_parts, *ws,
            out.data_ptr(), lse_out.data_ptr(), _ptr(status))
    return out, lse_out


def beam_select(logits, scores, k: int, finished=None, end_token: int = 0, out_scores=None,
                parents=None, tokens=None, status=None, stream=None):
    """The k best continuations of every request over its beams and the
    vocabulary; see mla_beam_select.

    logits bf16, fp16 or fp32 [B, W, V] with contiguous rows, scores fp32 [B, W]
    (summed log probabilities), finished bool or uint8 [B, W] or None.  Returns
    (scores fp32 [B, k], parents int32 [B, k] as rows b * W + w, tokens int32
    [B, k]), allocated unless given; parents go straight into pages_fork."""
    if logits.dim() != 3 or logits.dtype not in _LOGITS or (logits.stride(2) != 1 and logits.shape[2] > 1):
        raise ValueError(f"logits: expected bfloat16, float16 or float32 [B, W, V] with contiguous "
                         f"rows, got {logits.dtype} {tuple(logits.shape)} with strides {logits.stride()}")
    B, W, V = logits.shape
    _check_buffer(scores, "scores", _F32, B * W)
    if finished is not None and (finished.dtype not in (torch.bool, torch.uint8) or
                                 finished.numel() != B * W or not finished.is_contiguous()):
        raise ValueError(f"finished: expected {B * W} contiguous bool or uint8 values, got "
                         f"{finished.dtype} {tuple(finished.shape)}")
    _check_device(logits, "scores finished out_scores parents tokens status", scores, finished, out_scores, parents,
                  tokens, status)
    dev = logits.device
    if out_scores is None:
        out_scores = torch.empty((B, k), dtype=_F32, device=dev)
    if parents is None:
        parents = torch.empty((B, k), dtype=_I32, device=dev)
    if tokens is None:
        tokens = torch.empty((B, k), dtype=_I32, device=dev)
    for t, name, dtype in ((out_scores, "out_scores", _F32), (parents, "parents", _I32),
                           (tokens, "tokens", _I32)):
        _check_buffer(t, name, dtype, B * k)
    if status is not None:
        _check_buffer(status, "status", _I32, 1)
    _launch(logits, stream, library().mla_beam_select, logits.data_ptr(), _LOGITS[logits.dtype],
            logits.stride(0), logits.stride(1), scores.data_ptr(), _ptr(finished), B, W, V, end_token,
            k, out_scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(), _ptr(status))
    return out_scores, parents, tokens


def _table_arg(t: torch.Tensor, name: str, R: int):
    """An int32 page table [R, stride] with contiguous rows: address, row stride
    and entries a row."""
    if t.dtype is not _I32 or t.dim() != 2 or t.size(0) != R or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous int32 [{R}, stride], got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr(), t.size(1)


def pages_fork(table, lens, refs, free_count, parents=None, keep=None, grow=None, table_out=None,
               lens_out=None, copies=None, status=None, stream=None):
    """The page table of a step that may branch: row i takes keep[i] tokens of row
    parents[i] (-1: starts empty) and grows by grow[i]; see mla_pages_fork.

    table int32 [R, stride], lens int32 [R]; refs int32 [num_pages] and free_count
    int32 [1] are updated.  Returns (table_out int32 [R, stride], lens_out int32
    [R], copies int32 [3, R]), allocated unless given (table_out zeroed); run
    kv_copy(pool, copies[0], copies[1], scale, tokens=copies[2]) on every layer's
    pool."""
    R = table.shape[0]
    _check_device(table, "lens refs free_count parents keep grow table_out lens_out copies status", lens, refs,
                  free_count, parents, keep, grow, table_out, lens_out, copies, status)
    if table_out is None:
        table_out = torch.zeros_like(table)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    if copies is None:
        copies = torch.empty((3, R), dtype=_I32, device=table.device)
    elif copies.dtype is not _I32 or copies.shape != (3, R) or not copies.is_contiguous():
        raise _not_a_buffer(copies, "copies", _I32, 3 * R)
    rows = [None if t is None else _int32_arg(t, name, R)
            for t, name in ((parents, "parents"), (keep, "keep"), (grow, "grow"))]
    _check_buffer(refs, "refs", _I32, 1)
    _check_buffer(free_count, "free_count", _I32, 1)
    if status is not None:
        _check_buffer(status, "status", _I32, 1)
    _launch(table, stream, library().mla_pages_fork, *_table_arg(table, "table", R),
            _int32_arg(lens, "lens", R), *rows, R, refs.data_ptr(), refs.numel(),
            free_count.data_ptr(), *_table_arg(table_out, "table_out", R),
            _int32_arg(lens_out, "lens_out", R), copies.data_ptr(), _ptr(status))
    return table_out, lens_out, copies


def pages_compact(table, lens, refs, max_moves: Optional[int] = None, table_out=None, src=None,
                  dst=None, count=None, status=None, stream=None):
    """Move a pool's highest live pages into its lowest holes; see
    mla_pages_compact.  At most max_moves pages (the length of src and dst if
    those are given, else the pool's pages); refs is updated, table_out may be
    table.  Returns (table_out, src int32 [max_moves], dst, count int32 [1]),
    allocated unless given; run kv_copy(pool, src, dst, scale, count=count) on
    every layer's pool."""
    R = table.shape[0]
    _check_device(table, "lens refs table_out src dst count status", lens, refs, table_out, src, dst, count, status)
    _check_buffer(refs, "refs", _I32, 1)
    if max_moves is None:
        max_moves = src.numel() if src is not None else refs.numel()
    if table_out is None:
        table_out = torch.zeros_like(table)
    if src is None:
        src = torch.empty(max_moves, dtype=_I32, device=table.device)
    if dst is None:
        dst = torch.empty(max_moves, dtype=_I32, device=table.device)
    if count is None:
        count = torch.empty(1, dtype=_I32, device=table.device)
    _check_buffer(count, "count", _I32, 1)
    if status is not None:
        _check_buffer(status, "status", _I32, 1)
    table_args = _table_arg(table, "table", R)
    _launch(table, stream, library().mla_pages_compact, *table_args, _int32_arg(lens, "lens", R), R,
            refs.data_ptr(), refs.numel(), *_table_arg(table_out, "table_out", R),
            _int32_arg(src, "src", max_moves), _int32_arg(dst, "dst", max_moves), max_moves,
            count.data_ptr(), _ptr(status))
    return table_out, src, dst, count


def kv_copy(kv, src, dst, kv_scale=None, tokens=None, count=None, status=None, stream=None):
    """Copy pages src[i] to dst[i] (int32 page numbers, a negative one: nothing) of
    a pool of any format, the first tokens[i] rows of each or all 64; only the
    first *count entries where count (int32 [1]) is given.  See mla_kv_copy."""
    n = src.numel()
    kv_ptr, kind, scale_ptr, slots = _pool_args(kv, kv_scale)
    _check_device(kv, "src dst kv_scale tokens count status", src, dst, kv_scale, tokens, count, status)
    if count is not None:
        _check_buffer(count, "count", _I32, 1)
    if status is not None:
        _check_buffer(status, "status", _I32, 1)
    _launch(kv, stream, library().mla_kv_copy, kv_ptr, kind, scale_ptr, slots,
            _int32_arg(src, "src", n), _int32_arg(dst, "dst", n),
            None if tokens is None else _int32_arg(tokens, "tokens", n), _ptr(count), n, _ptr(status))


def debug_gather(kv, req_to_token, seq_lens, row_offset, total_rows: int,
                 stream=None):
    """Raw-byte gather of every live token row through the TMA path."""
    out = torch.empty((max(total_rows, 1), ROW_DIM), dtype=kv.dtype, device=kv.device)
    _launch(kv, stream, library().mla_debug_gather, _ptr(kv), _kv_dtype(kv), kv.shape[0],
            _ptr(req_to_token), req_to_token.stride(0), _ptr(seq_lens), _ptr(row_offset),
            req_to_token.shape[0], PAGE_SIZE, _ptr(out))
    return out[:total_rows]


def debug_wait(mode: int, delay_us: int, status, elapsed_ns, stream=None):
    """Run the kernels' bounded wait on a barrier phase that nothing
    completes (mode 0), that another warp aborts (1) or completes (2) after
    delay_us; see mla_debug_wait.  `status` int32 [1], `elapsed_ns` int64 [1]
    (device)."""
    with _on(status):
        _check(library().mla_debug_wait(mode, delay_us, _ptr(status),
                                        _ptr(elapsed_ns), _stream(stream)))


def debug_quotients(counters, stream=None):
    """Exhaustive check of the FP8 cache write's division routine against the
    IEEE division (see mla_debug_quotients); `counters` int64 [2] on the
    device, zeroed: bit mismatches, code mismatches are added."""
    with _on(counters):
        _check(library().mla_debug_quotients(
            counters.data_ptr(), counters.data_ptr() + 8, _stream(stream)))


def decode(batch, num_splits: Optional[int] = None, simt: bool = False,
           status=None, stream=None, split_pages=None, fused: bool = False,
           work=None):
    """One decode step of a synth.Batch-like object: partial + combine (two
    launches, or one with fused=True).

    Without num_splits the work-balanced scheduler chooses the parts and the
    launch order (mla_plan_sched; the CUDA-core path takes the parts only);
    with num_splits and no split_pages the pages are dealt uniformly.
    Returns (out bf16 [B, q, H, 512], lse fp32 [B, q, H], num_splits).

    Planning reads the lengths back from the device and uploads the plan
    synchronously, so the host waits for earlier work on the stream.  A
    serving loop keeps the lengths on the host and calls plan_sched,
    decode_partial and lse_combine itself, with the plan uploaded from pinned
    memory on its own stream (bench.py's end-to-end loop does that).
    """
    wl = batch.wl
    if num_splits is None and wl.num_splits:
        num_splits = wl.num_splits
    if num_splits is None:
        num_splits, bnd, wk, _ = plan_sched(
            wl.B, wl.q_len, wl.H, batch_lengths(batch), wl.num_shards,
            kv_dtype=wl.kv_dtype)
        split_pages = torch.from_numpy(bnd).to(batch.q_nope.device)
        if not simt:
            work = torch.from_numpy(wk).to(batch.q_nope.device)
    if fused:
        out, lse = decode_fused(
            batch.q_nope, batch.q_rope, batch.kv, batch.kv_scale,
            batch.req_to_token, batch.seq_lens, batch.kv_limit, num_splits,
            wl.sm_scale, num_shards=wl.num_shards, status=status, stream=stream,
            split_pages=split_pages, work=work)
        return out, lse, num_splits
    O_part, LSE_part = decode_partial(
        batch.q_nope, batch.q_rope, batch.kv, batch.kv_scale,
        batch.req_to_token, batch.seq_lens, batch.kv_limit, num_splits,
        wl.sm_scale, num_shards=wl.num_shards, status=status, simt=simt,
        stream=stream, split_pages=split_pages, work=work)
    out, lse = lse_combine(O_part, LSE_part, stream=stream)
    return out, lse, num_splits


def batch_lengths(batch):
    """Host list of the (virtual) request lengths of a batch."""
    return [int(x) for x in batch.seq_lens.tolist()]


def debug_beam_math(x, y, stream=None):
    """beam_select's e^x (x <= 0) and ln y (y >= 1) of float32 arrays, as float64;
    see mla_debug_beam_math."""
    n = x.numel()
    _check_device(x, "y", y)
    _check_buffer(x, "x", _F32, n)
    _check_buffer(y, "y", _F32, n)
    exp_x, log_y = (torch.empty(n, dtype=torch.float64, device=x.device) for _ in range(2))
    _launch(x, stream, library().mla_debug_beam_math, x.data_ptr(), y.data_ptr(), n, exp_x.data_ptr(), log_y.data_ptr())
    return exp_x, log_y
