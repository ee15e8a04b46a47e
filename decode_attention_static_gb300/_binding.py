"""ctypes binding of libdecode_attn.so: argument marshalling only.

Every function here takes torch tensors that already live on the GPU, checks
that their shapes agree, and passes raw pointers, sizes and the current CUDA
stream to the C entry point of the same name. All computation happens in the
library's kernels. If the library has not been built, every call raises
``LibraryNotBuilt`` — there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import pathlib
import threading
import warnings

import torch

LIBRARY = pathlib.Path(__file__).resolve().parent / "libdecode_attn.so"

DA_F16 = 0
DA_BF16 = 1
DA_DEVERR_KV_LEN = 1
DA_DEVERR_POSITION = 2
DA_DEVERR_TIMEOUT = 4
DA_DEVERR_WORKSPACE = 8
DA_DEVERR_PAGE = 16
DA_DEVERR_TOKENS = 32
DA_DEVERR_SEQUENCE = 64
DA_DEVERR_FULL = 128
DA_DEVERR_POOL = 256
DA_MAX_ROPE_AXES = 4
DA_TREE_MAX_TOKENS = 256
DA_POOL_HEADER = 4

_DTYPE_CODE = {torch.float16: DA_F16, torch.bfloat16: DA_BF16}


class LibraryNotBuilt(RuntimeError):
    pass


class DecodeAttnError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn} failed with status {status}: {message}")
        self.status = status


_lib = None
_fast = None  # the fast path's module; False where there is none

_vp = ctypes.c_void_p
_i = ctypes.c_int
_SIGNATURES = {
    "da_status_string": ([_i], ctypes.c_char_p),
    "da_version": ([], _i),
    "decode_attn_plan_splits": ([_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_i)], _i),
    "decode_attn_workspace_size": ([_i, _i, _i, _i, _i], ctypes.c_size_t),
    "decode_attn_workspace_init": ([_vp, ctypes.c_size_t, _vp], _i),
    "decode_attn_splits_for": ([_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_i)], _i),
    "decode_attn_kernel_for": ([_i, _i, _i, _i, _i, _i, _i, _i], _i),
    "da_set_timing_events": ([_vp, _vp], _i),
    "kvcache_append": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp], _i),
    "decode_attn_fwd": ([_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _vp, _vp, ctypes.c_size_t, _i, _i,
                         _vp, _vp], _i),
    "decode_attn_fwd_static_scratch": ([_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _vp, _i, _i, _vp,
                                        _vp], _i),
    "decode_step_fwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _vp, _vp, ctypes.c_size_t,
                         _i, _i, _vp, _vp], _i),
    "da_test_skip_slot": ([_i], _i),
    "da_set_prefix_ready": ([_i], _i),
    "decode_attn_shard_heads": ([_i, _i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i),
                                 ctypes.POINTER(_i)], _i),
    "decode_step_layers_fwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.c_float, _vp, _vp,
                                ctypes.c_size_t, _i, _i, _vp, _vp], _i),
    "decode_step_rope_fwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _vp, _vp,
                              ctypes.c_size_t, _i, _i, _vp, _vp], _i),
    "kvcache_append_paged": ([_vp] * 8 + [_i] + [_vp] * 3 + [_i] * 9 + [_vp, _vp], _i),
    "kvcache_append_paged_q8": ([_vp] * 10 + [_i] + [_vp] * 3 + [_i] * 9 + [_vp, _vp], _i),
    "decode_attn_paged_workspace_size": ([_i, _i, _i], ctypes.c_size_t),
    "decode_attn_paged_fwd": ([_vp] * 5 + [_i] * 9 + [ctypes.c_float, _vp, _vp, ctypes.c_size_t, _i, _vp, _vp], _i),
    "decode_attn_paged_q8_fwd": ([_vp] * 7 + [_i] * 9 + [ctypes.c_float, _vp, _vp, ctypes.c_size_t, _i, _vp, _vp], _i),
    "decode_attn_window_fwd": ([_vp] * 4 + [_i] * 7 + [ctypes.c_float, _vp, _vp, ctypes.c_size_t, _i, _vp, _vp], _i),
    "kvcache_append_paged_axes": ([_vp] * 8 + [_i] + [_vp] * 2 + [_i] + [_vp] * 3 + [_i] * 9 + [_vp, _vp], _i),
    "kvcache_append_paged_q8_axes": ([_vp] * 10 + [_i] + [_vp] * 2 + [_i] + [_vp] * 3 + [_i] * 9 + [_vp, _vp], _i),
    "decode_attn_tree_workspace_size": ([_i, _i, _i], ctypes.c_size_t),
    "decode_attn_tree_fwd": ([_vp] * 7 + [_i] * 9 + [ctypes.c_float, _vp, _vp, ctypes.c_size_t, _i, _vp, _vp], _i),
    "decode_attn_tree_q8_fwd": ([_vp] * 9 + [_i] * 9 + [ctypes.c_float, _vp, _vp, ctypes.c_size_t, _i, _vp, _vp], _i),
    "kvcache_pool_init": ([_vp, _i, _vp], _i),
    "kvcache_resize_paged": ([_vp] * 4 + [_i] * 4 + [_vp, _vp], _i),
    "kvcache_fork_paged": ([_vp] * 6 + [_i] * 5 + [_vp, _vp], _i),
    "kvcache_copy_pages": ([_vp] * 5 + [_i] * 7 + [_vp, _vp], _i),
    "kvcache_compact_paged": ([_vp] * 6 + [_i] * 8 + [_vp, _vp], _i),
    "kvcache_compact_paged_q8": ([_vp] * 8 + [_i] * 8 + [_vp, _vp], _i),
}


def library_path() -> pathlib.Path:
    return LIBRARY


def load_library() -> ctypes.CDLL:
    """Load the CUDA library (once). Raises LibraryNotBuilt if it is missing."""
    global _lib
    if _lib is None:
        if not LIBRARY.exists():
            raise LibraryNotBuilt(f"{LIBRARY} is missing: build it with decode_attention_static_gb300.build")
        lib = ctypes.CDLL(str(LIBRARY))
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _load_fast():
    """The binding's fast path (csrc/fastcall.cpp), bound to the library; False
    where it has not been built or does not load (then with a warning). Its
    functions return NotImplemented for calls that they leave to the Python path."""
    global _fast
    lib = load_library()
    try:
        from .build import fastcall_path

        path = fastcall_path()
        if not path.exists():
            _fast = False
            return _fast
        loader = importlib.machinery.ExtensionFileLoader("_fastcall", str(path))
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fastcall", loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "decode_attn_paged_fwd", "decode_attn_paged_q8_fwd", "decode_attn_window_fwd", "kvcache_append_paged",
            "kvcache_append_paged_q8", "kvcache_append_paged_axes", "kvcache_append_paged_q8_axes",
            "decode_attn_tree_fwd", "decode_attn_tree_q8_fwd", "kvcache_resize_paged", "kvcache_fork_paged",
            "kvcache_copy_pages", "kvcache_compact_paged", "kvcache_compact_paged_q8")))
        _fast = module
    except (ImportError, OSError, AttributeError) as e:
        _fast = False
        warnings.warn(f"the binding's fast path does not load, calls are made from Python: {e}")
    return _fast


def exported_symbols() -> list[str]:
    return list(_SIGNATURES)


def status_string(status: int) -> str:
    return load_library().da_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise DecodeAttnError(fn, status, status_string(status))


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


# Fast accessors of torch's current device and raw current stream (plain
# integers, no Python objects), with the public API as the fallback.
_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device_index = getattr(torch._C, "_cuda_getDevice", None)


def _raw_stream(index: int) -> int:
    if _raw_stream_of is not None:
        return _raw_stream_of(index)
    return torch.cuda.current_stream(index).cuda_stream


def _device_now() -> int:
    return _current_device_index() if _current_device_index is not None else torch.cuda.current_device()


def _same_device_contiguous(index: int, names: tuple, tensors: tuple) -> None:
    """Every tensor is a contiguous CUDA tensor on device `index` (one pass;
    the detailed check runs only to name the offending tensor)."""
    for name, t in zip(names, tensors):
        if t.get_device() != index or not t.is_contiguous():
            _on(torch.device("cuda", index), **{name: t})
            raise ValueError(f"{name} must be a contiguous CUDA tensor on cuda:{index}")


def _call_on(fn: str, index: int, *args) -> None:
    """_call for a device given by index."""
    f = getattr(load_library(), fn)
    if _device_now() == index:
        st = f(*args)
    else:
        with torch.cuda.device(index):
            st = f(*args)
    if st != 0:
        _check(fn, st)


def _code_for(dtype: torch.dtype) -> int:
    if dtype not in _DTYPE_CODE:
        raise TypeError(f"dtype {dtype} is not supported (float16 or bfloat16)")
    return _DTYPE_CODE[dtype]


def _dtype_code(t: torch.Tensor) -> int:
    return _code_for(t.dtype)


def _require(cond: bool, msg) -> None:
    """Raise ValueError(msg) unless cond; msg may be a callable giving the
    message (so that it is only formatted on failure)."""
    if not cond:
        raise ValueError(msg() if callable(msg) else msg)


def _int32(name: str, value) -> int:
    """value as the C int that it is passed as (ctypes would drop its upper bits)."""
    value = int(value)
    _require(-(1 << 31) <= value < 1 << 31, lambda: f"{name} = {value} does not fit 32 bits")
    return value


def _cuda_contig(name: str, t: torch.Tensor) -> None:
    _require(t.is_cuda, lambda: f"{name} must be a CUDA tensor")
    _require(t.is_contiguous(), lambda: f"{name} must be contiguous")


def _on(device: torch.device, **tensors: torch.Tensor) -> None:
    """Every named tensor is a contiguous CUDA tensor on `device`."""
    for name, t in tensors.items():
        _cuda_contig(name, t)
        _require(t.device == device, lambda: f"{name} is on {t.device}, the inputs on {device}")


def _err_ptr(err_flag: torch.Tensor | None, device: torch.device):
    if err_flag is None:
        return None
    _on(device, err_flag=err_flag)
    _require(err_flag.dtype == torch.int32 and err_flag.numel() >= 1, "err_flag must be int32 with one element")
    return _ptr(err_flag)


def _workspace(workspace: torch.Tensor, device: torch.device):
    """(pointer, size in bytes) of a caller workspace."""
    _on(device, workspace=workspace)
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def _call(fn: str, device: torch.device, *args) -> None:
    """Call entry point `fn` with `device` current (the library launches on
    the current device, on the stream passed in `args`)."""
    f = getattr(load_library(), fn)
    index = device.index if device.index is not None else torch.cuda.current_device()
    if torch.cuda.current_device() == index:
        st = f(*args)
    else:
        with torch.cuda.device(device):
            st = f(*args)
    _check(fn, st)


def plan_splits(B: int, n_kv_head: int, head_dim: int, max_kv_len: int, num_sms: int, ctas_per_sm: int,
                cluster_max: int = 16) -> tuple[int, int]:
    """(splits, cluster size) of the host split plan."""
    cs = ctypes.c_int(0)
    s = load_library().decode_attn_plan_splits(B, n_kv_head, head_dim, max_kv_len, num_sms, ctas_per_sm,
                                               cluster_max, ctypes.byref(cs))
    _check("decode_attn_plan_splits", s if s < 0 else 0)
    return s, cs.value


def decode_attn_workspace_size(B: int, n_head: int, n_kv_head: int, head_dim: int, capacity: int) -> int:
    n = load_library().decode_attn_workspace_size(B, n_head, n_kv_head, head_dim, capacity)
    if n == ctypes.c_size_t(-1).value:
        raise DecodeAttnError("decode_attn_workspace_size", -2, "invalid sizes or device query failed")
    return int(n)


def alloc_workspace(B: int, n_head: int, n_kv_head: int, head_dim: int, capacity: int, device=None) -> torch.Tensor:
    """A zero-filled device byte buffer of decode_attn_workspace_size() bytes (torch owns it)."""
    n = decode_attn_workspace_size(B, n_head, n_kv_head, head_dim, capacity)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def workspace_init(workspace: torch.Tensor) -> None:
    """Zero-fill a workspace on the current stream (needed once before first use)."""
    ws, ws_bytes = _workspace(workspace, workspace.device)
    _call("decode_attn_workspace_init", workspace.device, ws, ws_bytes, _stream(workspace))


def splits_for(B: int, n_head: int, n_kv_head: int, head_dim: int, capacity: int, max_kv_len_hint: int = 0,
               dtype: torch.dtype = torch.bfloat16) -> tuple[int, int]:
    """(splits, cluster size) decode_attn_fwd will use for these sizes on the current device."""
    cs = ctypes.c_int(0)
    s = load_library().decode_attn_splits_for(B, n_head, n_kv_head, head_dim, capacity, int(max_kv_len_hint),
                                              _code_for(dtype), ctypes.byref(cs))
    _check("decode_attn_splits_for", s if s < 0 else 0)
    return s, cs.value


# decode_attn_kernel_for results
KERNEL_NAMES = {0: "cuda_cores", 1: "tensor_cores", 2: "tensor_cores_paired"}


def kernel_for(B: int, n_head: int, n_kv_head: int, head_dim: int, capacity: int, max_kv_len_hint: int = 0,
               dtype: torch.dtype = torch.bfloat16, rotary: bool = False) -> str:
    """The decode kernel a call with these sizes launches on the current device:
    "cuda_cores", "tensor_cores" or "tensor_cores_paired" (for the layers call
    pass layers * B as B)."""
    k = load_library().decode_attn_kernel_for(B, n_head, n_kv_head, head_dim, capacity, int(max_kv_len_hint),
                                              _code_for(dtype), 1 if rotary else 0)
    _check("decode_attn_kernel_for", k if k < 0 else 0)
    return KERNEL_NAMES[k]


def shard_heads(n_head: int, n_kv_head: int, world: int, rank: int) -> tuple[int, int, int, int]:
    """(kv_head0, n_kv_local, head0, n_head_local) of rank `rank` in the
    KV-head partition of decode_attn_shard_heads (host only)."""
    out = [ctypes.c_int(0) for _ in range(4)]
    st = load_library().decode_attn_shard_heads(n_head, n_kv_head, world, rank, *(ctypes.byref(o) for o in out))
    _check("decode_attn_shard_heads", st)
    return tuple(o.value for o in out)


def set_timing_events(before: "torch.cuda.Event | None", after: "torch.cuda.Event | None") -> None:
    """Record `before`/`after` around the decode kernel of every later call on
    this thread (both None turns it off). Events need timing enabled."""
    if before is None or after is None:
        load_library().da_set_timing_events(None, None)
        return
    load_library().da_set_timing_events(ctypes.c_void_p(before.cuda_event), ctypes.c_void_p(after.cuda_event))


def kvcache_append(k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                   position_ids: torch.Tensor, err_flag: torch.Tensor | None = None) -> None:
    """k_cache[b, g, position_ids[b]] = k_new[b, g] (and V), in place."""
    _cuda_contig("k_cache", k_cache)
    dev = k_cache.device
    _on(dev, v_cache=v_cache, k_new=k_new, v_new=v_new, position_ids=position_ids)
    _require(k_cache.dim() == 4 and v_cache.shape == k_cache.shape, "caches must be [B, n_kv_head, capacity, D]")
    B, Hkv, cap, D = k_cache.shape
    _require(tuple(k_new.shape) == (B, Hkv, D) and v_new.shape == k_new.shape, "k_new/v_new must be [B, n_kv_head, D]")
    _require(position_ids.dtype == torch.int32 and position_ids.numel() == B, "position_ids must be int32 [B]")
    _require(k_new.dtype == k_cache.dtype == v_cache.dtype == v_new.dtype, "dtypes differ")
    _call("kvcache_append", dev, _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(position_ids), B, Hkv,
          D, cap, _dtype_code(k_cache), _err_ptr(err_flag, dev), _stream(k_cache))


def _attn_shapes(q, k_cache, v_cache, out):
    _cuda_contig("q", q)
    _on(q.device, k_cache=k_cache, v_cache=v_cache, out=out)
    _require(q.dim() == 3, "q must be [B, n_head, D]")
    _require(k_cache.dim() == 4 and v_cache.shape == k_cache.shape, "caches must be [B, n_kv_head, capacity, D]")
    B, H, D = q.shape
    _require(k_cache.shape[0] == B and k_cache.shape[3] == D, "cache batch/head_dim must match q")
    _require(out.shape == q.shape, "out must be [B, n_head, D]")
    _require(q.dtype == k_cache.dtype == v_cache.dtype == out.dtype, "dtypes differ")
    return B, H, k_cache.shape[1], D, k_cache.shape[2]


def decode_attn_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: torch.Tensor,
                    out: torch.Tensor | None = None, scale: float | None = None,
                    workspace: torch.Tensor | None = None, max_kv_len_hint: int = 0,
                    err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """softmax(scale * q K[:kv_len]^T) V[:kv_len] per head; returns out [B, n_head, D]."""
    if out is None:
        out = torch.empty_like(q)
    _cuda_contig("q", q)
    index = q.get_device()
    _require(q.dim() == 3, "q must be [B, n_head, D]")
    _require(k_cache.dim() == 4 and v_cache.shape == k_cache.shape, "caches must be [B, n_kv_head, capacity, D]")
    B, H, D = q.shape
    _, Hkv, cap, Dk = k_cache.shape
    _require(k_cache.shape[0] == B and Dk == D, "cache batch/head_dim must match q")
    _require(out.shape == q.shape, "out must be [B, n_head, D]")
    _require(q.dtype == k_cache.dtype == v_cache.dtype == out.dtype, "dtypes differ")
    _require(kv_len.dtype == torch.int32 and kv_len.numel() == B, "kv_len must be int32 [B]")
    if workspace is None:
        workspace = alloc_workspace(B, H, Hkv, D, cap, q.device)
    names = ("k_cache", "v_cache", "out", "kv_len", "workspace")
    tensors = (k_cache, v_cache, out, kv_len, workspace)
    if err_flag is not None:
        _require(err_flag.dtype == torch.int32 and err_flag.numel() >= 1, "err_flag must be int32 with one element")
        names, tensors = names + ("err_flag",), tensors + (err_flag,)
    _same_device_contiguous(index, names, tensors)
    _call_on("decode_attn_fwd", index, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kv_len.data_ptr(), B, H,
             Hkv, D, cap, float(D ** -0.5 if scale is None else scale), out.data_ptr(), workspace.data_ptr(),
             workspace.numel() * workspace.element_size(), int(max_kv_len_hint), _code_for(q.dtype),
             None if err_flag is None else err_flag.data_ptr(), _raw_stream(index))
    return out


def _step_inputs(q, k_cache, v_cache, k_new, v_new, position_ids, out, lead=()):
    """Shapes of a fused step: q [*lead, B, H, D], caches [*lead, B, Hkv, cap, D],
    k_new/v_new [*lead, B, Hkv, D], position_ids int32 [B]."""
    n = len(lead)
    B, H, Hkv, D, cap = _attn_shapes(q[(0,) * n], k_cache[(0,) * n], v_cache[(0,) * n], out[(0,) * n])
    _on(q.device, q=q, k_cache=k_cache, v_cache=v_cache, out=out, k_new=k_new, v_new=v_new,
        position_ids=position_ids)
    _require(tuple(k_new.shape) == (*lead, B, Hkv, D) and v_new.shape == k_new.shape,
             "k_new/v_new must be [" + "layers, " * n + "B, n_kv_head, D]")
    _require(k_new.dtype == v_new.dtype == q.dtype, "dtypes differ")
    _require(position_ids.dtype == torch.int32 and position_ids.numel() == B, "position_ids must be int32 [B]")
    return B, H, Hkv, D, cap


def decode_step_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor,
                    v_new: torch.Tensor, position_ids: torch.Tensor, out: torch.Tensor | None = None,
                    scale: float | None = None, workspace: torch.Tensor | None = None, max_kv_len_hint: int = 0,
                    err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """Fused append at position_ids then attention over [0, position_ids]."""
    if out is None:
        out = torch.empty_like(q)
    _cuda_contig("q", q)
    index = q.get_device()
    _require(q.dim() == 3, "q must be [B, n_head, D]")
    _require(k_cache.dim() == 4 and v_cache.shape == k_cache.shape, "caches must be [B, n_kv_head, capacity, D]")
    B, H, D = q.shape
    _, Hkv, cap, Dk = k_cache.shape
    _require(k_cache.shape[0] == B and Dk == D, "cache batch/head_dim must match q")
    _require(out.shape == q.shape, "out must be [B, n_head, D]")
    _require(k_new.shape == (B, Hkv, D) and v_new.shape == k_new.shape, "k_new/v_new must be [B, n_kv_head, D]")
    _require(q.dtype == k_cache.dtype == v_cache.dtype == out.dtype == k_new.dtype == v_new.dtype, "dtypes differ")
    _require(position_ids.dtype == torch.int32 and position_ids.numel() == B, "position_ids must be int32 [B]")
    if workspace is None:
        workspace = alloc_workspace(B, H, Hkv, D, cap, q.device)
    names = ("k_cache", "v_cache", "out", "k_new", "v_new", "position_ids", "workspace")
    tensors = (k_cache, v_cache, out, k_new, v_new, position_ids, workspace)
    if err_flag is not None:
        _require(err_flag.dtype == torch.int32 and err_flag.numel() >= 1, "err_flag must be int32 with one element")
        names, tensors = names + ("err_flag",), tensors + (err_flag,)
    _same_device_contiguous(index, names, tensors)
    _call_on("decode_step_fwd", index, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_new.data_ptr(),
             v_new.data_ptr(), position_ids.data_ptr(), B, H, Hkv, D, cap, float(D ** -0.5 if scale is None else scale),
             out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
             int(max_kv_len_hint), _code_for(q.dtype), None if err_flag is None else err_flag.data_ptr(),
             _raw_stream(index))
    return out


def decode_step_rope_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor,
                         v_new: torch.Tensor, rope_cos: torch.Tensor, rope_sin: torch.Tensor,
                         position_ids: torch.Tensor, out: torch.Tensor | None = None, scale: float | None = None,
                         workspace: torch.Tensor | None = None, max_kv_len_hint: int = 0,
                         err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """decode_step_fwd with the rotary embedding of q and k_new at
    position_ids (tables rope_cos/rope_sin fp32 [rows, D], rows >= capacity)."""
    if out is None:
        out = torch.empty_like(q)
    B, H, Hkv, D, cap = _step_inputs(q, k_cache, v_cache, k_new, v_new, position_ids, out)
    dev = q.device
    _on(dev, rope_cos=rope_cos, rope_sin=rope_sin)
    _require(rope_cos.dtype == torch.float32 and rope_sin.dtype == torch.float32 and rope_cos.dim() == 2
             and rope_cos.shape == rope_sin.shape and rope_cos.shape[1] == D, "rope tables must be fp32 [rows, D]")
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        workspace = alloc_workspace(B, H, Hkv, D, cap, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _call("decode_step_rope_fwd", dev, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
          _ptr(rope_cos), _ptr(rope_sin), rope_cos.shape[0], _ptr(position_ids), B, H, Hkv, D, cap, float(scale),
          _ptr(out), ws, ws_bytes, int(max_kv_len_hint), _dtype_code(q), _err_ptr(err_flag, dev), _stream(q))
    return out


def decode_step_layers_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor,
                           v_new: torch.Tensor, position_ids: torch.Tensor, out: torch.Tensor | None = None,
                           scale: float | None = None, workspace: torch.Tensor | None = None,
                           max_kv_len_hint: int = 0, err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """decode_step_fwd for every layer of [layers, ...]-stacked inputs and
    caches in one launch (layer l uses q[l], k_cache[l], ..., writes out[l]);
    the layers are independent, a batch of layers * B sequences. A workspace
    must hold decode_attn_workspace_size(layers * B, ...) bytes."""
    if out is None:
        out = torch.empty_like(q)
    _require(q.dim() == 4 and k_cache.dim() == 5, "q must be [layers, B, H, D] and caches [layers, B, Hkv, cap, D]")
    layers = q.shape[0]
    if layers == 0:
        return out
    _require(k_cache.shape[0] == layers and v_cache.shape == k_cache.shape and out.shape == q.shape,
             "every tensor needs the same leading layer count")
    B, H, Hkv, D, cap = _step_inputs(q, k_cache, v_cache, k_new, v_new, position_ids, out, lead=(layers,))
    dev = q.device
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        workspace = alloc_workspace(layers * B, H, Hkv, D, cap, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _call("decode_step_layers_fwd", dev, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
          _ptr(position_ids), layers, B, H, Hkv, D, cap, float(scale), _ptr(out), ws, ws_bytes,
          int(max_kv_len_hint), _dtype_code(q), _err_ptr(err_flag, dev), _stream(q))
    return out


_thread_state = threading.local()  # mirror of the library's per-thread ordering promise


def set_prefix_ready(on: bool) -> None:
    """Ordering promise of this thread's later decode calls (see
    da_set_prefix_ready in the C header): with B == 1 and a length bound, no
    kernel still running when a call's kernel starts writes the cache rows the
    call reads, so the kernel may copy its first tiles before waiting for the
    previous kernel on the stream."""
    load_library().da_set_prefix_ready(1 if on else 0)
    _thread_state.prefix_ready = bool(on)


@contextlib.contextmanager
def prefix_ready():
    """set_prefix_ready(True) for the calls (or the stream capture) inside the
    block; the thread's previous setting comes back on exit (blocks nest)."""
    before = getattr(_thread_state, "prefix_ready", False)
    set_prefix_ready(True)
    try:
        yield
    finally:
        set_prefix_ready(before)


def test_skip_slot(slot: int) -> None:
    """Failure-detection test hook: with slot >= 0, later decode (and tree) calls of
    this thread leave that ring slot of one CTA unfilled, so its bounded waits
    expire and the call reports DA_DEVERR_TIMEOUT (-1 turns it off)."""
    load_library().da_test_skip_slot(int(slot))


STATIC_SCRATCH_BYTES = 1 << 20  # DA_STATIC_SCRATCH_BYTES of the C header


def decode_attn_fwd_static_scratch(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   kv_len: torch.Tensor, out: torch.Tensor | None = None,
                                   scale: float | None = None, max_kv_len_hint: int = 0,
                                   err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """decode_attn_fwd without a caller workspace: the library's own fixed
    device scratch array holds the split partials (for callers that may not
    allocate GPU memory). ``out`` must be given by such callers; when it is
    None this helper creates it with torch for convenience."""
    if out is None:
        out = torch.empty_like(q)
    B, H, Hkv, D, cap = _attn_shapes(q, k_cache, v_cache, out)
    dev = q.device
    _on(dev, kv_len=kv_len)
    _require(kv_len.dtype == torch.int32 and kv_len.numel() == B, "kv_len must be int32 [B]")
    if scale is None:
        scale = D ** -0.5
    _call("decode_attn_fwd_static_scratch", dev, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), B, H, Hkv, D,
          cap, float(scale), _ptr(out), int(max_kv_len_hint), _dtype_code(q), _err_ptr(err_flag, dev), _stream(q))
    return out


def decode_attn_paged_workspace_size(n_head: int, n_kv_head: int, head_dim: int) -> int:
    """Scratch bytes of one paged or sliding-window attention call on the
    current device (the same for every batch, length and page size)."""
    n = load_library().decode_attn_paged_workspace_size(n_head, n_kv_head, head_dim)
    if n == ctypes.c_size_t(-1).value:
        raise DecodeAttnError("decode_attn_paged_workspace_size", -2, "invalid sizes or device query failed")
    return int(n)


def alloc_paged_workspace(n_head: int, n_kv_head: int, head_dim: int, device=None) -> torch.Tensor:
    """A zero-filled device byte buffer of decode_attn_paged_workspace_size() bytes (torch owns it)."""
    with torch.cuda.device(device):
        n = decode_attn_paged_workspace_size(n_head, n_kv_head, head_dim)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device or "cuda")


_I32, _F32, _E4M3 = torch.int32, torch.float32, torch.float8_e4m3fn

# The entry points below check their tensors in one expression (a call costs
# more host time in checks than in the library); only when it fails do the
# _explain functions look for what is wrong, to say it.


def _explain_device(index, named):
    for name, t in named.items():
        if t is not None:
            _on(torch.device("cuda", index), **{name: t})
            _require(t.get_device() == index, f"{name} must be a contiguous CUDA tensor on cuda:{index}")


def _explain_pool(k_pages, v_pages, k_scale, v_scale, dtype, eight):
    """Shape of a page pool, and checks of its types (and scales)."""
    _require(k_pages.dim() == 4 and v_pages.shape == k_pages.shape,
             "k_pages/v_pages must be [num_pages, n_kv_head, page_size, D]")
    want = torch.float8_e4m3fn if eight else dtype
    if k_pages.dtype != want or v_pages.dtype != want:
        raise TypeError(f"pages must be {want}")
    if eight:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _require(t.dtype == torch.float32 and t.shape == k_pages.shape[:2],
                     f"{name} must be float32 [num_pages, n_kv_head]")


def _explain_err_flag(err_flag):
    _require(err_flag is None or (err_flag.dtype == torch.int32 and err_flag.numel() >= 1),
             "err_flag must be int32 with one element")


def _explain_append(k_pages, v_pages, k_scale, v_scale, eight, k_new, v_new, page_table, position_ids, token_start,
                    rope_cos, rope_sin, q, q_out, err_flag, turns=None):
    _cuda_contig("k_new", k_new)
    _code_for(k_new.dtype)
    _explain_pool(k_pages, v_pages, k_scale, v_scale, k_new.dtype, eight)
    Hkv, D = k_pages.shape[1], k_pages.shape[3]
    _require(k_new.dim() == 3 and k_new.shape[1] == Hkv and k_new.shape[2] == D and v_new.shape == k_new.shape
             and v_new.dtype == k_new.dtype, "k_new/v_new must be [tokens, n_kv_head, D] of one type")
    _require(page_table.dtype == torch.int32 and page_table.dim() == 2, "page_table must be int32 [B, max_pages]")
    B = page_table.shape[0]
    _require(position_ids.dtype == torch.int32 and position_ids.numel() == B, "position_ids must be int32 [B]")
    if token_start is not None:
        _require(token_start.dtype == torch.int32 and token_start.numel() == B + 1, "token_start must be int32 [B + 1]")
    else:
        _require(k_new.shape[0] == B, "without token_start there is one token per sequence")
    _require((rope_cos is None) == (rope_sin is None), "rope_cos and rope_sin come together")
    if rope_cos is not None:
        _require(rope_cos.dtype == torch.float32 and rope_sin.dtype == torch.float32 and rope_cos.dim() == 2
                 and rope_cos.shape == rope_sin.shape and rope_cos.shape[1] == D, "rope tables must be fp32 [rows, D]")
    if q is not None:
        _require(rope_cos is not None, "rotating q needs the rope tables")
        _require(q.dim() == 3 and q.shape[0] == k_new.shape[0] and q.shape[2] == D and q.dtype == k_new.dtype,
                 "q must be [tokens, n_head, D] of the type of k_new")
        _require(q_out is None or (q_out.shape == q.shape and q_out.dtype == q.dtype), "q_out must match q")
    else:
        _require(q_out is None, "q_out comes with q")
    _explain_err_flag(err_flag)
    others = {}
    if turns is not None:
        rope_position_ids, rope_axis = turns
        _require(rope_cos is not None, "rotary positions need the rope tables")
        _require(rope_position_ids.dtype == torch.int32 and rope_position_ids.dim() == 2
                 and 1 <= rope_position_ids.shape[0] <= DA_MAX_ROPE_AXES
                 and rope_position_ids.shape[1] == k_new.shape[0],
                 f"rope_position_ids must be int32 [axes, tokens], at most {DA_MAX_ROPE_AXES} axes")
        _require(rope_axis is None or (rope_axis.dtype == torch.int32 and rope_axis.numel() == D // 2),
                 "rope_axis must be int32 [D / 2]")
        others = dict(rope_position_ids=rope_position_ids, rope_axis=rope_axis)
    _explain_device(k_new.get_device(), dict(
        v_new=v_new, k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale, page_table=page_table,
        position_ids=position_ids, token_start=token_start, rope_cos=rope_cos, rope_sin=rope_sin, q=q, q_out=q_out,
        err_flag=err_flag, **others))
    raise ValueError("inconsistent arguments")


def _append_paged(fn, k_pages, v_pages, k_scale, v_scale, eight, k_new, v_new, page_table, position_ids, token_start,
                  rope_cos, rope_sin, q, q_out, err_flag, turns=None):
    dtype, pool, new, table = k_new.dtype, k_pages.shape, k_new.shape, page_table.shape
    code, store = _DTYPE_CODE.get(dtype), _E4M3 if eight else dtype
    ix = k_new.get_device()
    ok = (ix >= 0 and code is not None and len(pool) == 4 and len(new) == 3 and len(table) == 2
          and new[1] == pool[1] and new[2] == pool[3] and v_new.shape == new and v_pages.shape == pool
          and v_new.dtype == dtype and k_pages.dtype == store and v_pages.dtype == store and page_table.dtype == _I32
          and position_ids.dtype == _I32 and position_ids.numel() == table[0]
          and v_new.get_device() == ix and k_pages.get_device() == ix and v_pages.get_device() == ix
          and page_table.get_device() == ix and position_ids.get_device() == ix
          and k_new.is_contiguous() and v_new.is_contiguous() and k_pages.is_contiguous() and v_pages.is_contiguous()
          and page_table.is_contiguous() and position_ids.is_contiguous()
          and (not eight or (k_scale.dtype == _F32 and v_scale.dtype == _F32 and k_scale.shape == (pairs := pool[:2])
                               and v_scale.shape == pairs and k_scale.get_device() == ix
                             and v_scale.get_device() == ix and k_scale.is_contiguous() and v_scale.is_contiguous()))
          and (new[0] == table[0] if token_start is None else
               (token_start.dtype == _I32 and token_start.numel() == table[0] + 1 and token_start.get_device() == ix
                and token_start.is_contiguous()))
          and (rope_cos is None) == (rope_sin is None) and (q is not None or q_out is None)
          and (err_flag is None or (err_flag.dtype == _I32 and err_flag.numel() >= 1 and err_flag.get_device() == ix
                                    and err_flag.is_contiguous())))
    rope_rows = n_head = 0
    cos_ptr = sin_ptr = q_ptr = out_ptr = None
    if ok and rope_cos is not None:
        rope = rope_cos.shape
        ok = (len(rope) == 2 and rope[1] == new[2] and rope_sin.shape == rope and rope_cos.dtype == _F32
              and rope_sin.dtype == _F32 and rope_cos.get_device() == ix and rope_sin.get_device() == ix
              and rope_cos.is_contiguous() and rope_sin.is_contiguous())
        if ok:
            rope_rows, cos_ptr, sin_ptr = rope[0], rope_cos.data_ptr(), rope_sin.data_ptr()
    if ok and q is not None:
        qs = q.shape
        ok = (rope_cos is not None and len(qs) == 3 and qs[0] == new[0] and qs[2] == new[2] and q.dtype == dtype
              and q.get_device() == ix and q.is_contiguous())
        if ok:
            if q_out is None:
                q_out = torch.empty_like(q)
            else:
                ok = (q_out.shape == qs and q_out.dtype == dtype and q_out.get_device() == ix
                      and q_out.is_contiguous())
            n_head, q_ptr, out_ptr = qs[1], q.data_ptr(), q_out.data_ptr()
    turn_args = ()
    if ok and turns is not None:
        rows, axis = turns
        ok = (rope_cos is not None and rows.dtype == _I32 and rows.dim() == 2
              and 1 <= rows.shape[0] <= DA_MAX_ROPE_AXES and rows.shape[1] == new[0] and rows.get_device() == ix
              and rows.is_contiguous()
              and (axis is None or (axis.dtype == _I32 and axis.numel() == new[2] // 2 and axis.get_device() == ix
                                    and axis.is_contiguous())))
        if ok:
            turn_args = (rows.data_ptr(), None if axis is None else axis.data_ptr(), rows.shape[0])
    if not ok:
        _explain_append(k_pages, v_pages, k_scale, v_scale, eight, k_new, v_new, page_table, position_ids,
                        token_start, rope_cos, rope_sin, q, q_out, err_flag, turns)
    tail = (k_new.data_ptr(), v_new.data_ptr(), q_ptr, out_ptr, cos_ptr, sin_ptr, rope_rows, *turn_args,
            page_table.data_ptr(),
            position_ids.data_ptr(), None if token_start is None else token_start.data_ptr(), table[0], new[0],
            n_head, pool[1], pool[3], pool[0], pool[2], table[1], code,
            None if err_flag is None else err_flag.data_ptr(), _raw_stream(ix))
    if eight:
        _call_on(fn, ix, k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *tail)
    else:
        _call_on(fn, ix, k_pages.data_ptr(), v_pages.data_ptr(), *tail)
    return q_out


def kvcache_append_paged(k_pages: torch.Tensor, v_pages: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                         page_table: torch.Tensor, position_ids: torch.Tensor,
                         token_start: torch.Tensor | None = None, rope_cos: torch.Tensor | None = None,
                         rope_sin: torch.Tensor | None = None, q: torch.Tensor | None = None,
                         q_out: torch.Tensor | None = None,
                         err_flag: torch.Tensor | None = None) -> torch.Tensor | None:
    """Append packed new rows to a paged cache, keys (and q) rotated on the way.

    Pools [num_pages, n_kv_head, page_size, D]; page_table int32 [B,
    max_pages]; k_new/v_new [tokens, n_kv_head, D], sequence b owning tokens
    [token_start[b], token_start[b + 1]) from position position_ids[b] on
    (token_start None: one token per sequence). With rope tables the keys are
    rotated at their positions, and q [tokens, n_head, D] into q_out (may be
    q), which is returned."""
    fast = _load_fast() if _fast is None else _fast
    if fast:
        r = fast.append(k_pages, v_pages, None, None, k_new, v_new, page_table, position_ids, token_start, rope_cos,
                        rope_sin, q, q_out, err_flag)
        if r is not NotImplemented:
            return r
    return _append_paged("kvcache_append_paged", k_pages, v_pages, None, None, False, k_new, v_new, page_table,
                         position_ids, token_start, rope_cos, rope_sin, q, q_out, err_flag)


def kvcache_append_paged_q8(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                            v_scale: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                            page_table: torch.Tensor, position_ids: torch.Tensor,
                            token_start: torch.Tensor | None = None, rope_cos: torch.Tensor | None = None,
                            rope_sin: torch.Tensor | None = None, q: torch.Tensor | None = None,
                            q_out: torch.Tensor | None = None,
                            err_flag: torch.Tensor | None = None) -> torch.Tensor | None:
    """kvcache_append_paged into float8_e4m3fn pools with one power-of-two
    scale per page and KV head (k_scale/v_scale float32 [num_pages, n_kv_head],
    updated in place; a page whose scale grows has its earlier rows rounded to
    the new one)."""
    fast = _load_fast() if _fast is None else _fast
    if fast and k_scale is not None:
        r = fast.append(k_pages, v_pages, k_scale, v_scale, k_new, v_new, page_table, position_ids, token_start,
                        rope_cos, rope_sin, q, q_out, err_flag)
        if r is not NotImplemented:
            return r
    return _append_paged("kvcache_append_paged_q8", k_pages, v_pages, k_scale, v_scale, True, k_new, v_new,
                         page_table, position_ids, token_start, rope_cos, rope_sin, q, q_out, err_flag)


def _explain_attn(q, k_pages, v_pages, k_scale, v_scale, eight, page_table, kv_len, out, workspace, err_flag):
    _cuda_contig("q", q)
    _require(q.dim() == 3, "q must be [B, n_head, D]")
    _code_for(q.dtype)
    B, _, D = q.shape
    _explain_pool(k_pages, v_pages, k_scale, v_scale, q.dtype, eight)
    _require(k_pages.shape[3] == D, "head_dim of the pages must match q")
    _require(page_table.dtype == torch.int32 and page_table.dim() == 2 and page_table.shape[0] == B,
             "page_table must be int32 [B, max_pages]")
    _explain_attn_tail(q, kv_len, out, workspace, err_flag, k_pages=k_pages, v_pages=v_pages, k_scale=k_scale,
                       v_scale=v_scale, page_table=page_table)


def _explain_attn_tail(q, kv_len, out, workspace, err_flag, **others):
    _require(kv_len.dtype == torch.int32 and kv_len.numel() == q.shape[0], "kv_len must be int32 [B]")
    _require(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    _explain_err_flag(err_flag)
    _explain_device(q.get_device(), dict(kv_len=kv_len, out=out, workspace=workspace, err_flag=err_flag, **others))
    raise ValueError("inconsistent arguments")


def _attn_paged(fn, q, k_pages, v_pages, k_scale, v_scale, eight, page_table, kv_len, window, sinks, out, scale,
                workspace, err_flag):
    window, sinks = _int32("window", window), _int32("sinks", sinks)
    dtype, shape, pool, table = q.dtype, q.shape, k_pages.shape, page_table.shape
    code, store = _DTYPE_CODE.get(dtype), _E4M3 if eight else dtype
    ix = q.get_device()
    if out is None:
        out = torch.empty_like(q)
    if not (ix >= 0 and code is not None and len(shape) == 3 and len(pool) == 4 and len(table) == 2
            and pool[3] == shape[2] and table[0] == shape[0] and v_pages.shape == pool and k_pages.dtype == store
            and v_pages.dtype == store and page_table.dtype == _I32 and kv_len.dtype == _I32
            and kv_len.numel() == shape[0] and out.shape == shape and out.dtype == dtype
            and k_pages.get_device() == ix and v_pages.get_device() == ix and page_table.get_device() == ix
            and kv_len.get_device() == ix and out.get_device() == ix and q.is_contiguous()
            and k_pages.is_contiguous() and v_pages.is_contiguous() and page_table.is_contiguous()
            and kv_len.is_contiguous() and out.is_contiguous()
            and (workspace is None or (workspace.get_device() == ix and workspace.is_contiguous()))
            and (not eight or (k_scale.dtype == _F32 and v_scale.dtype == _F32
                               and k_scale.shape == (pairs := pool[:2])
                               and v_scale.shape == pairs
                               and k_scale.get_device() == ix and v_scale.get_device() == ix
                               and k_scale.is_contiguous() and v_scale.is_contiguous()))
            and (err_flag is None or (err_flag.dtype == torch.int32 and err_flag.numel() >= 1
                                      and err_flag.get_device() == ix and err_flag.is_contiguous()))):
        _explain_attn(q, k_pages, v_pages, k_scale, v_scale, eight, page_table, kv_len, out, workspace, err_flag)
    if workspace is None:
        workspace = alloc_paged_workspace(shape[1], pool[1], shape[2], q.device)
    tail = (page_table.data_ptr(), kv_len.data_ptr(), shape[0], shape[1], pool[1], shape[2], pool[0], pool[2],
            table[1], window, sinks, shape[2] ** -0.5 if scale is None else float(scale), out.data_ptr(),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), code,
            None if err_flag is None else err_flag.data_ptr(), _raw_stream(ix))
    if eight:
        _call_on(fn, ix, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(),
                 v_scale.data_ptr(), *tail)
    else:
        _call_on(fn, ix, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), *tail)
    return out


def decode_attn_paged_fwd(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                          kv_len: torch.Tensor, window: int = 0, sinks: int = 0, out: torch.Tensor | None = None,
                          scale: float | None = None, workspace: torch.Tensor | None = None,
                          err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """Decode attention of q [B, n_head, D] over the first kv_len[b] rows of a
    paged cache (or, with window > 0, over the last `window` of them and the
    first `sinks`); kv_len[b] == 0 gives zeros. A workspace comes from
    alloc_paged_workspace (reuse it across calls)."""
    fast = _load_fast() if _fast is None else _fast
    if fast:
        r = fast.attn_paged(q, k_pages, v_pages, None, None, page_table, kv_len, window, sinks, out, scale, workspace,
                            err_flag)
        if r is not NotImplemented:
            return r
    return _attn_paged("decode_attn_paged_fwd", q, k_pages, v_pages, None, None, False, page_table, kv_len, window,
                       sinks, out, scale, workspace, err_flag)


def decode_attn_paged_q8_fwd(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                             v_scale: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, window: int = 0,
                             sinks: int = 0, out: torch.Tensor | None = None, scale: float | None = None,
                             workspace: torch.Tensor | None = None,
                             err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """decode_attn_paged_fwd over float8_e4m3fn pools with their scales
    float32 [num_pages, n_kv_head]."""
    fast = _load_fast() if _fast is None else _fast
    if fast and k_scale is not None:
        r = fast.attn_paged(q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, window, sinks, out, scale,
                            workspace, err_flag)
        if r is not NotImplemented:
            return r
    return _attn_paged("decode_attn_paged_q8_fwd", q, k_pages, v_pages, k_scale, v_scale, True, page_table, kv_len,
                       window, sinks, out, scale, workspace, err_flag)


def decode_attn_window_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: torch.Tensor,
                           window: int, sinks: int = 0, out: torch.Tensor | None = None, scale: float | None = None,
                           workspace: torch.Tensor | None = None,
                           err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """Decode attention over the last `window` of the first kv_len[b] rows of a
    static cache and its first `sinks` rows; nothing else is read."""
    fast = _load_fast() if _fast is None else _fast
    if fast:
        r = fast.attn_window(q, k_cache, v_cache, kv_len, window, sinks, out, scale, workspace, err_flag)
        if r is not NotImplemented:
            return r
    window, sinks = _int32("window", window), _int32("sinks", sinks)
    dtype, shape, cache = q.dtype, q.shape, k_cache.shape
    code, ix = _DTYPE_CODE.get(dtype), q.get_device()
    if out is None:
        out = torch.empty_like(q)
    if not (ix >= 0 and code is not None and len(shape) == 3 and len(cache) == 4 and cache[0] == shape[0]
            and cache[3] == shape[2] and v_cache.shape == cache and k_cache.dtype == dtype and v_cache.dtype == dtype
            and kv_len.dtype == torch.int32 and kv_len.numel() == shape[0] and out.shape == shape
            and out.dtype == dtype and k_cache.get_device() == ix and v_cache.get_device() == ix
            and kv_len.get_device() == ix and out.get_device() == ix and q.is_contiguous()
            and k_cache.is_contiguous() and v_cache.is_contiguous() and kv_len.is_contiguous()
            and out.is_contiguous()
            and (workspace is None or (workspace.get_device() == ix and workspace.is_contiguous()))
            and (err_flag is None or (err_flag.dtype == torch.int32 and err_flag.numel() >= 1
                                      and err_flag.get_device() == ix and err_flag.is_contiguous()))):
        _cuda_contig("q", q)
        _code_for(dtype)
        _require(len(shape) == 3, "q must be [B, n_head, D]")
        _require(len(cache) == 4 and v_cache.shape == cache, "caches must be [B, n_kv_head, capacity, D]")
        _require(cache[0] == shape[0] and cache[3] == shape[2], "cache batch/head_dim must match q")
        _require(k_cache.dtype == dtype and v_cache.dtype == dtype, "dtypes differ")
        _explain_attn_tail(q, kv_len, out, workspace, err_flag, k_cache=k_cache, v_cache=v_cache)
    if workspace is None:
        workspace = alloc_paged_workspace(shape[1], cache[1], shape[2], q.device)
    _call_on("decode_attn_window_fwd", ix, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kv_len.data_ptr(),
             shape[0], shape[1], cache[1], shape[2], cache[2], window, sinks,
             shape[2] ** -0.5 if scale is None else float(scale), out.data_ptr(), workspace.data_ptr(),
             workspace.numel() * workspace.element_size(), code, None if err_flag is None else err_flag.data_ptr(),
             _raw_stream(ix))
    return out


def kvcache_append_paged_axes(k_pages: torch.Tensor, v_pages: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                              page_table: torch.Tensor, position_ids: torch.Tensor, rope_position_ids: torch.Tensor,
                              rope_cos: torch.Tensor, rope_sin: torch.Tensor, rope_axis: torch.Tensor | None = None,
                              token_start: torch.Tensor | None = None, q: torch.Tensor | None = None,
                              q_out: torch.Tensor | None = None,
                              err_flag: torch.Tensor | None = None) -> torch.Tensor | None:
    """kvcache_append_paged with rotary positions of their own: element pair i
    of token t is rotated by row rope_position_ids[rope_axis[i], t] of the
    tables (rope_position_ids int32 [axes, tokens], at most 4 axes; rope_axis
    int32 [D / 2], None: the first axis for all)."""
    fast = _load_fast() if _fast is None else _fast
    if fast:
        r = fast.append(k_pages, v_pages, None, None, k_new, v_new, page_table, position_ids, token_start, rope_cos,
                        rope_sin, q, q_out, err_flag, rope_position_ids, rope_axis)
        if r is not NotImplemented:
            return r
    return _append_paged("kvcache_append_paged_axes", k_pages, v_pages, None, None, False, k_new, v_new, page_table,
                         position_ids, token_start, rope_cos, rope_sin, q, q_out, err_flag,
                         (rope_position_ids, rope_axis))


def kvcache_append_paged_q8_axes(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                                 v_scale: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                 page_table: torch.Tensor, position_ids: torch.Tensor,
                                 rope_position_ids: torch.Tensor, rope_cos: torch.Tensor, rope_sin: torch.Tensor,
                                 rope_axis: torch.Tensor | None = None, token_start: torch.Tensor | None = None,
                                 q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                                 err_flag: torch.Tensor | None = None) -> torch.Tensor | None:
    """kvcache_append_paged_axes into float8_e4m3fn pools with their scales."""
    fast = _load_fast() if _fast is None else _fast
    if fast and k_scale is not None:
        r = fast.append(k_pages, v_pages, k_scale, v_scale, k_new, v_new, page_table, position_ids, token_start,
                        rope_cos, rope_sin, q, q_out, err_flag, rope_position_ids, rope_axis)
        if r is not NotImplemented:
            return r
    return _append_paged("kvcache_append_paged_q8_axes", k_pages, v_pages, k_scale, v_scale, True, k_new, v_new,
                         page_table, position_ids, token_start, rope_cos, rope_sin, q, q_out, err_flag,
                         (rope_position_ids, rope_axis))


def decode_attn_tree_workspace_size(n_head: int, n_kv_head: int, head_dim: int) -> int:
    """Scratch bytes of one tree attention call on the current device (the same
    for every batch, length, tree and page size)."""
    n = load_library().decode_attn_tree_workspace_size(n_head, n_kv_head, head_dim)
    if n == ctypes.c_size_t(-1).value:
        raise DecodeAttnError("decode_attn_tree_workspace_size", -2, "invalid sizes or device query failed")
    return int(n)


def alloc_tree_workspace(n_head: int, n_kv_head: int, head_dim: int, device=None) -> torch.Tensor:
    """A zero-filled device byte buffer of decode_attn_tree_workspace_size() bytes (torch owns it)."""
    with torch.cuda.device(device):
        n = decode_attn_tree_workspace_size(n_head, n_kv_head, head_dim)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def _explain_tree(q, k_pages, v_pages, k_scale, v_scale, eight, page_table, kv_len, token_start, tree_mask, out,
                  workspace, err_flag):
    _cuda_contig("q", q)
    _require(q.dim() == 3, "q must be [tokens, n_head, D]")
    _code_for(q.dtype)
    _explain_pool(k_pages, v_pages, k_scale, v_scale, q.dtype, eight)
    _require(k_pages.shape[3] == q.shape[2], "head_dim of the pages must match q")
    _require(page_table.dtype == torch.int32 and page_table.dim() == 2, "page_table must be int32 [B, max_pages]")
    B = page_table.shape[0]
    _require(kv_len.dtype == torch.int32 and kv_len.numel() == B, "kv_len must be int32 [B]")
    if token_start is not None:
        _require(token_start.dtype == torch.int32 and token_start.numel() == B + 1, "token_start must be int32 [B + 1]")
    else:
        _require(q.shape[0] == B, "without token_start there is one token per sequence")
    _require(tree_mask is None or (tree_mask.dtype == torch.int64 and tree_mask.dim() == 2
                                   and tree_mask.shape[0] == q.shape[0]
                                   and 1 <= tree_mask.shape[1] <= DA_TREE_MAX_TOKENS // 64),
             "tree_mask must be int64 [tokens, words], at most 4 words")
    _require(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    _explain_err_flag(err_flag)
    _explain_device(q.get_device(), dict(
        k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale, page_table=page_table, kv_len=kv_len,
        token_start=token_start, tree_mask=tree_mask, out=out, workspace=workspace, err_flag=err_flag))
    raise ValueError("inconsistent arguments")


def _attn_tree(fn, q, k_pages, v_pages, k_scale, v_scale, eight, page_table, kv_len, token_start, tree_mask, out,
               scale, workspace, err_flag):
    dtype, shape, pool, table = q.dtype, q.shape, k_pages.shape, page_table.shape
    code, store, ix = _DTYPE_CODE.get(dtype), _E4M3 if eight else dtype, q.get_device()
    if out is None:
        out = torch.empty_like(q)
    if not (ix >= 0 and code is not None and len(shape) == 3 and len(pool) == 4 and len(table) == 2
            and pool[3] == shape[2] and v_pages.shape == pool and k_pages.dtype == store and v_pages.dtype == store
            and page_table.dtype == _I32 and kv_len.dtype == _I32 and kv_len.numel() == table[0]
            and out.shape == shape and out.dtype == dtype
            and k_pages.get_device() == ix and v_pages.get_device() == ix and page_table.get_device() == ix
            and kv_len.get_device() == ix and out.get_device() == ix and q.is_contiguous()
            and k_pages.is_contiguous() and v_pages.is_contiguous() and page_table.is_contiguous()
            and kv_len.is_contiguous() and out.is_contiguous()
            and (shape[0] == table[0] if token_start is None else
                 (token_start.dtype == _I32 and token_start.numel() == table[0] + 1
                  and token_start.get_device() == ix and token_start.is_contiguous()))
            and (tree_mask is None or (tree_mask.dtype == torch.int64 and tree_mask.dim() == 2
                                       and tree_mask.shape[0] == shape[0]
                                       and 1 <= tree_mask.shape[1] <= DA_TREE_MAX_TOKENS // 64
                                       and tree_mask.get_device() == ix and tree_mask.is_contiguous()))
            and (workspace is None or (workspace.get_device() == ix and workspace.is_contiguous()))
            and (not eight or (k_scale.dtype == _F32 and v_scale.dtype == _F32
                               and k_scale.shape == pool[:2] and v_scale.shape == pool[:2]
                               and k_scale.get_device() == ix and v_scale.get_device() == ix
                               and k_scale.is_contiguous() and v_scale.is_contiguous()))
            and (err_flag is None or (err_flag.dtype == _I32 and err_flag.numel() >= 1
                                      and err_flag.get_device() == ix and err_flag.is_contiguous()))):
        _explain_tree(q, k_pages, v_pages, k_scale, v_scale, eight, page_table, kv_len, token_start, tree_mask, out,
                      workspace, err_flag)
    if workspace is None:
        workspace = alloc_tree_workspace(shape[1], pool[1], shape[2], q.device)
    tail = (page_table.data_ptr(), kv_len.data_ptr(), None if token_start is None else token_start.data_ptr(),
            None if tree_mask is None else tree_mask.data_ptr(), 0 if tree_mask is None else tree_mask.shape[1],
            table[0], shape[0], shape[1], pool[1], shape[2], pool[0], pool[2], table[1],
            shape[2] ** -0.5 if scale is None else float(scale), out.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), code, None if err_flag is None else err_flag.data_ptr(),
            _raw_stream(ix))
    if eight:
        _call_on(fn, ix, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(),
                 v_scale.data_ptr(), *tail)
    else:
        _call_on(fn, ix, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), *tail)
    return out


def decode_attn_tree_fwd(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                         kv_len: torch.Tensor, token_start: torch.Tensor | None = None,
                         tree_mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         scale: float | None = None, workspace: torch.Tensor | None = None,
                         err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of several new tokens of each sequence over a paged cache that
    holds their rows already: q [tokens, n_head, D] packed, sequence b owning
    tokens [token_start[b], token_start[b + 1]) (None: one each), which are the
    last of its kv_len[b] rows. A token sees every row before them, and of them
    those whose bit is set in its row of tree_mask (int64 [tokens, words], bit
    i % 64 of word i / 64 for the sequence's i-th token; None: those up to
    itself). A workspace comes from alloc_tree_workspace (reuse it)."""
    fast = _load_fast() if _fast is None else _fast
    if fast:
        r = fast.attn_tree(q, k_pages, v_pages, None, None, page_table, kv_len, token_start, tree_mask, out, scale,
                           workspace, err_flag)
        if r is not NotImplemented:
            return r
    return _attn_tree("decode_attn_tree_fwd", q, k_pages, v_pages, None, None, False, page_table, kv_len, token_start,
                      tree_mask, out, scale, workspace, err_flag)


def decode_attn_tree_q8_fwd(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                            v_scale: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                            token_start: torch.Tensor | None = None, tree_mask: torch.Tensor | None = None,
                            out: torch.Tensor | None = None, scale: float | None = None,
                            workspace: torch.Tensor | None = None,
                            err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """decode_attn_tree_fwd over float8_e4m3fn pools with their scales float32
    [num_pages, n_kv_head]."""
    fast = _load_fast() if _fast is None else _fast
    if fast and k_scale is not None:
        r = fast.attn_tree(q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, token_start, tree_mask, out, scale,
                           workspace, err_flag)
        if r is not NotImplemented:
            return r
    return _attn_tree("decode_attn_tree_q8_fwd", q, k_pages, v_pages, k_scale, v_scale, True, page_table, kv_len,
                      token_start, tree_mask, out, scale, workspace, err_flag)


def _ints(index: int, **tensors) -> None:
    """Every given tensor is a contiguous int32 one on device `index`."""
    for name, (t, shape) in tensors.items():
        if t is None:
            continue
        _require(t.dtype == _I32 and tuple(t.shape) == tuple(shape), lambda: f"{name} must be int32 {list(shape)}")
        if t.get_device() != index or not t.is_contiguous():
            _explain_device(index, {name: t})


def _pool_pages(pool: torch.Tensor) -> int:
    """Pages of a pool's state."""
    _cuda_contig("pool", pool)
    _require(pool.dtype == _I32 and pool.dim() == 1 and pool.numel() > DA_POOL_HEADER
             and (pool.numel() - DA_POOL_HEADER) % 2 == 0,
             f"pool must be int32 [{DA_POOL_HEADER} + 2 * num_pages]")
    return (pool.numel() - DA_POOL_HEADER) // 2


def alloc_page_pool(num_pages: int, device=None) -> torch.Tensor:
    """State of a pool of num_pages pages, all free, for kvcache_resize_paged and kvcache_fork_paged."""
    _require(num_pages >= 1, "a pool needs a page")
    pool = torch.empty(DA_POOL_HEADER + 2 * num_pages, dtype=torch.int32, device=device or "cuda")
    _call_on("kvcache_pool_init", pool.get_device(), pool.data_ptr(), num_pages, _raw_stream(pool.get_device()))
    return pool


def page_pool_views(pool: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(free [1], counts [num_pages], list [num_pages]) of a pool's state: views
    of how many pages are free, how many table entries hold each page, and the
    free pages (the list's first free[0] entries)."""
    n = _pool_pages(pool)
    return pool[:1], pool[DA_POOL_HEADER:DA_POOL_HEADER + n], pool[DA_POOL_HEADER + n:]


def kvcache_resize_paged(page_table: torch.Tensor, held_len: torch.Tensor, wanted_len: torch.Tensor,
                         pool: torch.Tensor, page_size: int, err_flag: torch.Tensor | None = None) -> None:
    """Sequences whose first held_len[b] rows have pages become sequences of
    wanted_len[b] rows: pages are released to the pool's state, then taken from
    it (page_table int32 [B, max_pages], lengths int32 [B], pool from
    alloc_page_pool; all updated in place)."""
    fast = _load_fast() if _fast is None else _fast
    if fast and fast.resize(page_table, held_len, wanted_len, pool, page_size, err_flag) is not NotImplemented:
        return
    pages, ix = _pool_pages(pool), pool.get_device()
    _require(page_table.dim() == 2, "page_table must be int32 [B, max_pages]")
    B, most = page_table.shape
    _ints(ix, page_table=(page_table, (B, most)), held_len=(held_len, (B,)), wanted_len=(wanted_len, (B,)))
    _err_ptr(err_flag, pool.device)
    _call_on("kvcache_resize_paged", ix, page_table.data_ptr(), held_len.data_ptr(), wanted_len.data_ptr(),
             pool.data_ptr(), B, pages, _int32("page_size", page_size), most,
             None if err_flag is None else err_flag.data_ptr(), _raw_stream(ix))


def kvcache_fork_paged(page_table: torch.Tensor, kv_len: torch.Tensor, parent: torch.Tensor, child: torch.Tensor,
                       pool: torch.Tensor, page_size: int, copies: torch.Tensor | None = None,
                       err_flag: torch.Tensor | None = None) -> torch.Tensor:
    """Sequence child[i] becomes a copy of sequence parent[i] (int32 [forks]):
    whole pages are shared, a partly filled last one is replaced by a page of
    the pool. Returns copies int32 [3, forks] (source page, target page, rows),
    for kvcache_copy_pages on every layer's pools; page_table, kv_len and pool
    are updated in place."""
    fast = _load_fast() if _fast is None else _fast
    if fast:
        r = fast.fork(page_table, kv_len, parent, child, pool, page_size, copies, err_flag)
        if r is not NotImplemented:
            return r
    pages, ix = _pool_pages(pool), pool.get_device()
    _require(page_table.dim() == 2, "page_table must be int32 [B, max_pages]")
    (B, most), n = page_table.shape, parent.numel()
    if copies is None:
        copies = torch.empty((3, n), dtype=torch.int32, device=pool.device)
    _ints(ix, page_table=(page_table, (B, most)), kv_len=(kv_len, (B,)), parent=(parent, (n,)), child=(child, (n,)),
          copies=(copies, (3, n)))
    _err_ptr(err_flag, pool.device)
    _call_on("kvcache_fork_paged", ix, page_table.data_ptr(), kv_len.data_ptr(), parent.data_ptr(), child.data_ptr(),
             pool.data_ptr(), copies.data_ptr(), n, B, pages, _int32("page_size", page_size), most,
             None if err_flag is None else err_flag.data_ptr(), _raw_stream(ix))
    return copies


def _stacked_pools(k_pages, v_pages, k_scale, v_scale):
    """(layers, pages, heads, page size, D, element size) of the pools of one
    layer [num_pages, ...] or of several [layers, num_pages, ...]."""
    _cuda_contig("k_pages", k_pages)
    _on(k_pages.device, v_pages=v_pages)
    _require(k_pages.dim() in (4, 5) and v_pages.shape == k_pages.shape and v_pages.dtype == k_pages.dtype,
             "k_pages/v_pages must be [num_pages, n_kv_head, page_size, D], with a leading layer axis or without")
    if k_pages.dtype not in (torch.float16, torch.bfloat16, _E4M3):
        raise TypeError(f"pages of {k_pages.dtype} are not supported (float16, bfloat16 or float8_e4m3fn)")
    _require((k_scale is None) == (v_scale is None), "k_scale and v_scale come together")
    if k_scale is not None:
        _on(k_pages.device, k_scale=k_scale, v_scale=v_scale)
        _require(k_pages.dtype == _E4M3, "scales come with pages of float8_e4m3fn")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _require(t.dtype == _F32 and t.shape == k_pages.shape[:-2], lambda: f"{name} must be float32 "
                     f"{list(k_pages.shape[:-2])}")
    layers = k_pages.shape[0] if k_pages.dim() == 5 else 1
    return (layers, *k_pages.shape[-4:], k_pages.element_size())


def kvcache_copy_pages(k_pages: torch.Tensor, v_pages: torch.Tensor, copies: torch.Tensor,
                       k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                       err_flag: torch.Tensor | None = None) -> None:
    """Copy rows [0, copies[2, i]) of page copies[0, i] to page copies[1, i] in
    the pools of one layer or (with a leading layer axis) of several, in place;
    pages of 8 bits with their scales. Entries below 0 are skipped."""
    fast = _load_fast() if _fast is None else _fast
    if fast and fast.copy_pages(k_pages, v_pages, k_scale, v_scale, copies, err_flag) is not NotImplemented:
        return
    layers, pages, Hkv, size, D, element = _stacked_pools(k_pages, v_pages, k_scale, v_scale)
    _require(copies.dim() == 2 and copies.shape[0] == 3, "copies must be int32 [3, n]")
    n, ix = copies.shape[1], k_pages.get_device()
    _ints(ix, copies=(copies, (3, n)))
    _err_ptr(err_flag, k_pages.device)
    _call_on("kvcache_copy_pages", ix, k_pages.data_ptr(), v_pages.data_ptr(),
             None if k_scale is None else k_scale.data_ptr(), None if v_scale is None else v_scale.data_ptr(),
             copies.data_ptr(), n, layers, pages, Hkv, size, D, element,
             None if err_flag is None else err_flag.data_ptr(), _raw_stream(ix))


def _compact(fn, k_pages, v_pages, k_scale, v_scale, eight, page_table, keep, keep_start, position_ids, err_flag):
    fast = _load_fast() if _fast is None else _fast
    if fast and (k_scale is not None) == eight and fast.compact(
            k_pages, v_pages, k_scale, v_scale, page_table, keep, keep_start, position_ids, err_flag) is not NotImplemented:
        return
    if (k_pages.dtype == _E4M3) != eight:
        raise TypeError("pages must be float8_e4m3fn" if eight else "pages must be float16 or bfloat16")
    layers, pages, Hkv, size, D, _ = _stacked_pools(k_pages, v_pages, k_scale, v_scale)
    _require(page_table.dim() == 2, "page_table must be int32 [B, max_pages]")
    (B, most), ix = page_table.shape, k_pages.get_device()
    _ints(ix, page_table=(page_table, (B, most)), keep=(keep, (keep.numel(),)), keep_start=(keep_start, (B + 1,)),
          position_ids=(position_ids, (B,)))
    _err_ptr(err_flag, k_pages.device)
    scales = (k_scale.data_ptr(), v_scale.data_ptr()) if eight else ()
    _call_on(fn, ix, k_pages.data_ptr(), v_pages.data_ptr(), *scales, page_table.data_ptr(), keep.data_ptr(),
             keep_start.data_ptr(), position_ids.data_ptr(), B, keep.numel(), layers, Hkv, D, pages, size, most,
             None if err_flag is None else err_flag.data_ptr(), _raw_stream(ix))


def kvcache_compact_paged(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, keep: torch.Tensor,
                          keep_start: torch.Tensor, position_ids: torch.Tensor,
                          err_flag: torch.Tensor | None = None) -> None:
    """Move row keep[keep_start[b] + i] of sequence b to row position_ids[b] + i
    (rising rows, none moves up), in the pools of one layer or (with a leading
    layer axis) of several, in place: accepted drafts behind the prefix."""
    _compact("kvcache_compact_paged", k_pages, v_pages, None, None, False, page_table, keep, keep_start, position_ids,
             err_flag)


def kvcache_compact_paged_q8(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                             v_scale: torch.Tensor, page_table: torch.Tensor, keep: torch.Tensor,
                             keep_start: torch.Tensor, position_ids: torch.Tensor,
                             err_flag: torch.Tensor | None = None) -> None:
    """kvcache_compact_paged over float8_e4m3fn pools: a page that takes rows of
    pages with larger scales gets the largest one, its rows rounded to it."""
    _require(k_scale is not None and v_scale is not None, "pages of 8 bits need their scales")
    _compact("kvcache_compact_paged_q8", k_pages, v_pages, k_scale, v_scale, True, page_table, keep, keep_start,
             position_ids, err_flag)
