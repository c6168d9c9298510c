"""Build and load libblockattn.so (CUDA, sm_103a) and bind its C ABI.

The binding only marshals arguments: torch tensors become device pointers and
element strides, outputs and workspace are allocated with torch, and every
step of the computation runs in the library's kernels.  There is no other
implementation behind these functions; if the library cannot be built or
loaded they raise.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
_CSRC = os.path.join(_PKG, "csrc")
_BUILD = os.path.join(_PKG, "_build")
LIB_PATH = os.path.join(_BUILD, "libblockattn.so")
FASTCALL_PATH = os.path.join(_BUILD, f"_fastcall_torch{torch.__version__}.so")   # (its ABI is that of one version)
_SOURCES = ["api.cu", "attn_simt.cu", "attn_tc.cu", "attn_bwd.cu", "attn_bwd_tc.cu", "ulysses.cu", "decode.cu",
            "decode_group.cu", "kv4.cu", "qk_norm.cu", "attn_window_simt.cu"]
_HEADERS = ["common.cuh", "internal.h", "epilogue.cuh", "tc_ptx.cuh"]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]

BA_OK, BA_ERR_ARG, BA_ERR_SHAPE, BA_ERR_CUDA, BA_ERR_TIMEOUT, BA_ERR_UNSUPPORTED, BA_ERR_WORKSPACE = \
    0, -1, -2, -3, -4, -5, -6
BA_ERR_NOALLOC_LIMIT = -7
BA_NOALLOC_MAX_CLASS_BYTES = 1 << 20
BA_F32, BA_BF16 = 0, 1
PARTITIONS = {"contiguous": 0, "zigzag": 1, "striped": 2}
MODES = {"stepwise": 0, "fused": 1}
BA_TILE_EMPTY, BA_TILE_FULL, BA_TILE_PARTIAL = 0, 1, 2

_lib = None
_fast = None   # the module of csrc/fastcall.cpp, where it could be built


class BlockAttnError(RuntimeError):
    def __init__(self, fn, code):
        msg = _lib.ba_strerror(code).decode() if _lib is not None else str(code)
        super().__init__(f"{fn} failed: {msg} ({code})")
        self.code = code


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = [os.path.join(_CSRC, f) for f in _SOURCES + _HEADERS]
    deps.append(os.path.join(_ROOT, "include", "blockattn.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def _build_fastcall(force):
    """Compile csrc/fastcall.cpp against torch, where the headers of both are installed.  A torch whose
    C++ interface differs is warned of: every call then goes through the Python binding."""
    src, header = os.path.join(_CSRC, "fastcall.cpp"), os.path.join(_ROOT, "include", "blockattn.h")
    python = sysconfig.get_paths()["include"]
    torch_dir = os.path.dirname(torch.__file__)
    torch_header = os.path.join(torch_dir, "include", "torch", "csrc", "autograd", "python_variable.h")
    if not (os.path.exists(os.path.join(python, "Python.h")) and os.path.exists(torch_header)):
        return
    if not force and os.path.exists(FASTCALL_PATH) and \
            os.path.getmtime(FASTCALL_PATH) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return
    os.makedirs(_BUILD, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    includes = [os.path.join(_ROOT, "include"), python, os.path.join(torch_dir, "include"), cuda]
    libs = os.path.join(torch_dir, "lib")
    tmp = FASTCALL_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{p}" for p in includes), src, "-o", tmp,
           f"-L{libs}", f"-Wl,-rpath,{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(FASTCALL_PATH):   # of other sources
            os.remove(FASTCALL_PATH)
        warnings.warn(f"{src} did not compile, calls are marshalled in Python:\n{r.stderr}")
        return
    os.replace(tmp, FASTCALL_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA sources for sm_103a and the call marshalling (in parallel) and link the shared library."""
    with ThreadPoolExecutor(1) as ex:
        fastcall = ex.submit(_build_fastcall, force)
        _build_library(force, verbose)
        fastcall.result()
    return LIB_PATH


def _build_library(force, verbose):
    if not force and not _stale():
        return
    os.makedirs(_BUILD, exist_ok=True)
    nvcc = _nvcc()
    common = [nvcc, *ARCH_FLAGS, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", os.path.join(_ROOT, "include")]

    def compile_one(src):
        obj = os.path.join(_BUILD, src.replace(".cu", ".o"))
        cmd = common + ["-c", os.path.join(_CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(len(_SOURCES)) as ex:
        objs = list(ex.map(compile_one, _SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


class ba_tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("sB", ctypes.c_int64), ("sH", ctypes.c_int64),
                ("sT", ctypes.c_int64)]


class ba_kv4(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("codes_sB", ctypes.c_int64), ("codes_sH", ctypes.c_int64),
                ("codes_sT", ctypes.c_int64), ("scales_sB", ctypes.c_int64), ("scales_sH", ctypes.c_int64),
                ("scales_sT", ctypes.c_int64), ("k_exp", ctypes.c_int), ("v_exp", ctypes.c_int)]


EXPORTED = ["attn_block_fwd", "attn_block_fwd_workspace_size", "attn_merge", "ring_attn_fwd",
            "ring_attn_fwd_workspace_size", "rope_apply", "ba_tile_classes", "ba_index_maps",
            "ba_sync_status", "ba_debug_wait_timeout", "ba_strerror", "attn_block_fwd_noalloc",
            "attn_block_bwd", "attn_block_bwd_workspace_size", "ring_attn_bwd", "ring_attn_bwd_workspace_size",
            "ulysses_all_to_all", "ulysses_attn_fwd", "ulysses_attn_fwd_workspace_size",
            "attn_decode_fwd", "attn_decode_workspace_size", "ba_pair_schedule",
            "attn_window_fwd", "attn_window_fwd_workspace_size", "attn_window_bwd",
            "attn_window_bwd_workspace_size", "attn_window_decode_fwd", "attn_window_decode_workspace_size",
            "kv4_append", "kv4_read", "attn_decode_kv4_fwd", "attn_decode_kv4_workspace_size",
            "qk_norm_rope_fwd", "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_size"]


def load(path: str | None = None):
    """Load the library (building it first when needed) and declare signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = build()
    lib = ctypes.CDLL(path)
    i, i64, sz, vp, f = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    T = ba_tensor
    lib.ba_strerror.restype = ctypes.c_char_p
    lib.ba_strerror.argtypes = [i]
    lib.attn_block_fwd_workspace_size.restype = sz
    lib.attn_block_fwd_workspace_size.argtypes = [i, i, i, i]
    lib.attn_block_fwd.restype = i
    lib.attn_block_fwd.argtypes = [T, T, T, i, i, i, i, i, i, i64, i64, vp, i64, vp, i64, i, f, vp, i, vp, i,
                                   vp, sz, vp]
    lib.attn_block_fwd_noalloc.restype = i
    lib.attn_block_fwd_noalloc.argtypes = [T, T, T, i, i, i, i, i, i, i64, i64, vp, i64, vp, i64, i, f, vp, i, vp,
                                           i, vp]
    lib.attn_merge.restype = i
    lib.attn_merge.argtypes = [vp, vp, vp, vp, i64, i, vp]
    lib.ring_attn_fwd_workspace_size.restype = sz
    lib.ring_attn_fwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i, i, i, i]
    lib.ring_attn_fwd.restype = i
    lib.ring_attn_fwd.argtypes = [T, T, T, i, i, i, i, i, i, i, i, vp, i64, vp, i64, i, f, i, f, vp, i, vp, vp,
                                  vp, sz, vp]
    lib.rope_apply.restype = i
    lib.rope_apply.argtypes = [T, T, i, i, i, i, i, vp, f, f, vp, vp, vp]
    lib.ba_tile_classes.restype = i
    lib.ba_tile_classes.argtypes = [i, i, i, i64, i64, vp, i64, vp, i64, i, vp, vp]
    lib.ba_index_maps.restype = i
    lib.ba_index_maps.argtypes = [i, i, i, vp, vp]
    lib.ba_pair_schedule.restype = i
    lib.ba_pair_schedule.argtypes = [i, i, i, i, i, i, i, vp, ctypes.c_int64]
    lib.ba_sync_status.restype = i
    lib.ba_sync_status.argtypes = [vp]
    lib.ba_debug_wait_timeout.restype = i
    lib.ba_debug_wait_timeout.argtypes = [i64, vp]
    lib.attn_block_bwd_workspace_size.restype = sz
    lib.attn_block_bwd_workspace_size.argtypes = [i, i, i]
    lib.attn_block_bwd.restype = i
    lib.attn_block_bwd.argtypes = [T, T, T, T, T, vp, i, i, i, i, i, i, i64, i64, vp, i64, vp, i64, i, f,
                                   vp, vp, vp, i, vp, sz, vp]
    lib.ring_attn_bwd_workspace_size.restype = sz
    lib.ring_attn_bwd_workspace_size.argtypes = [i, i, i]
    lib.ring_attn_bwd.restype = i
    lib.ring_attn_bwd.argtypes = [T, T, T, T, T, vp, i, i, i, i, i, i, i, i, vp, i64, vp, i64, i, f,
                                  vp, vp, vp, vp, sz, vp]
    lib.ulysses_all_to_all.restype = i
    lib.ulysses_all_to_all.argtypes = [vp, vp, i, i, i, i, i, i, i, vp]
    lib.ulysses_attn_fwd_workspace_size.restype = sz
    lib.ulysses_attn_fwd_workspace_size.argtypes = [i, i, i, i, i, i, i]
    lib.ulysses_attn_fwd.restype = i
    lib.ulysses_attn_fwd.argtypes = [vp, vp, vp, i, i, i, i, i, i, vp, i64, vp, i64, i, f, vp, vp, vp, sz, vp]
    lib.attn_decode_workspace_size.restype = sz
    lib.attn_decode_workspace_size.argtypes = [i, i, i, i, i]
    lib.attn_decode_fwd.restype = i
    lib.attn_decode_fwd.argtypes = [T, T, T, i, i, i, i, i, vp, i, f, vp, i, vp, vp, sz, vp]
    lib.attn_window_fwd_workspace_size.restype = sz
    lib.attn_window_fwd_workspace_size.argtypes = [i, i, i, i, i]
    lib.attn_window_fwd.restype = i
    lib.attn_window_fwd.argtypes = [T, T, T, i, i, i, i, i, i, i, i64, i, i, vp, i64, f, vp, i, vp, vp, sz, vp]
    lib.attn_window_bwd_workspace_size.restype = sz
    lib.attn_window_bwd_workspace_size.argtypes = [i, i, i, i, i, i, i64, i, i]
    lib.attn_window_bwd.restype = i
    lib.attn_window_bwd.argtypes = [T, T, T, T, T, vp, i, i, i, i, i, i, i, i64, i, i, vp, i64, f, vp, vp, vp, i,
                                    vp, sz, vp]
    for fn in (lib.attn_window_decode_workspace_size, lib.attn_decode_kv4_workspace_size):
        fn.restype = sz
        fn.argtypes = [i, i, i, i, i, i, i]
    lib.attn_window_decode_fwd.restype = i
    lib.attn_window_decode_fwd.argtypes = [T, T, T, i, i, i, i, i, i, vp, i, i, f, vp, i, vp, vp, sz, vp]
    lib.kv4_append.restype = i
    lib.kv4_append.argtypes = [T, T, ba_kv4, i, i, i, i, i, i, vp, vp, vp]
    lib.kv4_read.restype = i
    lib.kv4_read.argtypes = [ba_kv4, i, i, i, i, i, i, i, vp, vp, vp]
    lib.attn_decode_kv4_fwd.restype = i
    lib.attn_decode_kv4_fwd.argtypes = [T, ba_kv4, i, i, i, i, i, i, vp, i, i, f, vp, i, vp, vp, sz, vp]
    lib.qk_norm_rope_fwd.restype = i
    lib.qk_norm_rope_fwd.argtypes = [T, T, vp, vp, i, i, i, i, i, i, i, f, vp, i64, f, f, vp, vp, vp]
    lib.qk_norm_rope_bwd_workspace_size.restype = sz
    lib.qk_norm_rope_bwd_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.qk_norm_rope_bwd.restype = i
    lib.qk_norm_rope_bwd.argtypes = [T, T, vp, vp, i, T, T, i, i, i, i, i, i, i, f, vp, i64, f, f, vp, vp, vp, vp, vp, sz,
                                     vp]
    _lib = lib
    if os.path.exists(FASTCALL_PATH):
        _load_fastcall(lib)
    return lib


def _load_fastcall(lib):
    global _fast
    spec = importlib.util.spec_from_file_location("_fastcall", FASTCALL_PATH)
    fast = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fast)
    fast.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in EXPORTED})
    _fast = fast


def _check(fn, rc):
    if rc != BA_OK:
        raise BlockAttnError(fn, rc)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return BA_F32
    if t == torch.bfloat16:
        return BA_BF16
    raise TypeError(f"unsupported dtype {t}")


def _tensor(x: torch.Tensor) -> ba_tensor:
    if x.dim() != 4 or x.stride(-1) != 1:
        raise ValueError("expected a (B, H, T, d) tensor with a contiguous last axis")
    if not x.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return ba_tensor(x.data_ptr(), x.stride(0), x.stride(1), x.stride(2))


def _mask(m, rows, cols, name="mask"):
    """(pointer, ld) of a 2-D uint8 mask.  The library indexes masks at global
    positions and sees only the pointer and the row stride, so the binding
    checks here that the mask covers every row (batch item for the key-padding
    mask, query position for attn_mask) and every key position a launch reads."""
    if m is None:
        return None, 0
    if m.dtype != torch.uint8 or m.dim() != 2 or m.stride(1) != 1:
        raise ValueError("masks are 2-D uint8 CUDA tensors with a contiguous last axis")
    if m.shape[0] < rows or m.shape[1] < cols:
        raise ValueError(f"{name} of shape {tuple(m.shape)} does not cover the ({rows}, {cols}) "
                         f"rows and key positions the call reads")
    if m.shape[0] > 1 and m.stride(0) < cols:
        raise ValueError(f"{name} rows overlap (stride {m.stride(0)} < {cols} key positions)")
    if not m.is_cuda:
        raise ValueError("masks are 2-D uint8 CUDA tensors with a contiguous last axis")
    return ctypes.c_void_p(m.data_ptr()), m.stride(0)


def _masks(key_padding_mask, attn_mask, B, q_rows, k_cols):
    """Both masks of a call whose queries reach global position q_rows - 1 and
    whose keys reach k_cols - 1."""
    kpm, kpm_ld = _mask(key_padding_mask, B, k_cols, "key_padding_mask")
    am, am_ld = _mask(attn_mask, q_rows, k_cols, "attn_mask")
    return kpm, kpm_ld, am, am_ld


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_out(out, lse, shape):
    """Outputs are written as contiguous (B, H, L, d) and (B, H, L) buffers."""
    if tuple(out.shape) != tuple(shape) or not out.is_contiguous() or not out.is_cuda:
        raise ValueError(f"out must be a contiguous CUDA tensor of shape {tuple(shape)}")
    if tuple(lse.shape) != tuple(shape[:3]) or not lse.is_contiguous() or lse.dtype != torch.float32:
        raise ValueError(f"lse must be a contiguous float32 CUDA tensor of shape {tuple(shape[:3])}")


def attn_block_fwd(q, k, v, *, q_off=0, k_off=0, key_padding_mask=None, attn_mask=None, causal=False,
                   scale=None, out=None, out_dtype=None, lse=None, accumulate=False, workspace=None,
                   stream=None):
    """One attention block with per-row natural-log LSE; see include/blockattn.h."""
    lib = load()
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    dt = _dtype_code(q.dtype)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out is None:
        out = torch.empty((B, H, Lq, d), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device)
    _check_out(out, lse, (B, H, Lq, d))
    kpm, kpm_ld, am, am_ld = _masks(key_padding_mask, attn_mask, B, q_off + Lq, k_off + Lk)
    need = lib.attn_block_fwd_workspace_size(B, Lq, Lk, int(kpm is not None or am is not None))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    rc = lib.attn_block_fwd(_tensor(q), _tensor(k), _tensor(v), B, H, Lq, Lk, d, dt, q_off, k_off, kpm, kpm_ld,
                            am, am_ld, int(bool(causal)), 0.0 if scale is None else float(scale),
                            _ptr(out), _dtype_code(out.dtype), _ptr(lse), int(bool(accumulate)),
                            _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream))
    _check("attn_block_fwd", rc)
    return out, lse


def attn_block_fwd_noalloc(q, k, v, out, lse, *, q_off=0, k_off=0, key_padding_mask=None, attn_mask=None,
                           causal=False, scale=None, accumulate=False, stream=None):
    """attn_block_fwd for callers that cannot allocate device memory: the caller
    passes out and lse, and the library allocates nothing (its tile-class scratch
    is a fixed device array of BA_NOALLOC_MAX_CLASS_BYTES).  Returns (out, lse)."""
    lib = load()
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    _check_out(out, lse, (B, H, Lq, d))
    kpm, kpm_ld, am, am_ld = _masks(key_padding_mask, attn_mask, B, q_off + Lq, k_off + Lk)
    rc = lib.attn_block_fwd_noalloc(_tensor(q), _tensor(k), _tensor(v), B, H, Lq, Lk, d, _dtype_code(q.dtype),
                                    q_off, k_off, kpm, kpm_ld, am, am_ld, int(bool(causal)),
                                    0.0 if scale is None else float(scale), _ptr(out), _dtype_code(out.dtype),
                                    _ptr(lse), int(bool(accumulate)), _stream(stream))
    _check("attn_block_fwd_noalloc", rc)
    return out, lse


def attn_merge(out_a, lse_a, out_b, lse_b, stream=None):
    """In place: (out_a, lse_a) <- LSE merge of (out_a, lse_a) and (out_b, lse_b)."""
    lib = load()
    for t in (out_a, lse_a, out_b, lse_b):
        if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("attn_merge takes contiguous fp32 CUDA tensors")
    d = out_a.shape[-1]
    rows = lse_a.numel()
    if out_a.numel() != rows * d or out_b.numel() != rows * d or lse_b.numel() != rows:
        raise ValueError("shape mismatch")
    _check("attn_merge", lib.attn_merge(_ptr(out_a), _ptr(lse_a), _ptr(out_b), _ptr(lse_b), rows, d,
                                        _stream(stream)))
    return out_a, lse_a


def ring_attn_fwd_workspace_size(B, H, T, d, dtype, P, partition="contiguous", mode="fused", has_masks=False,
                                 rope=False, out_dtype=None):
    lib = load()
    dt = _dtype_code(dtype)
    odt = dt if out_dtype is None else _dtype_code(out_dtype)
    return lib.ring_attn_fwd_workspace_size(B, H, T, d, dt, P, PARTITIONS[partition], MODES[mode],
                                            int(bool(has_masks)), int(bool(rope)), odt)


def ring_attn_fwd(q, k, v, *, P, partition="contiguous", mode="fused", key_padding_mask=None, attn_mask=None,
                  causal=False, scale=None, rope=False, rope_base=10000.0, out=None, out_dtype=None, lse=None,
                  return_index_maps=False, workspace=None, stream=None):
    """Ring Attention over P emulated ranks; see include/blockattn.h.
    Returns (out, lse) or (out, lse, tok_of (P, T/P), schedule (P, P))."""
    lib = load()
    B, H, T, d = q.shape
    dt = _dtype_code(q.dtype)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out is None:
        out = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    _check_out(out, lse, (B, H, T, d))
    kpm, kpm_ld, am, am_ld = _masks(key_padding_mask, attn_mask, B, T, T)
    masks = kpm is not None or am is not None
    need = ring_attn_fwd_workspace_size(B, H, T, d, q.dtype, P, partition, mode, masks, rope, out.dtype)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    maps = None
    if return_index_maps:
        maps = (ctypes.c_int32 * (T + P * P))()
    rc = lib.ring_attn_fwd(_tensor(q), _tensor(k), _tensor(v), B, H, T, d, dt, P, PARTITIONS[partition],
                           MODES[mode], kpm, kpm_ld, am, am_ld, int(bool(causal)),
                           0.0 if scale is None else float(scale), int(bool(rope)), float(rope_base),
                           _ptr(out), _dtype_code(out.dtype), _ptr(lse),
                           None if maps is None else ctypes.cast(maps, ctypes.c_void_p),
                           _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream))
    _check("ring_attn_fwd", rc)
    if return_index_maps:
        import numpy as np
        arr = np.ctypeslib.as_array(maps).copy()
        return out, lse, arr[:T].reshape(P, T // P), arr[T:].reshape(P, P)
    return out, lse


def _grads(B, H, Lq, Lk, d, device, dq, dk, dv):
    shapes = ((dq, (B, H, Lq, d)), (dk, (B, H, Lk, d)), (dv, (B, H, Lk, d)))
    res = []
    for t, shape in shapes:
        if t is None:
            t = torch.empty(shape, dtype=torch.float32, device=device)
        elif t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != shape or not t.is_cuda:
            raise ValueError(f"gradient buffers must be contiguous fp32 CUDA tensors of shape {shape}")
        res.append(t)
    return res


def _check_bwd_inputs(q, out, dout, lse):
    if out.dtype != q.dtype or dout.dtype != q.dtype:
        raise TypeError("out and dout must have the dtype of q")
    if out.shape != q.shape or dout.shape != q.shape:
        raise ValueError("out and dout must have the shape of q")
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != tuple(q.shape[:3]):
        raise ValueError("lse must be a contiguous fp32 tensor of shape (B, H, L)")


def attn_block_bwd(q, k, v, out, dout, lse, *, q_off=0, k_off=0, key_padding_mask=None, attn_mask=None,
                   causal=False, scale=None, dq=None, dk=None, dv=None, accumulate=False, workspace=None,
                   stream=None):
    """Gradients (dq, dk, dv) (fp32) of one attention block given the forward
    out and lse of the whole rows; see include/blockattn.h."""
    lib = load()
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    _check_bwd_inputs(q, out, dout, lse)
    dq, dk, dv = _grads(B, H, Lq, Lk, d, q.device, dq, dk, dv)
    kpm, kpm_ld, am, am_ld = _masks(key_padding_mask, attn_mask, B, q_off + Lq, k_off + Lk)
    need = lib.attn_block_bwd_workspace_size(B, H, Lq)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    rc = lib.attn_block_bwd(_tensor(q), _tensor(k), _tensor(v), _tensor(out), _tensor(dout), _ptr(lse), B, H, Lq,
                            Lk, d, _dtype_code(q.dtype), q_off, k_off, kpm, kpm_ld, am, am_ld, int(bool(causal)),
                            0.0 if scale is None else float(scale), _ptr(dq), _ptr(dk), _ptr(dv),
                            int(bool(accumulate)), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                            _stream(stream))
    _check("attn_block_bwd", rc)
    return dq, dk, dv


def ring_attn_bwd(q, k, v, out, dout, lse, *, P, partition="contiguous", mode="fused", key_padding_mask=None,
                  attn_mask=None, causal=False, scale=None, dq=None, dk=None, dv=None, workspace=None,
                  stream=None):
    """Ring Attention backward over P emulated ranks: (dq, dk, dv) fp32 in global
    token order; see include/blockattn.h."""
    lib = load()
    B, H, T, d = q.shape
    _check_bwd_inputs(q, out, dout, lse)
    dq, dk, dv = _grads(B, H, T, T, d, q.device, dq, dk, dv)
    kpm, kpm_ld, am, am_ld = _masks(key_padding_mask, attn_mask, B, T, T)
    need = lib.ring_attn_bwd_workspace_size(B, H, T)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    rc = lib.ring_attn_bwd(_tensor(q), _tensor(k), _tensor(v), _tensor(out), _tensor(dout), _ptr(lse), B, H, T, d,
                           _dtype_code(q.dtype), P, PARTITIONS[partition], MODES[mode], kpm, kpm_ld, am, am_ld,
                           int(bool(causal)), 0.0 if scale is None else float(scale), _ptr(dq), _ptr(dk),
                           _ptr(dv), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                           _stream(stream))
    _check("ring_attn_bwd", rc)
    return dq, dk, dv


A2A = {"token_to_head": 0, "head_to_token": 1}


def ulysses_all_to_all(x, P, direction, *, out=None, stream=None):
    """One Ulysses exchange of a contiguous stacked array: token_to_head takes
    (P, H, B, T/P, d) to (P, H/P, B, T, d); head_to_token is the inverse."""
    lib = load()
    if not x.is_contiguous() or not x.is_cuda:
        raise ValueError("ulysses_all_to_all takes a contiguous CUDA tensor")
    if direction == "token_to_head":
        P_, H, B, Tl, d = x.shape
        shape, T = (P, H // P, B, Tl * P, d), Tl * P
    elif direction == "head_to_token":
        P_, hl, B, T, d = x.shape
        H = hl * P
        shape = (P, H, B, T // P, d)
    else:
        raise ValueError(direction)
    if P_ != P:
        raise ValueError("leading axis must be P")
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    elif tuple(out.shape) != shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous tensor of shape {shape}")
    rc = lib.ulysses_all_to_all(_ptr(x), _ptr(out), P, H, B, T, d, x.element_size(), A2A[direction],
                                _stream(stream))
    _check("ulysses_all_to_all", rc)
    return out


def ulysses_attn_fwd(q_tok, k_tok, v_tok, *, key_padding_mask=None, attn_mask=None, causal=False, scale=None,
                     out=None, lse=None, workspace=None, stream=None):
    """Ulysses attention over P emulated ranks from token shards (P, H, B, T/P, d):
    returns (out (P, H, B, T/P, d), lse (P, H, B, T/P) fp32); see include/blockattn.h."""
    lib = load()
    for t in (q_tok, k_tok, v_tok):
        if not t.is_contiguous() or not t.is_cuda or t.shape != q_tok.shape or t.dtype != q_tok.dtype:
            raise ValueError("q_tok, k_tok, v_tok must be contiguous CUDA tensors of one shape and dtype")
    P, H, B, Tl, d = q_tok.shape
    T = P * Tl
    if out is None:
        out = torch.empty_like(q_tok)
    if lse is None:
        lse = torch.empty((P, H, B, Tl), dtype=torch.float32, device=q_tok.device)
    if tuple(out.shape) != tuple(q_tok.shape) or out.dtype != q_tok.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous, of the shape and dtype of q_tok")
    if tuple(lse.shape) != (P, H, B, Tl) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor of shape (P, H, B, T/P)")
    kpm, kpm_ld, am, am_ld = _masks(key_padding_mask, attn_mask, B, T, T)
    dt = _dtype_code(q_tok.dtype)
    need = lib.ulysses_attn_fwd_workspace_size(P, H, B, T, d, dt, int(kpm is not None or am is not None))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_tok.device)
    rc = lib.ulysses_attn_fwd(_ptr(q_tok), _ptr(k_tok), _ptr(v_tok), P, H, B, T, d, dt, kpm, kpm_ld, am, am_ld,
                              int(bool(causal)), 0.0 if scale is None else float(scale), _ptr(out), _ptr(lse),
                              _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream))
    _check("ulysses_attn_fwd", rc)
    return out, lse


# Helpers of the entry points below.  A single-token call is over on the GPU in a few
# microseconds, so a call that leaves its outputs, workspace and stream to the binding is
# marshalled in C++ (csrc/fastcall.cpp), which answers None to whatever is out of the ordinary.
# That, and everything that is to be refused, goes on here: one stride() per tensor, devices
# and streams as integers, sizes of workspaces remembered.

_DTYPES = {torch.float32: BA_F32, torch.bfloat16: BA_BF16}


def _code(dtype):
    c = _DTYPES.get(dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return c


def _view(name, x):
    """(pointer, strides) of a (B, H, T, d) tensor."""
    s = x.stride()
    if len(s) != 4 or s[3] != 1 and x.shape[3] > 1:
        raise ValueError(f"{name}: expected a (B, H, T, d) tensor with a contiguous last axis")
    return ba_tensor(x.data_ptr(), s[0], s[1], s[2])


def _device(ref, **tensors):
    """Index of ref's device: the current one (launches and torch's streams go there), and every tensor's."""
    dev = ref.get_device()
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{dev}, but the current device is cuda:{torch._C._cuda_getDevice()}")
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    return dev


def _on_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _kv_heads(q, k, v):
    """Checks k, v (B, Hkv, L, d) against q (B, Hq, .., d) and returns (B, Hq, Lq, d, Hkv, L)."""
    qs, ks = q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4 or ks != v.shape:
        raise ValueError("expected q (B, Hq, L, d) and k, v (B, Hkv, L, d) of one shape")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share a dtype")
    B, Hq, Lq, d = qs
    Bk, Hkv, Lk, dk = ks
    if Bk != B or dk != d:
        raise ValueError(f"k, v of shape {tuple(ks)} do not match q of shape {tuple(qs)}")
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads are not a multiple of {Hkv} key heads")
    return B, Hq, Lq, d, Hkv, Lk


def _empty(ref, shape, dtype, stream):
    """A new tensor beside ref, from the memory of the stream that the call runs on (so that
    nothing still pending on another stream uses the memory, and its reuse waits for this call)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=ref.device)   # (ref.new_empty takes 1 us more)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=ref.device)


def _buffer(ref, name, t, shape, dtype, stream):
    """An output: t checked (contiguous, of the shape and dtype, on ref's device), or a new one."""
    if t is None:
        return _empty(ref, shape, dtype, stream)
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.get_device() != ref.get_device():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {ref.device}")
    return t


def _out_pair(q, shape, out, out_dtype, lse, stream):
    """out and lse of an attention call on q of the given shape, and out's dtype code."""
    if out_dtype is None:
        out_dtype = q.dtype if out is None else out.dtype
    code = _DTYPES.get(out_dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {out_dtype}")
    if out is None and lse is None and stream is None:
        dev = q.device
        return (torch.empty(shape, dtype=out_dtype, device=dev), torch.empty(shape[:3], dtype=torch.float32, device=dev),
                code)
    return (_buffer(q, "out", out, shape, out_dtype, stream), _buffer(q, "lse", lse, shape[:3], torch.float32, stream),
            code)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(fn, dev, *sizes):
    """Bytes that a *_workspace_size query gives for these sizes on device dev (the current one)."""
    return getattr(load(), fn)(*sizes)


def _scratch(ref, need, workspace, stream):
    """(pointer, bytes, tensor) of a workspace: the caller's or a new one (the tensor is kept until the launch)."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = _empty(ref, (need,), torch.uint8, stream)
    elif not workspace.is_contiguous() or workspace.dtype != torch.uint8 or workspace.get_device() != ref.get_device():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace.data_ptr(), workspace.numel(), workspace


def _c_int(name, x, lo):
    if not lo <= x < 2147483648 or int(x) != x:
        raise ValueError(f"{name} = {x} is not an integer in [{lo}, 2^31)")
    return int(x)


def attn_window_fwd(q, k, v, *, window, sinks=0, q_off=0, key_padding_mask=None, scale=None, out=None, out_dtype=None,
                    lse=None, workspace=None, stream=None):
    """Causal attention with a sliding window and `sinks` first keys that stay visible:
    q (B, Hq, Lq, d) at positions q_off + i against k, v (B, Hkv, Lk, d) at positions
    0 .. Lk - 1, Hkv dividing Hq; see include/blockattn.h.  Returns (out, lse)."""
    lib = load()
    if _fast is not None and out is out_dtype is lse is workspace is stream is None:
        r = _fast.attn_window_fwd(q, k, v, window, sinks, q_off, key_padding_mask, scale)
        if r is not None:
            return r
    B, Hq, Lq, d, Hkv, Lk = _kv_heads(q, k, v)
    window, sinks, q_off = _c_int("window", window, 1), _c_int("sinks", sinks, 0), _c_int("q_off", q_off, 0)
    dt = _code(q.dtype)
    dev = _device(q, k=k, v=v, key_padding_mask=key_padding_mask)
    out, lse, odt = _out_pair(q, (B, Hq, Lq, d), out, out_dtype, lse, stream)
    kpm, kpm_ld = _mask(key_padding_mask, B, Lk, "key_padding_mask")
    need = _workspace_bytes("attn_window_fwd_workspace_size", dev, B, Hq, Lq, d, dt)
    ws, ws_bytes, keep = _scratch(q, need, workspace, stream)
    rc = lib.attn_window_fwd(_view("q", q), _view("k", k), _view("v", v), B, Hq, Hkv, Lq, Lk, d, dt, q_off, window, sinks,
                             kpm, kpm_ld, 0.0 if scale is None else float(scale), out.data_ptr(), odt,
                             lse.data_ptr(), ws, ws_bytes, _on_stream(stream, dev))
    _check("attn_window_fwd", rc)
    return out, lse


def attn_window_bwd(q, k, v, out, dout, lse, *, window, sinks=0, q_off=0, key_padding_mask=None, scale=None, dq=None,
                    dk=None, dv=None, grad_dtype=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of attn_window_fwd from its out and lse; of q's dtype
    unless grad_dtype (or the given buffers) say float32; see include/blockattn.h."""
    lib = load()
    if _fast is not None and dq is dk is dv is grad_dtype is workspace is stream is None:
        r = _fast.attn_window_bwd(q, k, v, out, dout, lse, window, sinks, q_off, key_padding_mask, scale)
        if r is not None:
            return r
    B, Hq, Lq, d, Hkv, Lk = _kv_heads(q, k, v)
    window, sinks, q_off = _c_int("window", window, 1), _c_int("sinks", sinks, 0), _c_int("q_off", q_off, 0)
    dt = _code(q.dtype)
    _check_bwd_inputs(q, out, dout, lse)
    dev = _device(q, k=k, v=v, out=out, dout=dout, lse=lse, key_padding_mask=key_padding_mask)
    if grad_dtype is None:
        grad_dtype = next((t.dtype for t in (dq, dk, dv) if t is not None), q.dtype)
    dq = _buffer(q, "dq", dq, q.shape, grad_dtype, stream)
    dk = _buffer(q, "dk", dk, k.shape, grad_dtype, stream)
    dv = _buffer(q, "dv", dv, v.shape, grad_dtype, stream)
    kpm, kpm_ld = _mask(key_padding_mask, B, Lk, "key_padding_mask")
    need = _workspace_bytes("attn_window_bwd_workspace_size", dev, B, Hq, Hkv, Lq, Lk, d, q_off, window, sinks)
    ws, ws_bytes, keep = _scratch(q, need, workspace, stream)
    rc = lib.attn_window_bwd(_view("q", q), _view("k", k), _view("v", v), _view("out", out), _view("dout", dout),
                             lse.data_ptr(), B, Hq, Hkv, Lq, Lk, d, dt, q_off, window, sinks, kpm, kpm_ld,
                             0.0 if scale is None else float(scale), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                             _code(grad_dtype), ws, ws_bytes, _on_stream(stream, dev))
    _check("attn_window_bwd", rc)
    return dq, dk, dv


def attn_decode_fwd(q, k_cache, v_cache, *, lengths=None, num_splits=0, scale=None, out=None, out_dtype=None,
                    lse=None, workspace=None, stream=None):
    """Decode attention of q (B, H, 1, d) against k_cache, v_cache (B, H, S, d),
    split along the keys and merged by the LSE rule; lengths: int32 (B) CUDA
    tensor of valid cache lengths or None.  Returns (out, lse)."""
    lib = load()
    B, H, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes one query per (b, h): q of shape (B, H, 1, d)")
    S = k_cache.shape[2]
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out is None:
        out = torch.empty((B, H, 1, d), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, 1), dtype=torch.float32, device=q.device)
    _check_out(out, lse, (B, H, 1, d))
    if lengths is not None and (lengths.dtype != torch.int32 or not lengths.is_cuda or lengths.numel() != B):
        raise ValueError("lengths must be an int32 CUDA tensor of B entries")
    need = lib.attn_decode_workspace_size(B, H, S, d, int(num_splits))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    rc = lib.attn_decode_fwd(_tensor(q), _tensor(k_cache), _tensor(v_cache), B, H, S, d, _dtype_code(q.dtype),
                             _ptr(lengths), int(num_splits), 0.0 if scale is None else float(scale), _ptr(out),
                             _dtype_code(out.dtype), _ptr(lse), _ptr(workspace),
                             0 if workspace is None else workspace.numel(), _stream(stream))
    _check("attn_decode_fwd", rc)
    return out, lse


def _per_sequence(name, t, B, dev):
    """Pointer of an int32 entry for each sequence, or None."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.get_device() != dev or t.numel() != B or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {B} entries on cuda:{dev}")
    return t.data_ptr()


def attn_window_decode_fwd(q, k_cache, v_cache, *, window, sinks=0, lengths=None, scale=None, out=None, out_dtype=None,
                           lse=None, workspace=None, stream=None):
    """Single-token form of attn_window_fwd: q (B, Hq, 1, d) at position lengths[b] - 1
    against the caches (B, Hkv, S, d), Hkv dividing Hq; lengths: int32 (B) or None (S).
    Returns (out, lse)."""
    lib = load()
    if _fast is not None and out is out_dtype is lse is workspace is stream is None:
        r = _fast.attn_window_decode_fwd(q, k_cache, v_cache, window, sinks, lengths, scale)
        if r is not None:
            return r
    B, Hq, one, d, Hkv, S = _kv_heads(q, k_cache, v_cache)
    if one != 1:
        raise ValueError("decode takes one query per (b, h): q of shape (B, Hq, 1, d)")
    window, sinks = _c_int("window", window, 1), _c_int("sinks", sinks, 0)
    dt = _code(q.dtype)
    dev = _device(q, k_cache=k_cache, v_cache=v_cache)
    lens = _per_sequence("lengths", lengths, B, dev)
    out, lse, odt = _out_pair(q, (B, Hq, 1, d), out, out_dtype, lse, stream)
    need = _workspace_bytes("attn_window_decode_workspace_size", dev, B, Hq, Hkv, S, d, window, sinks)
    ws, ws_bytes, keep = _scratch(q, need, workspace, stream)
    rc = lib.attn_window_decode_fwd(_view("q", q), _view("k_cache", k_cache), _view("v_cache", v_cache), B, Hq, Hkv, S, d,
                                    dt, lens, window, sinks, 0.0 if scale is None else float(scale), out.data_ptr(),
                                    odt, lse.data_ptr(), ws, ws_bytes, _on_stream(stream, dev))
    _check("attn_window_decode_fwd", rc)
    return out, lse


class KV4Cache:
    """A KV cache held in 4 bits: codes (B, H, S, d / 2) and scales (B, H, S, d / 16), uint8,
    of K and of V, with the tensors' powers of two; see include/blockattn.h (ba_kv4)."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "k_exp", "v_exp", "shape", "dev", "_c")

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_exp=0, v_exp=0):
        dev = k_codes.get_device()
        for t in (k_codes, k_scales, v_codes, v_scales):
            if t.dtype != torch.uint8 or t.dim() != 4 or t.get_device() != dev or dev < 0:
                raise ValueError("codes and scales are 4-D uint8 CUDA tensors on one device")
        B, H, S, half = shape = k_codes.shape
        cs, ss = k_codes.stride(), k_scales.stride()
        if half != 64 and half != 32:
            raise ValueError(f"codes of {half} bytes a row: rows of d = 64 or 128 values take 32 or 64")
        if v_codes.shape != shape or k_scales.shape != (B, H, S, half // 8) or v_scales.shape != k_scales.shape:
            raise ValueError("codes (B, H, S, d / 2) and scales (B, H, S, d / 16) of K and V must match")
        if v_codes.stride() != cs or v_scales.stride() != ss or cs[3] != 1 or ss[3] != 1:
            raise ValueError("K and V must have the same strides, and contiguous last axes")
        if not (-100 <= k_exp <= 100 and -100 <= v_exp <= 100 and int(k_exp) == k_exp and int(v_exp) == v_exp):
            raise ValueError(f"exponents {k_exp}, {v_exp} are not integers in [-100, 100]")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_exp, self.v_exp, self.shape, self.dev = int(k_exp), int(v_exp), (B, H, S, 2 * half), dev
        self._c = ba_kv4(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                         cs[0], cs[1], cs[2], ss[0], ss[1], ss[2], self.k_exp, self.v_exp)

    @classmethod
    def empty(cls, B, H, S, d, *, device="cuda", k_exp=0, v_exp=0):
        """A new cache of S slots per (b, h); its slots hold zeros."""
        def new(n):
            return torch.zeros((B, H, S, n), dtype=torch.uint8, device=device)
        return cls(new(d // 2), new(d // 16), new(d // 2), new(d // 16), k_exp, v_exp)


def kv4_append(cache, k, v, *, start=None, counts=None, stream=None):
    """Quantise k, v (B, H, T, d) into the slots start[b] + t of a KV4Cache (t < counts[b]);
    start, counts: int32 (B) CUDA tensors or None (0, T).  Slots outside the cache are dropped."""
    lib = load()
    if _fast is not None and stream is None:
        r = _fast.kv4_append(cache, k, v, start, counts)
        if r is not None:
            return r
    B, H, S, d = cache.shape
    shape = k.shape
    if len(shape) != 4 or shape != v.shape or k.dtype != v.dtype or shape[0] != B or shape[1] != H or shape[3] != d:
        raise ValueError(f"k, v of shape {tuple(shape)} do not match a cache of {cache.shape}")
    dev = _device(k, v=v, cache=cache.k_codes)
    rc = lib.kv4_append(_view("k", k), _view("v", v), cache._c, B, H, shape[2], S, d, _code(k.dtype),
                        _per_sequence("start", start, B, dev), _per_sequence("counts", counts, B, dev),
                        _on_stream(stream, dev))
    _check("kv4_append", rc)
    return cache


def kv4_read(cache, T, *, first=0, dtype=torch.bfloat16, out_k=None, out_v=None, stream=None):
    """The values of slots first .. first + T - 1 of a KV4Cache: (k, v), each (B, H, T, d)."""
    lib = load()
    if _fast is not None and out_k is out_v is stream is None:
        r = _fast.kv4_read(cache, T, first, dtype)
        if r is not None:
            return r
    B, H, S, d = cache.shape
    T, first, dt = _c_int("T", T, 0), _c_int("first", first, 0), _code(dtype)
    codes = cache.k_codes
    dev = _device(codes)
    k = _buffer(codes, "out_k", out_k, (B, H, T, d), dtype, stream)
    v = _buffer(codes, "out_v", out_v, (B, H, T, d), dtype, stream)
    rc = lib.kv4_read(cache._c, B, H, S, d, first, T, dt, k.data_ptr(), v.data_ptr(), _on_stream(stream, dev))
    _check("kv4_read", rc)
    return k, v


def attn_decode_kv4_fwd(q, cache, *, lengths=None, window=0, sinks=0, scale=None, out=None, out_dtype=None, lse=None,
                        workspace=None, stream=None):
    """Single-token attention of q (B, Hq, 1, d) bf16 over a KV4Cache of (B, Hkv, S, d), over
    every key (window = 0) or a window with sinks; see include/blockattn.h.  Returns (out, lse)."""
    lib = load()
    if _fast is not None and out is out_dtype is lse is workspace is stream is None:
        r = _fast.attn_decode_kv4_fwd(q, cache, lengths, window, sinks, scale)
        if r is not None:
            return r
    B, Hkv, S, d = cache.shape
    shape = tuple(q.shape)
    if len(shape) != 4 or shape[0] != B or shape[2] != 1 or shape[3] != d or Hkv == 0 or shape[1] % Hkv:
        raise ValueError(f"q of shape {tuple(shape)} does not match a cache of {cache.shape}")
    Hq = shape[1]
    window, sinks = _c_int("window", window, 0), _c_int("sinks", sinks, 0)
    dev = _device(q, cache=cache.k_codes)
    lens = _per_sequence("lengths", lengths, B, dev)
    out, lse, odt = _out_pair(q, (B, Hq, 1, d), out, out_dtype, lse, stream)
    need = _workspace_bytes("attn_decode_kv4_workspace_size", dev, B, Hq, Hkv, S, d, window, sinks)
    ws, ws_bytes, keep = _scratch(q, need, workspace, stream)
    rc = lib.attn_decode_kv4_fwd(_view("q", q), cache._c, B, Hq, Hkv, S, d, _code(q.dtype), lens, window, sinks,
                                 0.0 if scale is None else float(scale), out.data_ptr(), odt,
                                 lse.data_ptr(), ws, ws_bytes, _on_stream(stream, dev))
    _check("attn_decode_kv4_fwd", rc)
    return out, lse


def rope_apply(x, *, x2=None, base=10000.0, positions=None, pos_scale=1.0, out=None, out2=None, stream=None):
    """Rotary position embedding of x (B, H, T, d) into a contiguous output; with
    x2 given, rotates x2 by the same launch and returns (y, y2).  pos_scale is
    the Position Interpolation factor applied to the position index."""
    lib = load()
    B, H, T, d = x.shape
    if out is None:
        out = torch.empty((B, H, T, d), dtype=x.dtype, device=x.device)
    if x2 is not None:
        if x2.shape != x.shape or x2.dtype != x.dtype:
            raise ValueError("x2 must match x")
        if out2 is None:
            out2 = torch.empty((B, H, T, d), dtype=x.dtype, device=x.device)
    if positions is not None and (positions.dtype != torch.int32 or not positions.is_cuda):
        raise ValueError("positions: int32 CUDA tensor")
    t2 = _tensor(x2) if x2 is not None else ba_tensor(None, 0, 0, 0)
    _check("rope_apply", lib.rope_apply(_tensor(x), t2, B, H, T, d, _dtype_code(x.dtype), _ptr(positions),
                                        float(base), float(pos_scale), _ptr(out), _ptr(out2), _stream(stream)))
    return out if x2 is None else (out, out2)


def _norm_inputs(q, k, wq, wk, positions):
    """Checks of qk_norm_rope_*: ((B, Hq, Hkv, T, d), weight dtype code, positions pointer, ld)."""
    B, Hq, T, d = q.shape
    Bk, Hkv, Tk, dk = k.shape
    if Bk != B or Tk != T or dk != d:
        raise ValueError(f"k of shape {tuple(k.shape)} does not match q of shape {tuple(q.shape)}")
    if k.dtype != q.dtype or wq.dtype != wk.dtype or (wq.dtype != q.dtype and wq.dtype != torch.float32):
        raise TypeError("q and k share a dtype; the weights have it too or are float32")
    if wq.shape != (d,) or wk.shape != (d,) or not wq.is_contiguous() or not wk.is_contiguous():
        raise ValueError(f"wq and wk must be contiguous tensors of {d} entries")
    if positions is None:
        return (B, Hq, Hkv, T, d), _code(wq.dtype), None, 0
    shape, s, ld = positions.shape, positions.stride(), 0
    if positions.dtype != torch.int32 or len(shape) not in (1, 2) or shape[-1] != T or (T > 1 and s[-1] != 1) or \
            (len(shape) == 2 and shape[0] not in (1, B)):
        raise ValueError(f"positions must be an int32 CUDA tensor (T,) or (B, T) with T = {T}")
    if len(shape) == 2 and shape[0] == B and B > 1 and s[0] != 0:   # (an expanded row is shared by all)
        ld = s[0]
        if ld < T:
            raise ValueError("the rows of positions overlap")
    return (B, Hq, Hkv, T, d), _code(wq.dtype), positions.data_ptr(), ld


def qk_norm_rope_fwd(q, k, wq, wk, *, eps=1e-6, positions=None, base=10000.0, pos_scale=1.0, out_q=None, out_k=None,
                     stream=None):
    """Per-head RMS norm and rotation of q (B, Hq, T, d) and k (B, Hkv, T, d) in one pass;
    wq, wk (d); positions: int32 (T,) or (B, T), None: 0 .. T - 1; see include/blockattn.h.
    Returns (yq, yk), contiguous."""
    lib = load()
    if _fast is not None and out_q is out_k is stream is None:
        r = _fast.qk_norm_rope_fwd(q, k, wq, wk, eps, positions, base, pos_scale)
        if r is not None:
            return r
    tq, tk = _view("q", q), _view("k", k)
    sizes, wdt, pos, ld = _norm_inputs(q, k, wq, wk, positions)
    dev = _device(q, k=k, wq=wq, wk=wk, positions=positions)
    yq, yk = _buffer(q, "out_q", out_q, q.shape, q.dtype, stream), _buffer(q, "out_k", out_k, k.shape, q.dtype, stream)
    rc = lib.qk_norm_rope_fwd(tq, tk, wq.data_ptr(), wk.data_ptr(), wdt, *sizes, _code(q.dtype), float(eps), pos, ld,
                              float(base), float(pos_scale), yq.data_ptr(), yk.data_ptr(), _on_stream(stream, dev))
    _check("qk_norm_rope_fwd", rc)
    return yq, yk


def qk_norm_rope_bwd(q, k, wq, wk, dyq, dyk, *, eps=1e-6, positions=None, base=10000.0, pos_scale=1.0, dq=None, dk=None,
                     workspace=None, stream=None):
    """Gradients (dq, dk, dwq, dwk) of qk_norm_rope_fwd for dyq, dyk (of q's dtype or
    float32): dq, dk of q's dtype, dwq, dwk float32."""
    lib = load()
    if _fast is not None and dq is dk is workspace is stream is None:
        r = _fast.qk_norm_rope_bwd(q, k, wq, wk, eps, positions, base, pos_scale, dyq, dyk)
        if r is not None:
            return r
    tensors = _view("q", q), _view("k", k), _view("dyq", dyq), _view("dyk", dyk)
    sizes, wdt, pos, ld = _norm_inputs(q, k, wq, wk, positions)
    if dyq.shape != q.shape or dyk.shape != k.shape:
        raise ValueError("dyq and dyk must have the shapes of q and k")
    if dyq.dtype != dyk.dtype or (dyq.dtype != q.dtype and dyq.dtype != torch.float32):
        raise TypeError("dyq and dyk have the dtype of q or are float32")
    dev = _device(q, k=k, wq=wq, wk=wk, positions=positions, dyq=dyq, dyk=dyk)
    dt, d = _code(q.dtype), sizes[4]
    dq, dk = _buffer(q, "dq", dq, q.shape, q.dtype, stream), _buffer(q, "dk", dk, k.shape, q.dtype, stream)
    dwq, dwk = _empty(q, (2, d), torch.float32, stream).unbind(0)
    ws, ws_bytes, keep = _scratch(q, _workspace_bytes("qk_norm_rope_bwd_workspace_size", dev, *sizes, dt), workspace, stream)
    rc = lib.qk_norm_rope_bwd(tensors[0], tensors[1], wq.data_ptr(), wk.data_ptr(), wdt, tensors[2], tensors[3],
                              _code(dyq.dtype), *sizes, dt, float(eps), pos, ld, float(base), float(pos_scale),
                              dq.data_ptr(), dk.data_ptr(), dwq.data_ptr(), dwk.data_ptr(), ws, ws_bytes,
                              _on_stream(stream, dev))
    _check("qk_norm_rope_bwd", rc)
    return dq, dk, dwq, dwk


def tile_classes(B, Lq, Lk, *, q_off=0, k_off=0, key_padding_mask=None, attn_mask=None, causal=False,
                 device="cuda", stream=None):
    """int8 (B, ceil(Lq/128), ceil(Lk/128)) tile classes computed on the device."""
    lib = load()
    out = torch.empty((B, -(-Lq // 128), -(-Lk // 128)), dtype=torch.int8, device=device)
    kpm, kpm_ld, am, am_ld = _masks(key_padding_mask, attn_mask, B, q_off + Lq, k_off + Lk)
    _check("ba_tile_classes", lib.ba_tile_classes(B, Lq, Lk, q_off, k_off, kpm, kpm_ld, am, am_ld,
                                                  int(bool(causal)), _ptr(out), _stream(stream)))
    return out


def index_maps(T, P, partition="contiguous"):
    """Host, exact: (tok_of (P, T/P) int32, schedule (P, P) int32)."""
    import numpy as np
    lib = load()
    tok = np.zeros(T, dtype=np.int32)
    sch = np.zeros(P * P, dtype=np.int32)
    _check("ba_index_maps", lib.ba_index_maps(T, P, PARTITIONS[partition], tok.ctypes.data_as(ctypes.c_void_p),
                                              sch.ctypes.data_as(ctypes.c_void_p)))
    return tok.reshape(P, T // P), sch.reshape(P, P)


def pair_schedule(B, H, T, P, partition="zigzag", causal=True, num_sms=152):
    """Host, exact: the tensor-core forward kernel's work items for a ring_attn_fwd
    launch without masks, in dealing order, as an (n, 8) int32 array of
    (b, h, tile-0 row0, tile-0 rows, tile-1 row0, tile-1 rows, key tiles, phase)."""
    import numpy as np
    lib = load()
    n = lib.ba_pair_schedule(B, H, T, P, PARTITIONS[partition], int(causal), num_sms, None, 0)
    _check("ba_pair_schedule", min(n, 0))
    items = np.zeros((max(n, 0), 8), dtype=np.int32)
    if n > 0:
        _check("ba_pair_schedule", min(lib.ba_pair_schedule(B, H, T, P, PARTITIONS[partition], int(causal), num_sms,
                                                            items.ctypes.data_as(ctypes.c_void_p), n), 0))
    return items


def sync_status(stream=None) -> int:
    """Synchronise and return BA_OK, or BA_ERR_TIMEOUT when a bounded device wait expired."""
    return load().ba_sync_status(_stream(stream))


def debug_wait_timeout(timeout_ns: int, stream=None):
    _check("ba_debug_wait_timeout", load().ba_debug_wait_timeout(int(timeout_ns), _stream(stream)))
