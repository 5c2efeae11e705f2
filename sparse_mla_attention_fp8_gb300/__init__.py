"""Sparse MLA attention over the 656-byte FP8 cache, for GB300 (sm_103a).

Thin Python binding of the C-ABI library ``libsmla.so`` (declared in
``include/smla.h``).  Every function here only marshals torch tensors into
pointers and sizes and calls the same-named C entry point (the paged and MXFP8
operators through a compiled module, csrc/smla_binding.cpp); all the work runs in the
library's CUDA kernels.  There is no CPU fallback: if the library has
not been built, or a tensor is not on a CUDA device, the call raises.

Entry points (see include/smla.h for layouts and semantics):
  sparse_mla_decode_fp8, sparse_mla_prefill_bf16, mla_cache_store_fp8,
  sparse_mla_translate_indices, the separate-mode FP8 prefill
  (sparse_mla_prefill_fp8 with its steps sparse_mla_gather_upconvert_fp8 and
  sparse_mla_translate_indices_workspace, and the host-side
  sparse_mla_prefill_chunks), plus workspace-size and status helpers.
The paged 8-bit K/V cache of layers with separate K and V heads:
  paged_blocks_extend and paged_blocks_release (block tables and slot maps
  from request lengths), kv_cache_store_fp8, paged_attention_fp8.
What a decoder layer does around its attention, in MXFP8 (e4m3 codes with a
power-of-two scale per 32 values):
  mxfp8_quantize, rms_norm_mxfp8 (with the residual's addition), linear_mxfp8
  (with bias, activation, residual), moe_route and moe_mxfp8 (mixture of
  experts for few tokens).
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import threading
from concurrent.futures import ThreadPoolExecutor
from typing import Any, NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
_CSRC = os.path.join(_PKG, "csrc")
_BUILD = os.path.join(_PKG, "_build")
LIB_PATH = os.path.join(_PKG, "libsmla.so")
HEADER = os.path.join(_ROOT, "include", "smla.h")
BINDING_PATH = os.path.join(_PKG, "_binding.so")
_BINDING_STAMP = os.path.join(_BUILD, "binding.txt")  # what it was compiled against

SOURCES = ["smla_decode.cu", "smla_attn.cu", "smla_wide.cu", "smla_wide8.cu", "smla_store.cu", "smla_nvfp4.cu", "smla_absorb.cu",
           "smla_blocks.cu", "smla_kvstore.cu", "smla_paged_attn.cu", "smla_paged_prefill.cu",
           "smla_mxnorm.cu", "smla_linear.cu", "smla_moe.cu", "smla_route.cu", "smla_api.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]

SMLA_OK = 0
_lock = threading.Lock()
_lib = None
_binding = None


class SmlaError(RuntimeError):
    pass


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    deps = [src] + [os.path.join(_CSRC, f) for f in os.listdir(_CSRC) if f.endswith((".cuh", ".h"))] + [HEADER]
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA sources for sm_103a (in parallel) and link libsmla.so
    in place, and the Python binding of the paged and MXFP8 operators where torch is
    installed (the library itself needs nvcc alone).  Works without a GPU
    (nvcc cross-compiles)."""
    os.makedirs(_BUILD, exist_ok=True)
    nvcc = _nvcc()

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise SmlaError(f"{cmd[0]} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)

    def bind():
        tmp = BINDING_PATH + f".tmp{os.getpid()}"
        run(_binding_command(tmp))
        os.replace(tmp, BINDING_PATH)
        with open(_BINDING_STAMP, "w") as f:
            f.write(stamp)

    objs, jobs = [], []
    for s in SOURCES:
        src = os.path.join(_CSRC, s)
        objs.append(os.path.join(_BUILD, s.replace(".cu", ".o")))
        if force or _stale(objs[-1], src):
            jobs.append([nvcc, *NVCC_FLAGS, "-c", src, "-o", objs[-1]])
    stamp = _binding_stamp()
    binds = stamp is not None and (force or _binding_stale(stamp))
    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        binding = ex.submit(bind) if binds else None
        list(ex.map(run, jobs))
        if force or jobs or not os.path.exists(LIB_PATH):
            tmp = LIB_PATH + f".tmp{os.getpid()}"
            run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", *objs, "-o", tmp])
            os.replace(tmp, LIB_PATH)
        if binding is not None:
            binding.result()  # raises what went wrong there, the library being in place
    return LIB_PATH


def _binding_stamp():
    """What the Python binding is compiled against; None without torch."""
    import importlib.util
    import sys
    from importlib import metadata
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = metadata.version("torch")
    except metadata.PackageNotFoundError:  # a source tree on the path
        import torch
        version = torch.__version__
    return f"torch {version}, python {sys.version}"


def _binding_stale(stamp: str) -> bool:
    if _stale(BINDING_PATH, os.path.join(_CSRC, "smla_binding.cpp")) or not os.path.exists(_BINDING_STAMP):
        return True
    with open(_BINDING_STAMP) as f:
        return f.read() != stamp


def _binding_command(out: str) -> list:
    """The compiler call for the Python binding of the paged and MXFP8 operators (host
    code only, by the host compiler that nvcc finds, against the installed
    torch's headers)."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    return [_nvcc(), "-shared", "-O2", "-std=c++17", "-cudart", "none", "-Xcompiler", "-fPIC,-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-I" + sysconfig.get_path("include"), "-isystem", os.path.join(root, "include"), "-isystem",
            os.path.join(root, "include", "torch", "csrc", "api", "include"),
            os.path.join(_CSRC, "smla_binding.cpp"), "-o", out, "-L" + os.path.join(root, "lib"),
            "-Xlinker", "-rpath", "-Xlinker", os.path.join(root, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise SmlaError(f"{LIB_PATH} is missing: run sparse_mla_attention_fp8_gb300.build() first")
            L = ctypes.CDLL(LIB_PATH)
            P, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
            L.sparse_mla_decode_fp8.argtypes = [P, P, P, P, P, f32, i32, P, P, i32, i32, i32, i32, i32, i32, P, sz, P]
            L.sparse_mla_decode_fp8.restype = i32
            L.sparse_mla_decode_fp8_qfp8.argtypes = L.sparse_mla_decode_fp8.argtypes
            L.sparse_mla_decode_fp8_qfp8.restype = i32
            L.sparse_mla_decode_nvfp4.argtypes = L.sparse_mla_decode_fp8.argtypes
            L.sparse_mla_decode_nvfp4.restype = i32
            L.sparse_mla_decode_nvfp4_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.sparse_mla_decode_nvfp4_workspace_bytes.restype = sz
            L.mla_cache_store_nvfp4.argtypes = [P, P, P, i32, i32, P]
            L.mla_cache_store_nvfp4.restype = i32
            L.sparse_mla_decode_fp8_noalloc.argtypes = [P, P, P, P, P, f32, i32, P, P, i32, i32, i32, i32, i32, i32, P]
            L.sparse_mla_decode_fp8_noalloc.restype = i32
            L.sparse_mla_decode_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.sparse_mla_decode_workspace_bytes.restype = sz
            L.sparse_mla_prefill_bf16.argtypes = [P, P, P, f32, i32, P, P, i32, i32, i32, i32, P, sz, P]
            L.sparse_mla_prefill_bf16.restype = i32
            L.sparse_mla_prefill_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.sparse_mla_prefill_workspace_bytes.restype = sz
            L.sparse_mla_attention_plan.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
            L.sparse_mla_attention_plan.restype = i32
            L.mla_cache_store_fp8.argtypes = [P, P, P, i32, i32, P]
            L.mla_cache_store_fp8.restype = i32
            L.sparse_mla_translate_indices.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, P]
            L.sparse_mla_translate_indices.restype = i32
            L.smla_read_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_int), P]
            L.smla_read_device_status.restype = i32
            L.sparse_mla_prefill_fp8.argtypes = [P, P, P, P, P, P, P, f32, i32, P, P, i32, i32, i32, i32, i32, i32,
                                                 P, i32, P, sz, P]
            L.sparse_mla_prefill_fp8.restype = i32
            L.sparse_mla_prefill_fp8_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.sparse_mla_prefill_fp8_workspace_bytes.restype = sz
            L.sparse_mla_gather_upconvert_fp8.argtypes = [P, P, P, P, i32, i32, i32, P, i32, P]
            L.sparse_mla_gather_upconvert_fp8.restype = i32
            L.sparse_mla_translate_indices_workspace.argtypes = [P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, P]
            L.sparse_mla_translate_indices_workspace.restype = i32
            L.sparse_mla_prefill_chunks.argtypes = [P, i32, ctypes.c_int64, P, P, ctypes.POINTER(i32)]
            L.sparse_mla_prefill_chunks.restype = i32
            L.mla_absorb_q.argtypes = [P, P, P, i32, i32, i32, P, sz, P]
            L.mla_absorb_q.restype = i32
            L.mla_v_up_proj.argtypes = [P, P, P, i32, i32, i32, P, sz, P]
            L.mla_v_up_proj.restype = i32
            L.paged_blocks_extend.argtypes = [P] * 12 + [i32] * 5 + [P]
            L.paged_blocks_extend.restype = i32
            L.paged_blocks_release.argtypes = [P] * 7 + [i32] * 4 + [P]
            L.paged_blocks_release.restype = i32
            i64 = ctypes.c_int64
            L.kv_cache_store_fp8.argtypes = [P, i64, P, i64, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, P]
            L.kv_cache_store_fp8.restype = i32
            L.paged_attention_fp8.argtypes = [P, i64, P, P, P, P, P, P, P, f32, i32, i32, f32, P, P, P, P, P,
                                              i32, i32, i32, i32, i32, i32, i32, P, sz, P]
            L.paged_attention_fp8.restype = i32
            L.paged_attention_fp8_workspace_bytes.argtypes = [i32] * 6
            L.paged_attention_fp8_workspace_bytes.restype = sz
            L.mxfp8_quantize.argtypes = [P, i32, i64, P, P, i64, i32, i32, P]
            L.mxfp8_quantize.restype = i32
            L.rms_norm_mxfp8.argtypes = [P, i64, P, i64, P, i32, f32, P, P, i64, P, P, i32, i32, P]
            L.rms_norm_mxfp8.restype = i32
            L.linear_mxfp8.argtypes = [P, i64, P, i64, P, P, i64, P, i32, i32, P, i64, P, P, P, i64, i32, i32, i32, P]
            L.linear_mxfp8.restype = i32
            L.moe_route.argtypes = [P, i32, P, i32, i32, f32, i32, i32, P, P, i32, i32, i32, P]
            L.moe_route.restype = i32
            L.moe_mxfp8.argtypes = [P, i64, P, i64, P, P, P, P, i64, P, P, i64, P, i64, P, i32, i32, i32, i32, i32, P,
                                    sz, P]
            L.moe_mxfp8.restype = i32
            L.moe_mxfp8_workspace_bytes.argtypes = [i32] * 4
            L.moe_mxfp8_workspace_bytes.restype = sz
            L.smla_paged_wait_check.argtypes = [i32, P, P]
            L.smla_paged_wait_check.restype = i32
            L.smla_mxfp8_wait_check.argtypes = [i32, P]
            L.smla_mxfp8_wait_check.restype = i32
            L.smla_mxfp8_give_up.argtypes = [i32]
            L.smla_mxfp8_give_up.restype = None
            L.smla_read_noalloc_status.argtypes = [ctypes.POINTER(ctypes.c_int), P]
            L.smla_read_noalloc_status.restype = i32
            L.smla_last_error.argtypes = []
            L.smla_last_error.restype = ctypes.c_char_p
            L.smla_version.argtypes = []
            L.smla_version.restype = i32
            _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != SMLA_OK:
        msg = lib().smla_last_error().decode(errors="replace")
        raise SmlaError(f"{what} failed with status {rc}: {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(*tensors):
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise SmlaError("all tensors must be CUDA tensors (there is no CPU path)")
        if not t.is_contiguous():
            raise SmlaError("all tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise SmlaError("all tensors must be on the same device")
    return dev


def _expect(t, dtype, shape, name):
    if t.dtype != dtype:
        raise SmlaError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise SmlaError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def decode_workspace_bytes(T: int, H: int, K: int, num_splits: int = 0) -> int:
    return int(lib().sparse_mla_decode_workspace_bytes(T, H, K, num_splits))


def decode_nvfp4_workspace_bytes(T: int, H: int, K: int, num_splits: int = 0) -> int:
    return int(lib().sparse_mla_decode_nvfp4_workspace_bytes(T, H, K, num_splits))


def prefill_workspace_bytes(T: int, H: int, K: int, num_splits: int = 0) -> int:
    return int(lib().sparse_mla_prefill_workspace_bytes(T, H, K, num_splits))


def attention_plan(fp8: bool, T: int, H: int, K: int, num_splits: int = 0) -> tuple:
    """(kernel launches, attention-kernel CTAs) of one decode (fp8=True) or
    prefill call with these sizes on the current device."""
    launches, ctas = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().sparse_mla_attention_plan(int(bool(fp8)), T, H, K, num_splits, ctypes.byref(launches),
                                           ctypes.byref(ctas)), "sparse_mla_attention_plan")
    return int(launches.value), int(ctas.value)


def sparse_mla_decode_fp8(q, kv_cache, indices, block_table, req_id_per_token, sm_scale: float,
                          num_splits: int = 0, out=None, lse=None, workspace=None, stream=None):
    """FP8 sparse decode.  q bf16 [T,H,576]; kv_cache uint8 [NB,64,656];
    indices int32 [T,K] (logical, <0 = none); block_table int32 [R,MB];
    req_id_per_token int32 [T].  Returns (out bf16 [T,H,512], lse fp32 [T,H]).
    With H < 128, q, indices, block_table and req_id_per_token must not be
    written by a kernel of this library directly before the call, but by
    paged_blocks_extend, or by linear_mxfp8 in bf16 rows of a multiple of 576
    values (so q may be)."""
    return _decode("sparse_mla_decode_fp8", q, kv_cache, indices, block_table, req_id_per_token, sm_scale,
                   num_splits, out, lse, workspace, stream)


def sparse_mla_decode_fp8_qfp8(q, kv_cache, indices, block_table, req_id_per_token, sm_scale: float,
                               num_splits: int = 0, out=None, lse=None, workspace=None, stream=None):
    """sparse_mla_decode_fp8 with the query quantized to FP8 (two e4m3 terms)
    and both products on the FP8 tensor path; at H = 128 a kernel of its own
    (slower than sparse_mla_decode_fp8's on GB300).  Same arguments and results."""
    return _decode("sparse_mla_decode_fp8_qfp8", q, kv_cache, indices, block_table, req_id_per_token, sm_scale,
                   num_splits, out, lse, workspace, stream)


def sparse_mla_decode_nvfp4(q, kv_cache, indices, block_table, req_id_per_token, sm_scale: float,
                            num_splits: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Sparse decode over the NVFP4 cache (kv_cache uint8 [NB,64,352]); the
    other arguments and the results as for sparse_mla_decode_fp8."""
    return _decode("sparse_mla_decode_nvfp4", q, kv_cache, indices, block_table, req_id_per_token, sm_scale,
                   num_splits, out, lse, workspace, stream, row_bytes=352)


def _decode(name, q, kv_cache, indices, block_table, req_id_per_token, sm_scale, num_splits, out, lse, workspace,
            stream, row_bytes=656):
    import torch
    dev = _dev(q, kv_cache, indices, block_table, req_id_per_token, out, lse, workspace)
    T, H, D = q.shape
    NB = kv_cache.shape[0]
    K = indices.shape[1]
    R, MB = block_table.shape
    _expect(q, torch.bfloat16, (T, H, 576), "q")
    _expect(kv_cache, torch.uint8, (NB, 64, row_bytes), "kv_cache")
    _expect(indices, torch.int32, (T, K), "indices")
    _expect(req_id_per_token, torch.int32, (T,), "req_id_per_token")
    if block_table.dtype != torch.int32:
        raise SmlaError("block_table must be int32")
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    _expect(out, torch.bfloat16, (T, H, 512), "out")
    _expect(lse, torch.float32, (T, H), "lse")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = getattr(lib(), name)(_ptr(q), _ptr(kv_cache), _ptr(indices), _ptr(block_table), _ptr(req_id_per_token),
                              float(sm_scale), int(num_splits), _ptr(out), _ptr(lse), T, H, K, R, MB, NB,
                              _ptr(workspace), ws_bytes, _stream_ptr(stream, dev))
    _check(rc, name)
    return out, lse


def sparse_mla_decode_fp8_noalloc(q, kv_cache, indices, block_table, req_id_per_token, sm_scale: float,
                                  num_splits: int = 0, out=None, lse=None, stream=None):
    """sparse_mla_decode_fp8 for callers that cannot allocate device memory
    at call time (code under CUDA graph capture, allocation-free serving
    loops): the library's fixed 32 MiB per-device scratch replaces the
    workspace.  Pass preallocated `out` and `lse` to keep the call free of
    allocations on the Python side too.  The first call on a device should
    come before any stream capture; calls that overlap on the GPU race on the
    shared scratch.  Raises SmlaError if the work split needs more scratch."""
    import torch
    dev = _dev(q, kv_cache, indices, block_table, req_id_per_token, out, lse)
    T, H, D = q.shape
    NB = kv_cache.shape[0]
    K = indices.shape[1]
    R, MB = block_table.shape
    _expect(q, torch.bfloat16, (T, H, 576), "q")
    _expect(kv_cache, torch.uint8, (NB, 64, 656), "kv_cache")
    _expect(indices, torch.int32, (T, K), "indices")
    _expect(req_id_per_token, torch.int32, (T,), "req_id_per_token")
    if block_table.dtype != torch.int32:
        raise SmlaError("block_table must be int32")
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    _expect(out, torch.bfloat16, (T, H, 512), "out")
    _expect(lse, torch.float32, (T, H), "lse")
    rc = lib().sparse_mla_decode_fp8_noalloc(_ptr(q), _ptr(kv_cache), _ptr(indices), _ptr(block_table),
                                             _ptr(req_id_per_token), float(sm_scale), int(num_splits), _ptr(out),
                                             _ptr(lse), T, H, K, R, MB, NB, _stream_ptr(stream, dev))
    _check(rc, "sparse_mla_decode_fp8_noalloc")
    return out, lse


def sparse_mla_prefill_bf16(q, kv, indices, sm_scale: float, num_splits: int = 0, out=None, lse=None,
                            workspace=None, stream=None):
    """BF16 sparse prefill.  q bf16 [T,H,576]; kv bf16 [N,576]; indices int32
    [T,K] rows of kv (<0 or >=N = none).  Returns (out, lse)."""
    import torch
    dev = _dev(q, kv, indices, out, lse, workspace)
    T, H, D = q.shape
    N = kv.shape[0]
    K = indices.shape[1]
    _expect(q, torch.bfloat16, (T, H, 576), "q")
    _expect(kv, torch.bfloat16, (N, 576), "kv")
    _expect(indices, torch.int32, (T, K), "indices")
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    _expect(out, torch.bfloat16, (T, H, 512), "out")
    _expect(lse, torch.float32, (T, H), "lse")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sparse_mla_prefill_bf16(_ptr(q), _ptr(kv), _ptr(indices), float(sm_scale), int(num_splits),
                                       _ptr(out), _ptr(lse), T, H, N, K, _ptr(workspace), ws_bytes,
                                       _stream_ptr(stream, dev))
    _check(rc, "sparse_mla_prefill_bf16")
    return out, lse


def prefill_fp8_workspace_bytes(T: int, H: int, K: int, num_splits: int = 0) -> int:
    return int(lib().sparse_mla_prefill_fp8_workspace_bytes(T, H, K, num_splits))


def sparse_mla_prefill_fp8(q, kv_cache, indices, block_table, req_id_per_token, seq_lens, workspace_starts,
                           kv_workspace, sm_scale: float, num_splits: int = 0, out=None, lse=None, workspace=None,
                           stream=None):
    """Separate-mode FP8 prefill of one chunk of prefill requests: the
    requests' cache rows up-converted into kv_workspace (bf16 [N, 576]), the
    logical indices mapped to its rows, then the bf16 prefill.  q bf16
    [T,H,576]; kv_cache uint8 [NB,64,656]; indices int32 [T,K]; block_table
    int32 [R,MB]; req_id_per_token int32 [T]; seq_lens, workspace_starts int32
    [R].  Returns (out bf16 [T,H,512], lse fp32 [T,H])."""
    import torch
    dev = _dev(q, kv_cache, indices, block_table, req_id_per_token, seq_lens, workspace_starts, kv_workspace, out,
               lse, workspace)
    T, H, _ = q.shape
    NB = kv_cache.shape[0]
    K = indices.shape[1]
    R, MB = block_table.shape
    N = kv_workspace.shape[0]
    _expect(q, torch.bfloat16, (T, H, 576), "q")
    _expect(kv_cache, torch.uint8, (NB, 64, 656), "kv_cache")
    _expect(indices, torch.int32, (T, K), "indices")
    _expect(req_id_per_token, torch.int32, (T,), "req_id_per_token")
    _expect(seq_lens, torch.int32, (R,), "seq_lens")
    _expect(workspace_starts, torch.int32, (R,), "workspace_starts")
    _expect(kv_workspace, torch.bfloat16, (N, 576), "kv_workspace")
    if block_table.dtype != torch.int32:
        raise SmlaError("block_table must be int32")
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    _expect(out, torch.bfloat16, (T, H, 512), "out")
    _expect(lse, torch.float32, (T, H), "lse")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sparse_mla_prefill_fp8(_ptr(q), _ptr(kv_cache), _ptr(indices), _ptr(block_table),
                                      _ptr(req_id_per_token), _ptr(seq_lens), _ptr(workspace_starts),
                                      float(sm_scale), int(num_splits), _ptr(out), _ptr(lse), T, H, K, R, MB, NB,
                                      _ptr(kv_workspace), N, _ptr(workspace), ws_bytes, _stream_ptr(stream, dev))
    _check(rc, "sparse_mla_prefill_fp8")
    return out, lse


def sparse_mla_gather_upconvert_fp8(kv_cache, block_table, seq_lens, workspace_starts, kv_workspace, stream=None):
    """Up-convert positions 0 .. seq_lens[r] - 1 of each request into
    kv_workspace (bf16 [N, 576]) rows workspace_starts[r] + p."""
    import torch
    dev = _dev(kv_cache, block_table, seq_lens, workspace_starts, kv_workspace)
    R, MB = block_table.shape
    _expect(kv_workspace, torch.bfloat16, (kv_workspace.shape[0], 576), "kv_workspace")
    rc = lib().sparse_mla_gather_upconvert_fp8(_ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
                                               _ptr(workspace_starts), R, MB, kv_cache.shape[0], _ptr(kv_workspace),
                                               kv_workspace.shape[0], _stream_ptr(stream, dev))
    _check(rc, "sparse_mla_gather_upconvert_fp8")
    return kv_workspace


def sparse_mla_translate_indices_workspace(indices, block_table, req_id_per_token, prefill_request_id,
                                           workspace_starts, num_blocks: int, out=None, stream=None):
    """Logical top-k indices -> cache slots (decode tokens) or prefill
    workspace rows (prefill tokens), int32 [T, K], -1 = none."""
    import torch
    dev = _dev(indices, block_table, req_id_per_token, prefill_request_id, workspace_starts, out)
    T, K = indices.shape
    R, MB = block_table.shape
    if out is None:
        out = torch.empty((T, K), dtype=torch.int32, device=dev)
    rc = lib().sparse_mla_translate_indices_workspace(_ptr(indices), _ptr(block_table), _ptr(req_id_per_token),
                                                      _ptr(prefill_request_id), _ptr(workspace_starts),
                                                      workspace_starts.numel(), _ptr(out), T, K, R, MB,
                                                      int(num_blocks), _stream_ptr(stream, dev))
    _check(rc, "sparse_mla_translate_indices_workspace")
    return out


def sparse_mla_prefill_chunks(seq_lens, workspace_rows: int):
    """Host-side chunking of prefill requests (a sequence of ints) into
    workspaces of ``workspace_rows`` rows: returns (list of (start, end)
    request ranges, list of chunk-local workspace starts)."""
    R = len(seq_lens)
    sl = (ctypes.c_int32 * max(R, 1))(*[int(v) for v in seq_lens])
    ends = (ctypes.c_int32 * max(R, 1))()
    starts = (ctypes.c_int32 * max(R, 1))()
    n = ctypes.c_int32(0)
    _check(lib().sparse_mla_prefill_chunks(ctypes.cast(sl, ctypes.c_void_p), R, int(workspace_rows),
                                           ctypes.cast(ends, ctypes.c_void_p), ctypes.cast(starts, ctypes.c_void_p),
                                           ctypes.byref(n)), "sparse_mla_prefill_chunks")
    bounds, b = [], 0
    for i in range(n.value):
        bounds.append((b, int(ends[i])))
        b = int(ends[i])
    return bounds, [int(starts[i]) for i in range(R)]


def mla_absorb_q(q, w_uk_t, out=None, workspace=None, stream=None):
    """Attention-ready query from q bf16 [T,H,P+64] and W_UK_T bf16 [H,P,512]:
    bf16 [T,H,576] = (q_nope x W_UK_T per head) ++ q_pe."""
    import torch
    dev = _dev(q, w_uk_t, out, workspace)
    T, H, D = q.shape
    P = D - 64
    _expect(w_uk_t, torch.bfloat16, (H, P, 512), "w_uk_t")
    if q.dtype != torch.bfloat16:
        raise SmlaError("q must be bf16")
    if out is None:
        out = torch.empty((T, H, 576), dtype=torch.bfloat16, device=dev)
    _expect(out, torch.bfloat16, (T, H, 576), "out")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().mla_absorb_q(_ptr(q), _ptr(w_uk_t), _ptr(out), T, H, P, _ptr(workspace), ws_bytes,
                              _stream_ptr(stream, dev)), "mla_absorb_q")
    return out


def mla_v_up_proj(attn_out, w_uv, out=None, workspace=None, stream=None):
    """Per-head value up-projection: attn_out bf16 [T,H,512] x W_UV bf16
    [H,512,V] -> bf16 [T,H,V]."""
    import torch
    dev = _dev(attn_out, w_uv, out, workspace)
    T, H, _ = attn_out.shape
    V = w_uv.shape[2]
    _expect(attn_out, torch.bfloat16, (T, H, 512), "attn_out")
    _expect(w_uv, torch.bfloat16, (H, 512, V), "w_uv")
    if out is None:
        out = torch.empty((T, H, V), dtype=torch.bfloat16, device=dev)
    _expect(out, torch.bfloat16, (T, H, V), "out")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().mla_v_up_proj(_ptr(attn_out), _ptr(w_uv), _ptr(out), T, H, V, _ptr(workspace), ws_bytes,
                               _stream_ptr(stream, dev)), "mla_v_up_proj")
    return out


def mla_cache_store_fp8(kv_new, slot_mapping, kv_cache, stream=None):
    """Quantize bf16 [T,576] rows into kv_cache uint8 [NB,64,656] at
    slot_mapping int64 [T] (<0 skips).  Modifies kv_cache in place.  kv_new and
    slot_mapping must not be written by a kernel of this library directly before
    the call, but by paged_blocks_extend, or by linear_mxfp8 in bf16 rows of a
    multiple of 576 values (so kv_new may be)."""
    import torch
    dev = _dev(kv_new, slot_mapping, kv_cache)
    T = kv_new.shape[0]
    NB = kv_cache.shape[0]
    _expect(kv_new, torch.bfloat16, (T, 576), "kv_new")
    _expect(slot_mapping, torch.int64, (T,), "slot_mapping")
    _expect(kv_cache, torch.uint8, (NB, 64, 656), "kv_cache")
    rc = lib().mla_cache_store_fp8(_ptr(kv_new), _ptr(slot_mapping), _ptr(kv_cache), T, NB, _stream_ptr(stream, dev))
    _check(rc, "mla_cache_store_fp8")
    return kv_cache


def mla_cache_store_nvfp4(kv_new, slot_mapping, kv_cache, stream=None):
    """Quantize bf16 [T,576] rows into the NVFP4 kv_cache uint8 [NB,64,352] at
    slot_mapping int64 [T] (<0 skips).  Modifies kv_cache in place."""
    import torch
    dev = _dev(kv_new, slot_mapping, kv_cache)
    T = kv_new.shape[0]
    NB = kv_cache.shape[0]
    _expect(kv_new, torch.bfloat16, (T, 576), "kv_new")
    _expect(slot_mapping, torch.int64, (T,), "slot_mapping")
    _expect(kv_cache, torch.uint8, (NB, 64, 352), "kv_cache")
    rc = lib().mla_cache_store_nvfp4(_ptr(kv_new), _ptr(slot_mapping), _ptr(kv_cache), T, NB, _stream_ptr(stream, dev))
    _check(rc, "mla_cache_store_nvfp4")
    return kv_cache


def sparse_mla_translate_indices(indices, block_table, req_id_per_token, num_blocks: int, out=None, stream=None):
    """Logical top-k indices -> physical cache slots (int32 [T,K], -1 = none)."""
    import torch
    dev = _dev(indices, block_table, req_id_per_token, out)
    T, K = indices.shape
    R, MB = block_table.shape
    if out is None:
        out = torch.empty((T, K), dtype=torch.int32, device=dev)
    rc = lib().sparse_mla_translate_indices(_ptr(indices), _ptr(block_table), _ptr(req_id_per_token), _ptr(out),
                                            T, K, R, MB, int(num_blocks), _stream_ptr(stream, dev))
    _check(rc, "sparse_mla_translate_indices")
    return out


# ---- paged 8-bit K/V cache

class PagedBatch(NamedTuple):
    """What paged_blocks_extend makes of a batch's lengths."""
    query_start: Any       # int32 [R + 1]
    seq_lens: Any          # int32 [R]
    req_id_per_token: Any  # int32 [T]
    positions: Any         # int32 [T]
    slot_mapping: Any      # int64 [T]
    free_count: Any        # int32 [1]
    missing: Any           # int32 [1]


def _bound():
    """The compiled binding of the paged and the MXFP8 operators, on the loaded library."""
    global _binding
    if _binding is None:
        import importlib.util

        import torch  # noqa: F401  (its libraries first)
        L = lib()
        with _lock:
            if _binding is None:
                if not os.path.exists(BINDING_PATH):
                    raise SmlaError(f"{BINDING_PATH} is missing: run sparse_mla_attention_fp8_gb300.build() first")
                spec = importlib.util.spec_from_file_location(__name__ + "._binding", BINDING_PATH)
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
                module.init(SmlaError, *(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in (
                    "paged_blocks_extend", "paged_blocks_release", "kv_cache_store_fp8", "paged_attention_fp8",
                    "paged_attention_fp8_workspace_bytes", "smla_last_error", "mxfp8_quantize", "rms_norm_mxfp8",
                    "linear_mxfp8", "moe_route", "moe_mxfp8", "moe_mxfp8_workspace_bytes")))
                _binding = module
    return _binding


def _on(stream, tensor, call, *args):
    """call(*args) on a stream that the caller names: it is made current, so
    that what the call allocates belongs to it."""
    import torch
    if tensor.is_cuda and stream.device != tensor.device:
        raise SmlaError("the stream must be on the tensors' device")
    with torch.cuda.stream(stream):
        return call(*args)


def paged_blocks_extend(context_lens, query_lens, block_table, free_blocks, free_count, num_tokens: int,
                        num_blocks: int, out=None, stream=None):
    """Block tables, slot maps and positions of a batch from its requests'
    lengths (int32 [R] each): the blocks that the new tokens need are taken
    from the stack free_blocks[:free_count] (int32 [F], [1]) into block_table
    (int32 [R, MB], modified in place).  num_tokens: rows of the batch, at
    least the new tokens' number; num_blocks: blocks of the cache.  Returns a
    PagedBatch (`out`, if given; its seq_lens may be context_lens and its
    free_count the argument, which are then updated)."""
    args = (context_lens, query_lens, block_table, free_blocks, free_count, num_tokens, num_blocks, out)
    call = (_binding or _bound()).extend
    made = call(*args) if stream is None else _on(stream, block_table, call, *args)
    return made if type(made) is PagedBatch else PagedBatch._make(made)


def paged_blocks_release(release, seq_lens, block_table, free_blocks, free_count, num_blocks: int, context_lens=None,
                         free_count_out=None, stream=None):
    """The blocks of the requests with release set (bool or uint8 [R]) back on
    the stack (free_blocks modified in place).  Returns (context_lens int32
    [R]: 0 for them, seq_lens for the others; free_count int32 [1]); both may
    be written over the arguments of those meanings."""
    args = (release, seq_lens, block_table, free_blocks, free_count, num_blocks, context_lens, free_count_out)
    call = (_binding or _bound()).release
    return call(*args) if stream is None else _on(stream, block_table, call, *args)


def kv_cache_store_fp8(k, v, query_start, seq_lens, block_table, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Quantize a batch's new K and V rows (bf16 [T,HK,D], slices of longer
    rows allowed) into the paged e4m3 caches (uint8 [NB,HK,64,D], scales fp32
    [NB,HK]), modified in place.  query_start int32 [R+1], seq_lens int32 [R],
    block_table int32 [R,MB]."""
    args = (k, v, query_start, seq_lens, block_table, k_cache, v_cache, k_scale, v_scale)
    call = (_binding or _bound()).store
    call(*args) if stream is None else _on(stream, block_table, call, *args)
    return k_cache, v_cache, k_scale, v_scale


def paged_attention_fp8_workspace_bytes(T: int, H: int, HK: int, D: int, R: int, max_query_len: int) -> int:
    return int(lib().paged_attention_fp8_workspace_bytes(T, H, HK, D, R, max_query_len))


def paged_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, query_start, sm_scale: float,
                        max_query_len=None, window: int = 0, softcap: float = 0.0, alibi_slopes=None,
                        prefix_lens=None, doc_start=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of a ragged batch over the paged e4m3 caches.  q bf16 [T,H,D]
    (slices of longer rows allowed); the cache as for kv_cache_store_fp8;
    causal, with a sliding window, capped scores (softcap 0 or from 1e-20 to
    1e30), distance biases (fp32 [H]), a prefix that all tokens of a request
    see, in whichever document (int32 [R]), and documents (int32 [T]: first
    position of the token's document) as asked.  max_query_len: an estimate of
    the most new tokens of a request (default: T - R + 1, which takes the
    padding rows of a batch for tokens of one: give it there).  The
    workspace, if none is given, is allocated for the call; read_device_status()
    tells whether a call has failed, with either.  Returns (out bf16 [T,H,D],
    lse fp32 [T,H]); rows of no request are left as they were."""
    args = (q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, query_start, sm_scale, max_query_len, window,
            softcap, alibi_slopes, prefix_lens, doc_start, out, lse, workspace)
    call = (_binding or _bound()).attention
    return call(*args) if stream is None else _on(stream, block_table, call, *args)


# ---- MXFP8 operators

class MxNorm(NamedTuple):
    """What rms_norm_mxfp8 makes; None for what was not asked for."""
    codes: Any     # uint8 [T, K]
    scales: Any    # uint8 [T, K / 32]
    normed: Any    # bf16 [T, K]
    residual: Any  # bf16 [T, K]


_ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5}
_SCORINGS = {"softmax": 0, "sigmoid": 1}


def _choice(table: dict, name: str, what: str) -> int:
    if name not in table:
        raise SmlaError(f"{what}: {name!r} is none of {', '.join(table)}")
    return table[name]


def mxfp8_quantize(x, codes=None, scales=None, stream=None):
    """MXFP8 of x (bf16 or float32 [T,K], slices of longer rows allowed; K a
    multiple of 32): (codes uint8 [T,K] of float8_e4m3, scales uint8 [T,K/32],
    the byte E + 127 for the scale 2^E of 32 values, in rows a multiple of 4
    bytes apart).  The form in which the other MXFP8 operators take activations
    and weights, as uint8 or viewed as float8_e4m3fn and float8_e8m0fnu."""
    args = (x, codes, scales)
    call = (_binding or _bound()).quantize
    return call(*args) if stream is None else _on(stream, x, call, *args)


def rms_norm_mxfp8(x, weight=None, eps: float = 1e-6, residual=None, normed=False, quantized: bool = True,
                   residual_out=None, codes=None, scales=None, stream=None):
    """RMS norm of h = x + residual (bf16 [T,K], slices of longer rows allowed)
    with a weight (bf16 or float32 [K]), quantized from its float32 values.
    Returns an MxNorm: codes and scales as mxfp8_quantize's (if `quantized`);
    the norm in bf16, if `normed` is True or a tensor for it; and h rounded to
    bf16, if a residual is given (in `residual_out`, which may be the residual
    itself, or a new tensor)."""
    args = (x, weight, eps, residual, normed, quantized, residual_out, codes, scales)
    call = (_binding or _bound()).norm
    return MxNorm._make(call(*args) if stream is None else _on(stream, x, call, *args))


def linear_mxfp8(x, x_scale, weight, weight_scale, bias=None, activation: str = "none", residual=None,
                 quantized: bool = False, out=None, out_scale=None, stream=None):
    """y = act(x W^T + bias) + residual on MXFP8 operands: x [T,K] (slices of
    longer rows allowed), weight [N,K], bias bf16 or float32 [N], residual bf16
    [T,N].  activation: "none", "relu", "silu", "gelu", "gelu_tanh", or "swiglu":
    silu(first half) * second half of a product with 2 N rows.  Returns y in bf16
    [T,N], or, if `quantized` (N a multiple of 32, no residual), its codes and
    scales as mxfp8_quantize's.  out may be the residual.  Rows of a multiple of
    576 values in bf16 (q, kv_new) may go directly to the latent cache's decode
    and store; what the other MXFP8 operators write may not be these calls' q,
    kv_new, indices, tables or slots without another kernel between."""
    args = (x, x_scale, weight, weight_scale, bias, _choice(_ACTIVATIONS, activation, "activation"), residual, quantized,
            out, out_scale)
    call = (_binding or _bound()).linear
    return call(*args) if stream is None else _on(stream, x, call, *args)


def moe_route(logits, topk: int, scoring: str = "softmax", bias=None, renormalize: bool = True, scale: float = 1.0,
              num_groups: int = 1, topk_groups: int = 1, ids=None, weights=None, stream=None):
    """The topk experts of each token from its router logits (bf16 or float32
    [T,E]): the largest scores ("softmax" over the logits, or "sigmoid" of each)
    plus bias (fp32 [E]), with num_groups > 1 among the topk_groups groups of
    experts whose two largest have the largest sums; ties go to the lowest index.
    Returns (ids int32 [T,topk], weights fp32 [T,topk]: the scores, divided by
    their sum if `renormalize`, times scale).  Logits of -infinity mask an
    expert; where too few are left, id -1 with weight 0."""
    args = (logits, topk, _choice(_SCORINGS, scoring, "scoring"), bias, renormalize, scale, num_groups, topk_groups, ids,
            weights)
    call = (_binding or _bound()).route
    return call(*args) if stream is None else _on(stream, logits, call, *args)


def moe_mxfp8_workspace_bytes(T: int, E: int, topk: int, F: int) -> int:
    return int(lib().moe_mxfp8_workspace_bytes(T, E, topk, F))


def moe_mxfp8(x, x_scale, topk_ids, topk_weights, w13, w13_scale, w2, w2_scale, residual=None, out=None,
              workspace=None, stream=None):
    """Mixture-of-experts layer of a batch of few tokens: each token's experts
    (int32 [T,topk], ids outside [0,E) skipped) with their weights (fp32
    [T,topk]); w13 [E,2F,K]: an expert's gate and up projections, w2 [E,K,F], all
    MXFP8.  The weighted silu(gate) * up is rounded to MXFP8 between the
    products.  Returns bf16 [T,K], with the residual (bf16 [T,K]) added if given;
    out may be the residual."""
    args = (x, x_scale, topk_ids, topk_weights, w13, w13_scale, w2, w2_scale, residual, out, workspace)
    call = (_binding or _bound()).moe
    return call(*args) if stream is None else _on(stream, x, call, *args)


def read_noalloc_status(stream=None) -> int:
    """Synchronize and read/clear the status word of the allocation-free
    decode's fixed scratch on the current device (0 = ok)."""
    import torch
    st = ctypes.c_int(0)
    dev = torch.device("cuda", torch.cuda.current_device())
    _check(lib().smla_read_noalloc_status(ctypes.byref(st), _stream_ptr(stream, dev)), "smla_read_noalloc_status")
    return int(st.value)


def paged_wait_check(workspace, many_rows: bool = False, stream=None) -> None:
    """Let one device thread wait in vain until the kernels' time limit (2 s)
    and report it as paged_attention_fp8 does (in its kernel for few or for
    many rows): for tests of a caller's failure handling."""
    import torch
    dev = _dev(workspace)
    if workspace.nbytes < 256:
        raise SmlaError(f"workspace has {workspace.nbytes} bytes, 256 needed")
    with torch.cuda.device(dev):
        _check(lib().smla_paged_wait_check(int(many_rows), _ptr(workspace), _stream_ptr(stream, dev)),
               "smla_paged_wait_check")


def mxfp8_wait_check(experts: bool = False, stream=None) -> None:
    """The same on the current device, as linear_mxfp8 or moe_mxfp8 reports it
    (to read_device_status())."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device())
    _check(lib().smla_mxfp8_wait_check(int(experts), _stream_ptr(stream, dev)), "smla_mxfp8_wait_check")


def mxfp8_give_up(on: bool) -> None:
    """While on, this thread's linear_mxfp8 and moe_mxfp8 calls unwind as if
    their kernels' waits ran out at once, and report it: for tests of a caller's
    failure handling."""
    lib().smla_mxfp8_give_up(int(on))


def read_device_status(workspace=None, stream=None) -> int:
    """Synchronize and read/clear the kernels' device status word (0 = ok).
    Without a workspace: that of the library's own workspace on the current
    device, and whether a paged_attention_fp8, linear_mxfp8 or moe_mxfp8 call on
    it has failed, whichever workspace it had."""
    import torch
    st = ctypes.c_int(0)
    dev = workspace.device if workspace is not None else torch.device("cuda", torch.cuda.current_device())
    rc = lib().smla_read_device_status(_ptr(workspace), ctypes.byref(st), _stream_ptr(stream, dev))
    _check(rc, "smla_read_device_status")
    return int(st.value)
