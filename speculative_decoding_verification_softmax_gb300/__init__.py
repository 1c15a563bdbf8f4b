"""GB300-native speculative-decoding verification.

Thin ctypes binding over ``libspecv.so`` (C ABI declared in ``include/specv.h``).
Every step of verification and scheduling runs in the library's CUDA kernels;
this module only checks tensor properties, allocates outputs/workspaces with
PyTorch and passes pointers and the current CUDA stream.  There is no CPU
fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import threading
from concurrent.futures import ThreadPoolExecutor

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
_CSRC = os.path.join(_HERE, "csrc")
LIB_PATH = os.path.join(_HERE, "libspecv.so")
SOURCES = ["specv_verify.cu", "specv_sched.cu", "specv_api.cu", "specv_static.cu", "specv_pages.cu",
           "specv_append.cu", "specv_append_rows.cu", "specv_attend.cu", "specv_attend_simt.cu", "specv_attend_mma16.cu",
           "specv_attend_mma8.cu", "specv_attend_tc.cu", "specv_share.cu", "specv_share_f32.cu", "specv_share_mma.cu", "specv_share_tc.cu"]
HEADERS = ["specv_common.cuh", "specv_rowstats.cuh", "specv_cache.cuh", "specv_append.cuh", "specv_attend.cuh", "specv_attend_mma.cuh", "specv_attend_tc.cuh",
           "specv_attend_tc_launch.cuh", "specv_trace.h"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]

# status codes (include/specv.h)
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_TEMPERATURE = 0, -1, -2, -3, -4
ERR_VERIFY_LEN, ERR_TOKEN, ERR_WORKSPACE, ERR_COST_TABLE = -5, -6, -7, -8
ERR_NONFINITE, ERR_TIMEOUT, ERR_CUDA, ERR_UNIFORM, ERR_CONFIDENCE = -9, -10, -11, -12, -13
ERR_ROW_INDEX, ERR_POOL, ERR_CACHE_LEN, ERR_PAGE, ERR_REQUEST = -14, -15, -16, -17, -18
ERR_PLAN = -19
F32, BF16, F16, E4M3 = 0, 1, 2, 3
SCHED_EXACT, SCHED_ALGORITHM1, SCHED_DCUT = 0, 1, 2
MAX_BATCH, MAX_GAMMA, MAX_SCHED_CANDIDATES = 4096, 32, 16384

EXPORTED = ["spec_verify_workspace_bytes", "spec_verify", "spec_verify_stats",
            "spec_schedule_workspace_bytes", "spec_schedule", "spec_read_status",
            "spec_status_string", "spec_profile_events", "spec_verify_kernel_count",
            "spec_verify_static", "spec_schedule_static", "spec_sts_fit", "spec_verify_packed",
            "spec_pack_rows", "spec_selftest_wait", "spec_selftest_expire_first_wait",
            "spec_cache_workspace_bytes", "spec_attend_workspace_bytes", "spec_attend", "spec_append_kv",
            "spec_reserve_pages", "spec_commit_pages", "spec_free_pages", "spec_fork_pages",
            "spec_compact_pages", "spec_share_plan_bytes", "spec_share_plan",
            "spec_attend_shared_workspace_bytes", "spec_attend_shared", "spec_append_rows", "spec_map_rows"]
STATIC_WORKSPACE_BYTES = 8 << 20


class SpecError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (code {code})" if where else status_string(code))


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu for sm_103a into libspecv.so (in-tree, parallel TUs)."""
    srcs = [os.path.join(_CSRC, s) for s in SOURCES]
    deps = srcs + [os.path.join(_CSRC, h) for h in HEADERS] + [os.path.join(_ROOT, "include", "specv.h")]
    if (not force and os.path.exists(LIB_PATH)
            and all(os.path.getmtime(LIB_PATH) >= os.path.getmtime(d) for d in deps)):
        return LIB_PATH
    bdir = os.path.join(_HERE, "_build")
    os.makedirs(bdir, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


_lib = None
_lock = threading.Lock()


def lib():
    """The loaded libspecv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() "
                                       "(or speculative_decoding_verification_softmax_gb300.build())")
                L = ctypes.CDLL(LIB_PATH)
                vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
                L.spec_verify_workspace_bytes.argtypes = [i32, i32, i32, i32]
                L.spec_verify_workspace_bytes.restype = sz
                L.spec_verify.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, f32, vp, vp, vp, vp, sz, vp]
                L.spec_verify.restype = i32
                L.spec_verify_stats.argtypes = [vp, sz, i32, i32, i32, i32, vp, vp, vp, vp, vp]
                L.spec_verify_stats.restype = i32
                L.spec_schedule_workspace_bytes.argtypes = [i32, i32]
                L.spec_schedule_workspace_bytes.restype = sz
                L.spec_schedule.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, vp, sz, vp]
                L.spec_schedule_static.argtypes = [vp, i32, i32, f32, i32, i32, vp, vp, vp, sz, vp]
                L.spec_schedule_static.restype = i32
                L.spec_sts_fit.argtypes = [vp, vp, i32, i32, vp, vp]
                L.spec_sts_fit.restype = i32
                L.spec_schedule.restype = i32
                L.spec_read_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
                L.spec_read_status.restype = i32
                L.spec_status_string.argtypes = [i32]
                L.spec_status_string.restype = ctypes.c_char_p
                L.spec_profile_events.argtypes = [vp, vp]
                L.spec_profile_events.restype = i32
                L.spec_verify_kernel_count.argtypes = [i32, f32]
                L.spec_verify_kernel_count.restype = i32
                L.spec_verify_static.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, f32, vp, vp, vp, vp]
                L.spec_verify_static.restype = i32
                L.spec_verify_packed.argtypes = [vp, i32, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, f32, vp,
                                                 vp, vp, vp, sz, vp]
                L.spec_verify_packed.restype = i32
                L.spec_pack_rows.argtypes = [vp, i32, i32, vp, vp, vp, vp]
                L.spec_pack_rows.restype = i32
                L.spec_selftest_wait.argtypes = [ctypes.c_longlong, vp, vp, vp]
                L.spec_selftest_wait.restype = i32
                L.spec_selftest_expire_first_wait.argtypes = [i32]
                L.spec_selftest_expire_first_wait.restype = i32
                ll, cp = ctypes.c_longlong, ctypes.POINTER(Cache)
                L.spec_cache_workspace_bytes.argtypes = [i32, i32]
                L.spec_cache_workspace_bytes.restype = sz
                L.spec_attend_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
                L.spec_attend_workspace_bytes.restype = sz
                L.spec_attend.argtypes = [vp, ll, ll, i32, i32, cp, vp, i32, vp, vp, vp, i32, i32, i32, f32, i32,
                                          i32, vp, vp, vp, sz, vp]
                L.spec_append_kv.argtypes = [vp, ll, ll, vp, vp, ll, ll, ll, ll, i32, i32, cp, vp, i32, vp, vp, vp,
                                             i32, i32, i32, vp, i32, i32, f32, vp, vp, sz, vp]
                L.spec_reserve_pages.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, sz, vp]
                L.spec_commit_pages.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, sz, vp]
                L.spec_free_pages.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, vp, sz, vp]
                L.spec_fork_pages.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, cp, vp, vp, sz, vp]
                L.spec_compact_pages.argtypes = [vp, vp, vp, i32, i32, cp, vp, vp, vp, vp, sz, vp]
                L.spec_share_plan_bytes.argtypes = [i32, i32, i32]
                L.spec_share_plan_bytes.restype = sz
                L.spec_share_plan.argtypes = [vp, i32, i32, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]
                L.spec_attend_shared_workspace_bytes.argtypes = [i32] * 6
                L.spec_attend_shared_workspace_bytes.restype = sz
                L.spec_attend_shared.argtypes = [vp, ll, ll, i32, i32, cp, vp, i32, vp, sz, i32, i32, i32, f32, vp, vp,
                                                 vp, sz, vp]
                L.spec_append_rows.argtypes = [vp, ll, ll, vp, vp, ll, ll, ll, ll, i32, i32, cp, vp, vp, i32, vp, i32, i32,
                                               f32, vp, vp, sz, vp]
                L.spec_map_rows.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
                for f in (L.spec_append_rows, L.spec_map_rows, L.spec_share_plan, L.spec_attend_shared, L.spec_attend, L.spec_append_kv, L.spec_reserve_pages, L.spec_commit_pages,
                          L.spec_free_pages, L.spec_fork_pages, L.spec_compact_pages):
                    f.restype = i32
                _lib = L
    return _lib


class Cache(ctypes.Structure):
    """spec_cache: where the pages of a key-value cache are."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dt", ctypes.c_int), ("layers", ctypes.c_int),
                ("pages", ctypes.c_int), ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("layer_stride", ctypes.c_longlong), ("page_stride", ctypes.c_longlong),
                ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class CostTable(ctypes.Structure):
    """spec_cost_table: piecewise-linear round cost, knots (tokens[i], cost_ms[i])."""
    _fields_ = [("n", ctypes.c_int), ("tokens", ctypes.c_double * 32), ("cost_ms", ctypes.c_double * 32)]

    @classmethod
    def from_knots(cls, tokens, cost_ms) -> "CostTable":
        t = cls()
        t.n = len(tokens)
        if len(cost_ms) != t.n or not 1 <= t.n <= 32:
            t.n = 0 if t.n == 0 else 33  # rejected by the library
            return t
        for i, (a, b) in enumerate(zip(tokens, cost_ms)):
            t.tokens[i] = float(a)
            t.cost_ms[i] = float(b)
        return t


def status_string(code: int) -> str:
    try:
        return lib().spec_status_string(int(code)).decode()
    except RuntimeError:
        return f"status {code}"


def _check(rc: int, where: str):
    if rc != OK:
        raise SpecError(rc, where)


# ------------------------------------------------------------ torch helpers
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _check_tensor(name, t, dtype, shape, required=True):
    """A contiguous tensor of `dtype` and `shape` on the current CUDA device
    (the device whose current stream the call uses), or None if allowed."""
    torch = _torch()
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_verify_inputs(B, gamma, V, ldtype, draft_logits, draft_shape, draft_tokens, verify_len, temperature,
                         uniforms, out_tokens, out_accept_len):
    """Shapes, dtypes and devices of every tensor a verify call reads or writes
    (the library reads them with the sizes it is given, so a mismatch here
    would be an out-of-bounds access on the device)."""
    torch = _torch()
    greedy = float(temperature) == 0.0
    _check_tensor("draft_logits", draft_logits, ldtype, draft_shape, required=not greedy and gamma > 0)
    _check_tensor("draft_tokens", draft_tokens, torch.int32, (B, gamma), required=gamma > 0)
    _check_tensor("verify_len", verify_len, torch.int32, (B,), required=False)
    _check_tensor("uniforms", uniforms, torch.float32, (B, gamma + 2), required=not greedy)
    _check_tensor("out_tokens", out_tokens, torch.int32, (B, gamma + 1), required=False)
    _check_tensor("out_accept_len", out_accept_len, torch.int32, (B,), required=False)


def verify_workspace_bytes(B: int, gamma: int, V: int, dtype_code: int) -> int:
    return int(lib().spec_verify_workspace_bytes(B, gamma, V, dtype_code))


def alloc_verify_workspace(B: int, gamma: int, V: int, dtype_code: int, device=None):
    """A verification workspace (its contents need no initialisation)."""
    torch = _torch()
    n = verify_workspace_bytes(B, gamma, V, dtype_code)
    if n == 0:
        raise SpecError(ERR_SHAPE, "spec_verify_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def verify(target_logits, draft_logits, draft_tokens, verify_len, temperature: float, uniforms,
           *, out_tokens=None, out_accept_len=None, workspace=None, stream=None):
    """Run spec_verify on device tensors (see include/specv.h).

    target_logits [B, gamma+1, V] and draft_logits [B, gamma, V] (bf16 or fp32,
    contiguous), draft_tokens [B, gamma] int32, verify_len [B] int32 or None,
    uniforms [B, gamma+2] fp32 (None at temperature 0).  Returns
    (out_tokens [B, gamma+1] int32, out_accept_len [B] int32, workspace).
    """
    torch = _torch()
    B, G1, V = target_logits.shape
    gamma = G1 - 1
    dt = _dtype_code(target_logits)
    dev = target_logits.device
    _check_tensor("target_logits", target_logits, target_logits.dtype, (B, G1, V))
    _check_verify_inputs(B, gamma, V, target_logits.dtype, draft_logits, (B, gamma, V), draft_tokens, verify_len,
                         temperature, uniforms, out_tokens, out_accept_len)
    if workspace is not None:
        _check_tensor("workspace", workspace, torch.uint8, (workspace.numel(),))
    if out_tokens is None:
        out_tokens = torch.empty((B, G1), dtype=torch.int32, device=dev)
    if out_accept_len is None:
        out_accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_verify_workspace(B, gamma, V, dt, dev)
    rc = lib().spec_verify(_ptr(target_logits), _ptr(draft_logits), dt, B, gamma, V, _ptr(draft_tokens),
                           _ptr(verify_len), ctypes.c_float(temperature), _ptr(uniforms), _ptr(out_tokens),
                           _ptr(out_accept_len), _ptr(workspace), workspace.numel(),
                           _stream_handle(stream))
    _check(rc, "spec_verify")
    return out_tokens, out_accept_len, workspace


def verify_static(target_logits, draft_logits, draft_tokens, verify_len, temperature: float, uniforms,
                  *, out_tokens=None, out_accept_len=None, stream=None):
    """spec_verify_static: verification without a workspace, for callers that
    cannot allocate device memory where they verify.  The scratch is a fixed
    8 MiB array on the device (shared by all calls; order overlapping calls on
    one stream).  Only the outputs, if not given, are allocated here.
    Returns (out_tokens, out_accept_len)."""
    torch = _torch()
    B, G1, V = target_logits.shape
    gamma = G1 - 1
    dt = _dtype_code(target_logits)
    dev = target_logits.device
    _check_tensor("target_logits", target_logits, target_logits.dtype, (B, G1, V))
    _check_verify_inputs(B, gamma, V, target_logits.dtype, draft_logits, (B, gamma, V), draft_tokens, verify_len,
                         temperature, uniforms, out_tokens, out_accept_len)
    if out_tokens is None:
        out_tokens = torch.empty((B, G1), dtype=torch.int32, device=dev)
    if out_accept_len is None:
        out_accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    rc = lib().spec_verify_static(_ptr(target_logits), _ptr(draft_logits), dt, B, gamma, V, _ptr(draft_tokens),
                                  _ptr(verify_len), ctypes.c_float(temperature), _ptr(uniforms),
                                  _ptr(out_tokens), _ptr(out_accept_len), _stream_handle(stream))
    _check(rc, "spec_verify_static")
    return out_tokens, out_accept_len


def verify_packed(target_logits, draft_logits, target_row, draft_row, draft_tokens, verify_len,
                  temperature: float, uniforms, *, out_tokens=None, out_accept_len=None, workspace=None,
                  stream=None):
    """Run spec_verify_packed: target_logits [K_target, V] and draft_logits
    [K_draft, V] (bf16 or fp32, contiguous; draft may be None at temperature 0),
    the row index target_row / draft_row [B] int32, draft_tokens [B, gamma]
    int32, verify_len [B] int32 or None, uniforms [B, gamma+2] fp32.
    Returns (out_tokens [B, gamma+1], out_accept_len [B], workspace)."""
    torch = _torch()
    Kt, V = target_logits.shape
    B, gamma = draft_tokens.shape
    Kd = draft_logits.shape[0] if draft_logits is not None else 0
    dt = _dtype_code(target_logits)
    dev = target_logits.device
    _check_tensor("target_logits", target_logits, target_logits.dtype, (Kt, V))
    _check_verify_inputs(B, gamma, V, target_logits.dtype, draft_logits, (Kd, V), draft_tokens, verify_len,
                         temperature, uniforms, out_tokens, out_accept_len)
    _check_tensor("target_row", target_row, torch.int32, (B,))
    _check_tensor("draft_row", draft_row, torch.int32, (B,), required=float(temperature) != 0.0 and gamma > 0)
    if workspace is not None:
        _check_tensor("workspace", workspace, torch.uint8, (workspace.numel(),))
    if out_tokens is None:
        out_tokens = torch.empty((B, gamma + 1), dtype=torch.int32, device=dev)
    if out_accept_len is None:
        out_accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_verify_workspace(B, gamma, V, dt, dev)
    rc = lib().spec_verify_packed(_ptr(target_logits), Kt, _ptr(draft_logits), Kd, _ptr(target_row),
                                  _ptr(draft_row), dt, B, gamma, V, _ptr(draft_tokens), _ptr(verify_len),
                                  ctypes.c_float(temperature), _ptr(uniforms), _ptr(out_tokens),
                                  _ptr(out_accept_len), _ptr(workspace), workspace.numel(),
                                  _stream_handle(stream))
    _check(rc, "spec_verify_packed")
    return out_tokens, out_accept_len, workspace


def pack_rows(verify_len, gamma: int, *, target_row=None, draft_row=None, totals=None, stream=None):
    """Run spec_pack_rows on verify_len [B] int32 (CUDA): the dense request-major
    row index.  Returns (target_row [B], draft_row [B], totals [2] = (K_target,
    K_draft)), all int32 on the device."""
    torch = _torch()
    B = verify_len.shape[0]
    dev = verify_len.device
    _check_tensor("verify_len", verify_len, torch.int32, (B,))
    for name, t, shp in (("target_row", target_row, (B,)), ("draft_row", draft_row, (B,)), ("totals", totals, (2,))):
        _check_tensor(name, t, torch.int32, shp, required=False)
    if target_row is None:
        target_row = torch.empty((B,), dtype=torch.int32, device=dev)
    if draft_row is None:
        draft_row = torch.empty((B,), dtype=torch.int32, device=dev)
    if totals is None:
        totals = torch.empty((2,), dtype=torch.int32, device=dev)
    rc = lib().spec_pack_rows(_ptr(verify_len), B, gamma, _ptr(target_row), _ptr(draft_row), _ptr(totals),
                              _stream_handle(stream))
    _check(rc, "spec_pack_rows")
    return target_row, draft_row, totals


def verify_stats(workspace, B: int, gamma: int, V: int, dtype_code: int, stream=None):
    """Diagnostics of the last verify on `workspace`: (px, qx, resid_mass, status)."""
    torch = _torch()
    dev = workspace.device
    px = torch.empty((B, gamma), dtype=torch.float64, device=dev)
    qx = torch.empty((B, gamma), dtype=torch.float64, device=dev)
    mass = torch.empty((B,), dtype=torch.float64, device=dev)
    st = torch.empty((B,), dtype=torch.int32, device=dev)
    rc = lib().spec_verify_stats(_ptr(workspace), workspace.numel(), B, gamma, V, dtype_code, _ptr(px),
                                 _ptr(qx), _ptr(mass), _ptr(st), _stream_handle(stream))
    _check(rc, "spec_verify_stats")
    return px, qx, mass, st


def _sts_arg(sts, gamma):
    if sts is None:
        return None, None
    import numpy as np
    arr = np.ascontiguousarray(np.asarray(sts, dtype=np.float32).reshape(-1))
    if arr.size != gamma:
        raise ValueError("sts temperatures need one value per draft position")
    return arr, arr.ctypes.data_as(ctypes.c_void_p)


def schedule(confidence, cost, min_len: int = 0, mode: int = SCHED_EXACT, *, sts=None, out_verify_len=None,
             workspace=None, stream=None):
    """Run spec_schedule: confidence [B, gamma] fp32 CUDA tensor, cost = (tokens, cost_ms)
    knots or a CostTable (for SCHED_DCUT: (ratios, costs)); sts = per-position STS
    temperatures or None.  Returns (out_verify_len [B] int32, workspace)."""
    torch = _torch()
    B, gamma = confidence.shape
    _check_tensor("confidence", confidence, torch.float32, (B, gamma))
    _check_tensor("out_verify_len", out_verify_len, torch.int32, (B,), required=False)
    table = cost if isinstance(cost, CostTable) else CostTable.from_knots(*cost)
    if out_verify_len is None:
        out_verify_len = torch.empty((B,), dtype=torch.int32, device=confidence.device)
    if workspace is None:
        workspace = torch.zeros(max(256, int(lib().spec_schedule_workspace_bytes(B, gamma))),
                                dtype=torch.uint8, device=confidence.device)
    keep, sts_p = _sts_arg(sts, gamma)
    rc = lib().spec_schedule(_ptr(confidence), B, gamma, ctypes.byref(table), min_len, mode, sts_p,
                             _ptr(out_verify_len), _ptr(workspace), workspace.numel(),
                             _stream_handle(stream))
    _check(rc, "spec_schedule")
    return out_verify_len, workspace


def schedule_static(confidence, threshold: float, max_len: int, min_len: int = 0, *, sts=None,
                    out_verify_len=None, workspace=None, stream=None):
    """Run spec_schedule_static: leading positions with confidence >= threshold,
    clamped to [min_len, max_len] (threshold <= 0: fixed length max_len)."""
    torch = _torch()
    B, gamma = confidence.shape
    _check_tensor("confidence", confidence, torch.float32, (B, gamma), required=threshold > 0)
    _check_tensor("out_verify_len", out_verify_len, torch.int32, (B,), required=False)
    if out_verify_len is None:
        out_verify_len = torch.empty((B,), dtype=torch.int32, device=confidence.device)
    if workspace is None:
        workspace = torch.zeros(256, dtype=torch.uint8, device=confidence.device)
    keep, sts_p = _sts_arg(sts, gamma)
    rc = lib().spec_schedule_static(_ptr(confidence), B, gamma, ctypes.c_float(threshold), max_len, min_len, sts_p,
                                    _ptr(out_verify_len), _ptr(workspace), workspace.numel(),
                                    _stream_handle(stream))
    _check(rc, "spec_schedule_static")
    return out_verify_len, workspace


def sts_fit(confidence, accept_len):
    """spec_sts_fit on host arrays: confidences [n, gamma] and the accept lengths
    observed at verify_len = gamma.  Returns (temperatures [gamma] fp32, ece [gamma])."""
    import numpy as np
    c = np.ascontiguousarray(confidence, np.float32)
    al = np.ascontiguousarray(accept_len, np.int32)
    n, gamma = c.shape
    T = np.empty(gamma, np.float32)
    e = np.empty(gamma, np.float64)
    rc = lib().spec_sts_fit(c.ctypes.data_as(ctypes.c_void_p), al.ctypes.data_as(ctypes.c_void_p), n, gamma,
                            T.ctypes.data_as(ctypes.c_void_p), e.ctypes.data_as(ctypes.c_void_p))
    _check(rc, "spec_sts_fit")
    return T, e


def selftest_wait(limit_ns: int = 1_000_000, stream=None):
    """Run spec_selftest_wait: returns ((status_blocked, status_completed),
    (elapsed_ns_blocked, elapsed_ns_completed)) after synchronising."""
    torch = _torch()
    st = torch.full((2,), 99, dtype=torch.int32, device="cuda")
    el = torch.zeros((2,), dtype=torch.int64, device="cuda")
    _check(lib().spec_selftest_wait(int(limit_ns), _ptr(st), _ptr(el), _stream_handle(stream)), "spec_selftest_wait")
    torch.cuda.synchronize()
    return tuple(int(v) for v in st.cpu()), tuple(int(v) for v in el.cpu())


def selftest_expire_first_wait(on: bool) -> None:
    """Test hook: while on, the first copy wait of every streaming warp in later
    verify calls, and the first one of a tensor-core attention, counts as expired
    (the timeout paths; see include/specv.h)."""
    _check(lib().spec_selftest_expire_first_wait(1 if on else 0), "spec_selftest_expire_first_wait")


def read_status(workspace, stream=None) -> int:
    """Synchronise the stream, read and clear the workspace's device status word."""
    v = ctypes.c_int(0)
    _check(lib().spec_read_status(_ptr(workspace), _stream_handle(stream), ctypes.byref(v)),
           "spec_read_status")
    return v.value


def profile_events(before=None, after=None):
    """Register torch.cuda.Event pair recorded around the row-statistics kernel."""
    b = ctypes.c_void_p(before.cuda_event) if before is not None else None
    a = ctypes.c_void_p(after.cuda_event) if after is not None else None
    _check(lib().spec_profile_events(b, a), "spec_profile_events")


def kernel_count(B: int, temperature: float) -> int:
    return int(lib().spec_verify_kernel_count(B, ctypes.c_float(temperature)))


# ------------------------------------------------------- the key-value cache
# These calls run many times a token (per layer), and a small batch's kernels
# take a few microseconds: what they check is checked in one expression per
# tensor, and the message is looked for only when it fails.
_codes = {}


def _dtype_codes():
    torch = _torch()
    if not _codes:
        _codes.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32, torch.float8_e4m3fn: E4M3})
    return _codes


def _row_dtype(name, t) -> int:
    code = _dtype_codes().get(t.dtype)
    if code is None or code == E4M3:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _on_device(name, t, dev):
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")


def _want(name, t, dtype, shape, dev):
    """_check_tensor of a required tensor, the device already known."""
    if t is not None and t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return
    _check_tensor(name, t, dtype, shape)


def _current_device(t):
    """The current device; a host tensor is refused later, with its name."""
    return _torch().cuda.current_device() if t.is_cuda else 0


def _raw_stream(stream, dev):
    return _torch()._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _address(t):
    return None if t is None else t.data_ptr()


def _made_on(stream, make, *args, **kw):
    """make(*args) on the stream that the call runs on: what is allocated, zeroed
    and later freed there is in order with the call's kernels."""
    if stream is None:
        return make(*args, **kw)
    with _torch().cuda.stream(stream):
        return make(*args, **kw)


def _cache_arg(k_cache, v_cache, k_scale, v_scale, dev, layered=False):
    """spec_cache of [pages, page_size, kv_heads, head_dim] tensors (with
    `layered` also [layers, pages, ...]) of any strides with adjacent values."""
    dt = _dtype_codes().get(k_cache.dtype)
    if dt is None:
        raise TypeError(f"k_cache must be bfloat16, float16, float32 or float8_e4m3fn, got {k_cache.dtype}")
    if v_cache.dtype is not k_cache.dtype:
        raise TypeError(f"v_cache must be {k_cache.dtype}, got {v_cache.dtype}")
    shape, strides = k_cache.shape, k_cache.stride()
    dims = len(shape)
    if dims != 4 and not (layered and dims == 5):
        raise ValueError(f"k_cache must be {'[layers, ' if layered else '['}pages, page_size, kv_heads, head_dim], "
                         f"got {tuple(shape)}")
    if v_cache.shape != shape or v_cache.stride() != strides:
        raise ValueError("v_cache must have the shape and strides of k_cache")
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        _on_device("k_cache", k_cache, dev)
        _on_device("v_cache", v_cache, dev)
    P, page, H, D = shape[-4:]
    if strides[-1] != 1 and D != 1:
        raise ValueError("the head_dim values of k_cache must be adjacent")
    # a dimension of one entry has no stride of its own
    unit = 64
    ls = strides[0] if dims == 5 and shape[0] > 1 else unit
    ps, ts, hs = strides[-4] if P > 1 else unit, strides[-3] if page > 1 else unit, strides[-2] if H > 1 else unit
    if k_scale is not None or v_scale is not None:
        torch = _torch()
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None:
                if dt != E4M3:
                    raise ValueError(f"{name} belongs to a float8_e4m3fn cache")
                _want(name, s, torch.float32, (H,), dev)
    return Cache(k_cache.data_ptr(), v_cache.data_ptr(), dt, shape[0] if dims == 5 else 1, P, page, H, D, ls,
                 ps, ts, hs, _address(k_scale), _address(v_scale))


def _row_strides(name, t, dtype, heads, dim, B, gamma, packed, dev):
    """(rows, row stride, head stride) of query-like rows: [B, gamma+1, heads,
    dim] (padded) or [rows, heads, dim] (packed)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        _on_device(name, t, dev)
    shape, s = t.shape, t.stride()
    if packed:
        if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
            raise ValueError(f"{name} must have shape [rows, {heads}, {dim}] with a row index, got {tuple(shape)}")
        rows, rs = shape[0], s[0]
    else:
        if shape != (B, gamma + 1, heads, dim):
            raise ValueError(f"{name} must have shape {(B, gamma + 1, heads, dim)}, got {tuple(shape)}")
        rows, rs = B * (gamma + 1), s[1] if gamma > 0 else s[0]
        if gamma > 0 and B > 1 and s[0] != (gamma + 1) * s[1]:
            raise ValueError(f"the rows of {name} must be equally spaced")
    if s[-1] != 1 and dim != 1:
        raise ValueError(f"the head_dim values of {name} must be adjacent")
    return rows, rs if rows > 1 else heads * dim, s[-2] if heads > 1 else dim


def _tables(page_table, cache_len, verify_len, row, dev):
    i32 = _torch().int32
    B, slots = page_table.shape
    _want("page_table", page_table, i32, (B, slots), dev)
    _want("cache_len", cache_len, i32, (B,), dev)
    if verify_len is not None:
        _want("verify_len", verify_len, i32, (B,), dev)
    if row is not None:
        _want("row", row, i32, (B,), dev)


def _workspace_bytes(workspace, dev):
    _want("workspace", workspace, _torch().uint8, (workspace.numel(),), dev)
    return workspace.numel()


def _gamma_of(q, row, gamma):
    if row is None:
        if q.dim() != 4:
            raise ValueError("q must be [B, gamma+1, heads, head_dim] without a row index")
        if gamma is not None and gamma != q.shape[1] - 1:
            raise ValueError(f"q has {q.shape[1]} rows a request, gamma is {gamma}")
        return q.shape[1] - 1
    if q.dim() != 3:
        raise ValueError("q must be [rows, heads, head_dim] with a row index")
    if gamma is None:
        raise ValueError("packed rows need gamma")
    return int(gamma)


def alloc_attend_workspace(B: int, gamma: int, q_heads: int, kv_heads: int, head_dim: int, device=None):
    """A workspace of attend (zeroed; its status word is sticky until read_status)."""
    torch = _torch()
    n = int(lib().spec_attend_workspace_bytes(B, gamma, q_heads, kv_heads, head_dim))
    if n == 0:
        raise SpecError(ERR_SHAPE, "spec_attend_workspace_bytes")
    w = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    w[:256].zero_()
    return w


def alloc_cache_workspace(B: int, pages: int = 0, device=None):
    """A workspace of append_kv and the page calls (compact_pages needs the
    number of pages), zeroed."""
    torch = _torch()
    n = int(lib().spec_cache_workspace_bytes(B, pages))
    if n == 0:
        raise SpecError(ERR_SHAPE, "spec_cache_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def attend(q, k_cache, v_cache, page_table, cache_len, verify_len=None, row=None, *, gamma=None, scale=None,
           window: int = 0, sinks: int = 0, k_scale=None, v_scale=None, out=None, out_lse=None, workspace=None,
           stream=None):
    """Run spec_attend: attention of the tested tokens over a paged cache.

    q [B, gamma+1, heads, head_dim], or packed [rows, heads, head_dim] with row
    [B] int32 (the target rows of pack_rows) and gamma; bf16, fp16 or fp32,
    heads and rows at any 16-byte strides.  k_cache and v_cache [pages,
    page_size, kv_heads, head_dim] of q's type or float8_e4m3fn (with k_scale,
    v_scale [kv_heads] fp32 or None).  page_table [B, max_pages], cache_len [B],
    verify_len [B] or None (gamma for all), int32.  scale defaults to 1 /
    sqrt(head_dim).  out like q (contiguous; rows that no request has are left
    as they were, and undefined in an out made here), out_lse like q without
    head_dim, fp32.  Returns (out, workspace)."""
    torch = _torch()
    dt = _row_dtype("q", q)
    gamma = _gamma_of(q, row, gamma)
    dev = _current_device(q)
    cache = _cache_arg(k_cache, v_cache, k_scale, v_scale, dev)
    B, slots = page_table.shape
    heads, dim = q.shape[-2], k_cache.shape[-1]
    rows, rs, hs = _row_strides("q", q, q.dtype, heads, dim, B, gamma, row is not None, dev)
    _tables(page_table, cache_len, verify_len, row, dev)
    if out is None:
        out = _made_on(stream, torch.empty, q.shape, dtype=q.dtype, device=q.device)
    else:
        _want("out", out, q.dtype, q.shape, dev)
    if out_lse is not None:
        _want("out_lse", out_lse, torch.float32, q.shape[:-1], dev)
    if workspace is None:
        workspace = _made_on(stream, alloc_attend_workspace, B, gamma, heads, k_cache.shape[-2], dim, q.device)
    rc = lib().spec_attend(q.data_ptr(), rs, hs, dt, heads, cache, page_table.data_ptr(), slots,
                           cache_len.data_ptr(), _address(verify_len), _address(row), rows, B, gamma,
                           dim ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(), _address(out_lse),
                           workspace.data_ptr(), _workspace_bytes(workspace, dev), _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_attend")
    return out, workspace


def alloc_share_plan(B: int, gamma: int, rows: int | None = None, device=None):
    """A plan of share_plan; rows: the packed rows, B * (gamma + 1) by default."""
    torch = _torch()
    n = int(lib().spec_share_plan_bytes(B, gamma, B * (gamma + 1) if rows is None else rows))
    if n == 0:
        raise SpecError(ERR_SHAPE, "spec_share_plan_bytes")
    w = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    w[:256].zero_()
    return w


def alloc_attend_shared_workspace(B: int, gamma: int, q_heads: int, kv_heads: int, head_dim: int,
                                  rows: int | None = None, device=None):
    """A workspace of attend_shared (its status word zeroed, sticky until read_status)."""
    torch = _torch()
    n = int(lib().spec_attend_shared_workspace_bytes(B, gamma, B * (gamma + 1) if rows is None else rows, q_heads,
                                                     kv_heads, head_dim))
    if n == 0:
        raise SpecError(ERR_SHAPE, "spec_attend_shared_workspace_bytes")
    w = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    w[:256].zero_()
    return w


def share_plan(page_table, cache_len, verify_len=None, row=None, *, gamma: int, page_size: int,
               rows: int | None = None, least: int = 256, out_leader=None, out_shared=None, plan=None, stream=None):
    """Run spec_share_plan: groups of requests whose page tables begin with the
    same pages, for attend_shared.  page_table, cache_len, verify_len and row as for
    attend; rows: those of q where they are packed (with `row`).  The plan serves all
    layers of a round, and is made again when lengths, rows or shared entries change.
    It pays from about 16,000 saved positions a group on, (members - 1) * shared, with
    one to five rows a request, and from about 100,000 with 17; below, attend is faster.
    Returns (plan, out_leader [B], out_shared [B])."""
    torch = _torch()
    dev = _current_device(page_table)
    B, slots = page_table.shape
    _tables(page_table, cache_len, verify_len, row, dev)
    if rows is None:
        if row is not None:
            raise ValueError("packed rows need rows")
        rows = B * (gamma + 1)
    elif row is None and rows != B * (gamma + 1):
        raise ValueError(f"padded rows are {B * (gamma + 1)}, got {rows}")
    for name, t in (("out_leader", out_leader), ("out_shared", out_shared)):
        if t is not None:
            _want(name, t, torch.int32, (B,), dev)
    if out_leader is None:
        out_leader = _made_on(stream, torch.empty, (B,), dtype=torch.int32, device=page_table.device)
    if out_shared is None:
        out_shared = _made_on(stream, torch.empty, (B,), dtype=torch.int32, device=page_table.device)
    if plan is None:
        plan = _made_on(stream, alloc_share_plan, B, gamma, rows, page_table.device)
    _want("plan", plan, torch.uint8, (plan.numel(),), dev)
    rc = lib().spec_share_plan(page_table.data_ptr(), slots, page_size, cache_len.data_ptr(), _address(verify_len),
                               _address(row), rows, B, gamma, least, out_leader.data_ptr(), out_shared.data_ptr(),
                               plan.data_ptr(), plan.numel(), _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_share_plan")
    return plan, out_leader, out_shared


def attend_shared(q, k_cache, v_cache, page_table, plan, *, gamma=None, scale=None, k_scale=None, v_scale=None,
                  out=None, out_lse=None, workspace=None, stream=None):
    """Run spec_attend_shared: attend without a window, for a batch that shares
    prefixes by the plan of share_plan, which holds the lengths and rows.  q [B,
    gamma+1, heads, head_dim], or packed [rows, heads, head_dim] with gamma; other
    arguments as for attend.  Returns (out, workspace)."""
    torch = _torch()
    dt = _row_dtype("q", q)
    packed = q.dim() == 3
    gamma = _gamma_of(q, True if packed else None, gamma)
    dev = _current_device(q)
    cache = _cache_arg(k_cache, v_cache, k_scale, v_scale, dev)
    B, slots = page_table.shape
    heads, dim = q.shape[-2], k_cache.shape[-1]
    rows, rs, hs = _row_strides("q", q, q.dtype, heads, dim, B, gamma, packed, dev)
    _want("page_table", page_table, torch.int32, (B, slots), dev)
    _want("plan", plan, torch.uint8, (plan.numel(),), dev)
    if out is None:
        out = _made_on(stream, torch.empty, q.shape, dtype=q.dtype, device=q.device)
    else:
        _want("out", out, q.dtype, q.shape, dev)
    if out_lse is not None:
        _want("out_lse", out_lse, torch.float32, q.shape[:-1], dev)
    if workspace is None:
        workspace = _made_on(stream, alloc_attend_shared_workspace, B, gamma, heads, k_cache.shape[-2], dim, rows,
                             q.device)
    rc = lib().spec_attend_shared(q.data_ptr(), rs, hs, dt, heads, cache, page_table.data_ptr(), slots,
                                  plan.data_ptr(), plan.numel(), rows, B, gamma, dim ** -0.5 if scale is None else scale,
                                  out.data_ptr(), _address(out_lse), workspace.data_ptr(),
                                  _workspace_bytes(workspace, dev), _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_attend_shared")
    return out, workspace


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     context: int = 0, low: float = 1.0, high: float = 4.0):
    """Angle per token of each of the rotary_dim / 2 pairs, base^(-2i / rotary_dim),
    as a float64 array for rope_table.  For contexts longer than trained:

    scaling="linear": every frequency divided by `factor`;
    scaling="base": the base times factor^(rotary_dim / (rotary_dim - 2)), which
    keeps the highest frequency and divides the lowest by `factor`;
    scaling="banded": with w the wavelength in tokens, frequencies with
    context / w below `low` are divided by `factor`, those with context / w above
    `high` are kept, and those between are blended linearly in context / w."""
    import numpy as np
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    half = rotary_dim // 2
    if scaling == "base":
        if rotary_dim > 2:
            base = base * factor ** (rotary_dim / (rotary_dim - 2))
    elif scaling not in (None, "linear", "banded"):
        raise ValueError(f"unknown scaling {scaling!r}")
    f = base ** (-np.arange(half, dtype=np.float64) / half)
    if scaling == "linear":
        f = f / factor
    if scaling == "banded":
        if context < 1 or not high > low:
            raise ValueError("banded scaling needs the trained context and low < high")
        keep = np.clip((context * f / (2.0 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = (1.0 - keep) * f / factor + keep * f
    return f


def rope_table(frequencies, device=None):
    """The `turns` of append_kv for these angles per token (any array of
    float64): each as a fraction of 2^64 of a turn, int64 on the device."""
    import numpy as np
    torch = _torch()
    f = np.asarray(frequencies, dtype=np.float64).reshape(-1)
    if not np.all(np.isfinite(f)):
        raise ValueError("frequencies must be finite")
    turns = [int(round(float(x) / (2.0 * np.pi) * 2.0 ** 64)) % 2 ** 64 for x in f]
    return torch.from_numpy(np.array(turns, dtype=np.uint64).view(np.int64)).to(device or "cuda")


def append_kv(q, k, v, k_cache, v_cache, page_table, cache_len, verify_len=None, row=None, *, gamma=None,
              turns=None, interleaved: bool = False, mscale: float = 1.0, k_scale=None, v_scale=None, out_q=None,
              workspace=None, stream=None):
    """Run spec_append_kv: rotary positions, and the tested tokens' keys and
    values into their pages.

    q as for attend, k and v like it with kv_heads; any 16-byte strides (slices
    of one projection are fine).  turns: rope_table's, for 2 * len(turns)
    rotated values of each head, or None (no rotation).  out_q like q and
    contiguous (q itself is allowed where it is contiguous).  Other arguments as
    for attend.  Returns (out_q, workspace)."""
    torch = _torch()
    dt = _row_dtype("q", q)
    gamma = _gamma_of(q, row, gamma)
    dev = _current_device(q)
    cache = _cache_arg(k_cache, v_cache, k_scale, v_scale, dev)
    B, slots = page_table.shape
    heads, H, dim = q.shape[-2], k_cache.shape[-2], k_cache.shape[-1]
    packed = row is not None
    rows, rs, hs = _row_strides("q", q, q.dtype, heads, dim, B, gamma, packed, dev)
    krows, krs, khs = _row_strides("k", k, q.dtype, H, dim, B, gamma, packed, dev)
    vrows, vrs, vhs = _row_strides("v", v, q.dtype, H, dim, B, gamma, packed, dev)
    if krows != rows or vrows != rows:
        raise ValueError(f"q, k and v must have the same rows, got {rows}, {krows} and {vrows}")
    _tables(page_table, cache_len, verify_len, row, dev)
    n = 0
    if turns is not None:
        n = turns.numel()
        _want("turns", turns, torch.int64, (n,), dev)
    if out_q is None:
        out_q = _made_on(stream, torch.empty, q.shape, dtype=q.dtype, device=q.device)
    else:
        _want("out_q", out_q, q.dtype, q.shape, dev)
    if workspace is None:
        workspace = _made_on(stream, alloc_cache_workspace, B, 0, q.device)
    rc = lib().spec_append_kv(q.data_ptr(), rs, hs, k.data_ptr(), v.data_ptr(), krs, khs, vrs, vhs, dt, heads, cache,
                              page_table.data_ptr(), slots, cache_len.data_ptr(), _address(verify_len), _address(row),
                              rows, B, gamma, _address(turns), 2 * n, 1 if interleaved else 0, mscale,
                              out_q.data_ptr(), workspace.data_ptr(), _workspace_bytes(workspace, dev),
                              _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_append_kv")
    return out_q, workspace


def append_rows(q, k, v, k_cache, v_cache, position, slot, *, turns=None, interleaved: bool = False,
                mscale: float = 1.0, k_scale=None, v_scale=None, out_q=None, workspace=None, stream=None):
    """Run spec_append_rows: rotary positions, and keys and values of any rows into
    their slots.

    q [rows, heads, head_dim] (None: no queries), k and v [rows, kv_heads, head_dim];
    any 16-byte strides.  position [rows] int32 and slot [rows] int64 as map_rows
    writes them (a position below 0: no row; a slot below 0: not stored).  Other
    arguments as for append_kv.  Returns (out_q, workspace)."""
    torch = _torch()
    dt = _row_dtype("k", k)
    if k.dim() != 3 or (q is not None and q.dim() != 3):
        raise ValueError("q, k and v must be [rows, heads, head_dim]")
    dev = _current_device(k)
    cache = _cache_arg(k_cache, v_cache, k_scale, v_scale, dev)
    H, dim = k_cache.shape[-2], k_cache.shape[-1]
    rows, krs, khs = _row_strides("k", k, k.dtype, H, dim, 0, 0, True, dev)
    vrows, vrs, vhs = _row_strides("v", v, k.dtype, H, dim, 0, 0, True, dev)
    heads, rs, hs = 0, 0, 0
    if q is not None:
        heads = q.shape[1]
        qrows, rs, hs = _row_strides("q", q, k.dtype, heads, dim, 0, 0, True, dev)
        if qrows != rows:
            raise ValueError(f"q and k must have the same rows, got {qrows} and {rows}")
        if out_q is None:
            out_q = _made_on(stream, torch.empty, q.shape, dtype=q.dtype, device=q.device)
        else:
            _want("out_q", out_q, q.dtype, q.shape, dev)
    if vrows != rows:
        raise ValueError(f"k and v must have the same rows, got {rows} and {vrows}")
    _want("position", position, torch.int32, (rows,), dev)
    _want("slot", slot, torch.int64, (rows,), dev)
    n = 0
    if turns is not None:
        n = turns.numel()
        _want("turns", turns, torch.int64, (n,), dev)
    if workspace is None:
        workspace = _made_on(stream, alloc_cache_workspace, 1, 0, k.device)
    rc = lib().spec_append_rows(_address(q), rs, hs, k.data_ptr(), v.data_ptr(), krs, khs, vrs, vhs, dt, heads, cache,
                                position.data_ptr(), slot.data_ptr(), rows, _address(turns), 2 * n,
                                1 if interleaved else 0, mscale, _address(out_q), workspace.data_ptr(),
                                _workspace_bytes(workspace, dev), _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_append_rows")
    return out_q, workspace


def _page_state(page_table, num_pages, ref_count, cache_len=None):
    """(device, B, max_pages, pages) of tensors that belong together."""
    i32 = _torch().int32
    dev = _current_device(page_table)
    B, slots = page_table.shape
    pages = ref_count.numel()
    _want("page_table", page_table, i32, (B, slots), dev)
    _want("num_pages", num_pages, i32, (B,), dev)
    _want("ref_count", ref_count, i32, (pages,), dev)
    if cache_len is not None:
        _want("cache_len", cache_len, i32, (B,), dev)
    return dev, B, slots, pages


def reserve_pages(page_table, num_pages, ref_count, cache_len, verify_len=None, *, gamma: int, page_size: int,
                  out_status=None, workspace=None, stream=None):
    """Run spec_reserve_pages: pages for positions cache_len[b] .. cache_len[b]
    + verify_len[b] of every request.  page_table [B, max_pages], num_pages [B]
    and ref_count [pages] are updated.  Returns (out_status [B], workspace)."""
    i32 = _torch().int32
    dev, B, slots, pages = _page_state(page_table, num_pages, ref_count, cache_len)
    if verify_len is not None:
        _want("verify_len", verify_len, i32, (B,), dev)
    if out_status is not None:
        _want("out_status", out_status, i32, (B,), dev)
    if out_status is None:
        out_status = _made_on(stream, _torch().empty, (B,), dtype=i32, device=page_table.device)
    if workspace is None:
        workspace = _made_on(stream, alloc_cache_workspace, B, 0, page_table.device)
    rc = lib().spec_reserve_pages(page_table.data_ptr(), num_pages.data_ptr(), ref_count.data_ptr(), pages,
                                  cache_len.data_ptr(), _address(verify_len), B, gamma, slots, page_size,
                                  out_status.data_ptr(), workspace.data_ptr(), _workspace_bytes(workspace, dev),
                                  _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_reserve_pages")
    return out_status, workspace


def map_rows(page_table, num_pages, ref_count, cache_len, new_len, *, rows: int, page_size: int, out_first=None,
             out_request=None, out_position=None, out_slot=None, out_status=None, workspace=None, stream=None):
    """Run spec_map_rows: pages for new_len[b] ([B] int32, any number) positions
    behind cache_len[b], and the request, position and slot of each of their rows,
    one request behind the other, in arrays of `rows`.  page_table, num_pages and
    ref_count are updated.  Returns (out_first [B+1], out_request [rows],
    out_position [rows], out_slot [rows] int64, out_status [B], workspace)."""
    torch = _torch()
    i32 = torch.int32
    dev, B, slots, pages = _page_state(page_table, num_pages, ref_count, cache_len)
    _want("new_len", new_len, i32, (B,), dev)
    outs = []
    for name, t, dtype, n in (("out_first", out_first, i32, B + 1), ("out_request", out_request, i32, rows),
                              ("out_position", out_position, i32, rows), ("out_slot", out_slot, torch.int64, rows),
                              ("out_status", out_status, i32, B)):
        if t is None:
            t = _made_on(stream, torch.empty, (n,), dtype=dtype, device=page_table.device)
        else:
            _want(name, t, dtype, (n,), dev)
        outs.append(t)
    if workspace is None:
        workspace = _made_on(stream, alloc_cache_workspace, B, 0, page_table.device)
    rc = lib().spec_map_rows(page_table.data_ptr(), num_pages.data_ptr(), ref_count.data_ptr(), pages,
                             cache_len.data_ptr(), new_len.data_ptr(), B, slots, page_size, rows,
                             *[t.data_ptr() for t in outs], workspace.data_ptr(), _workspace_bytes(workspace, dev),
                             _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_map_rows")
    return (*outs, workspace)


def commit_pages(page_table, num_pages, ref_count, cache_len, accept_len, *, page_size: int, window: int = 0,
                 sinks: int = 0, out_cache_len=None, workspace=None, stream=None):
    """Run spec_commit_pages: cache_len + accept_len + 1 into out_cache_len (by
    default cache_len itself), and pages behind it, or left by the window, given
    back.  Returns (out_cache_len, workspace)."""
    i32 = _torch().int32
    dev, B, slots, pages = _page_state(page_table, num_pages, ref_count, cache_len)
    _want("accept_len", accept_len, i32, (B,), dev)
    if out_cache_len is not None:
        _want("out_cache_len", out_cache_len, i32, (B,), dev)
    if out_cache_len is None:
        out_cache_len = cache_len
    if workspace is None:
        workspace = _made_on(stream, alloc_cache_workspace, B, 0, page_table.device)
    rc = lib().spec_commit_pages(page_table.data_ptr(), num_pages.data_ptr(), ref_count.data_ptr(), pages,
                                 cache_len.data_ptr(), accept_len.data_ptr(), B, slots, page_size, window, sinks,
                                 out_cache_len.data_ptr(), workspace.data_ptr(), _workspace_bytes(workspace, dev),
                                 _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_commit_pages")
    return out_cache_len, workspace


def free_pages(page_table, num_pages, ref_count, cache_len, requests, *, workspace=None, stream=None):
    """Run spec_free_pages: the requests named in `requests` [n] int32 end and
    give their pages back.  Returns the workspace."""
    i32 = _torch().int32
    dev, B, slots, pages = _page_state(page_table, num_pages, ref_count, cache_len)
    n = requests.numel()
    _want("requests", requests, i32, (n,), dev)
    if workspace is None:
        workspace = _made_on(stream, alloc_cache_workspace, B, 0, page_table.device)
    rc = lib().spec_free_pages(page_table.data_ptr(), num_pages.data_ptr(), ref_count.data_ptr(), pages,
                               cache_len.data_ptr(), requests.data_ptr(), n, B, slots, workspace.data_ptr(),
                               _workspace_bytes(workspace, dev), _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_free_pages")
    return workspace


def fork_pages(page_table, num_pages, ref_count, cache_len, src, dst, k_cache, v_cache, *, out_status=None,
               workspace=None, stream=None):
    """Run spec_fork_pages: request dst[i] becomes a copy of request src[i] (src,
    dst [n] int32), sharing full pages and copying the partial last one in every
    layer of k_cache and v_cache ([layers, pages, page_size, kv_heads, head_dim],
    or without layers).  Returns (out_status [n], workspace)."""
    i32 = _torch().int32
    dev, B, slots, pages = _page_state(page_table, num_pages, ref_count, cache_len)
    n = src.numel()
    _want("src", src, i32, (n,), dev)
    _want("dst", dst, i32, (n,), dev)
    if out_status is not None:
        _want("out_status", out_status, i32, (n,), dev)
    cache = _cache_arg(k_cache, v_cache, None, None, dev, layered=True)
    if cache.pages != pages:
        raise ValueError(f"the cache has {cache.pages} pages, ref_count {pages}")
    if out_status is None:
        out_status = _made_on(stream, _torch().empty, (n,), dtype=i32, device=page_table.device)
    if workspace is None:
        workspace = _made_on(stream, alloc_cache_workspace, B, 0, page_table.device)
    rc = lib().spec_fork_pages(page_table.data_ptr(), num_pages.data_ptr(), ref_count.data_ptr(),
                               cache_len.data_ptr(), src.data_ptr(), dst.data_ptr(), n, B, slots, cache,
                               out_status.data_ptr(), workspace.data_ptr(), _workspace_bytes(workspace, dev),
                               _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_fork_pages")
    return out_status, workspace


def compact_pages(page_table, num_pages, ref_count, k_cache, v_cache, *, out_page_table=None, out_ref_count=None,
                  out_total=None, workspace=None, stream=None):
    """Run spec_compact_pages: the N referenced pages move to the ids 0..N-1 in
    every layer of k_cache and v_cache.  The renamed table and counts go to
    out_page_table and out_ref_count (by default the inputs themselves).
    Returns (out_total [1] = N, workspace)."""
    i32 = _torch().int32
    dev, B, slots, pages = _page_state(page_table, num_pages, ref_count)
    if out_page_table is not None:
        _want("out_page_table", out_page_table, i32, (B, slots), dev)
    if out_ref_count is not None:
        _want("out_ref_count", out_ref_count, i32, (pages,), dev)
    if out_total is not None:
        _want("out_total", out_total, i32, (1,), dev)
    cache = _cache_arg(k_cache, v_cache, None, None, dev, layered=True)
    if cache.pages != pages:
        raise ValueError(f"the cache has {cache.pages} pages, ref_count {pages}")
    out_page_table = page_table if out_page_table is None else out_page_table
    out_ref_count = ref_count if out_ref_count is None else out_ref_count
    if out_total is None:
        out_total = _made_on(stream, _torch().empty, (1,), dtype=i32, device=page_table.device)
    if workspace is None:
        workspace = _made_on(stream, alloc_cache_workspace, B, pages, page_table.device)
    rc = lib().spec_compact_pages(page_table.data_ptr(), num_pages.data_ptr(), ref_count.data_ptr(), B, slots, cache,
                                  out_page_table.data_ptr(), out_ref_count.data_ptr(), out_total.data_ptr(),
                                  workspace.data_ptr(), _workspace_bytes(workspace, dev), _raw_stream(stream, dev))
    if rc != OK:
        raise SpecError(rc, "spec_compact_pages")
    return out_total, workspace
