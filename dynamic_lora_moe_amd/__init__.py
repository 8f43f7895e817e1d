"""MI355X (gfx950) hot path of token-level pre-gated dynamic LoRA adapters.

A thin ctypes binding of libdlm.so (declared in include/dlm.h).  It only
marshals torch tensors (device memory) and the current HIP stream into the
C ABI; every step of the path runs in the library's HIP kernels.  There is no
fallback: if the library is missing or fails to load, importing the ops raises.

  pregate(x, Wr)                  -> (idx [T][2] int32, g [T][2] fp32)
  route(logits, k, ...)           -> (idx [T][k] int32, g [T][k] fp32); route_backward
  Layers([(W, A, B), ...], E, r, scale).switch(old, new)   # in place, one launch
  sgmm(x, idx, g, A, B, y, scale)                          # y updated in place
  AdamW(params, grads, ...).step(lr)                       # many tensors at once
  Muon(params, grads, ...).step(lr)                        # orthogonalised momentum
  balance(logits, idx, ...)       -> (loss, counts, rows, probs); balance_backward
  Int8Group([(x, W, w_scale, y), ...]).run()               # a base in 8 bits; .backward()
  SgmmGroup([(x, A, B, y), ...], E, r, scale).run(idx, g)  # .bind_grads(...).backward(idx, g, dg)
"""
from __future__ import annotations

import ctypes as C
import functools
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdlm.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "dlm.h")

DLM_OK, DLM_EINVAL, DLM_ESHAPE, DLM_EDTYPE, DLM_EALIGN = 0, -1, -2, -3, -4
DLM_EWORKSPACE, DLM_EHIP, DLM_EDEVICE, DLM_ENOMEM = -5, -6, -7, -8
DLM_F32, DLM_BF16 = 0, 1
DLM_SOFTMAX, DLM_SIGMOID = 0, 1
STATUS_NAMES = {0: "DLM_OK", -1: "DLM_EINVAL", -2: "DLM_ESHAPE", -3: "DLM_EDTYPE",
                -4: "DLM_EALIGN", -5: "DLM_EWORKSPACE", -6: "DLM_EHIP", -7: "DLM_EDEVICE",
                -8: "DLM_ENOMEM"}


class DLMError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class dlm_proj(C.Structure):
    _fields_ = [("W", C.c_void_p), ("A", C.c_void_p), ("B", C.c_void_p),
                ("d_out", C.c_int64), ("d_in", C.c_int64)]


class dlm_sgmm_problem(C.Structure):
    _fields_ = [("x", C.c_void_p), ("A", C.c_void_p), ("B", C.c_void_p), ("y", C.c_void_p),
                ("d_in", C.c_int64), ("d_out", C.c_int64)]


class dlm_route_cfg(C.Structure):
    _fields_ = [("k", C.c_int32), ("score", C.c_int32), ("n_groups", C.c_int32), ("keep_groups", C.c_int32),
                ("group_top", C.c_int32), ("renorm", C.c_int32), ("scale", C.c_float)]


class dlm_adamw_param(C.Structure):
    _fields_ = [("p", C.c_void_p), ("g", C.c_void_p), ("master", C.c_void_p), ("m", C.c_void_p), ("v", C.c_void_p),
                ("m_scale", C.c_void_p), ("v_scale", C.c_void_p), ("n", C.c_int64), ("weight_decay", C.c_float)]


class dlm_balance_cfg(C.Structure):
    _fields_ = [("k", C.c_int32), ("score", C.c_int32), ("alpha", C.c_float), ("zeta", C.c_float)]


class dlm_adamw_cfg(C.Structure):
    _fields_ = [("lr", C.c_float), ("beta1", C.c_double), ("beta2", C.c_double), ("eps", C.c_float)]


class dlm_i8_problem(C.Structure):
    _fields_ = [("x", C.c_void_p), ("W", C.c_void_p), ("w_scale", C.c_void_p), ("y", C.c_void_p), ("d_in", C.c_int64),
                ("d_out", C.c_int64)]


class dlm_muon_param(C.Structure):
    _fields_ = [("p", C.c_void_p), ("g", C.c_void_p), ("master", C.c_void_p), ("m", C.c_void_p), ("count", C.c_int64),
                ("rows", C.c_int64), ("cols", C.c_int64), ("weight_decay", C.c_float), ("scale", C.c_float)]


MAX_MUON_STEPS, MAX_BALANCE_SEQS = 10, 65536


class dlm_muon_cfg(C.Structure):
    _fields_ = [("lr", C.c_float), ("momentum", C.c_double), ("nesterov", C.c_int32), ("eps", C.c_float), ("steps", C.c_int32),
                ("coefs", C.c_double * 3 * MAX_MUON_STEPS)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libdlm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with dynamic_lora_moe_amd/build.py")
    lib = C.CDLL(path)
    P, I64, I32, F = C.c_void_p, C.c_int64, C.c_int32, C.c_float
    sig = {
        "dlm_last_error": ([], C.c_char_p),
        "dlm_version": ([], C.c_char_p),
        "dlm_pregate": ([P, P, I64, I64, I32, I32, P, P, P], C.c_int),
        "dlm_pregate_centroid": ([P, P, I64, I64, I32, I32, I32, P, P, P], C.c_int),
        "dlm_route": ([P, I64, P, I64, I32, I32, P, P, P, P, P], C.c_int),
        "dlm_route_backward": ([P, I64, P, P, I64, I32, I32, P, P, I64, P], C.c_int),
        "dlm_balance_workspace_size": ([I64, I32, I32, P], C.c_int),
        "dlm_balance": ([P, I64, P, P, I32, I64, I32, I32, P, P, P, P, P, P, C.c_size_t, P], C.c_int),
        "dlm_balance_backward": ([P, I64, P, P, P, I32, I64, I32, I32, P, P, I32, P, I64, P], C.c_int),
        "dlm_sgmm_group_backward_workspace_size": ([P, I64, P], C.c_int),
        "dlm_sgmm_group_bind_grads": ([P, P, P, P, P], C.c_int),
        "dlm_sgmm_group_backward": ([P, P, P, P, I64, I32, P, C.c_size_t, P], C.c_int),
        "dlm_adamw_create": ([P, I32, I32, I32, I32, I64, C.c_uint32, P], C.c_int),
        "dlm_adamw_destroy": ([P], C.c_int),
        "dlm_adamw_step": ([P, P, P, P, P], C.c_int),
        "dlm_adamw_status": ([P, P, P, P], C.c_int),
        "dlm_adamw_read_state": ([P, P, P, P, I64, P, P, P], C.c_int),
        "dlm_i8_quantize": ([P, I64, I64, I32, P, P, P], C.c_int),
        "dlm_i8_group_create": ([P, I32, I32, P], C.c_int),
        "dlm_i8_group_destroy": ([P], C.c_int),
        "dlm_i8_group_workspace_size": ([P, I64, P], C.c_int),
        "dlm_i8_group_run": ([P, I64, P, C.c_size_t, P], C.c_int),
        "dlm_i8_group_bind_grads": ([P, P, P], C.c_int),
        "dlm_i8_group_backward_workspace_size": ([P, I64, P], C.c_int),
        "dlm_i8_group_backward": ([P, I64, I32, P, C.c_size_t, P], C.c_int),
        "dlm_muon_create": ([P, I32, I32, I32, P], C.c_int),
        "dlm_muon_destroy": ([P], C.c_int),
        "dlm_muon_step": ([P, P, P, P, P], C.c_int),
        "dlm_muon_status": ([P, P, P], C.c_int),
        "dlm_layers_create": ([P, I32, I32, I32, F, I32, P], C.c_int),
        "dlm_layers_destroy": ([P], C.c_int),
        "dlm_switch": ([P, P, P, P, P, P], C.c_int),
        "dlm_switch_launches": ([P], C.c_int),
        "dlm_layers_status": ([P, P, P], C.c_int),
        "dlm_sgmm_workspace_size": ([I64, I64, I32, I32, I32, P], C.c_int),
        "dlm_sgmm": ([P, P, P, P, P, P, I64, I64, I64, I32, I32, F, I32, P, C.c_size_t, P], C.c_int),
        "dlm_sgmm_noalloc": ([P, P, P, P, P, P, I64, I64, I64, I32, I32, F, I32, P, P], C.c_int),
        "dlm_sgmm_group_create": ([P, I32, I32, I32, F, I32, P], C.c_int),
        "dlm_sgmm_group_destroy": ([P], C.c_int),
        "dlm_layers_repack": ([P, P], C.c_int),
        "dlm_layers_bind_vectors": ([P, P, P], C.c_int),
        "dlm_gemv": ([P, P], C.c_int),
        "dlm_switch_gemv": ([P, P, P, P, P, P], C.c_int),
        "dlm_switch_gemv_launches": ([P], C.c_int),
        "dlm_gemv_unmerged": ([P, P, P, P], C.c_int),
        "dlm_gemv_unmerged_launches": ([P], C.c_int),
        "dlm_sgmm_launches": ([I64, I64, I32, I32, I32], C.c_int),
        "dlm_sgmm_group_repack": ([P, P], C.c_int),
        "dlm_sgmm_group_run": ([P, P, P, I64, P, C.c_size_t, P], C.c_int),
        "dlm_sgmm_status": ([P, P, P], C.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def header_functions(path: str = HEADER):
    """Names of the functions include/dlm.h declares."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(dlm_\w+)\s*\(", text, flags=re.M)))


def _check(rc: int, what: str):
    if rc != DLM_OK:
        raise DLMError(rc, f"{what}: {load().dlm_last_error().decode()}")


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DLM_F32
    if t.dtype == torch.bfloat16:
        return DLM_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _like(t: torch.Tensor, name: str, shape, dtype, device):
    """The library takes bare pointers and cannot see a tensor's extent: every
    buffer it reads or writes is checked here against the shape it will assume."""
    _need(t, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _sets_out(idx, g, T: int, k: int, device, what: str, stream):
    """Per-row expert sets: idx [T][k] int32 and g [T][k] fp32 (allocated when None)."""
    own_idx, own_g = idx is None, g is None
    if own_idx:
        idx = torch.empty((T, k), dtype=torch.int32, device=device)
    else:
        _like(idx, f"{what} idx", (T, k), torch.int32, device)
    if own_g:
        g = torch.empty((T, k), dtype=torch.float32, device=device)
    else:
        _like(g, f"{what} g", (T, k), torch.float32, device)
    if stream is not None:
        _fresh(stream, idx if own_idx else None, g if own_g else None)
    return idx, g


def _fresh(stream, *tensors):
    """Before a launch on `stream` into tensors made here on the current stream (a None
    was not): what the current stream still runs may use the memory they were given, so
    `stream` waits for it, and the allocator keeps them until the launch has ended."""
    made = [t for t in tensors if t is not None]
    if stream is None or not made:
        return
    current = torch.cuda.current_stream(made[0].device)
    if stream != current:
        stream.wait_stream(current)
        for t in made:
            t.record_stream(stream)


# ---- router -------------------------------------------------------------------

def pregate(x: torch.Tensor, Wr: torch.Tensor, idx=None, g=None, stream=None):
    """Top-2 pre-gate: x [T][d], Wr [d][E] -> idx [T][2] int32, g [T][2] fp32 (device)."""
    _need(x, "x")
    _need(Wr, "Wr")
    T, d = x.shape
    E = Wr.shape[1]
    _like(Wr, "Wr", (d, E), x.dtype, x.device)
    idx, g = _sets_out(idx, g, T, 2, x.device, "pregate", stream)
    _check(load().dlm_pregate(_p(x), _p(Wr), T, d, E, _dt(x), _p(idx), _p(g), _stream(stream)),
           "dlm_pregate")
    return idx, g


def pregate_centroid(x: torch.Tensor, C: torch.Tensor, idx=None, g=None, stream=None):
    """Nearest-centroid pre-gate: x [T][d], C [E][J][d] -> idx [T][2] int32 (slot 1
    empty), g [T][2] fp32 = (1, 0) (device)."""
    _need(x, "x")
    _need(C, "C")
    T, d = x.shape
    E, J, d2 = C.shape
    _like(C, "C", (E, J, d), x.dtype, x.device)
    idx, g = _sets_out(idx, g, T, 2, x.device, "pregate_centroid", stream)
    _check(load().dlm_pregate_centroid(_p(x), _p(C), T, d, E, J, _dt(x), _p(idx), _p(g), _stream(stream)),
           "dlm_pregate_centroid")
    return idx, g


_SCORES = {"softmax": DLM_SOFTMAX, "sigmoid": DLM_SIGMOID}


def _rows(t: torch.Tensor, name: str):
    """(T, E, row pitch) of a device matrix whose rows are contiguous, its pitch any."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    T, E = t.shape
    ld = t.stride(0) if T > 1 else max(E, 1)
    if ld < E:
        raise ValueError(f"{name} has overlapping rows (pitch {ld} of {E})")
    return T, E, ld


def _here(t: torch.Tensor, stream, name: str) -> int:
    """The library launches on the current device: tensors and stream belong to
    it.  Returns the stream's handle."""
    dev = torch._C._cuda_getDevice()
    if t.device.index != dev:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream belongs to {stream.device}, but the current device is cuda:{dev}")
    return stream.cuda_stream


@functools.lru_cache(maxsize=64)
def _route_cfg(k, score, n_groups, keep_groups, group_top, renorm, scale):
    if score not in _SCORES:
        raise ValueError(f"score is one of {sorted(_SCORES)}, got {score!r}")
    return C.byref(dlm_route_cfg(k, _SCORES[score], n_groups, keep_groups, group_top, 1 if renorm else 0, scale))


def _ptr(t):
    """A tensor's address as ctypes takes it, None for None."""
    return None if t is None else t.data_ptr()


def route(logits: torch.Tensor, k: int, score: str = "softmax", bias=None, n_groups: int = 1, keep_groups: int = 1,
          group_top: int = 1, renorm: bool = True, scale: float = 1.0, counts=None, idx=None, g=None, stream=None):
    """Routing from logits [T][E] (any row pitch): softmax or sigmoid scores, a
    selection bias [E] fp32, the best keep_groups of n_groups groups (by their
    best key or the sum of their best two), the top k, weights renormalised over
    the chosen or not -> idx [T][k] int32, g [T][k] fp32 (device).  -inf marks an
    expert the row may not use; counts [E] int32 is added to."""
    T, E, ld = _rows(logits, "logits")
    handle = _here(logits, stream, "logits")
    if bias is not None:
        _like(bias, "bias", (E,), torch.float32, logits.device)
    if counts is not None:
        _like(counts, "counts", (E,), torch.int32, logits.device)
    idx, g = _sets_out(idx, g, T, k, logits.device, "route", stream)
    cfg = _route_cfg(k, score, n_groups, keep_groups, group_top, bool(renorm), float(scale))
    _check(load().dlm_route(logits.data_ptr(), ld, _ptr(bias), T, E, _dt(logits), cfg, idx.data_ptr(), g.data_ptr(),
                            _ptr(counts), handle), "dlm_route")
    return idx, g


def route_backward(logits: torch.Tensor, idx: torch.Tensor, dg: torch.Tensor, score: str = "softmax",
                   renorm: bool = True, scale: float = 1.0, dlogits=None, stream=None):
    """dLoss/dlogits [T][E] (logits' dtype; returned) from dg [T][k] = dLoss/dg of
    route()'s weights for its choice idx [T][k]."""
    T, E, ld = _rows(logits, "logits")
    handle = _here(logits, stream, "logits")
    if idx.dim() != 2:
        raise ValueError("idx must be [T][k]")
    k = idx.shape[1]
    _like(idx, "idx", (T, k), torch.int32, logits.device)
    _like(dg, "dg", (T, k), torch.float32, logits.device)
    if dlogits is None:
        dlogits, ldd = torch.empty((T, E), dtype=logits.dtype, device=logits.device), max(E, 1)
        _fresh(stream, dlogits)
    else:
        Td, Ed, ldd = _rows(dlogits, "dlogits")
        if (Td, Ed) != (T, E) or dlogits.dtype != logits.dtype or dlogits.device != logits.device:
            raise ValueError("dlogits must have logits' shape, dtype and device")
    cfg = _route_cfg(k, score, 1, 1, 1, bool(renorm), float(scale))
    _check(load().dlm_route_backward(logits.data_ptr(), ld, idx.data_ptr(), dg.data_ptr(), T, E, _dt(logits), cfg,
                                     dlogits.data_ptr(), ldd, handle), "dlm_route_backward")
    return dlogits


@functools.lru_cache(maxsize=64)
def _balance_cfg(k, score, alpha, zeta):
    if score not in _SCORES:
        raise ValueError(f"score is one of {sorted(_SCORES)}, got {score!r}")
    return C.byref(dlm_balance_cfg(k, _SCORES[score], alpha, zeta))


def _sequences(offsets, device) -> int:
    """Sequences that offsets [S + 1] int32 cut the rows into (None: one)."""
    if offsets is None:
        return 1
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [sequences + 1], of at least one sequence")
    _like(offsets, "offsets", offsets.shape, torch.int32, device)
    return offsets.shape[0] - 1


@functools.lru_cache(maxsize=64)
def balance_workspace_size(T: int, E: int, n_seq: int = 1) -> int:
    b = C.c_size_t(0)
    _check(load().dlm_balance_workspace_size(T, E, n_seq, C.byref(b)), "dlm_balance_workspace_size")
    return b.value


def balance(logits: torch.Tensor, idx: torch.Tensor, score: str = "softmax", alpha: float = 1.0, zeta: float = 0.0,
            offsets=None, loss=None, counts=None, rows=None, probs=None, workspace=None, stream=None):
    """The balance loss of a routing: logits [T][E] (any row pitch), idx [T][k] route()'s
    choice, offsets [S + 1] int32 the packed sequences' borders (None: one sequence) ->
    loss [2] fp32 (alpha times the balance term, zeta times the squared log sums, both
    means over the sequences), counts [S][E] int32 and rows [S] int32 (what
    balance_backward() takes), probs [S][E] fp32 the mean scores (device)."""
    T, E, ld = _rows(logits, "logits")
    handle = _here(logits, stream, "logits")
    dev = logits.device
    if idx.dim() != 2:
        raise ValueError("idx must be [T][k]")
    k = idx.shape[1]
    _like(idx, "idx", (T, k), torch.int32, dev)
    S = _sequences(offsets, dev)
    cfg = _balance_cfg(k, score, float(alpha), float(zeta))
    made = []

    def out(t, name, shape, dtype):
        if t is None:
            made.append(t := torch.empty(shape, dtype=dtype, device=dev))
        else:
            _like(t, name, shape, dtype, dev)
        return t

    loss = out(loss, "loss", (2,), torch.float32)
    counts, rows = out(counts, "counts", (S, E), torch.int32), out(rows, "rows", (S,), torch.int32)
    probs = out(probs, "probs", (S, E), torch.float32)
    if workspace is None:
        made.append(workspace := torch.empty(balance_workspace_size(T, E, S), dtype=torch.uint8, device=dev))
    _fresh(stream, *made)
    _check(load().dlm_balance(logits.data_ptr(), ld, idx.data_ptr(), _ptr(offsets), S, T, E, _dt(logits), cfg,
                              loss.data_ptr(), counts.data_ptr(), rows.data_ptr(), probs.data_ptr(), workspace.data_ptr(),
                              _ws_bytes(workspace), handle), "dlm_balance")
    return loss, counts, rows, probs


def balance_backward(logits: torch.Tensor, counts: torch.Tensor, rows: torch.Tensor, k: int, score: str = "softmax",
                     alpha: float = 1.0, zeta: float = 0.0, offsets=None, dloss=None, dlogits=None,
                     accumulate: bool = False, stream=None):
    """dLoss/dlogits [T][E] (logits' dtype; returned) of balance()'s loss, weighted by
    dloss [2] fp32 (None: 1, 1), from its counts [S][E] and rows [S] for a choice of k
    experts a row.  accumulate adds to dlogits, as to route_backward()'s; rows of no
    sequence are left as they are (0 in a dlogits made here)."""
    T, E, ld = _rows(logits, "logits")
    handle = _here(logits, stream, "logits")
    dev = logits.device
    S = _sequences(offsets, dev)
    _like(counts, "counts", (S, E), torch.int32, dev)
    _like(rows, "rows", (S,), torch.int32, dev)
    if dloss is not None:
        _like(dloss, "dloss", (2,), torch.float32, dev)
    if dlogits is None:
        if accumulate:
            raise ValueError("accumulate needs the dlogits to add to")
        make = torch.empty if offsets is None else torch.zeros
        dlogits, ldd = make((T, E), dtype=logits.dtype, device=dev), max(E, 1)
        _fresh(stream, dlogits)
    else:
        Td, Ed, ldd = _rows(dlogits, "dlogits")
        if (Td, Ed) != (T, E) or dlogits.dtype != logits.dtype or dlogits.device != dev:
            raise ValueError("dlogits must have logits' shape, dtype and device")
    cfg = _balance_cfg(k, score, float(alpha), float(zeta))
    _check(load().dlm_balance_backward(logits.data_ptr(), ld, counts.data_ptr(), rows.data_ptr(), _ptr(offsets), S, T, E,
                                       _dt(logits), cfg, _ptr(dloss), 1 if accumulate else 0, dlogits.data_ptr(), ldd,
                                       handle), "dlm_balance_backward")
    return dlogits


# ---- fused switch ---------------------------------------------------------------

def _set_ptrs(s):
    if s is None:
        return None, None
    i, g = s
    _need(i, "set idx")
    _need(g, "set g")
    if i.dtype != torch.int32 or g.dtype != torch.float32 or i.numel() < 2 or g.numel() < 2:
        raise ValueError("a set is (int32 idx[2], fp32 g[2]) on the device")
    return _p(i), _p(g)


class Layers:
    """Every adapted weight of every layer, switched together by one launch."""

    def __init__(self, projs, E: int, r: int, scale: float):
        self._keep = list(projs)
        arr = (dlm_proj * len(self._keep))()
        dt = None
        for k, (W, A, B) in enumerate(self._keep):
            _need(W, f"weight {k} W")
            if W.dim() != 2:
                raise ValueError(f"weight {k}: W must be [d_out][d_in]")
            d_out, d_in = W.shape
            W0 = self._keep[0][0]
            _like(W, f"weight {k} W", (d_out, d_in), W0.dtype, W0.device)
            _like(A, f"weight {k} A", (E, r, d_in), W.dtype, W.device)
            _like(B, f"weight {k} B", (E, d_out, r), W.dtype, W.device)
            dt = _dt(W) if dt is None else dt
            arr[k] = dlm_proj(W.data_ptr(), A.data_ptr(), B.data_ptr(), W.shape[0], W.shape[1])
        h = C.c_void_p()
        _check(load().dlm_layers_create(arr, len(self._keep), E, r, float(scale), dt, C.byref(h)),
               "dlm_layers_create")
        self._h = h
        self.E, self.r, self.scale = E, r, scale

    def switch(self, old=None, new=None, stream=None):
        """old/new: (idx int32[2], g fp32[2]) device tensors, or None for the empty set."""
        oi, og = _set_ptrs(old)
        ni, ng = _set_ptrs(new)
        _check(load().dlm_switch(self._h, oi, og, ni, ng, _stream(stream)), "dlm_switch")

    def status(self, stream=None) -> int:
        code = C.c_int32(0)
        _check(load().dlm_layers_status(self._h, C.byref(code), _stream(stream)), "dlm_layers_status")
        return code.value

    def launches_per_switch(self) -> int:
        return load().dlm_switch_launches(self._h)

    def bind_vectors(self, xs, ys):
        """Bind an input x_i [d_in] (the weights' dtype) and an output y_i [d_out]
        (fp32) device tensor to every weight, for gemv() and switch_gemv()."""
        if not len(xs) == len(ys) == len(self._keep):
            raise ValueError("one x and one y per weight")
        for k, ((W, _, _), x, y) in enumerate(zip(self._keep, xs, ys)):
            _like(x, f"x {k}", (W.shape[1],), W.dtype, W.device)
            _like(y, f"y {k}", (W.shape[0],), torch.float32, W.device)
        xa = (C.c_void_p * len(xs))(*[x.data_ptr() for x in xs])
        ya = (C.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
        _check(load().dlm_layers_bind_vectors(self._h, xa, ya), "dlm_layers_bind_vectors")
        self._vecs = (list(xs), list(ys))

    def gemv(self, stream=None):
        """y_i = W_i x_i for every weight (bound vectors)."""
        _check(load().dlm_gemv(self._h, _stream(stream)), "dlm_gemv")

    def switch_gemv(self, old=None, new=None, stream=None):
        """switch(old, new), then y_i = W'_i x_i (bound vectors)."""
        oi, og = _set_ptrs(old)
        ni, ng = _set_ptrs(new)
        _check(load().dlm_switch_gemv(self._h, oi, og, ni, ng, _stream(stream)), "dlm_switch_gemv")

    def launches_per_switch_gemv(self) -> int:
        return load().dlm_switch_gemv_launches(self._h)

    def gemv_unmerged(self, new, stream=None):
        """y_i = W_i x_i + s sum_k g_k B_k (A_k x_i) for the set new = (idx
        int32[2], g fp32[2]) on the device (bound vectors); W is not modified."""
        ni, ng = _set_ptrs(new)
        if not ni:
            raise ValueError("gemv_unmerged needs a set (idx, g)")
        _check(load().dlm_gemv_unmerged(self._h, ni, ng, _stream(stream)), "dlm_gemv_unmerged")

    def launches_per_gemv_unmerged(self) -> int:
        return load().dlm_gemv_unmerged_launches(self._h)

    def repack(self, stream=None):
        """Refresh the packed A copy (ranks 17..64, bf16) after changing an A bank in place."""
        _check(load().dlm_layers_repack(self._h, _stream(stream)), "dlm_layers_repack")

    def close(self):
        if getattr(self, "_h", None):
            _check(load().dlm_layers_destroy(self._h), "dlm_layers_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


# ---- SGMM ------------------------------------------------------------------------

def sgmm_workspace_size(T: int, d_in_max: int, E: int, r: int, n_problems: int = 1) -> int:
    b = C.c_size_t(0)
    _check(load().dlm_sgmm_workspace_size(T, d_in_max, E, r, n_problems, C.byref(b)),
           "dlm_sgmm_workspace_size")
    return b.value


def sgmm_workspace(T: int, d_in_max: int, E: int, r: int, n_problems: int = 1,
                   device="cuda") -> torch.Tensor:
    n = sgmm_workspace_size(T, d_in_max, E, r, n_problems)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _clean(workspace):
    """The workspace with its status word cleared, for who may read it before a launch has written it."""
    workspace[:256].zero_()
    return workspace


def _ws_bytes(workspace) -> int:
    _need(workspace, "workspace")
    return workspace.numel() * workspace.element_size()


def sgmm(x, idx, g, A, B, y, scale: float, workspace=None, stream=None):
    """y += sum_k s g_k (x A_k^T) B_k^T row by row, in place (returns y).

    With a workspace the call only enqueues; read the device's decision on the
    sets with sgmm_status(workspace).  Without one it allocates a workspace,
    waits for the launches (so the temporary outlives them) and raises
    DLMError(DLM_EDEVICE) if the device rejected a set (y is then unchanged)."""
    _need(x, "x")
    _need(A, "A")
    _need(B, "B")
    T, d_in = x.shape
    E, r, _ = A.shape
    d_out = B.shape[1]
    _like(A, "A", (E, r, d_in), x.dtype, x.device)
    _like(B, "B", (E, d_out, r), x.dtype, x.device)
    _like(y, "y", (T, d_out), x.dtype, x.device)
    _like(idx, "idx", (T, 2), torch.int32, x.device)
    _like(g, "g", (T, 2), torch.float32, x.device)
    own = workspace is None
    if own:
        workspace = sgmm_workspace(T, d_in, E, r, 1, x.device)
        _fresh(stream, workspace)
    _check(load().dlm_sgmm(_p(x), _p(idx), _p(g), _p(A), _p(B), _p(y), T, d_in, d_out, E, r,
                           float(scale), _dt(x), _p(workspace), _ws_bytes(workspace), _stream(stream)),
           "dlm_sgmm")
    if own and T > 0 and sgmm_status(workspace, stream) != DLM_OK:
        raise DLMError(DLM_EDEVICE, "dlm_sgmm: the device rejected an expert set (index outside [-1, E) or "
                                    "a non-finite gate); y is unchanged")
    return y


def sgmm_noalloc(x, idx, g, A, B, y, scale: float, status=None, stream=None):
    """sgmm() with the workspace in the library's own scratch array (no device
    allocation by the call; calls overlapping on one device race).  status: an
    optional int32 [1] device tensor receiving 0, or nonzero if a set was rejected."""
    _need(x, "x")
    _need(A, "A")
    _need(B, "B")
    T, d_in = x.shape
    E, r, _ = A.shape
    d_out = B.shape[1]
    _like(A, "A", (E, r, d_in), x.dtype, x.device)
    _like(B, "B", (E, d_out, r), x.dtype, x.device)
    _like(y, "y", (T, d_out), x.dtype, x.device)
    _like(idx, "idx", (T, 2), torch.int32, x.device)
    _like(g, "g", (T, 2), torch.float32, x.device)
    if status is not None:
        _like(status, "status", (1,), torch.int32, x.device)
    _check(load().dlm_sgmm_noalloc(_p(x), _p(idx), _p(g), _p(A), _p(B), _p(y), T, d_in, d_out, E, r,
                                   float(scale), _dt(x), _p(status), _stream(stream)), "dlm_sgmm_noalloc")
    return y


def sgmm_launches(T: int, d_in_max: int, r: int, n_problems: int = 1, dtype=torch.bfloat16) -> int:
    """Kernel launches of one sgmm / sgmm_noalloc (n_problems = 1) or
    SgmmGroup.run call at rank r."""
    dt = {torch.float32: DLM_F32, torch.bfloat16: DLM_BF16}.get(dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {dtype}")
    n = load().dlm_sgmm_launches(T, d_in_max, r, n_problems, dt)
    if n < 0:
        raise DLMError(DLM_EINVAL, load().dlm_last_error().decode())
    return n


def sgmm_status(workspace, stream=None) -> int:
    code = C.c_int32(0)
    _check(load().dlm_sgmm_status(_p(workspace), C.byref(code), _stream(stream)), "dlm_sgmm_status")
    return code.value


class SgmmGroup:
    """Many (x, A, B, y) problems run on the same rows' expert sets (decide once)."""

    def __init__(self, problems, E: int, r: int, scale: float):
        self._keep = list(problems)
        arr = (dlm_sgmm_problem * len(self._keep))()
        dt = None
        x0 = self._keep[0][0]
        _need(x0, "problem 0 x")
        for k, (x, A, B, y) in enumerate(self._keep):
            _need(x, f"problem {k} x")
            _need(B, f"problem {k} B")
            if x.dim() != 2 or B.dim() != 3:
                raise ValueError(f"problem {k}: x must be [T][d_in] and B [E][d_out][r]")
            T_k, d_in = x.shape
            d_out = B.shape[1]
            _like(x, f"problem {k} x", (T_k, d_in), x0.dtype, x0.device)
            _like(A, f"problem {k} A", (E, r, d_in), x.dtype, x.device)
            _like(B, f"problem {k} B", (E, d_out, r), x.dtype, x.device)
            _like(y, f"problem {k} y", (T_k, d_out), x.dtype, x.device)
            dt = _dt(x) if dt is None else dt
            arr[k] = dlm_sgmm_problem(x.data_ptr(), A.data_ptr(), B.data_ptr(), y.data_ptr(),
                                      x.shape[1], y.shape[1])
        h = C.c_void_p()
        _check(load().dlm_sgmm_group_create(arr, len(self._keep), E, r, float(scale), dt, C.byref(h)),
               "dlm_sgmm_group_create")
        self._h = h
        self.E, self.r, self.n = E, r, len(self._keep)
        self.d_in_max = max(x.shape[1] for x, _, _, _ in self._keep)
        self.rows = min(x.shape[0] for x, _, _, _ in self._keep)  # rows every problem holds
        self.device = x0.device

    def workspace(self, T: int, device="cuda"):
        return sgmm_workspace(T, self.d_in_max, self.E, self.r, self.n, device)

    def repack(self, stream=None):
        """Refresh the packed A copies after the A banks were changed in place."""
        _check(load().dlm_sgmm_group_repack(self._h, _stream(stream)), "dlm_sgmm_group_repack")

    def run(self, idx, g, T: int | None = None, workspace=None, stream=None):
        """Run every problem on rows [0, T) of (idx, g); returns the workspace,
        whose status word sgmm_status() reads (a rejected set leaves every y
        unchanged)."""
        _need(idx, "idx")
        T = idx.shape[0] if T is None else T
        if not 0 <= T <= self.rows:
            raise ValueError(f"T={T} rows, but the group's problems hold {self.rows}")
        _like(idx[:T], "idx", (T, 2), torch.int32, self.device)
        _like(g[:T], "g", (T, 2), torch.float32, self.device)
        if workspace is None:
            workspace = self.workspace(T, idx.device) if T else _clean(self.workspace(T, idx.device))
            _fresh(stream, workspace)
        _check(load().dlm_sgmm_group_run(self._h, _p(idx), _p(g), T, _p(workspace),
                                         _ws_bytes(workspace), _stream(stream)), "dlm_sgmm_group_run")
        return workspace

    def bind_grads(self, dys, dxs, dAs, dBs):
        """Bind the buffers of backward(): per problem dy [T][d_out] and dx [T][d_in]
        (the problems' dtype; dxs or an entry of it may be None, and problems that
        share an x may share a dx), dA [E][r][d_in] and dB [E][d_out][r] fp32."""
        _here(self._keep[0][0], None, "problem 0 x")
        n = self.n
        dys, dAs, dBs = list(dys), list(dAs), list(dBs)
        dxs = [None] * n if dxs is None else list(dxs)
        if not len(dys) == len(dxs) == len(dAs) == len(dBs) == n:
            raise ValueError("one dy, dx (or None), dA and dB per problem")
        for k, ((x, A, B, y), dy, dx, dA, dB) in enumerate(zip(self._keep, dys, dxs, dAs, dBs)):
            _like(dy, f"dy {k}", y.shape, x.dtype, x.device)
            if dx is not None:
                _like(dx, f"dx {k}", x.shape, x.dtype, x.device)
            _like(dA, f"dA {k}", A.shape, torch.float32, x.device)
            _like(dB, f"dB {k}", B.shape, torch.float32, x.device)
        ptrs = lambda ts: (C.c_void_p * n)(*[None if t is None else t.data_ptr() for t in ts])  # noqa: E731
        _check(load().dlm_sgmm_group_bind_grads(self._h, ptrs(dys), ptrs(dxs), ptrs(dAs), ptrs(dBs)),
               "dlm_sgmm_group_bind_grads")
        self._grads = (dys, dxs, dAs, dBs)

    def backward_workspace(self, T: int):
        """A workspace of backward() for T rows (once the buffers are bound)."""
        b = C.c_size_t(0)
        _check(load().dlm_sgmm_group_backward_workspace_size(self._h, T, C.byref(b)),
               "dlm_sgmm_group_backward_workspace_size")
        return torch.empty(b.value, dtype=torch.uint8, device=self.device)

    def backward(self, idx, g, dg=None, accumulate: bool = False, T: int | None = None, workspace=None, stream=None):
        """The gradients of run() for rows [0, T) of (idx, g) into the bound buffers:
        dx is added to in place, dA and dB are written (or added to), and dg [T][2]
        fp32, if given, is the gradient of g.  Returns the workspace, whose status
        word sgmm_status() reads (a rejected set leaves every buffer unchanged)."""
        _need(idx, "idx")
        handle = _here(idx, stream, "idx")
        T = idx.shape[0] if T is None else T
        if not 0 <= T <= self.rows:
            raise ValueError(f"T={T} rows, but the group's problems hold {self.rows}")
        _like(idx[:T], "idx", (T, 2), torch.int32, self.device)
        _like(g[:T], "g", (T, 2), torch.float32, self.device)
        if dg is not None:
            _like(dg[:T], "dg", (T, 2), torch.float32, self.device)
        if workspace is None:
            workspace = self.backward_workspace(T) if T else _clean(self.backward_workspace(T))
            _fresh(stream, workspace)
        _check(load().dlm_sgmm_group_backward(self._h, _ptr(idx), _ptr(g), _ptr(dg), T, 1 if accumulate else 0,
                                              _ptr(workspace), _ws_bytes(workspace), handle), "dlm_sgmm_group_backward")
        return workspace

    def close(self):
        if getattr(self, "_h", None):
            _check(load().dlm_sgmm_group_destroy(self._h), "dlm_sgmm_group_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass


# ---- 8-bit products -----------------------------------------------------------------

def quantize_rows(x: torch.Tensor, q=None, scale=None, stream=None):
    """Rows [T][d] as 8-bit codes and a scale each: (q [T][d] int8, scale [T] fp32), 127
    for a row's largest magnitude.  A weight [d_out][d_in] so becomes what Int8Group takes."""
    _need(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T][d]")
    handle = _here(x, stream, "x")
    T, d = x.shape
    own_q, own_s = q is None, scale is None
    q = torch.empty((T, d), dtype=torch.int8, device=x.device) if own_q else q
    scale = torch.empty(T, dtype=torch.float32, device=x.device) if own_s else scale
    _like(q, "q", (T, d), torch.int8, x.device)
    _like(scale, "scale", (T,), torch.float32, x.device)
    _fresh(stream, q if own_q else None, scale if own_s else None)
    _check(load().dlm_i8_quantize(_p(x), T, d, _dt(x), _p(q), _p(scale), handle), "dlm_i8_quantize")
    return q, scale


class Int8Group:
    """A frozen base's products in 8 bits, many at once: y = s_x w_scale (codes of x) W^T.

    problems: [(x [T][d_in], W [d_out][d_in] int8, w_scale [d_out] fp32, y [T][d_out])], x
    and y fixed buffers of one dtype (bf16 or fp32).  W and w_scale are copied here; x is
    coded at every run, once where problems share it.  Run it before the SgmmGroup of the
    same problems, which adds the adapters to y."""

    def __init__(self, problems):
        problems = list(problems)
        n = len(problems)
        if not n:
            raise ValueError("at least one problem")
        x0 = problems[0][0]
        _need(x0, "problem 0 x")
        arr = (dlm_i8_problem * n)()
        for k, (x, W, w_scale, y) in enumerate(problems):
            if x.dim() != 2 or W.dim() != 2:
                raise ValueError(f"problem {k}: x must be [T][d_in] and W [d_out][d_in]")
            T, d_in = x.shape
            d_out = W.shape[0]
            _like(x, f"problem {k} x", (T, d_in), x0.dtype, x0.device)
            _like(W, f"problem {k} W", (d_out, d_in), torch.int8, x0.device)
            _like(w_scale, f"problem {k} w_scale", (d_out,), torch.float32, x0.device)
            _like(y, f"problem {k} y", (T, d_out), x0.dtype, x0.device)
            arr[k] = dlm_i8_problem(x.data_ptr(), W.data_ptr(), w_scale.data_ptr(), y.data_ptr(), d_in, d_out)
        dt = _dt(x0)
        _here(x0, None, "problem 0 x")
        h = C.c_void_p()
        _check(load().dlm_i8_group_create(arr, n, dt, C.byref(h)), "dlm_i8_group_create")
        self._h = h
        self._keep = [(x, y) for x, _, _, y in problems]
        self.n, self.device = n, x0.device
        self.rows = min(x.shape[0] for x, _ in self._keep)  # rows every problem holds
        self._sizes = {}

    def _size(self, T: int, what: str) -> int:
        if (T, what) not in self._sizes:
            b = C.c_size_t(0)
            _check(getattr(load(), what)(self._h, T, C.byref(b)), what)
            self._sizes[T, what] = b.value
        return self._sizes[T, what]

    def workspace(self, T: int):
        """A workspace of run() for T rows."""
        return torch.empty(self._size(T, "dlm_i8_group_workspace_size"), dtype=torch.uint8, device=self.device)

    def backward_workspace(self, T: int):
        """A workspace of backward() for T rows (once the buffers are bound)."""
        return torch.empty(self._size(T, "dlm_i8_group_backward_workspace_size"), dtype=torch.uint8, device=self.device)

    def _call(self, T, workspace, stream, make):
        handle = _here(self._keep[0][0], stream, "problem 0 x")
        T = self.rows if T is None else T
        if not 0 <= T <= self.rows:
            raise ValueError(f"T={T} rows, but the group's problems hold {self.rows}")
        if workspace is None:
            workspace = make(T)
            _fresh(stream, workspace)
        return handle, T, workspace

    def run(self, T: int | None = None, workspace=None, stream=None):
        """Write rows [0, T) of every y (None: every row)."""
        handle, T, workspace = self._call(T, workspace, stream, self.workspace)
        _check(load().dlm_i8_group_run(self._h, T, _ptr(workspace), _ws_bytes(workspace), handle), "dlm_i8_group_run")
        return workspace

    def bind_grads(self, dys, dxs):
        """Bind the buffers of backward(): per problem dy [T][d_out] and dx [T][d_in] (the
        problems' dtype; dxs or an entry of it may be None, with its dy: not wanted).
        Problems that share an input share its dx, which is then their sum."""
        _here(self._keep[0][0], None, "problem 0 x")
        dys, dxs = list(dys), [None] * self.n if dxs is None else list(dxs)
        if not len(dys) == len(dxs) == self.n:
            raise ValueError("one dy and dx (or None) per problem")
        for k, ((x, y), dy, dx) in enumerate(zip(self._keep, dys, dxs)):
            if dy is not None:
                _like(dy, f"dy {k}", y.shape, x.dtype, x.device)
            if dx is not None:
                _like(dx, f"dx {k}", x.shape, x.dtype, x.device)
        ptrs = lambda ts: (C.c_void_p * self.n)(*[None if t is None else t.data_ptr() for t in ts])  # noqa: E731
        _check(load().dlm_i8_group_bind_grads(self._h, ptrs(dys), ptrs(dxs)), "dlm_i8_group_bind_grads")
        self._grads = (dys, dxs)
        self._sizes.clear()

    def backward(self, accumulate: bool = False, T: int | None = None, workspace=None, stream=None):
        """dx of rows [0, T) from the bound dy: written, or with accumulate added to."""
        handle, T, workspace = self._call(T, workspace, stream, self.backward_workspace)
        _check(load().dlm_i8_group_backward(self._h, T, 1 if accumulate else 0, _ptr(workspace), _ws_bytes(workspace), handle),
               "dlm_i8_group_backward")
        return workspace

    def close(self):
        if getattr(self, "_h", None):
            _check(load().dlm_i8_group_destroy(self._h), "dlm_i8_group_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass


# ---- AdamW -------------------------------------------------------------------------

ADAMW_BLOCK = 256  # elements that share a scale of the 8-bit moments


class AdamW:
    """AdamW over many tensors at once (params updated in place).

    params / grads: device tensors of one dtype each (fp32 or bf16), any shapes.  A
    step reads the gradients from these buffers.
    masters: per parameter an fp32 copy that the step updates (a bf16 parameter
    then becomes its rounding), or None.  state_bits 32: moments fp32; 8: codes
    with a scale per 256 elements.  states: per parameter (m, v), or with 8 bits
    (m int8, v uint8, m_scale, v_scale), flat; zeros are made when None.
    weight_decay: one value, or one per parameter.  step: steps already taken."""

    def __init__(self, params, grads, masters=None, state_bits: int = 32, states=None, beta1: float = 0.9,
                 beta2: float = 0.999, eps: float = 1e-8, weight_decay=0.01, step: int = 0, seed: int = 0):
        self.params, self.grads = list(params), list(grads)
        n = len(self.params)
        if not n or len(self.grads) != n:
            raise ValueError("one gradient per parameter, at least one parameter")
        self.masters = [None] * n if masters is None else list(masters)
        wd = [float(w) for w in weight_decay] if isinstance(weight_decay, (list, tuple)) else [float(weight_decay)] * n
        if state_bits not in (32, 8):
            raise ValueError("state_bits is 32 or 8")
        if states is None:
            states = [self._zeros(p, state_bits) for p in self.params]
            if self.params[0].is_cuda:  # steps may run on any stream
                torch.cuda.current_stream(self.params[0].device).synchronize()
        self.states = [tuple(st) for st in states]
        if not len(self.masters) == len(wd) == len(self.states) == n:
            raise ValueError("one master (or None), weight decay and state per parameter")
        p0, g0 = self.params[0], self.grads[0]
        arr = (dlm_adamw_param * n)()
        for k, (p, g, w, st) in enumerate(zip(self.params, self.grads, self.masters, self.states)):
            _like(p, f"parameter {k}", p.shape, p0.dtype, p0.device)
            _like(g, f"gradient {k}", p.shape, g0.dtype, p0.device)
            if w is not None:
                _like(w, f"master {k}", p.shape, torch.float32, p0.device)
            ne = p.numel()
            nb = -(-ne // ADAMW_BLOCK)
            want = [torch.float32, torch.float32] if state_bits == 32 else \
                [torch.int8, torch.uint8, torch.float32, torch.float32]
            if len(st) != len(want):
                raise ValueError(f"state {k} has {len(st)} tensors, expected {len(want)}")
            for t, dt, m, name in zip(st, want, (ne, ne, nb, nb), ("m", "v", "m_scale", "v_scale")):
                if t.numel() != m:
                    raise ValueError(f"state {k} {name} has {t.numel()} elements, expected {m}")
                _like(t, f"state {k} {name}", t.shape, dt, p0.device)
            ptr = [t.data_ptr() for t in st] + [None, None]
            arr[k] = dlm_adamw_param(p.data_ptr(), g.data_ptr(), None if w is None else w.data_ptr(), ptr[0], ptr[1],
                                     ptr[2], ptr[3], ne, wd[k])
        _here(p0, None, "parameter 0")
        h = C.c_void_p()
        _check(load().dlm_adamw_create(arr, n, _dt(p0), _dt(g0), state_bits, int(step), seed & 0xFFFFFFFF, C.byref(h)),
               "dlm_adamw_create")
        self._h = h
        self.state_bits, self.device = state_bits, p0.device
        self.beta1, self.beta2, self.eps = float(beta1), float(beta2), float(eps)

    @staticmethod
    def _zeros(p, bits):
        z = lambda n, dt: torch.zeros(n, dtype=dt, device=p.device)  # noqa: E731
        n = p.numel()
        if bits == 32:
            return z(n, torch.float32), z(n, torch.float32)
        nb = -(-n // ADAMW_BLOCK)
        return z(n, torch.int8), z(n, torch.uint8), z(nb, torch.float32), z(nb, torch.float32)

    def step(self, lr: float, lr_scale=None, grad_scale=None, stream=None):
        """One step.  lr_scale / grad_scale: optional fp32 [1] device tensors that
        multiply lr / the gradients, read when the step runs."""
        handle = _here(self.params[0], stream, "parameter 0")
        for t, name in ((lr_scale, "lr_scale"), (grad_scale, "grad_scale")):
            if t is not None:
                _like(t, name, (1,), torch.float32, self.device)
        cfg = dlm_adamw_cfg(float(lr), self.beta1, self.beta2, self.eps)
        _check(load().dlm_adamw_step(self._h, C.byref(cfg), _ptr(lr_scale), _ptr(grad_scale), handle), "dlm_adamw_step")

    def status(self, stream=None):
        """(steps taken, DLM_OK or DLM_EDEVICE: some gradient was not finite); clears the error."""
        handle = _here(self.params[0], stream, "parameter 0")
        step, code = C.c_int64(0), C.c_int32(0)
        _check(load().dlm_adamw_status(self._h, C.byref(step), C.byref(code), handle), "dlm_adamw_status")
        return step.value, code.value

    def read_state(self, k: int, stream=None):
        """(m, v) of parameter k as fp32 tensors of its shape."""
        st, shape = self.states[k], self.params[k].shape
        if self.state_bits == 32:
            return st[0].view(shape), st[1].view(shape)
        m, v = adamw_read_state(*st, stream=stream)
        return m.view(shape), v.view(shape)

    def close(self):
        if getattr(self, "_h", None):
            _check(load().dlm_adamw_destroy(self._h), "dlm_adamw_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass


def adamw_read_state(m, v, m_scale, v_scale, m_out=None, v_out=None, stream=None):
    """The fp32 values (m, v) that 8-bit moments stand for: flat codes and one scale per 256 elements."""
    n = m.numel()
    nb = -(-n // ADAMW_BLOCK)
    _like(m, "m", (n,), torch.int8, m.device)
    _like(v, "v", (n,), torch.uint8, m.device)
    _like(m_scale, "m_scale", (nb,), torch.float32, m.device)
    _like(v_scale, "v_scale", (nb,), torch.float32, m.device)
    handle = _here(m, stream, "m")
    own_m, own_v = m_out is None, v_out is None
    m_out = torch.empty(n, dtype=torch.float32, device=m.device) if own_m else m_out
    v_out = torch.empty(n, dtype=torch.float32, device=m.device) if own_v else v_out
    _like(m_out, "m_out", (n,), torch.float32, m.device)
    _like(v_out, "v_out", (n,), torch.float32, m.device)
    _fresh(stream, m_out if own_m else None, v_out if own_v else None)
    _check(load().dlm_adamw_read_state(_p(m), _p(v), _p(m_scale), _p(v_scale), n, _p(m_out), _p(v_out), handle),
           "dlm_adamw_read_state")
    return m_out, v_out


# ---- Muon -------------------------------------------------------------------------

class Muon:
    """Momentum orthogonalised by Newton-Schulz products, over the matrices of many
    tensors at once (params updated in place).

    params / grads: device tensors of one dtype each (fp32 or bf16) of two or more
    dimensions; the last two are a matrix, what is before them counts matrices (a bank
    [E][r][d] holds one per expert).  The smaller side is at most 512.
    masters: per parameter an fp32 copy that the step updates (a bf16 parameter then
    becomes its rounding), or None.  states: per parameter its momentum, fp32 of the
    parameter's shape; zeros are made when None.
    steps, coefs: the products X <- a X + (b A + c A^2) X, (a, b, c) for all or one triple
    per step.  scale: the update's factor: "shape" = sqrt(max(1, rows / cols)), which is
    sqrt(max(1, outputs / inputs)) for matrices stored outputs first, as A [r][d_in] and
    B [d_out][r] are (one stored inputs first, as a router's [d][E], takes the number
    max(1, cols / rows) ** 0.5), "rms" = 0.2 sqrt(max(rows, cols)) (an entry's size then is
    about AdamW's), a number, or one per parameter.  weight_decay: one value, or one per
    parameter."""

    def __init__(self, params, grads, masters=None, states=None, momentum: float = 0.95, nesterov: bool = True,
                 weight_decay=0.0, eps: float = 1e-7, steps: int = 5, coefs=(3.4445, -4.7750, 2.0315), scale="shape"):
        self.params, self.grads = list(params), list(grads)
        n = len(self.params)
        if not n or len(self.grads) != n:
            raise ValueError("one gradient per parameter, at least one parameter")
        self.masters = [None] * n if masters is None else list(masters)
        each = lambda v: list(v) if isinstance(v, (list, tuple)) else [v] * n  # noqa: E731
        wd, scales = each(weight_decay), each(scale)
        if states is None:
            states = [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in self.params]
            if self.params[0].is_cuda:  # steps may run on any stream
                torch.cuda.current_stream(self.params[0].device).synchronize()
        self.states = list(states)
        if not len(self.masters) == len(wd) == len(scales) == len(self.states) == n:
            raise ValueError("one master (or None), weight decay, scale and state per parameter")
        if not 1 <= int(steps) <= MAX_MUON_STEPS:
            raise ValueError(f"steps is 1 to {MAX_MUON_STEPS}, got {steps}")
        triples = [coefs] * int(steps) if not isinstance(coefs[0], (list, tuple)) else list(coefs)
        if len(triples) != steps or any(len(t) != 3 for t in triples):
            raise ValueError("coefs is one (a, b, c), or one for each step")
        p0, g0 = self.params[0], self.grads[0]
        arr = (dlm_muon_param * n)()
        for k, (p, g, w, m) in enumerate(zip(self.params, self.grads, self.masters, self.states)):
            if p.dim() < 2:
                raise ValueError(f"parameter {k} is no matrix: it has {p.dim()} dimension(s)")
            _like(p, f"parameter {k}", p.shape, p0.dtype, p0.device)
            _like(g, f"gradient {k}", p.shape, g0.dtype, p0.device)
            _like(m, f"state {k}", p.shape, torch.float32, p0.device)
            if w is not None:
                _like(w, f"master {k}", p.shape, torch.float32, p0.device)
            rows, cols = p.shape[-2:] if p.numel() else (1, 1)
            count = p.numel() // (rows * cols)
            arr[k] = dlm_muon_param(p.data_ptr(), g.data_ptr(), None if w is None else w.data_ptr(), m.data_ptr(), count,
                                    rows, cols, float(wd[k]), self._scale(scales[k], rows, cols))
        _here(p0, None, "parameter 0")
        h = C.c_void_p()
        _check(load().dlm_muon_create(arr, n, _dt(p0), _dt(g0), C.byref(h)), "dlm_muon_create")
        self._h = h
        self.device = p0.device
        self._cfg = dlm_muon_cfg(0.0, float(momentum), 1 if nesterov else 0, float(eps), int(steps))
        for k, t in enumerate(triples):
            for j in range(3):
                self._cfg.coefs[k][j] = float(t[j])

    @staticmethod
    def _scale(scale, rows, cols) -> float:
        if scale == "shape":
            return max(1.0, rows / max(cols, 1)) ** 0.5
        if scale == "rms":
            return 0.2 * max(rows, cols) ** 0.5
        if isinstance(scale, str):
            raise ValueError(f"scale is 'shape', 'rms' or a number, got {scale!r}")
        return float(scale)

    def step(self, lr: float, lr_scale=None, grad_scale=None, stream=None):
        """One step.  lr_scale / grad_scale: optional fp32 [1] device tensors that
        multiply lr / the gradients, read when the step runs."""
        handle = _here(self.params[0], stream, "parameter 0")
        for t, name in ((lr_scale, "lr_scale"), (grad_scale, "grad_scale")):
            if t is not None:
                _like(t, name, (1,), torch.float32, self.device)
        self._cfg.lr = float(lr)
        _check(load().dlm_muon_step(self._h, C.byref(self._cfg), _ptr(lr_scale), _ptr(grad_scale), handle), "dlm_muon_step")

    def status(self, stream=None) -> int:
        """DLM_OK, or DLM_EDEVICE if some matrix was not finite (and was left unchanged); clears the error."""
        handle = _here(self.params[0], stream, "parameter 0")
        code = C.c_int32(0)
        _check(load().dlm_muon_status(self._h, C.byref(code), handle), "dlm_muon_status")
        return code.value

    def close(self):
        if getattr(self, "_h", None):
            _check(load().dlm_muon_destroy(self._h), "dlm_muon_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass
