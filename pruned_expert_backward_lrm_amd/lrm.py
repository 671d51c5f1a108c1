"""ctypes binding of liblrm.so (the C ABI in include/lrm.h).

Argument marshalling only: every step of the pruned expert backward runs in
the HIP kernels behind the C ABI.  PyTorch provides device memory and the
stream.  Importing this module fails loudly when the library is not built;
there is no fallback implementation.
"""

from __future__ import annotations

import ctypes as C
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblrm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -m pruned_expert_backward_lrm_amd.build`")
_lib = C.CDLL(LIB_PATH)

# ------------------------------------------------------------------ constants
LRM_OK = 0
STATUS_NAMES = ["OK", "ERR_NULL", "ERR_SHAPE", "ERR_DTYPE", "ERR_LAYOUT", "ERR_ALIGN",
                "ERR_QUOTA", "ERR_WORKSPACE", "ERR_INDEX", "ERR_HIP", "ERR_UNSUPPORTED",
                "ERR_INFEASIBLE"]
LRM_ERR_INDEX, LRM_ERR_INFEASIBLE = 8, 11
LRM_F32, LRM_BF16 = 0, 1
LRM_ROWS_TOKEN, LRM_ROWS_PAIR = 0, 1
LRM_LINEAR, LRM_SWIGLU = 0, 1
LRM_KEEP_ALL = 1
LRM_DW_BF16 = 2
LRM_QUOTA_ON_DEVICE = 4
LRM_DEBUG_CHECKS = 8
LRM_GATHER_LOADS = 16
LRM_ROUTE_RENORM = 1
ROWS = {"token": LRM_ROWS_TOKEN, "pair": LRM_ROWS_PAIR}
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_RULES = {"max": 0, "top2": 1}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
LRM_MOMENTS_F32, LRM_MOMENTS_8BIT = 0, 1
MOMENTS = {"m": 0, "v": 1}


class LrmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.lrm_status_string(status).decode()
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{where}: LRM_{name} ({msg})")


# ------------------------------------------------------------------- structs
class lrm_pairs(C.Structure):
    _fields_ = [("T", C.c_int32), ("N", C.c_int32), ("E", C.c_int32), ("_pad", C.c_int32),
                ("token", C.c_void_p), ("expert", C.c_void_p), ("weight", C.c_void_p)]


class lrm_mat(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("dtype", C.c_int32), ("rows", C.c_int32),
                ("cols", C.c_int32), ("_pad", C.c_int32), ("ld", C.c_int64)]


class lrm_problem(C.Structure):
    _fields_ = [("kind", C.c_int32), ("flags", C.c_uint32), ("dtype", C.c_int32),
                ("_pad", C.c_int32), ("pairs", lrm_pairs), ("X", lrm_mat), ("G", lrm_mat),
                ("W", C.c_void_p), ("w_stride", C.c_int64), ("d_in", C.c_int32),
                ("d_out", C.c_int32), ("quota", C.c_void_p), ("A", lrm_mat), ("B", lrm_mat),
                ("W_gate", C.c_void_p), ("W_up", C.c_void_p), ("W_down", C.c_void_p),
                ("H", C.c_int32), ("I", C.c_int32), ("quota_down", C.c_void_p),
                ("quota_gate", C.c_void_p), ("quota_up", C.c_void_p), ("h_sumsq", C.c_void_p)]


class lrm_outputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "dW", "dW_gate", "dW_up", "dW_down", "dX", "score", "pos", "offsets", "score_gate",
        "score_up", "pos_gate", "pos_up", "offsets_gate", "offsets_up", "dH")]


class lrm_router(C.Structure):
    _fields_ = [("T", C.c_int32), ("E", C.c_int32), ("k", C.c_int32), ("score", C.c_int32),
                ("flags", C.c_uint32), ("n_group", C.c_int32), ("topk_group", C.c_int32),
                ("group_rule", C.c_int32), ("scale", C.c_float), ("dtype", C.c_int32),
                ("logits", C.c_void_p), ("ld", C.c_int64), ("bias", C.c_void_p),
                ("expert_mask", C.c_void_p), ("token_mask", C.c_void_p)]


class lrm_forward(C.Structure):
    _fields_ = [("kind", C.c_int32), ("act", C.c_int32), ("dtype", C.c_int32),
                ("_pad", C.c_int32), ("pairs", lrm_pairs), ("X", lrm_mat), ("R", lrm_mat),
                ("W", C.c_void_p), ("w_stride", C.c_int64), ("bias", C.c_void_p),
                ("d_in", C.c_int32), ("d_out", C.c_int32), ("W_gate", C.c_void_p),
                ("W_up", C.c_void_p), ("W_down", C.c_void_p), ("H", C.c_int32),
                ("I", C.c_int32)]


class lrm_forward_outputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("Y", "Yp", "Z", "A", "B", "h_sumsq")]


class lrm_pair_grad_problem(C.Structure):
    _fields_ = [("act", C.c_int32), ("dtype", C.c_int32), ("pairs", lrm_pairs), ("dY", lrm_mat),
                ("Z", lrm_mat)]


class lrm_pair_grad_outputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("dweight", "G", "dbias")]


class lrm_balance(C.Structure):
    _fields_ = [("router", lrm_router), ("expert", C.c_void_p), ("counts", C.c_void_p),
                ("seq", C.c_void_p), ("S", C.c_int32), ("coef", C.c_float), ("z_coef", C.c_float),
                ("_pad", C.c_int32)]


class lrm_param(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("p", "g", "master", "m", "v", "m_exp", "v_exp")] + \
        [("n", C.c_int64), ("lr", C.c_float), ("weight_decay", C.c_float)]


class lrm_params(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n", "p_dtype", "g_dtype", "moments", "masters", "_pad")] + \
        [("param", C.POINTER(lrm_param)), ("table", C.c_void_p), ("chunks", C.c_int64)]


class lrm_adamw_step(C.Structure):
    _fields_ = [(n, C.c_double) for n in ("lr", "beta1", "beta2", "eps", "grad_scale", "max_norm")] + \
        [("step", C.c_int64), ("seed", C.c_uint64), ("sumsq", C.c_void_p), ("n_sumsq", C.c_int32),
         ("_pad", C.c_int32), ("lr_dev", C.c_void_p), ("steps", C.c_void_p)]


_P = C.c_void_p
_SZ = C.c_size_t
_I32 = C.c_int32
_sigs = {
    "lrm_status_string": (C.c_char_p, [C.c_int]),
    "lrm_version": (_I32, []),
    "lrm_max_kept": (C.c_int64, [_I32, _I32, _P]),
    "lrm_score": (C.c_int, [C.POINTER(lrm_pairs), C.POINTER(lrm_mat), C.POINTER(lrm_mat), _P,
                            _P, _SZ, _P]),
    "lrm_score_workspace_size": (_SZ, [C.POINTER(lrm_pairs)]),
    "lrm_score_glu": (C.c_int, [C.POINTER(lrm_pairs), C.POINTER(lrm_mat), C.POINTER(lrm_mat),
                                C.POINTER(lrm_mat), _P, _P, _SZ, _P]),
    "lrm_select": (C.c_int, [C.POINTER(lrm_pairs), _P, _P, C.c_uint32, _P, _P, _P, _P, _SZ, _P]),
    "lrm_select_workspace_size": (_SZ, [C.POINTER(lrm_pairs)]),
    "lrm_compact": (C.c_int, [C.POINTER(lrm_pairs), _P, _P, _I32, C.POINTER(lrm_mat),
                              C.POINTER(lrm_mat), _P, _P, _P]),
    "lrm_compact_rows": (C.c_int, [C.POINTER(lrm_pairs), _P, _P, _I32, _P, C.POINTER(lrm_mat),
                                   C.POINTER(lrm_mat), _P, _P, _P]),
    "lrm_grouped_bwd": (C.c_int, [_I32, _P, _I32, _I32, _P, _P, _P, C.c_int64, _I32, _I32, _P, _P,
                                  _P, _SZ, _P]),
    "lrm_grouped_bwd_workspace_size": (_SZ, [_I32]),
    "lrm_unpermute": (C.c_int, [C.POINTER(lrm_pairs), _P, _P, _I32, _I32, _P, _P, _SZ, _P]),
    "lrm_unpermute_workspace_size": (_SZ, [C.POINTER(lrm_pairs)]),
    "lrm_expert_backward": (C.c_int, [C.POINTER(lrm_problem), C.POINTER(lrm_outputs), _P, _SZ,
                                      _P]),
    "lrm_expert_backward_events": (C.c_int, [C.POINTER(lrm_problem), C.POINTER(lrm_outputs), _P,
                                             _SZ, _P, C.POINTER(C.c_void_p), _I32]),
    "lrm_workspace_size": (_SZ, [C.POINTER(lrm_problem)]),
    "lrm_check_device_errors": (C.c_int, [_P, _P]),
    "lrm_select_static": (C.c_int, [C.POINTER(lrm_pairs), _P, _P, C.c_uint32, _P, _P, _P, _P]),
    "lrm_quota_waterfill": (C.c_int, [_I32, _P, C.c_int64, _P]),
    "lrm_quota_waterfill_device": (C.c_int, [C.POINTER(lrm_pairs), _P, C.c_int64, _P, _P, _SZ,
                                             _P]),
    "lrm_quota_waterfill_device_workspace_size": (_SZ, [C.POINTER(lrm_pairs)]),
    "lrm_redistribute": (C.c_int, [_I32, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ]),
    "lrm_redistribute_workspace_size": (_SZ, [_I32, _I32]),
    "lrm_receiver_layout": (C.c_int, [_I32, _I32, _P, _P, _I32, _P, _P, _P, _P, _SZ, _P]),
    "lrm_receiver_layout_workspace_size": (_SZ, [_I32, _I32]),
    "lrm_route": (C.c_int, [C.POINTER(lrm_router), _P, _P, _P, _P, _P, _SZ, _P]),
    "lrm_route_workspace_size": (_SZ, [C.POINTER(lrm_router)]),
    "lrm_route_bwd": (C.c_int, [C.POINTER(lrm_router), _P, _P, _P, C.c_int64, _P]),
    "lrm_route_share": (C.c_int, [_I32, _I32, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ,
                                  _P]),
    "lrm_route_share_workspace_size": (_SZ, [_I32, _I32]),
    "lrm_expert_forward": (C.c_int, [C.POINTER(lrm_forward), C.POINTER(lrm_forward_outputs), _P,
                                     _SZ, _P]),
    "lrm_forward_workspace_size": (_SZ, [C.POINTER(lrm_forward)]),
    "lrm_pair_grad": (C.c_int, [C.POINTER(lrm_pair_grad_problem),
                                C.POINTER(lrm_pair_grad_outputs), _P, _SZ, _P]),
    "lrm_pair_grad_workspace_size": (_SZ, [C.POINTER(lrm_pair_grad_problem)]),
    "lrm_balance_loss": (C.c_int, [C.POINTER(lrm_balance), _P, _P, _P, _P, _SZ, _P]),
    "lrm_balance_workspace_size": (_SZ, [C.POINTER(lrm_balance)]),
    "lrm_balance_bwd": (C.c_int, [C.POINTER(lrm_balance), _P, _P, _P, _P, C.c_int64, _P]),
    "lrm_params_table": (C.c_int, [C.POINTER(lrm_params), _SZ, _P]),
    "lrm_params_table_size": (_SZ, [_I32]),
    "lrm_grad_sumsq": (C.c_int, [C.POINTER(lrm_params), _P, _P, _SZ, _P]),
    "lrm_sumsq_workspace_size": (_SZ, [C.POINTER(lrm_params)]),
    "lrm_adamw": (C.c_int, [C.POINTER(lrm_params), C.POINTER(lrm_adamw_step), _P]),
    "lrm_moment_read": (C.c_int, [C.c_int64, _I32, _P, _P, _I32, _P, _P]),
}
for _name, (_res, _args) in _sigs.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sigs)


# ------------------------------------------------------------------- helpers
def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream=None, device=None) -> int:
    """The stream's handle; device: where the call's tensors are, which has to be
    the current GPU and the stream's."""
    if stream is None:
        if device is not None and device.index is None:
            raise ValueError(f"the tensors are on {device}, not on a GPU")
        stream = torch.cuda.current_stream()
        if device is not None and stream.device_index != device.index:
            raise ValueError(f"the tensors are on {device}, which is not the current device")
    elif device is not None and not stream.device_index == device.index == torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}: not a GPU, not the current device, or not "
                         "the stream's device")
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != LRM_OK:
        raise LrmError(status, where)


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LRM_BF16
    if t.dtype == torch.float32:
        return LRM_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


class Pairs:
    """The routed pairs of a layer call: device int32 token/expert, fp32 weight."""

    def __init__(self, token: torch.Tensor, expert: torch.Tensor, weight: torch.Tensor,
                 T: int, E: int):
        self.token, self.expert, self.weight = token, expert, weight
        self.T, self.E, self.N = int(T), int(E), int(token.shape[0])
        self.c = lrm_pairs(self.T, self.N, self.E, 0, _ptr(token), _ptr(expert), _ptr(weight))

    @classmethod
    def from_routing(cls, r, device) -> "Pairs":
        return cls(torch.as_tensor(r.token, dtype=torch.int32, device=device),
                   torch.as_tensor(r.expert, dtype=torch.int32, device=device),
                   torch.as_tensor(r.weight, dtype=torch.float32, device=device), r.T, r.E)


def mat(t: torch.Tensor | None, rows: str | int) -> lrm_mat:
    """Describe a row-major device matrix whose rows are addressed via the pairs."""
    if t is None:
        return lrm_mat(None, 0, 0, 0, 0, 0)
    r = ROWS[rows] if isinstance(rows, str) else int(rows)
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("matrices must be 2-D with unit column stride")
    m = lrm_mat(_ptr(t), dtype_code(t), r, t.shape[1], 0, t.stride(0))
    m._tensor = t  # the descriptor keeps its memory alive
    return m


def _scratch(nbytes: int, device, stream):
    """Device scratch for a call on `stream`, allocated on that stream: freed with
    its last reference, it goes to later work of the same stream only."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _ws(nbytes: int, device, ws, stream=None):
    return ws if ws is not None else _scratch(max(int(nbytes), 256), device, stream)


def _quota_arr(q):
    """Quotas as the C ABI takes them: a host int32 array, or (with
    LRM_QUOTA_ON_DEVICE) a contiguous int32 device tensor passed as it is."""
    if isinstance(q, torch.Tensor) and q.is_cuda:
        if q.dtype != torch.int32 or not q.is_contiguous():
            raise ValueError("device quotas must be a contiguous int32 tensor")
        return q
    return np.ascontiguousarray(np.asarray(q, dtype=np.int32))


# ---------------------------------------------------------------- the steps
def lrm_score(pairs: Pairs, X: lrm_mat, G: lrm_mat, score: torch.Tensor, ws=None, stream=None):
    need = _lib.lrm_score_workspace_size(C.byref(pairs.c))
    ws = _ws(need, score.device, ws, stream)
    _check(_lib.lrm_score(C.byref(pairs.c), C.byref(X), C.byref(G), _ptr(score), _ptr(ws),
                          ws.numel(), _stream(stream)), "lrm_score")


def lrm_score_glu(pairs: Pairs, A: lrm_mat, B: lrm_mat, G: lrm_mat, score: torch.Tensor,
                  ws=None, stream=None):
    need = _lib.lrm_score_workspace_size(C.byref(pairs.c))
    ws = _ws(need, score.device, ws, stream)
    _check(_lib.lrm_score_glu(C.byref(pairs.c), C.byref(A), C.byref(B), C.byref(G),
                              _ptr(score), _ptr(ws), ws.numel(), _stream(stream)),
           "lrm_score_glu")


def lrm_select(pairs: Pairs, score, quota, pos, offsets, kept, flags=0, ws=None, stream=None,
               device=None):
    need = _lib.lrm_select_workspace_size(C.byref(pairs.c))
    ws = _ws(need, device or offsets.device, ws, stream)
    q = _quota_arr(quota) if quota is not None else None
    _check(_lib.lrm_select(C.byref(pairs.c), _ptr(score), _ptr(q), flags, _ptr(pos),
                           _ptr(offsets), _ptr(kept), _ptr(ws), ws.numel(), _stream(stream)),
           "lrm_select")
    return ws


def lrm_select_static(pairs: Pairs, score, quota, pos, offsets, kept, flags=0, stream=None):
    """lrm_select with the library's own scratch array (no workspace, no
    allocation)."""
    q = _quota_arr(quota) if quota is not None else None
    _check(_lib.lrm_select_static(C.byref(pairs.c), _ptr(score), _ptr(q), flags, _ptr(pos),
                                  _ptr(offsets), _ptr(kept), _stream(stream)),
           "lrm_select_static")


def lrm_compact(pairs: Pairs, kept, offsets, max_rows: int, X: lrm_mat, G: lrm_mat, Xp, Gp,
                stream=None):
    _check(_lib.lrm_compact(C.byref(pairs.c), _ptr(kept), _ptr(offsets), int(max_rows),
                            C.byref(X), C.byref(G), _ptr(Xp), _ptr(Gp), _stream(stream)),
           "lrm_compact")


def lrm_compact_rows(pairs: Pairs, kept, offsets, max_rows: int, dst, X: lrm_mat, G: lrm_mat,
                     Xp, Gp, stream=None):
    """lrm_compact writing packed row m to row dst[m] (receiver-major rows)."""
    _check(_lib.lrm_compact_rows(C.byref(pairs.c), _ptr(kept), _ptr(offsets), int(max_rows),
                                 _ptr(dst), C.byref(X), C.byref(G), _ptr(Xp), _ptr(Gp),
                                 _stream(stream)),
           "lrm_compact_rows")


def lrm_grouped_bwd(E: int, offsets, max_rows: int, Gp, Xp, W, d_in: int, d_out: int, dW, dXp,
                    dtype=None, w_stride=None, ws=None, stream=None):
    dt = dtype if dtype is not None else dtype_code(Gp)
    if w_stride is None:
        w_stride = d_in * d_out
    need = _lib.lrm_grouped_bwd_workspace_size(int(E))
    ws = _ws(need, offsets.device, ws, stream)
    _check(_lib.lrm_grouped_bwd(int(E), _ptr(offsets), int(max_rows), dt, _ptr(Gp), _ptr(Xp),
                                _ptr(W), int(w_stride), int(d_in), int(d_out), _ptr(dW),
                                _ptr(dXp), _ptr(ws), ws.numel(), _stream(stream)),
           "lrm_grouped_bwd")


def lrm_unpermute(pairs: Pairs, pos, dXp, d_in: int, out_rows, dX, ws=None, stream=None):
    need = _lib.lrm_unpermute_workspace_size(C.byref(pairs.c))
    ws = _ws(need, dX.device, ws, stream)
    r = ROWS[out_rows] if isinstance(out_rows, str) else int(out_rows)
    _check(_lib.lrm_unpermute(C.byref(pairs.c), _ptr(pos), _ptr(dXp), int(d_in), r, _ptr(dX),
                              _ptr(ws), ws.numel(), _stream(stream)), "lrm_unpermute")


def lrm_max_kept(N: int, quota) -> int:
    q = _quota_arr(quota)
    return int(_lib.lrm_max_kept(int(N), int(q.shape[0]), q.ctypes.data))


def lrm_quota_waterfill(counts, budget: int) -> np.ndarray:
    """Host call: water-filling quotas [E] for candidate counts [E] under a
    pair budget."""
    n = np.ascontiguousarray(np.asarray(counts, dtype=np.int32))
    q = np.zeros_like(n)
    _check(_lib.lrm_quota_waterfill(int(n.shape[0]), _ptr(n), int(budget), _ptr(q)),
           "lrm_quota_waterfill")
    return q


def lrm_quota_waterfill_device(pairs: Pairs, budget: int, quota, counts=None, ws=None,
                               stream=None):
    """Device call: water-filling quotas written to the device int32 [E] tensor
    `quota`, from device counts [E] or (counts None) the pairs' own counts.
    Returns the workspace (its error word reports pairs out of range)."""
    need = _lib.lrm_quota_waterfill_device_workspace_size(C.byref(pairs.c))
    ws = _ws(need, quota.device, ws, stream)
    _check(_lib.lrm_quota_waterfill_device(C.byref(pairs.c), _ptr(counts), int(budget),
                                           _ptr(quota), _ptr(ws), ws.numel(), _stream(stream)),
           "lrm_quota_waterfill_device")
    return ws


def lrm_redistribute(kept, replica, base=None, cap=None):
    """Host call: the peak-minimising integer assignment of each expert's kept
    pairs to its replicas.  kept [E], replica [E][G] (bool), base/cap [G] or
    None.  Returns (peak, assign int32 [E][G]) as NumPy."""
    k = np.ascontiguousarray(np.asarray(kept, dtype=np.int32))
    rep = np.ascontiguousarray(np.asarray(replica).astype(np.uint8))
    E, G = rep.shape
    b = None if base is None else np.ascontiguousarray(np.asarray(base, dtype=np.int64))
    c = None if cap is None else np.ascontiguousarray(np.asarray(cap, dtype=np.int64))
    assign = np.zeros((E, G), np.int32)
    peak = np.zeros(1, np.int64)
    ws = np.empty(max(int(_lib.lrm_redistribute_workspace_size(E, G)), 64), np.uint8)
    _check(_lib.lrm_redistribute(E, G, _ptr(k), _ptr(rep), _ptr(b), _ptr(c), _ptr(assign),
                                 _ptr(peak), _ptr(ws), ws.nbytes), "lrm_redistribute")
    return int(peak[0]), assign


def lrm_receiver_layout(offsets, assign, max_rows: int, ws=None, stream=None):
    """Device call: receiver-major layout of the packed rows for a device
    assignment [E][G].  Returns (send_off [G+1], blk_off [G][E+1], dst
    [max_rows], ws) device int32 tensors."""
    E, G = int(assign.shape[0]), int(assign.shape[1])
    dev = offsets.device
    i32 = dict(dtype=torch.int32, device=dev)
    send_off = torch.empty(G + 1, **i32)
    blk_off = torch.empty(G, E + 1, **i32)
    dst = torch.empty(max(int(max_rows), 1), **i32)
    ws = _ws(_lib.lrm_receiver_layout_workspace_size(E, G), dev, ws, stream)
    _check(_lib.lrm_receiver_layout(E, G, _ptr(offsets), _ptr(assign), int(max_rows),
                                    _ptr(send_off), _ptr(blk_off), _ptr(dst), _ptr(ws),
                                    ws.numel(), _stream(stream)), "lrm_receiver_layout")
    return send_off, blk_off, dst, ws


def lrm_check_device_errors(ws, stream=None) -> int:
    return int(_lib.lrm_check_device_errors(_ptr(ws), _stream(stream)))


# ---------------------------------------------------------- the fused call
class Problem:
    """An lrm_problem plus the objects that keep its memory alive."""

    def __init__(self, kind: int, pairs: Pairs, dtype: int, flags: int = 0):
        self.keep = [pairs]
        self.c = lrm_problem()
        self.c.kind, self.c.flags, self.c.dtype = kind, flags, dtype
        self.c.pairs = pairs.c
        self.pairs = pairs

    def hold(self, *objs):
        self.keep.extend(objs)


def linear_problem(pairs: Pairs, X, x_rows, G, g_rows, W, quota, flags=0) -> Problem:
    pb = Problem(LRM_LINEAR, pairs, dtype_code(X), flags)
    q = _quota_arr(quota) if quota is not None else None
    pb.hold(X, G, W, q)
    c = pb.c
    c.X, c.G = mat(X, x_rows), mat(G, g_rows)
    c.W, c.w_stride = _ptr(W), W.stride(0)
    c.d_in, c.d_out = X.shape[1], G.shape[1]
    c.quota = _ptr(q)
    return pb


def swiglu_problem(pairs: Pairs, X, x_rows, G, g_rows, A, B, W_gate, W_up, W_down,
                   quota_down, quota_gate, quota_up, flags=0, h_sumsq=None) -> Problem:
    pb = Problem(LRM_SWIGLU, pairs, dtype_code(X), flags)
    qs = [(_quota_arr(q) if q is not None else None) for q in (quota_down, quota_gate, quota_up)]
    pb.hold(X, G, A, B, W_gate, W_up, W_down, *qs, h_sumsq)
    pb.c.h_sumsq = _ptr(h_sumsq)
    c = pb.c
    c.X, c.G = mat(X, x_rows), mat(G, g_rows)
    c.A, c.B = mat(A, "pair"), mat(B, "pair")
    c.W_gate, c.W_up, c.W_down = _ptr(W_gate), _ptr(W_up), _ptr(W_down)
    c.H, c.I = X.shape[1], A.shape[1]
    c.quota_down, c.quota_gate, c.quota_up = (_ptr(q) for q in qs)
    return pb


def lrm_workspace_size(pb: Problem) -> int:
    return int(_lib.lrm_workspace_size(C.byref(pb.c)))


def _outputs(outputs: dict) -> lrm_outputs:
    o = lrm_outputs()
    for k, v in outputs.items():
        setattr(o, k, _ptr(v))
    return o


def _fused_ws(pb: Problem, ws, stream=None):
    if ws is not None:
        return ws
    n = lrm_workspace_size(pb)
    if n == 0:
        raise LrmError(2, "lrm_workspace_size")
    return _scratch(n, pb.pairs.token.device, stream)


def lrm_expert_backward(pb: Problem, outputs: dict, ws=None, stream=None):
    o = _outputs(outputs)
    ws = _fused_ws(pb, ws, stream)
    _check(_lib.lrm_expert_backward(C.byref(pb.c), C.byref(o), _ptr(ws), ws.numel(),
                                    _stream(stream)), "lrm_expert_backward")
    return ws


def lrm_expert_backward_events(pb: Problem, outputs: dict, events, ws=None, stream=None):
    """The fused call recording torch.cuda.Event objects at stage boundaries
    (each event must have been recorded once so that its handle exists)."""
    o = _outputs(outputs)
    ws = _fused_ws(pb, ws, stream)
    arr = (C.c_void_p * len(events))(*[ev.cuda_event for ev in events])
    _check(_lib.lrm_expert_backward_events(C.byref(pb.c), C.byref(o), _ptr(ws), ws.numel(),
                                           _stream(stream), arr, len(events)),
           "lrm_expert_backward_events")
    return ws


# -------------------------------------------------------------- the router
class Router:
    """An lrm_router over logits [T][E] (fp32 or bf16, unit column stride) plus
    the tensors that keep its memory alive.  bias: fp32 [E]; expert_mask [E]
    and token_mask [T]: uint8 or bool, nonzero where the expert or token takes
    part."""

    def __init__(self, logits: torch.Tensor, k: int, score: str = "softmax", renorm: bool = True,
                 scale: float = 1.0, n_group: int = 1, topk_group: int = 1,
                 group_rule: str = "top2", bias=None, expert_mask=None, token_mask=None):
        if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
            raise ValueError("logits must be 2-D with unit column stride")
        T, E = logits.shape
        for name, t, n, dts in (("bias", bias, E, (torch.float32,)),
                                ("expert_mask", expert_mask, E, (torch.uint8, torch.bool)),
                                ("token_mask", token_mask, T, (torch.uint8, torch.bool))):
            if t is not None and (t.dtype not in dts or t.shape != (n,) or not t.is_contiguous()
                                  or t.device != logits.device):
                raise ValueError(f"{name} must be a contiguous {dts[0]} tensor of {n} entries "
                                 "on the logits' device")
        self.T, self.E, self.k = int(T), int(E), int(k)
        self.device = logits.device
        self.keep = [logits, bias, expert_mask, token_mask]
        ld = logits.stride(0) if T > 1 else max(logits.stride(0), E)
        self.c = lrm_router(self.T, self.E, self.k, SCORES[score],
                            LRM_ROUTE_RENORM if renorm else 0, int(n_group), int(topk_group),
                            GROUP_RULES[group_rule], float(scale), dtype_code(logits),
                            _ptr(logits), ld, _ptr(bias), _ptr(expert_mask), _ptr(token_mask))
        self.ws_bytes = int(_lib.lrm_route_workspace_size(C.byref(self.c)))


def _slots(name, t, n, dtype, device):
    """A dense array of at least n entries of a type on a device, or None."""
    if t is not None and (t.dtype != dtype or t.numel() < n or not t.is_contiguous()
                          or t.device != device):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {n} entries "
                         f"on {device}")


def lrm_route(r: Router, expert, weight, token=None, counts=None, ws=None, stream=None):
    """The k experts of every token (int32 [T*k], -1 in empty slots) and their
    weights (fp32 [T*k]); optionally the slots' tokens and the experts' counts."""
    n, on = r.T * r.k, r.device
    _slots("expert", expert, n, torch.int32, on)
    _slots("weight", weight, n, torch.float32, on)
    _slots("token", token, n, torch.int32, on)
    _slots("counts", counts, r.E, torch.int32, on)
    if counts is not None:
        ws = _ws(r.ws_bytes, counts.device, ws, stream)
    _check(_lib.lrm_route(C.byref(r.c), _ptr(expert), _ptr(weight), _ptr(token), _ptr(counts),
                          _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream, on)),
           "lrm_route")


def lrm_route_bwd(r: Router, expert, dweight, dlogits: torch.Tensor, stream=None):
    """Gradient of the logits (their dtype, [T][E]) from the gradient of the
    weights (fp32 [T*k]) of a choice (int32 [T*k])."""
    n = r.T * r.k
    _slots("expert", expert, n, torch.int32, r.device)
    _slots("dweight", dweight, n, torch.float32, r.device)
    if dlogits.shape != (r.T, r.E) or (r.E > 1 and dlogits.stride(1) != 1) or \
            dtype_code(dlogits) != r.c.dtype or dlogits.device != r.device:
        raise ValueError("dlogits must be [T][E] of the logits' dtype with unit column stride "
                         "on the logits' device")
    ldd = dlogits.stride(0) if r.T > 1 else max(dlogits.stride(0), r.E)
    _check(_lib.lrm_route_bwd(C.byref(r.c), _ptr(expert), _ptr(dweight), _ptr(dlogits), ldd,
                              _stream(stream, r.device)), "lrm_route_bwd")


def lrm_route_share(T: int, k: int, expert, weight, e0: int, E: int, out_token, out_expert,
                    out_weight, out_n, out_slot=None, ws=None, stream=None):
    """The pairs of the experts [e0, e0 + E), in slot order: token, local
    expert, weight and slot arrays [T*k] (the first out_n[0] entries)."""
    n = int(T) * int(k)
    for name, t, m, dt in (("expert", expert, n, torch.int32), ("weight", weight, n, torch.float32),
                           ("out_token", out_token, n, torch.int32),
                           ("out_expert", out_expert, n, torch.int32),
                           ("out_weight", out_weight, n, torch.float32),
                           ("out_slot", out_slot, n, torch.int32), ("out_n", out_n, 1, torch.int32)):
        _slots(name, t, m, dt, out_n.device)
    ws = _ws(_lib.lrm_route_share_workspace_size(int(T), int(k)), out_n.device, ws, stream)
    _check(_lib.lrm_route_share(int(T), int(k), _ptr(expert), _ptr(weight), int(e0), int(E),
                                _ptr(out_token), _ptr(out_expert), _ptr(out_weight),
                                _ptr(out_slot), _ptr(out_n), _ptr(ws), ws.numel(),
                                _stream(stream, out_n.device)), "lrm_route_share")


# ----------------------------------------------- balance of the experts' load
class Balance:
    """An lrm_balance over a Router plus the tensors that keep its memory alive.
    expert: int32 [T*k], the choice; counts: int32 [S][E] slots per expert (of
    lrm_route, or summed over GPUs), None: from the choice; seq: int32 [S+1],
    the sequences' offsets, None: one sequence of all tokens."""

    def __init__(self, router: Router, expert=None, counts=None, seq=None, coef: float = 0.01,
                 z_coef: float = 0.0):
        on = router.device
        _slots("expert", expert, router.T * router.k, torch.int32, on)
        if seq is not None:
            if seq.dim() != 1 or seq.numel() < 2:
                raise ValueError("seq must hold the offsets of one sequence at least")
            _slots("seq", seq, 2, torch.int32, on)
        self.S = 1 if seq is None else int(seq.numel()) - 1
        _slots("counts", counts, self.S * router.E, torch.int32, on)
        self.router = router
        self.keep = [router, expert, counts, seq]
        self.has_expert, self.has_counts = expert is not None, counts is not None
        self.c = lrm_balance(router.c, _ptr(expert), _ptr(counts), _ptr(seq), self.S, float(coef),
                             float(z_coef), 0)


def lrm_balance_workspace_size(b: Balance) -> int:
    return int(_lib.lrm_balance_workspace_size(C.byref(b.c)))


def lrm_balance_loss(b: Balance, loss, saved, counts=None, ws=None, stream=None):
    """The balance loss and the z loss (fp32 loss[2]), what their gradient needs
    (fp32 saved[S*E + 2]) and, where b has none, the counts (int32 [S][E])."""
    on = b.router.device
    _slots("loss", loss, 2, torch.float32, on)
    _slots("saved", saved, b.S * b.router.E + 2, torch.float32, on)
    _slots("counts", counts, b.S * b.router.E, torch.int32, on)
    if ws is None:
        ws = _grown(lrm_balance_workspace_size(b), on, stream)
    _check(_lib.lrm_balance_loss(C.byref(b.c), _ptr(loss), _ptr(saved), _ptr(counts), _ptr(ws),
                                 ws.numel() if ws is not None else 0, _stream(stream, on)),
           "lrm_balance_loss")


def lrm_balance_bwd(b: Balance, saved, dlogits: torch.Tensor, dloss=None, dweight=None, stream=None):
    """Gradient of the logits (their dtype, [T][E]): of both losses, from their
    gradients (fp32 dloss[2], None: ones), and with dweight (fp32 [T*k]) of the
    routing weights too, in place of lrm_route_bwd."""
    r = b.router
    _slots("saved", saved, b.S * r.E + 2, torch.float32, r.device)
    _slots("dloss", dloss, 2, torch.float32, r.device)
    _slots("dweight", dweight, r.T * r.k, torch.float32, r.device)
    if dlogits.shape != (r.T, r.E) or (r.E > 1 and dlogits.stride(1) != 1) or \
            dtype_code(dlogits) != r.c.dtype or dlogits.device != r.device:
        raise ValueError("dlogits must be [T][E] of the logits' dtype with unit column stride "
                         "on the logits' device")
    ldd = dlogits.stride(0) if r.T > 1 else max(dlogits.stride(0), r.E)
    _check(_lib.lrm_balance_bwd(C.byref(b.c), _ptr(saved), _ptr(dloss), _ptr(dweight), _ptr(dlogits),
                                ldd, _stream(stream, r.device)), "lrm_balance_bwd")


# ------------------------------------------------------ the experts forward
class Forward:
    """An lrm_forward plus the objects that keep its memory alive."""

    def __init__(self, kind: int, pairs: Pairs, X, x_rows, residual, act: str = "none"):
        _rows("X", X, x_rows, pairs)
        _rows("residual", residual, "token", pairs)
        self.pairs = pairs
        self.keep = [pairs, X, residual]
        self.c = lrm_forward()
        self.c.kind, self.c.act, self.c.dtype = kind, ACTS[act], dtype_code(X)
        self.c.pairs, self.c.X = pairs.c, mat(X, x_rows)
        self.c.R = mat(residual, "token")


def _rows(name, t, rows, pairs):
    """A row of t for every token or pair, on the pairs' device."""
    if t is None:
        return
    need = pairs.T if rows in ("token", ROWS["token"]) else pairs.N
    if t.shape[0] < need or t.device != pairs.token.device:
        raise ValueError(f"{name} must have at least {need} rows on the pairs' device")


def _dense(name, t, shape, dtype, device):
    if t.device != device:
        raise ValueError(f"{name} must be on the pairs' device")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def linear_forward(pairs: Pairs, X, x_rows, W, act="none", bias=None, residual=None) -> Forward:
    """y_p = act(W_e x_p + bias_e) with W [E][d_out][d_in], bias [E][d_out]."""
    if W.dim() != 3 or W.shape[0] != pairs.E or W.dtype != X.dtype or W.stride(2) != 1 or \
            W.stride(1) != W.shape[2] or W.shape[2] != X.shape[1] or \
            W.device != pairs.token.device:
        raise ValueError("W must be [E][d_out][d_in] of X's dtype, dense inside an expert, "
                         "on the pairs' device")
    # (the stride of one expert says nothing)
    stride = W.stride(0) if pairs.E > 1 else W.shape[1] * W.shape[2]
    if stride < W.shape[1] * W.shape[2]:
        raise ValueError("the experts of W must not share memory (an expanded W: call contiguous)")
    if bias is not None:
        _dense("bias", bias, W.shape[:2], X.dtype, pairs.token.device)
    f = Forward(LRM_LINEAR, pairs, X, x_rows, residual, act)
    f.keep += [W, bias]
    c = f.c
    c.W, c.w_stride = _ptr(W), stride
    c.bias = _ptr(bias)
    c.d_in, c.d_out = W.shape[2], W.shape[1]
    f.sizes = {"Y": (X.dtype, pairs.T * c.d_out), "Yp": (X.dtype, pairs.N * c.d_out),
               "Z": (X.dtype, pairs.N * c.d_out)}
    return f


def swiglu_forward(pairs: Pairs, X, W_gate, W_up, W_down, residual=None) -> Forward:
    """y_p = W_down (silu(W_gate x) * (W_up x)), weights as in swiglu_problem."""
    H, I = X.shape[1], W_gate.shape[1]  # noqa: E741
    for name, w, shape in (("W_gate", W_gate, (pairs.E, I, H)), ("W_up", W_up, (pairs.E, I, H)),
                           ("W_down", W_down, (pairs.E, H, I))):
        _dense(name, w, shape, X.dtype, pairs.token.device)
    f = Forward(LRM_SWIGLU, pairs, X, "token", residual)
    f.keep += [W_gate, W_up, W_down]
    c = f.c
    c.W_gate, c.W_up, c.W_down = _ptr(W_gate), _ptr(W_up), _ptr(W_down)
    c.H, c.I = H, I
    f.sizes = {"Y": (X.dtype, pairs.T * H), "Yp": (X.dtype, pairs.N * H),
               "A": (X.dtype, pairs.N * I), "B": (X.dtype, pairs.N * I),
               "h_sumsq": (torch.float64, pairs.N)}
    return f


def lrm_forward_workspace_size(f: Forward) -> int:
    return int(_lib.lrm_forward_workspace_size(C.byref(f.c)))


def _marshal(struct, outputs: dict):
    o = struct()
    o._fits = None  # the problem whose sizes were checked last
    o._tensors = dict(outputs)  # the descriptor keeps its memory alive
    for k, v in outputs.items():
        if v is not None and not v.is_contiguous():
            raise ValueError(f"output {k} must be contiguous")
        setattr(o, k, _ptr(v))
    return o


def _check_outputs(o, problem):
    """The outputs have the problem's types, sizes and device."""
    if o._fits is problem:
        return
    for k, t in o._tensors.items():
        if t is None or k not in problem.sizes:  # (the call refuses what its kind does not have)
            continue
        dtype, n = problem.sizes[k]
        if t.dtype != dtype or t.numel() != n or t.device != problem.pairs.token.device:
            raise ValueError(f"output {k} must be {n} elements of {dtype} on the pairs' device")
    o._fits = problem


def forward_outputs(outputs: dict) -> lrm_forward_outputs:
    """The outputs of lrm_expert_forward (Y, Yp, Z, A, B, h_sumsq), marshalled
    once for several calls."""
    return _marshal(lrm_forward_outputs, outputs)


def _grown(need, device, stream):
    return _scratch(need, device, stream) if need else None


def lrm_expert_forward(f: Forward, outputs, ws=None, stream=None):
    """The experts' forward pass; outputs: a dict or forward_outputs(dict)."""
    o = forward_outputs(outputs) if isinstance(outputs, dict) else outputs
    _check_outputs(o, f)
    if ws is None:
        ws = _grown(lrm_forward_workspace_size(f), f.pairs.token.device, stream)
    _check(_lib.lrm_expert_forward(C.byref(f.c), C.byref(o), _ptr(ws),
                                   ws.numel() if ws is not None else 0,
                                   _stream(stream, f.pairs.token.device)),
           "lrm_expert_forward")
    return ws


# -------------------------------------------------- the epilogue's backward
class PairGrad:
    """An lrm_pair_grad_problem plus the objects that keep its memory alive."""

    def __init__(self, pairs: Pairs, dY, dy_rows, Z, act: str):
        _rows("dY", dY, dy_rows, pairs)
        _rows("Z", Z, "pair", pairs)
        self.pairs = pairs
        self.keep = [pairs, dY, Z]
        d = Z.shape[1]
        self.sizes = {"dweight": (torch.float32, pairs.N), "G": (Z.dtype, pairs.N * d),
                      "dbias": (torch.float32, pairs.E * d)}
        self.c = lrm_pair_grad_problem(ACTS[act], dtype_code(Z), pairs.c, mat(dY, dy_rows),
                                       mat(Z, "pair"))


def pair_grad_problem(pairs: Pairs, dY, dy_rows, Z, act="none") -> PairGrad:
    return PairGrad(pairs, dY, dy_rows, Z, act)


def lrm_pair_grad_workspace_size(g: PairGrad) -> int:
    return int(_lib.lrm_pair_grad_workspace_size(C.byref(g.c)))


def pair_grad_outputs(outputs: dict) -> lrm_pair_grad_outputs:
    """The outputs of lrm_pair_grad (dweight, G, dbias), marshalled once."""
    return _marshal(lrm_pair_grad_outputs, outputs)


def lrm_pair_grad(g: PairGrad, outputs, ws=None, stream=None):
    """Gradients of the routing weights, the projection's output and the bias;
    outputs: a dict or pair_grad_outputs(dict)."""
    o = pair_grad_outputs(outputs) if isinstance(outputs, dict) else outputs
    _check_outputs(o, g)
    if ws is None:
        ws = _grown(lrm_pair_grad_workspace_size(g), g.pairs.token.device, stream)
    _check(_lib.lrm_pair_grad(C.byref(g.c), C.byref(o), _ptr(ws),
                              ws.numel() if ws is not None else 0,
                              _stream(stream, g.pairs.token.device)),
           "lrm_pair_grad")
    return ws


# ---------------------------------------------- update of the parameters
def _apart(spans):
    """Refuses arrays that share memory, where one of them is written.  spans:
    (name, addresses, bytes, written) a list of arrays."""
    lo = np.concatenate([p for _, p, _, _ in spans])
    hi = lo + np.concatenate([n for _, _, n, _ in spans])
    w = np.concatenate([np.full(len(p), x) for _, p, _, x in spans])
    at = np.nonzero(hi > lo)[0]
    at = at[np.argsort(lo[at], kind="stable")]
    lo, hi, w = lo[at], hi[at], w[at]
    # the end of what starts before: of everything, and of what is written
    end = np.concatenate([[0], np.maximum.accumulate(hi)[:-1]]) if len(hi) else hi
    end_w = np.concatenate([[0], np.maximum.accumulate(np.where(w, hi, 0))[:-1]]) if len(hi) else hi
    bad = np.nonzero(lo < np.where(w, end, end_w))[0]
    if len(bad):
        i = int(at[bad[0]])
        for name, p, _, _ in spans:
            if i < len(p):
                raise ValueError(f"{name}[{i}] shares memory with another tensor of the list")
            i -= len(p)


class Params:
    """Tensors that are updated together: an lrm_params, its table on the GPU
    (written on the given or the current stream) and the tensors themselves.

    g: their gradients (fp32 or bf16, all alike); p: the weights (fp32 or bf16);
    m, v: the moments, fp32, or uint8 codes with the blocks' exponents m_exp and
    v_exp (uint8 [(n + 31) // 32] each); master: fp32 weights behind bf16 p; lr,
    weight_decay: a number for all, or one each.  All lists have one entry a
    tensor; entries are contiguous.  With g alone: for lrm_grad_sumsq."""

    def __init__(self, g, p=None, m=None, v=None, master=None, m_exp=None, v_exp=None, lr=1.0,
                 weight_decay=0.0, stream=None):
        g = list(g)
        n = len(g)
        lists = {"p": p, "master": master, "m": m, "v": v, "m_exp": m_exp, "v_exp": v_exp}
        lists = {"g": g, **{k: list(x) for k, x in lists.items() if x is not None}}
        if not g:
            raise ValueError("at least one tensor is wanted")
        self.device = g[0].device
        eight = "m_exp" in lists
        moment = torch.uint8 if eight else torch.float32
        want = {"g": g[0].dtype, "p": lists["p"][0].dtype if lists.get("p") else None,
                "master": torch.float32, "m": moment, "v": moment, "m_exp": torch.uint8,
                "v_exp": torch.uint8}
        counts = [t.numel() for t in g]
        blocks = [(x + 31) // 32 for x in counts]
        self.param = (lrm_param * n)()
        rows = np.frombuffer(self.param, dtype=np.dtype(lrm_param))
        rows["n"] = counts
        spans = []
        for name, ts in lists.items():
            if len(ts) != n:
                raise ValueError(f"{name} must have {n} tensors, as g has")
            dt, sizes = want[name], blocks if name.endswith("_exp") else counts
            for i, (t, x) in enumerate(zip(ts, sizes)):
                if t.dtype is not dt or t.numel() != x or t.device != self.device or \
                        not t.is_contiguous():
                    raise ValueError(f"{name}[{i}] must be a contiguous {dt} tensor of {x} elements "
                                     f"on {self.device}")
            at = np.array([t.data_ptr() for t in ts], np.int64)
            rows[name] = at
            spans.append((name, at, np.array(sizes, np.int64) * ts[0].element_size(), name != "g"))
        # (what is written lies apart from everything; gradients may share memory)
        _apart(spans)

        def each(x, name):
            x = [float(y) for y in x] if isinstance(x, (list, tuple)) else [float(x)] * n
            if len(x) != n:
                raise ValueError(f"{name} must be a number or {n} of them")
            return x

        rows["lr"], rows["weight_decay"] = each(lr, "lr"), each(weight_decay, "weight_decay")
        self.n = n
        self.keep = lists
        self.table = _scratch(int(_lib.lrm_params_table_size(n)), self.device, stream)
        self.c = lrm_params(n, dtype_code(lists["p"][0]) if lists.get("p") else LRM_F32,
                            dtype_code(g[0]), LRM_MOMENTS_8BIT if eight else LRM_MOMENTS_F32,
                            int("master" in lists), 0, self.param, _ptr(self.table), 0)
        _check(_lib.lrm_params_table(C.byref(self.c), self.table.numel(),
                                     _stream(stream, self.device)), "lrm_params_table")


def lrm_sumsq_workspace_size(ps: Params) -> int:
    return int(_lib.lrm_sumsq_workspace_size(C.byref(ps.c)))


def lrm_grad_sumsq(ps: Params, sumsq, ws=None, stream=None):
    """The sum of squares of all gradients (fp64 sumsq[0])."""
    _slots("sumsq", sumsq, 1, torch.float64, ps.device)
    if ws is None:
        ws = _grown(lrm_sumsq_workspace_size(ps), ps.device, stream)
    _check(_lib.lrm_grad_sumsq(C.byref(ps.c), _ptr(sumsq), _ptr(ws),
                               ws.numel() if ws is not None else 0, _stream(stream, ps.device)),
           "lrm_grad_sumsq")


class AdamW:
    """An lrm_adamw_step: the settings of lrm_adamw, and the device tensors that
    it reads.  lr: a number, or an fp32 tensor of one entry on the GPU (read when
    the step runs); sumsq: fp64, sums of squares of the gradients (all entries are
    added): for clipping to max_norm (0: none), and a step whose sum is not
    finite is left out; steps: int64 tensor of one entry, counted by the calls."""

    def __init__(self, lr=1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 seed: int = 0, grad_scale: float = 1.0, max_norm: float = 0.0, sumsq=None,
                 steps=None):
        lr_dev = lr if isinstance(lr, torch.Tensor) else None
        for name, t, dt in (("lr", lr_dev, torch.float32), ("steps", steps, torch.int64)):
            if t is not None and (t.dtype != dt or t.numel() != 1):
                raise ValueError(f"{name} must be one {dt} value")
        if sumsq is not None and (sumsq.dtype != torch.float64 or not sumsq.is_contiguous()):
            raise ValueError("sumsq must be a contiguous torch.float64 tensor")
        self.keep = [t for t in (lr_dev, sumsq, steps) if t is not None]
        self.c = lrm_adamw_step(0.0 if lr_dev is not None else float(lr), float(beta1), float(beta2),
                                float(eps), float(grad_scale), float(max_norm), 0,
                                int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(sumsq),
                                0 if sumsq is None else sumsq.numel(), 0, _ptr(lr_dev), _ptr(steps))


def lrm_adamw(ps: Params, opt: AdamW, step: int = 0, stream=None):
    """One AdamW step over all tensors; step: its number, from 1 (not read where
    opt counts the steps on the GPU)."""
    for t in opt.keep:
        if t.device != ps.device:
            raise ValueError(f"the step's tensors must be on {ps.device}")
    opt.c.step = int(step)
    _check(_lib.lrm_adamw(C.byref(ps.c), C.byref(opt.c), _stream(stream, ps.device)), "lrm_adamw")


def lrm_moment_read(codes, exps, out, which: str, stream=None):
    """The values that 8-bit moments (uint8 codes [n], exponents [(n + 31) // 32])
    stand for; which: "m" or "v"; out: fp32 or bf16 [n]."""
    n = out.numel()
    _slots("codes", codes, n, torch.uint8, out.device)
    _slots("exps", exps, (n + 31) // 32, torch.uint8, out.device)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    _check(_lib.lrm_moment_read(n, MOMENTS[which], _ptr(codes), _ptr(exps), dtype_code(out), _ptr(out),
                                _stream(stream, out.device)), "lrm_moment_read")
