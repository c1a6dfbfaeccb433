"""Thin ctypes binding of libep.so (C ABI in include/ep.h).

The functions keep the C names and only marshal arguments. torch tensors
become device pointers, the current torch stream becomes `stream`, and a
non-OK status raises EpError. Every step of the path runs in the library's
CUDA kernels. Importing this module loads the library and raises
ImportError if it is missing: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m combine_top_group_b200.build` "
        "(nvcc, sm_100a). The library has no CPU fallback.")

_lib = ctypes.CDLL(LIB_PATH)

EP_OK, EP_ERR_INVALID, EP_ERR_CAPACITY, EP_ERR_OOM, EP_ERR_CUDA, EP_ERR_UNSUPPORTED, EP_ERR_DEVICE = range(7)
EP_DEVERR_EXPERT_ID, EP_DEVERR_ROW_BOUNDS, EP_DEVERR_TIMEOUT = 0x1, 0x2, 0x4
EP_FLAG_FP8 = 0x1
EP_FLAG_LOW_LATENCY = 0x2
EP_FLAG_DEDUP = 0x4
EP_FLAG_SHARD = 0x8
EP_ROUTE_SOFTMAX, EP_ROUTE_SOFTMAX_RENORM, EP_ROUTE_GROUP_SIGMOID = 0, 1, 2
EP_DTYPE_BF16, EP_DTYPE_FP32, EP_DTYPE_E4M3 = 0, 1, 2
EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
EP_ACT_NONE, EP_ACT_SILU, EP_ACT_GELU, EP_ACT_SWIGLU = 0, 1, 2, 3


class EpConfig(ctypes.Structure):
    _fields_ = [("num_ranks", ctypes.c_int32), ("max_tokens_per_rank", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class EpLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_idx", "topk_w", "is_token_in_rank", "num_tokens_per_rank", "cnt_src_expert",
        "num_tokens_per_expert", "expert_off", "rank_off", "src_off", "dst_row")]


class EpLinear(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "x", "x_scale", "w", "w_scale", "bias", "residual", "out", "out_scale")] + \
        [(n, ctypes.c_int32) for n in ("in_features", "out_features", "act", "out_type")]


_P = ctypes.c_void_p
_st = ctypes.c_int
_lib.ep_abi_version.restype = ctypes.c_int
_lib.ep_status_string.argtypes = [_st]
_lib.ep_status_string.restype = ctypes.c_char_p
_lib.ep_last_error_message.restype = ctypes.c_char_p
_lib.ep_default_config.argtypes = [ctypes.c_int] * 5
_lib.ep_default_config.restype = EpConfig
_lib.ep_buffer_workspace_bytes.argtypes = [ctypes.POINTER(EpConfig), ctypes.POINTER(ctypes.c_size_t)]
_lib.ep_buffer_workspace_bytes.restype = _st
_lib.ep_buffer_create.argtypes = [ctypes.POINTER(EpConfig), _P, ctypes.c_size_t, ctypes.POINTER(_P)]
_lib.ep_buffer_create.restype = _st
_lib.ep_buffer_destroy.argtypes = [_P]
_lib.ep_buffer_destroy.restype = _st
_lib.ep_buffer_set_num_sms.argtypes = [_P, ctypes.c_int]
_lib.ep_buffer_set_num_sms.restype = _st
_lib.ep_buffer_layout.argtypes = [_P, ctypes.POINTER(EpLayout)]
_lib.ep_buffer_layout.restype = _st
_lib.ep_buffer_recv.argtypes = [_P, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P),
                                ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_int64)]
_lib.ep_buffer_recv.restype = _st
_lib.ep_get_layout.argtypes = [_P, ctypes.c_int, _P, _P, _P, ctypes.c_int, ctypes.c_uint64, ctypes.c_float, _P]
_lib.ep_get_layout.restype = _st
_lib.ep_dispatch.argtypes = [_P, ctypes.c_int, _P, _P]
_lib.ep_dispatch.restype = _st
_lib.ep_combine.argtypes = [_P, ctypes.c_int, _P, _P, _P, _P]
_lib.ep_combine.restype = _st
_lib.ep_check_errors.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int, _P]
_lib.ep_check_errors.restype = _st
_lib.ep_get_layout_noalloc.argtypes = [ctypes.POINTER(EpConfig), ctypes.c_int, _P, _P, _P, ctypes.c_int,
                                       ctypes.c_uint64, ctypes.c_float, ctypes.POINTER(EpLayout), _P, _P]
_lib.ep_get_layout_noalloc.restype = _st
_lib.ep_buffer_dedup.argtypes = [_P] + [ctypes.POINTER(_P)] * 9 + [ctypes.POINTER(ctypes.c_int64)]
_lib.ep_buffer_dedup.restype = _st
_lib.ep_dispatch_dedup.argtypes = [_P, ctypes.c_int, _P, _P]
_lib.ep_dispatch_dedup.restype = _st
_lib.ep_permute.argtypes = [_P, ctypes.c_int, _P]
_lib.ep_permute.restype = _st
_lib.ep_local_reduce.argtypes = [_P, ctypes.c_int, _P, _P, _P]
_lib.ep_local_reduce.restype = _st
_lib.ep_combine_dedup.argtypes = [_P, ctypes.c_int, _P, _P]
_lib.ep_combine_dedup.restype = _st
_lib.ep_selftest_wait_timeout.argtypes = [_P, ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint32), _P]
_lib.ep_selftest_wait_timeout.restype = _st
_lib.ep_buffer_shard.argtypes = [_P] + [ctypes.POINTER(_P)] * 5
_lib.ep_buffer_shard.restype = _st
_lib.ep_shard_layout.argtypes = [_P, ctypes.c_int, ctypes.c_int, _P, _P, _P, ctypes.c_int, ctypes.c_uint64,
                                 ctypes.c_float, _P]
_lib.ep_shard_layout.restype = _st
_lib.ep_shard_place.argtypes = [_P, ctypes.c_int, ctypes.c_int, _P]
_lib.ep_shard_place.restype = _st
_lib.ep_shard_dispatch.argtypes = [_P, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P, _P, _P]
_lib.ep_shard_dispatch.restype = _st
_lib.ep_shard_combine.argtypes = [_P, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P]
_lib.ep_shard_combine.restype = _st
_i64, _int, _sz, _f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_lib.ep_rmsnorm.argtypes = [_i64, _int, _P, _P, _P, _int, _f32, _P, _P, _P, _P, _P, _P]
_lib.ep_rmsnorm.restype = _st
_lib.ep_rmsnorm_backward_workspace_bytes.argtypes = [_i64, _int, ctypes.POINTER(_sz)]
_lib.ep_rmsnorm_backward_workspace_bytes.restype = _st
_lib.ep_rmsnorm_backward.argtypes = [_i64, _int, _P, _P, _P, _int, _P, _P, _P, _P, _P, _sz, _P]
_lib.ep_rmsnorm_backward.restype = _st
_lib.ep_balance_loss_workspace_bytes.argtypes = [_i64, _int, _int, ctypes.POINTER(_sz)]
_lib.ep_balance_loss_workspace_bytes.restype = _st
_lib.ep_balance_loss.argtypes = [_i64, _int, _int, _int, _P, _P, _int, _P, _f32, _P, _P, _P, _P, _sz, _P, _P]
_lib.ep_balance_loss.restype = _st
_lib.ep_balance_loss_backward.argtypes = [_i64, _int, _int, _int, _P, _int, _P, _P, _f32, _P, _int, _P, _P]
_lib.ep_balance_loss_backward.restype = _st
_lib.ep_linear.argtypes = [_P, _i64, ctypes.POINTER(EpLinear), _P]
_lib.ep_linear.restype = _st
_lib.ep_expert_linear.argtypes = [_P, _int, ctypes.POINTER(EpLinear), _P]
_lib.ep_expert_linear.restype = _st

EXPORTED = ("ep_abi_version", "ep_status_string", "ep_last_error_message", "ep_default_config",
            "ep_buffer_workspace_bytes", "ep_buffer_create", "ep_buffer_destroy", "ep_buffer_set_num_sms",
            "ep_buffer_layout",
            "ep_buffer_recv", "ep_get_layout", "ep_dispatch", "ep_combine", "ep_check_errors",
            "ep_get_layout_noalloc", "ep_selftest_wait_timeout", "ep_buffer_dedup", "ep_dispatch_dedup",
            "ep_permute", "ep_local_reduce", "ep_combine_dedup", "ep_buffer_shard", "ep_shard_layout",
            "ep_shard_place", "ep_shard_dispatch", "ep_shard_combine",
            "ep_rmsnorm", "ep_rmsnorm_backward_workspace_bytes", "ep_rmsnorm_backward",
            "ep_balance_loss_workspace_bytes", "ep_balance_loss", "ep_balance_loss_backward",
            "ep_linear", "ep_expert_linear")


class EpError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str | None = None):
        self.status = status
        if msg is None:
            msg = _lib.ep_last_error_message().decode()
        super().__init__(f"{where}: {_lib.ep_status_string(status).decode()} ({msg})")


def _check(status: int, where: str) -> None:
    if status != EP_OK:
        raise EpError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class EpBuffer:
    """Handle plus the torch-owned workspace it lives in."""

    def __init__(self, handle: int, cfg: EpConfig, workspace: torch.Tensor):
        self.handle = handle
        self.cfg = cfg
        self.workspace = workspace

    @property
    def fp8(self) -> bool:
        return bool(self.cfg.flags & EP_FLAG_FP8)

    @property
    def shard(self) -> bool:
        return bool(self.cfg.flags & EP_FLAG_SHARD)

    def _view(self, ptr: int, dtype: torch.dtype, shape) -> torch.Tensor:
        off = ptr - self.workspace.data_ptr()
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        assert 0 <= off and off + nbytes <= self.workspace.numel()
        return self.workspace.narrow(0, off, nbytes).view(dtype).view(*shape)

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            _lib.ep_buffer_destroy(h)


def ep_abi_version() -> int:
    return _lib.ep_abi_version()


def ep_status_string(status: int) -> str:
    return _lib.ep_status_string(status).decode()


def ep_last_error_message() -> str:
    return _lib.ep_last_error_message().decode()


def ep_default_config(num_ranks: int, max_tokens_per_rank: int, hidden: int, num_experts: int,
                      topk: int) -> EpConfig:
    return _lib.ep_default_config(num_ranks, max_tokens_per_rank, hidden, num_experts, topk)


def ep_buffer_workspace_bytes(cfg: EpConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.ep_buffer_workspace_bytes(ctypes.byref(cfg), ctypes.byref(n)), "ep_buffer_workspace_bytes")
    return n.value


def ep_buffer_create(cfg: EpConfig, workspace: torch.Tensor | None = None, device=None) -> EpBuffer:
    """Wraps `workspace` (a uint8 CUDA tensor of at least
    ep_buffer_workspace_bytes(cfg) bytes), allocating it first if None."""
    nbytes = ep_buffer_workspace_bytes(cfg)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    h = _P()
    _check(_lib.ep_buffer_create(ctypes.byref(cfg), workspace.data_ptr(), workspace.numel(), ctypes.byref(h)),
           "ep_buffer_create")
    return EpBuffer(h.value, cfg, workspace)


def ep_buffer_destroy(buf: EpBuffer) -> None:
    h, buf.handle = buf.handle, None
    if h:
        _check(_lib.ep_buffer_destroy(h), "ep_buffer_destroy")


def ep_buffer_set_num_sms(buf: EpBuffer, num_sms: int) -> None:
    """SM budget of dispatch and combine (0 = all); Buffer.set_num_sms analogue."""
    _check(_lib.ep_buffer_set_num_sms(buf.handle, num_sms), "ep_buffer_set_num_sms")
    buf.cfg.num_sms = num_sms


def ep_buffer_layout(buf: EpBuffer, T: int) -> dict:
    """torch views of the layout arrays for T tokens per rank (one source rank,
    N = T, for an EP_FLAG_SHARD buffer)."""
    lay = EpLayout()
    _check(_lib.ep_buffer_layout(buf.handle, ctypes.byref(lay)), "ep_buffer_layout")
    c = buf.cfg
    R, E, K = c.num_ranks, c.num_experts, c.topk
    S = 1 if buf.shard else R
    N = S * T
    return dict(
        topk_idx=buf._view(lay.topk_idx, torch.int32, (N, K)),
        topk_w=buf._view(lay.topk_w, torch.float32, (N, K)),
        is_token_in_rank=buf._view(lay.is_token_in_rank, torch.uint8, (N, R)),
        num_tokens_per_rank=buf._view(lay.num_tokens_per_rank, torch.int32, (S, R)),
        cnt=buf._view(lay.cnt_src_expert, torch.int32, (S, E)),
        num_tokens_per_expert=buf._view(lay.num_tokens_per_expert, torch.int32, (E,)),
        expert_off=buf._view(lay.expert_off, torch.int32, (E + 1,)),
        rank_off=buf._view(lay.rank_off, torch.int32, (R + 1,)),
        src_off=buf._view(lay.src_off, torch.int32, (E, S)),
        dst_row=buf._view(lay.dst_row, torch.int32, (N, K)),
    )


def ep_buffer_recv(buf: EpBuffer) -> dict:
    """torch views of the receive buffers (M_max rows)."""
    px, ps, pr, pw = _P(), _P(), _P(), _P()
    m = ctypes.c_int64(0)
    _check(_lib.ep_buffer_recv(buf.handle, ctypes.byref(px), ctypes.byref(ps), ctypes.byref(pr),
                               ctypes.byref(pw), ctypes.byref(m)), "ep_buffer_recv")
    H, M = buf.cfg.hidden, m.value
    out = dict(max_rows=M,
               recv_src=buf._view(pr.value, torch.int32, (M,)),
               recv_w=buf._view(pw.value, torch.float32, (M,)))
    if buf.fp8:
        out["recv_x"] = buf._view(px.value, torch.uint8, (M, H))
        out["recv_scale"] = buf._view(ps.value, torch.float32, (M, H // 128))
    else:
        out["recv_x"] = buf._view(px.value, torch.bfloat16, (M, H))
        out["recv_scale"] = None
    return out


def ep_get_layout(buf: EpBuffer, T: int, logits=None, topk_idx=None, topk_w=None, route: int = 0,
                  mask_seed: int = 0, mask_frac: float = 0.0, stream=None) -> None:
    _check(_lib.ep_get_layout(buf.handle, T, _ptr(logits), _ptr(topk_idx), _ptr(topk_w), route,
                              mask_seed & 0xFFFF_FFFF_FFFF_FFFF, mask_frac, _stream(stream)), "ep_get_layout")


def ep_dispatch(buf: EpBuffer, T: int, x, stream=None) -> None:
    _check(_lib.ep_dispatch(buf.handle, T, _ptr(x), _stream(stream)), "ep_dispatch")


def ep_combine(buf: EpBuffer, T: int, y, y_scale, out, stream=None) -> None:
    _check(_lib.ep_combine(buf.handle, T, _ptr(y), _ptr(y_scale), _ptr(out), _stream(stream)), "ep_combine")


def ep_check_errors(buf: EpBuffer, clear: bool = True, stream=None) -> int:
    """Synchronises the stream and returns the device error word (0 = clean)."""
    w = ctypes.c_uint32(0)
    st = _lib.ep_check_errors(buf.handle, ctypes.byref(w), 1 if clear else 0, _stream(stream))
    if st not in (EP_OK, EP_ERR_DEVICE):
        _check(st, "ep_check_errors")
    return w.value


def ep_buffer_dedup(buf: EpBuffer, T: int) -> dict:
    """torch views of the deduplicated-receive layout and buffers."""
    ptrs = [_P() for _ in range(9)]
    d = ctypes.c_int64(0)
    _check(_lib.ep_buffer_dedup(buf.handle, *[ctypes.byref(q) for q in ptrs], ctypes.byref(d)), "ep_buffer_dedup")
    c = buf.cfg
    R, K, H, N, D = c.num_ranks, c.topk, c.hidden, c.num_ranks * T, d.value
    out = dict(max_rows=D,
               tok_row=buf._view(ptrs[0].value, torch.int32, (N, R)),
               rank_row_off=buf._view(ptrs[1].value, torch.int32, (R + 1,)),
               rank_src_off=buf._view(ptrs[2].value, torch.int32, (R, R)),
               dd_src=buf._view(ptrs[5].value, torch.int32, (D,)),
               dd_topk_idx=buf._view(ptrs[6].value, torch.int32, (D, K)),
               dd_topk_w=buf._view(ptrs[7].value, torch.float32, (D, K)),
               partial=buf._view(ptrs[8].value, torch.bfloat16, (D, H)))
    if buf.fp8:
        out["dd_x"] = buf._view(ptrs[3].value, torch.uint8, (D, H))
        out["dd_scale"] = buf._view(ptrs[4].value, torch.float32, (D, H // 128))
    else:
        out["dd_x"] = buf._view(ptrs[3].value, torch.bfloat16, (D, H))
        out["dd_scale"] = None
    return out


def ep_dispatch_dedup(buf: EpBuffer, T: int, x, stream=None) -> None:
    _check(_lib.ep_dispatch_dedup(buf.handle, T, _ptr(x), _stream(stream)), "ep_dispatch_dedup")


def ep_permute(buf: EpBuffer, T: int, stream=None) -> None:
    _check(_lib.ep_permute(buf.handle, T, _stream(stream)), "ep_permute")


def ep_local_reduce(buf: EpBuffer, T: int, y, y_scale, stream=None) -> None:
    _check(_lib.ep_local_reduce(buf.handle, T, _ptr(y), _ptr(y_scale), _stream(stream)), "ep_local_reduce")


def ep_combine_dedup(buf: EpBuffer, T: int, out, stream=None) -> None:
    _check(_lib.ep_combine_dedup(buf.handle, T, _ptr(out), _stream(stream)), "ep_combine_dedup")


def ep_selftest_wait_timeout(words, limit_ns: int, stream=None) -> int:
    """Runs bounded waits that can never be satisfied; returns the error
    bits they left (EP_DEVERR_TIMEOUT expected). `words`: 4-element int32/uint32
    CUDA tensor."""
    w = ctypes.c_uint32(0)
    _check(_lib.ep_selftest_wait_timeout(_ptr(words), limit_ns, ctypes.byref(w), _stream(stream)),
           "ep_selftest_wait_timeout")
    return w.value


def ep_get_layout_noalloc(cfg: EpConfig, T: int, out: dict, error_word, logits=None, topk_idx=None,
                          topk_w=None, route: int = 0, mask_seed: int = 0, mask_frac: float = 0.0,
                          stream=None) -> None:
    """Routing + layout into the caller's own tensors (`out` holds the
    ep_layout_t arrays by name, as ep_buffer_layout returns them;
    `error_word` is a 1-element int32/uint32 CUDA tensor). It uses the
    library's static scratch and allocates nothing."""
    lay = EpLayout(topk_idx=_ptr(out["topk_idx"]), topk_w=_ptr(out["topk_w"]),
                   is_token_in_rank=_ptr(out["is_token_in_rank"]),
                   num_tokens_per_rank=_ptr(out["num_tokens_per_rank"]), cnt_src_expert=_ptr(out["cnt"]),
                   num_tokens_per_expert=_ptr(out["num_tokens_per_expert"]),
                   expert_off=_ptr(out["expert_off"]), rank_off=_ptr(out["rank_off"]),
                   src_off=_ptr(out["src_off"]), dst_row=_ptr(out["dst_row"]))
    _check(_lib.ep_get_layout_noalloc(ctypes.byref(cfg), T, _ptr(logits), _ptr(topk_idx), _ptr(topk_w), route,
                                      mask_seed & 0xFFFF_FFFF_FFFF_FFFF, mask_frac, ctypes.byref(lay),
                                      _ptr(error_word), _stream(stream)), "ep_get_layout_noalloc")


# ---- one rank per GPU (EP_FLAG_SHARD) ------------------------------------------

def _table(entries):
    """Host array of device pointers (tensors or ints; None stays NULL)."""
    if entries is None:
        return None
    arr = (_P * len(entries))(*[_ptr(t) for t in entries])
    return arr


def ep_buffer_shard(buf: EpBuffer, T: int) -> dict:
    """torch views of the shard arrays: cnt_row [E], cnt_all [R, E],
    dst_rank [T, K], recv_count [E/R], recv_off [E/R + 1]."""
    ptrs = [_P() for _ in range(5)]
    _check(_lib.ep_buffer_shard(buf.handle, *[ctypes.byref(p) for p in ptrs]), "ep_buffer_shard")
    c = buf.cfg
    R, E, K = c.num_ranks, c.num_experts, c.topk
    L = E // R
    return dict(cnt_row=buf._view(ptrs[0].value, torch.int32, (E,)),
                cnt_all=buf._view(ptrs[1].value, torch.int32, (R, E)),
                dst_rank=buf._view(ptrs[2].value, torch.uint8, (T, K)),
                recv_count=buf._view(ptrs[3].value, torch.int32, (L,)),
                recv_off=buf._view(ptrs[4].value, torch.int32, (L + 1,)))


def ep_shard_layout(buf: EpBuffer, rank: int, T: int, logits=None, topk_idx=None, topk_w=None, route: int = 0,
                    mask_seed: int = 0, mask_frac: float = 0.0, stream=None) -> None:
    _check(_lib.ep_shard_layout(buf.handle, rank, T, _ptr(logits), _ptr(topk_idx), _ptr(topk_w), route,
                                mask_seed & 0xFFFF_FFFF_FFFF_FFFF, mask_frac, _stream(stream)), "ep_shard_layout")


def ep_shard_place(buf: EpBuffer, rank: int, T: int, stream=None) -> None:
    _check(_lib.ep_shard_place(buf.handle, rank, T, _stream(stream)), "ep_shard_place")


def ep_shard_dispatch(buf: EpBuffer, rank: int, T: int, x, peer_recv_x, peer_recv_scale, peer_recv_src,
                      peer_recv_w, stream=None) -> None:
    """peer_* are length-R lists of each rank's receive arrays (tensors or
    device pointers); peer_recv_scale is None without FP8."""
    tx, ts, tr, tw = (_table(peer_recv_x), _table(peer_recv_scale), _table(peer_recv_src),
                      _table(peer_recv_w))
    _check(_lib.ep_shard_dispatch(buf.handle, rank, T, _ptr(x), tx, ts, tr, tw, _stream(stream)),
           "ep_shard_dispatch")


def ep_shard_combine(buf: EpBuffer, rank: int, T: int, peer_y, peer_y_scale, out, stream=None) -> None:
    """peer_y: length-R list of each rank's expert output (bf16, or e4m3 with
    peer_y_scale for the fused dequantisation)."""
    ty, ts = _table(peer_y), _table(peer_y_scale)
    _check(_lib.ep_shard_combine(buf.handle, rank, T, ty, ts, _ptr(out), _stream(stream)), "ep_shard_combine")



# ---- the MoE block around dispatch and combine ----------------------------------
# These take torch tensors only, and check what a pointer cannot say: device,
# element type, shape and contiguity.

_BF16, _F32, _I32, _U8 = (torch.bfloat16,), (torch.float32,), (torch.int32,), (torch.uint8,)
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_GAMMA = (torch.bfloat16, torch.float32)
_OUT = (torch.bfloat16, torch.float32, *_E4M3)
_WORD = (torch.int32, torch.uint32)


def _refuse(where: str, why: str):
    raise EpError(EP_ERR_INVALID, where, why)


def _shape_of(where: str, name: str, t, dims: int):
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        _refuse(where, f"{name} is no tensor of {dims} dimension{'s' if dims > 1 else ''}")
    return t.shape


def _why_not(t, dtypes, dev: int, shape) -> str:
    if not isinstance(t, torch.Tensor):
        return "is no tensor"
    if t.dtype not in dtypes:
        return f"has dtype {t.dtype}, not {' or '.join(str(d) for d in dtypes)}"
    if t.get_device() != dev or dev < 0:
        return f"is on {t.device}, not on the CUDA device of the call"
    if not t.is_contiguous():
        return "is not contiguous"
    return f"has shape {tuple(t.shape)}, not {tuple(shape)}"


def _checked(where: str, dev: int, *wanted) -> None:
    """Each of `wanted` is (name, tensor or None, dtypes, shape or None). A
    tensor is contiguous, on CUDA device `dev`, and of that type and shape."""
    for name, t, dtypes, shape in wanted:
        # (get_device is -1 for host tensors)
        if t is not None and not (isinstance(t, torch.Tensor) and t.get_device() == dev >= 0 and t.dtype in dtypes and
                                  t.is_contiguous() and (shape is None or t.shape == shape)):
            _refuse(where, f"{name} {_why_not(t, dtypes, dev, shape if shape is not None else ())}")


def _required(where: str, *named) -> None:
    for name, t in named:
        if t is None:
            _refuse(where, f"{name} is None")


def _on(dev: int, fn, *args):
    """fn(*args) with `dev` the current device."""
    if torch._C._cuda_getDevice() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _stream_on(dev: int, stream):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def ep_rmsnorm_backward_workspace_bytes(N: int, H: int) -> int:
    n = _sz(0)
    _check(_lib.ep_rmsnorm_backward_workspace_bytes(N, H, ctypes.byref(n)), "ep_rmsnorm_backward_workspace_bytes")
    return n.value


def ep_rmsnorm(x, gamma, eps: float, residual=None, h=None, y=None, q=None, q_scale=None, rstd=None,
               stream=None) -> None:
    """Residual addition, RMS norm and e4m3 cast of x [N, H] into whichever
    of h, y, q + q_scale and rstd are given."""
    w = "ep_rmsnorm"
    shape = _shape_of(w, "x", x, 2)
    N, H = shape
    dev = x.get_device()
    _required(w, ("gamma", gamma))
    _checked(w, dev, ("x", x, _BF16, None), ("gamma", gamma, _GAMMA, (H,)), ("residual", residual, _BF16, shape),
             ("h", h, _BF16, shape), ("y", y, _BF16, shape), ("q", q, _E4M3, shape),
             ("q_scale", q_scale, _F32, (N, H // 128)), ("rstd", rstd, _F32, (N,)))
    _check(_on(dev, _lib.ep_rmsnorm, N, H, _ptr(x), _ptr(residual), _ptr(gamma), int(gamma.dtype is torch.float32), eps,
               _ptr(h), _ptr(y), _ptr(q), _ptr(q_scale), _ptr(rstd), _stream_on(dev, stream)), w)


def ep_rmsnorm_backward(h, rstd, gamma, dy, dx, dgamma, workspace, dh=None, stream=None) -> None:
    """Gradient of ep_rmsnorm; workspace: uint8, ep_rmsnorm_backward_workspace_bytes(N, H)."""
    w = "ep_rmsnorm_backward"
    shape = _shape_of(w, "h", h, 2)
    N, H = shape
    dev = h.get_device()
    _required(w, ("rstd", rstd), ("gamma", gamma), ("dy", dy), ("dx", dx), ("dgamma", dgamma),
              ("workspace", workspace))
    _checked(w, dev, ("h", h, _BF16, None), ("rstd", rstd, _F32, (N,)), ("gamma", gamma, _GAMMA, (H,)),
             ("dy", dy, _BF16, shape), ("dh", dh, _BF16, shape), ("dx", dx, _BF16, shape),
             ("dgamma", dgamma, _F32, (H,)), ("workspace", workspace, _U8, None))
    _check(_on(dev, _lib.ep_rmsnorm_backward, N, H, _ptr(h), _ptr(rstd), _ptr(gamma), int(gamma.dtype is torch.float32),
               _ptr(dy), _ptr(dh), _ptr(dx), _ptr(dgamma), _ptr(workspace), workspace.numel(),
               _stream_on(dev, stream)), w)


def ep_balance_loss_workspace_bytes(N: int, E: int, S: int = 1) -> int:
    n = _sz(0)
    _check(_lib.ep_balance_loss_workspace_bytes(N, E, S, ctypes.byref(n)), "ep_balance_loss_workspace_bytes")
    return n.value


def _sequences(where: str, seq_off) -> int:
    if seq_off is None:
        return 1
    n = _shape_of(where, "seq_off", seq_off, 1)[0]
    if n < 2:
        _refuse(where, "seq_off is not [S + 1] with S >= 1")
    return n - 1


def ep_balance_loss(logits, topk_idx, score: int, coef: float, loss, counts, workspace, error_word, seq_off=None,
                    prob=None, stream=None) -> None:
    """Balance loss of logits [N, E] and topk_idx [N, K] over the sequences of
    seq_off [S + 1] (None: one); fills loss [1], counts [S, E], prob [S, E]."""
    w = "ep_balance_loss"
    N, E = _shape_of(w, "logits", logits, 2)
    K, S, dev = _shape_of(w, "topk_idx", topk_idx, 2)[1], _sequences(w, seq_off), logits.get_device()
    _required(w, ("loss", loss), ("counts", counts), ("workspace", workspace), ("error_word", error_word))
    _checked(w, dev, ("logits", logits, _F32, None), ("topk_idx", topk_idx, _I32, (N, K)),
             ("seq_off", seq_off, _I32, None), ("loss", loss, _F32, (1,)), ("counts", counts, _I32, (S, E)),
             ("prob", prob, _F32, (S, E)), ("workspace", workspace, _U8, None),
             ("error_word", error_word, _WORD, (1,)))
    _check(_on(dev, _lib.ep_balance_loss, N, E, K, score, _ptr(logits), _ptr(topk_idx), S, _ptr(seq_off), coef,
               _ptr(loss), _ptr(counts), _ptr(prob), _ptr(workspace), workspace.numel(), _ptr(error_word),
               _stream_on(dev, stream)), w)


def ep_balance_loss_backward(logits, counts, topk: int, score: int, coef: float, dlogits, seq_off=None,
                             grad_loss=None, accumulate: bool = False, stream=None) -> None:
    """Gradient of ep_balance_loss for the logits, into (or added to) dlogits."""
    w = "ep_balance_loss_backward"
    shape = _shape_of(w, "logits", logits, 2)
    N, E = shape
    S, dev = _sequences(w, seq_off), logits.get_device()
    _required(w, ("counts", counts), ("dlogits", dlogits))
    _checked(w, dev, ("logits", logits, _F32, None), ("counts", counts, _I32, (S, E)), ("dlogits", dlogits, _F32, shape),
             ("seq_off", seq_off, _I32, None), ("grad_loss", grad_loss, _F32, (1,)))
    _check(_on(dev, _lib.ep_balance_loss_backward, N, E, topk, score, _ptr(logits), S, _ptr(seq_off), _ptr(counts), coef,
               _ptr(grad_loss), 1 if accumulate else 0, _ptr(dlogits), _stream_on(dev, stream)), w)


def _linear_args(where, dev, groups, rows, x, w, out, x_scale, w_scale, bias, residual, act, out_scale):
    """Checks the tensors of a linear layer on at least `rows` rows and
    returns the C struct."""
    have, cin = _shape_of(where, "x", x, 2)
    room, cout = _shape_of(where, "out", out, 2)
    _required(where, ("w", w))
    if (x_scale is None) != (w_scale is None):
        _refuse(where, "x_scale and w_scale go together")
    if min(have, room) < rows:
        _refuse(where, f"x and out hold {have} and {room} rows, the call needs {rows}")
    for name, t in (("x_scale", x_scale), ("residual", residual), ("out_scale", out_scale)):
        if t is not None and _shape_of(where, name, t, 2)[0] < rows:
            _refuse(where, f"{name} holds {t.shape[0]} rows, the call needs {rows}")
    parts = 2 if act == EP_ACT_SWIGLU else 1
    kind = _BF16 if x_scale is None else _E4M3
    _checked(where, dev, ("x", x, kind, None), ("w", w, kind, (groups, parts * cout, cin)), ("out", out, _OUT, None),
             ("bias", bias, _F32, (groups, parts * cout)))
    if x_scale is not None:
        _checked(where, dev, ("x_scale", x_scale, _F32, (x_scale.shape[0], cin // 128)),
                 ("w_scale", w_scale, _F32, (groups, parts * -(-cout // 128), cin // 128)))
    if residual is not None:
        _checked(where, dev, ("residual", residual, _BF16, (residual.shape[0], cout)))
    if out_scale is not None:
        _checked(where, dev, ("out_scale", out_scale, _F32, (out_scale.shape[0], cout // 128)))
    dt = out.dtype
    return EpLinear(_ptr(x), _ptr(x_scale), _ptr(w), _ptr(w_scale), _ptr(bias), _ptr(residual), _ptr(out),
                    _ptr(out_scale), cin, cout, act,
                    EP_DTYPE_BF16 if dt is torch.bfloat16 else EP_DTYPE_FP32 if dt is torch.float32 else EP_DTYPE_E4M3)


def ep_linear(buf: EpBuffer, x, w, out, x_scale=None, w_scale=None, bias=None, residual=None,
              act: int = EP_ACT_NONE, out_scale=None, stream=None) -> None:
    """out = act(x w[0]^T + bias) + residual on x [rows, in]; w [1, wide, in]."""
    rows, dev = _shape_of("ep_linear", "x", x, 2)[0], buf.workspace.get_device()
    a = _linear_args("ep_linear", dev, 1, rows, x, w, out, x_scale, w_scale, bias, residual, act, out_scale)
    _check(_lib.ep_linear(buf.handle, rows, ctypes.byref(a), _stream_on(dev, stream)), "ep_linear")


def ep_expert_linear(buf: EpBuffer, T: int, x, w, out, x_scale=None, w_scale=None, bias=None, residual=None,
                     act: int = EP_ACT_NONE, out_scale=None, stream=None) -> None:
    """The experts' layer on the receive rows of the last layout: x [rows, in],
    w [experts, wide, in] (a shard's own experts with EP_FLAG_SHARD)."""
    c, dev = buf.cfg, buf.workspace.get_device()
    E, R, flags = c.num_experts, c.num_ranks, c.flags
    rows = E * R * c.max_tokens_per_rank if flags & EP_FLAG_LOW_LATENCY else R * T * c.topk
    a = _linear_args("ep_expert_linear", dev, E // R if flags & EP_FLAG_SHARD else E, rows, x, w, out, x_scale, w_scale,
                     bias, residual, act, out_scale)
    _check(_lib.ep_expert_linear(buf.handle, T, ctypes.byref(a), _stream_on(dev, stream)), "ep_expert_linear")
