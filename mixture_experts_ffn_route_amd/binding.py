"""Thin Python binding of the C ABI in include/moe.h (argument marshalling only).

Every function has the name of the C entry point it calls.  Device buffers
are torch tensors (PyTorch provides the device memory and the stream); all
arithmetic happens in the HIP library.  There is no fallback: if the library
is not built, importing this module raises.
"""

import ctypes
import os

import numpy as np
import torch  # loaded first so the library binds to the same HIP runtime as torch

from dataclasses import replace

from .config import (ACT_QUANT, ACTIVATION, DTYPE, LAYOUT, ROUTE, SCORE, LinearConfig,
                     MoEConfig)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mi355x.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_HIP = -4
MOE_FLAG_TOKEN_ID_RANGE = 1
MOE_FLAG_EXPERT_RANGE = 2
MOE_NOALLOC_SCRATCH_BYTES = 64 << 20
MOE_FEW_MAX_TOKENS = 16

EXPORTED_SYMBOLS = (
    "moe_status_string", "moe_validate_config", "moe_build_tid2eid", "moe_workspace_layout",
    "moe_workspace_size", "moe_route", "moe_permute", "moe_forward", "moe_forward_profiled",
    "moe_pack_weights", "moe_build_tid2eid_multistart", "moe_update_bias", "moe_probe_read",
    "moe_probe_mfma", "moe_redequant_fp8", "moe_forward_ex", "moe_forward_noalloc",
    "moe_few_workspace_layout", "moe_few_workspace_size", "moe_forward_few",
    "moe_linear_workspace_size", "moe_linear", "moe_linear_backward", "moe_linear_path",
    "moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward",
    "moe_checkpoint_save", "moe_checkpoint_load", "moe_experts_workspace_size", "moe_experts",
    "moe_experts_backward", "moe_experts_path",
)
MOE_STAGES = ("route", "permute", "gemm1", "gemm2", "combine")


class MoeConfigC(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32), ("n_routed_experts", ctypes.c_int32),
        ("n_activated_experts", ctypes.c_int32), ("n_expert_groups", ctypes.c_int32),
        ("n_limited_groups", ctypes.c_int32), ("moe_inter_dim", ctypes.c_int32),
        ("n_shared_experts", ctypes.c_int32), ("score_func", ctypes.c_int32),
        ("route_scale", ctypes.c_float), ("renormalize", ctypes.c_int32),
        ("swiglu_limit", ctypes.c_float), ("route_mode", ctypes.c_int32),
        ("vocab_size", ctypes.c_int64), ("act_dtype", ctypes.c_int32),
        ("expert_dtype", ctypes.c_int32), ("weight_layout", ctypes.c_int32),
        ("act_quant", ctypes.c_int32),
    ]


class MoeWeightsC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "gate_w", "gate_bias", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
        "sh_gate", "sh_up", "sh_down", "tid2eid")]


class MoeWsLayoutC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "total_bytes", "route_weights", "route_indices", "counts", "offsets", "sorted_tok",
        "sorted_slot", "sorted_weight", "inverse", "tiles", "tile_count", "flags",
        "route_logits", "perm_hist", "xq", "xq_scales", "hq", "hq_scales", "h", "yrows")] + [
        ("max_tiles", ctypes.c_int32), ("tile_rows", ctypes.c_int32)]


class MoeFewLayoutC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "total_bytes", "route_weights", "route_indices", "flags", "scores", "plan_slots",
        "plan_experts", "plan_weights", "plan_rows", "plan_masks", "xq", "xq_scales", "hq",
        "hq_scales", "h", "h_lo", "yrows")]


class MoeLinearConfigC(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("in_dim", ctypes.c_int32), ("out_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("limit", ctypes.c_float),
        ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64), ("ld_residual", ctypes.c_int64),
    ]


class MoeLinearWeightsC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w", "w_up", "bias", "bias_up")]


class MoeLinearGradsC(ctypes.Structure):
    _fields_ = [*((n, ctypes.c_void_p) for n in ("dx", "dw", "dw_up", "dbias", "dbias_up")),
                ("ld_dx", ctypes.c_int64)]


class MoeLinearPathC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("path", "tile_rows", "tile_cols", "parts")]


class MoeExpertsSavedC(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in (
        "gate", "up", "gate_scales", "up_scales")]


class MoeExpertsPathC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tile_rows", "tile_cols", "streamed")]


class MoeExpertsGradsC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "dw_gate", "dw_up", "dw_down")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    cfgp, wp = ctypes.POINTER(MoeConfigC), ctypes.POINTER(MoeWeightsC)
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_validate_config.argtypes = [cfgp]
    lib.moe_build_tid2eid.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp]
    lib.moe_workspace_layout.argtypes = [cfgp, i64, ctypes.POINTER(MoeWsLayoutC)]
    lib.moe_workspace_size.restype = ctypes.c_size_t
    lib.moe_workspace_size.argtypes = [cfgp, i64]
    lib.moe_route.argtypes = [cfgp, wp, vp, vp, i64, vp, vp, vp]
    lib.moe_permute.argtypes = [cfgp, vp, i64, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_forward.argtypes = [cfgp, wp, vp, vp, i64, vp, vp, ctypes.c_size_t, vp]
    lib.moe_pack_weights.argtypes = [cfgp, wp, wp, vp]
    lib.moe_build_tid2eid_multistart.argtypes = [vp, i64, i32, i32, vp, i32, vp, vp, vp, vp, vp]
    lib.moe_update_bias.argtypes = [cfgp, vp, i64, ctypes.c_float, vp, vp, vp]
    lib.moe_probe_read.argtypes = [vp, i64, vp, vp]
    lib.moe_probe_mfma.argtypes = [i32, i32, vp, vp, vp]
    lib.moe_redequant_fp8.argtypes = [vp, vp, i64, i32, i32, vp, vp, vp, vp]
    lib.moe_forward_profiled.argtypes = [cfgp, wp, vp, vp, i64, vp, vp, ctypes.c_size_t,
                                         ctypes.POINTER(ctypes.c_void_p), vp]
    lib.moe_forward_ex.argtypes = [cfgp, wp, vp, vp, i64, vp, vp, ctypes.c_size_t,
                                   ctypes.POINTER(ctypes.c_void_p), vp, vp]
    lib.moe_forward_noalloc.argtypes = [cfgp, wp, vp, vp, i64, vp, vp]
    lib.moe_few_workspace_layout.argtypes = [cfgp, i64, ctypes.POINTER(MoeFewLayoutC)]
    lib.moe_few_workspace_size.restype = ctypes.c_size_t
    lib.moe_few_workspace_size.argtypes = [cfgp, i64]
    lib.moe_forward_few.argtypes = lib.moe_forward.argtypes
    lcp, lwp = ctypes.POINTER(MoeLinearConfigC), ctypes.POINTER(MoeLinearWeightsC)
    lib.moe_linear_workspace_size.restype = ctypes.c_size_t
    lib.moe_linear_workspace_size.argtypes = [lcp, i32]
    lib.moe_linear.argtypes = [lcp, lwp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.moe_linear_backward.argtypes = [lcp, lwp, vp, vp, vp, vp, ctypes.POINTER(MoeLinearGradsC),
                                        vp, ctypes.c_size_t, vp]
    lib.moe_linear_path.argtypes = [lcp, i32, ctypes.POINTER(MoeLinearPathC)]
    size = ctypes.c_size_t
    lib.moe_dispatch.argtypes = [cfgp, vp, vp, i64, i64, vp, vp]
    lib.moe_dispatch_backward.argtypes = lib.moe_dispatch.argtypes
    lib.moe_combine.argtypes = [cfgp, vp, vp, vp, vp, i64, i64, vp, vp]
    lib.moe_combine_backward.argtypes = [cfgp, vp, vp, vp, vp, i64, i64, vp, vp, vp]
    lib.moe_checkpoint_save.argtypes = [vp, i32, i64, i32, i64, ctypes.c_float, vp, vp, vp]
    lib.moe_checkpoint_load.argtypes = [vp, vp, i32, i64, i32, i64, vp, vp]
    sp = ctypes.POINTER(MoeExpertsSavedC)
    lib.moe_experts_workspace_size.restype = size
    lib.moe_experts_workspace_size.argtypes = [cfgp, i64, i32]
    lib.moe_experts.argtypes = [cfgp, wp, vp, vp, i64, vp, sp, vp, size, vp]
    lib.moe_experts_backward.argtypes = [cfgp, wp, vp, vp, i64, vp, sp,
                                         ctypes.POINTER(MoeExpertsGradsC), vp, size, vp]
    lib.moe_experts_path.argtypes = [cfgp, i64, i32, ctypes.POINTER(MoeExpertsPathC)]
    for f in ("moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward",
              "moe_experts_path",
              "moe_checkpoint_save", "moe_checkpoint_load", "moe_experts", "moe_experts_backward"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("moe_few_workspace_layout", "moe_forward_few", "moe_linear", "moe_linear_backward",
              "moe_linear_path"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("moe_validate_config", "moe_build_tid2eid", "moe_workspace_layout", "moe_route",
              "moe_permute", "moe_forward", "moe_forward_profiled", "moe_forward_ex",
              "moe_forward_noalloc",
              "moe_pack_weights",
              "moe_build_tid2eid_multistart", "moe_update_bias", "moe_probe_read",
              "moe_probe_mfma"):
        getattr(lib, f).restype = ctypes.c_int
    return lib


_lib = _load()


class MoEError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {moe_status_string(status)} ({status})")


def _check(status, where):
    if status != MOE_OK:
        raise MoEError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return ctypes.c_void_p(t.data_ptr())
    if isinstance(t, np.ndarray):
        return t.ctypes.data_as(ctypes.c_void_p)
    raise TypeError(type(t))


# The current stream's handle without a Stream object around it (3 us a call).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if isinstance(stream, int):              # a raw hipStream_t (0 = default stream)
        return ctypes.c_void_p(stream)
    if stream is None and _current_raw_stream is not None:
        return ctypes.c_void_p(_current_raw_stream(torch.cuda.current_device()))
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def config_c(cfg: MoEConfig) -> MoeConfigC:
    return MoeConfigC(
        cfg.dim, cfg.n_routed_experts, cfg.n_activated_experts, cfg.n_expert_groups,
        cfg.n_limited_groups, cfg.moe_inter_dim, cfg.n_shared_experts, SCORE[cfg.score_func],
        cfg.route_scale, cfg.renormalize, cfg.swiglu_limit, ROUTE[cfg.route_mode],
        cfg.vocab_size, DTYPE[cfg.act_dtype], DTYPE[cfg.expert_dtype], LAYOUT[cfg.weight_layout],
        ACT_QUANT[cfg.act_quant])


def weights_c(layer: dict) -> MoeWeightsC:
    return MoeWeightsC(*[_ptr(layer.get(n)) for n, _ in MoeWeightsC._fields_])


def moe_status_string(status: int) -> str:
    return _lib.moe_status_string(int(status)).decode()


def moe_validate_config(cfg: MoEConfig) -> int:
    return _lib.moe_validate_config(ctypes.byref(config_c(cfg)))


def moe_build_tid2eid(p, n: int, k: int):
    """Greedy table on the host.  Returns (tid2eid int32 [m,k], load [n], max_vio, min_vio)."""
    p = np.ascontiguousarray(p, dtype=np.float64)
    m = p.shape[0]
    table = np.empty((m, k), dtype=np.int32)
    load = np.empty(n, dtype=np.float64)
    mx, mn = ctypes.c_double(), ctypes.c_double()
    _check(_lib.moe_build_tid2eid(_ptr(p), m, n, k, _ptr(table), _ptr(load), ctypes.byref(mx),
                                  ctypes.byref(mn)), "moe_build_tid2eid")
    return table, load, mx.value, mn.value


def moe_build_tid2eid_multistart(p, n: int, k: int, orders):
    """Multi-start greedy on the host.  orders: int64 [S, m] token orders.
    Returns (tid2eid, load, max_vio, min_vio, best_start)."""
    p = np.ascontiguousarray(p, dtype=np.float64)
    orders = np.ascontiguousarray(orders, dtype=np.int64)
    m = p.shape[0]
    table = np.empty((m, k), dtype=np.int32)
    load = np.empty(n, dtype=np.float64)
    mx, mn, best = ctypes.c_double(), ctypes.c_double(), ctypes.c_int32()
    _check(_lib.moe_build_tid2eid_multistart(_ptr(p), m, n, k, _ptr(orders), orders.shape[0],
                                             _ptr(table), _ptr(load), ctypes.byref(mx),
                                             ctypes.byref(mn), ctypes.byref(best)),
           "moe_build_tid2eid_multistart")
    return table, load, mx.value, mn.value, best.value


def moe_update_bias(cfg: MoEConfig, counts, T: int, gamma: float, bias, stats=None, stream=None):
    """Sign step of the selection bias (device tensors; bias updated in place;
    stats: float64 [4] device tensor or None)."""
    _check(_lib.moe_update_bias(ctypes.byref(config_c(cfg)), _ptr(counts), T, gamma, _ptr(bias),
                                _ptr(stats), _stream(stream)), "moe_update_bias")


def moe_probe_read(buf, out, stream=None):
    _check(_lib.moe_probe_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(out),
                               _stream(stream)), "moe_probe_read")


def moe_probe_mfma(iters: int, out, shape=0, stream=None) -> float:
    """Launch the MFMA probe (shape 0: 16x16x32 bf16, 1: 32x32x16 bf16,
    2: scaled 16x16x128 E4M3 x E2M1, 3: the same E4M3 x E4M3); returns the
    flops the launch performs."""
    flops = ctypes.c_double()
    _check(_lib.moe_probe_mfma(iters, shape, _ptr(out), ctypes.byref(flops), _stream(stream)),
           "moe_probe_mfma")
    return flops.value


def moe_workspace_layout(cfg: MoEConfig, T: int) -> dict:
    lay = MoeWsLayoutC()
    _check(_lib.moe_workspace_layout(ctypes.byref(config_c(cfg)), T, ctypes.byref(lay)),
           "moe_workspace_layout")
    return {name: getattr(lay, name) for name, _ in MoeWsLayoutC._fields_}


def moe_workspace_size(cfg: MoEConfig, T: int) -> int:
    return _lib.moe_workspace_size(ctypes.byref(config_c(cfg)), T)


def moe_route(cfg: MoEConfig, layer: dict, x, token_ids, T: int, weights, indices, stream=None):
    _check(_lib.moe_route(ctypes.byref(config_c(cfg)), ctypes.byref(weights_c(layer)), _ptr(x),
                          _ptr(token_ids), T, _ptr(weights), _ptr(indices), _stream(stream)),
           "moe_route")


def moe_permute(cfg: MoEConfig, indices, T: int, counts, offsets, sorted_tok, sorted_slot,
                inverse, flags=None, stream=None):
    _check(_lib.moe_permute(ctypes.byref(config_c(cfg)), _ptr(indices), T, _ptr(counts),
                            _ptr(offsets), _ptr(sorted_tok), _ptr(sorted_slot), _ptr(inverse),
                            _ptr(flags), _stream(stream)), "moe_permute")


PACKED_MEMBERS = ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
                  "sh_gate", "sh_up", "sh_down")


def moe_pack_weights(cfg: MoEConfig, src: dict, dst: dict, stream=None):
    _check(_lib.moe_pack_weights(ctypes.byref(config_c(cfg)), ctypes.byref(weights_c(src)),
                                 ctypes.byref(weights_c(dst)), _stream(stream)),
           "moe_pack_weights")


def pack_layer(cfg: MoEConfig, layer: dict, stream=None):
    """(cfg with weight_layout "tiled", a copy of `layer` whose expert matrices
    are freshly allocated tiled copies written by moe_pack_weights)."""
    out = dict(layer)
    for n in PACKED_MEMBERS:
        if layer.get(n) is not None:
            out[n] = torch.empty_like(layer[n])
    moe_pack_weights(cfg, layer, out, stream)
    return replace(cfg, weight_layout="tiled"), out


def moe_redequant_fp8(codes, scales, n_mat: int, N: int, K: int, fp8, block_scales, lossy,
                      stream=None):
    """FP4 [n_mat, N, K/2] codes + [n_mat, N, K/32] scales -> E4M3 codes in the
    FP8 expert layout, [n_mat, N/128, K/128] block scales and lossy flags."""
    _check(_lib.moe_redequant_fp8(_ptr(codes), _ptr(scales), n_mat, N, K, _ptr(fp8),
                                  _ptr(block_scales), _ptr(lossy), _stream(stream)),
           "moe_redequant_fp8")


def redequant_layer(cfg: MoEConfig, layer: dict, stream=None):
    """(cfg with FP8 experts and tiled weights, a copy of the FP4 `layer` whose
    routed matrices are re-dequantised to FP8 by moe_redequant_fp8 and whose
    shared matrices are tiled by moe_pack_weights, total lossy block count)."""
    if cfg.expert_dtype != "fp4" or cfg.weight_layout != "rows":
        raise ValueError("redequant_layer takes an FP4 layer in the row layout")
    out = dict(layer)
    shared = {n: layer.get(n) for n in ("sh_gate", "sh_up", "sh_down")}
    if cfg.n_shared_experts:
        dst = {n: torch.empty_like(v) for n, v in shared.items()}
        moe_pack_weights(cfg, shared, dst, stream)
        out.update(dst)
    E, d, I = cfg.n_routed_experts, cfg.dim, cfg.moe_inter_dim
    dev = layer["w_gate"].device
    lossy_total = 0
    for n, sn, N, K in (("w_gate", "s_gate", I, d), ("w_up", "s_up", I, d),
                        ("w_down", "s_down", d, I)):
        codes = torch.empty((E, N, K), dtype=torch.uint8, device=dev)
        bsc = torch.empty((E, N // 128, K // 128), dtype=torch.uint8, device=dev)
        lossy = torch.empty_like(bsc)
        moe_redequant_fp8(layer[n], layer[sn], E, N, K, codes, bsc, lossy, stream)
        out[n], out[sn] = codes, bsc
        lossy_total += int(lossy.sum())
    return replace(cfg, expert_dtype="fp8", weight_layout="tiled"), out, lossy_total


def moe_forward(cfg: MoEConfig, layer: dict, x, token_ids, T: int, y, ws, stream=None,
                ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.moe_forward(ctypes.byref(config_c(cfg)), ctypes.byref(weights_c(layer)), _ptr(x),
                            _ptr(token_ids), T, _ptr(y), _ptr(ws), ws_bytes, _stream(stream)),
           "moe_forward")


def moe_forward_profiled(cfg: MoEConfig, layer: dict, x, token_ids, T: int, y, ws, events,
                         stream=None):
    """events: len(MOE_STAGES) + 1 raw hipEvent_t handles (see HipEvents)."""
    arr = (ctypes.c_void_p * len(events))(*events)
    _check(_lib.moe_forward_profiled(ctypes.byref(config_c(cfg)), ctypes.byref(weights_c(layer)),
                                     _ptr(x), _ptr(token_ids), T, _ptr(y), _ptr(ws),
                                     ws.numel() * ws.element_size(), arr, _stream(stream)),
           "moe_forward_profiled")


def moe_forward_ex(cfg: MoEConfig, layer: dict, x, token_ids, T: int, y, ws, events=None,
                   stream=None, side_stream=None):
    """events: None or len(MOE_STAGES) + 1 raw hipEvent_t handles; side_stream:
    None, or a torch stream / raw handle other than `stream`."""
    arr = (ctypes.c_void_p * len(events))(*events) if events is not None else None
    side = None if side_stream is None else _stream(side_stream)
    _check(_lib.moe_forward_ex(ctypes.byref(config_c(cfg)), ctypes.byref(weights_c(layer)),
                               _ptr(x), _ptr(token_ids), T, _ptr(y), _ptr(ws),
                               ws.numel() * ws.element_size(), arr, _stream(stream), side),
           "moe_forward_ex")


def moe_forward_noalloc(cfg: MoEConfig, layer: dict, x, token_ids, T: int, y, stream=None):
    """moe_forward on the library's own device array (no workspace argument)."""
    _check(_lib.moe_forward_noalloc(ctypes.byref(config_c(cfg)), ctypes.byref(weights_c(layer)),
                                    _ptr(x), _ptr(token_ids), T, _ptr(y), _stream(stream)),
           "moe_forward_noalloc")


def _config_ref(cfg):
    """byref of a configuration given as MoEConfig or as config_c of one."""
    return ctypes.byref(cfg if isinstance(cfg, MoeConfigC) else config_c(cfg))


def moe_few_workspace_layout(cfg, T: int) -> dict:
    lay = MoeFewLayoutC()
    _check(_lib.moe_few_workspace_layout(_config_ref(cfg), T, ctypes.byref(lay)),
           "moe_few_workspace_layout")
    return {name: getattr(lay, name) for name, _ in MoeFewLayoutC._fields_}


def moe_few_workspace_size(cfg, T: int) -> int:
    return _lib.moe_few_workspace_size(_config_ref(cfg), T)


def _ws_check(where, ws, device):
    """A workspace is memory of the call's device in one piece (None: the library
    refuses it where it needs one)."""
    if ws is None:
        return
    if not ws.is_contiguous():
        raise ValueError(f"{where}: ws is not contiguous")
    if ws.device != device:
        raise ValueError(f"{where}: ws is on {ws.device}, others on {device}")


def _few_check(c: MoeConfigC, layer, x, token_ids, T, y, ws):
    """Types, sizes, contiguity and devices of a call's tensors (None: the library
    refuses it where it needs one); of weights_c's addresses nothing is known."""
    where, device = "moe_forward_few", None
    dt = torch.float32 if c.act_dtype == DTYPE["f32"] else torch.bfloat16
    ids = {ROUTE["hash"]: 1, ROUTE["ngram"]: 2}.get(c.route_mode)
    for name, t, dtype, width in (("x", x, dt, c.dim), ("y", y, dt, c.dim),
                                  ("token_ids", token_ids if ids else None, torch.int32, ids)):
        if t is None:
            continue
        if t.dtype is not dtype:
            raise ValueError(f"{where}: {name} is {t.dtype}, expected {dtype}")
        if t.numel() < T * width or (dtype is dt and t.shape[-1] != width):
            raise ValueError(f"{where}: {name} holds {tuple(t.shape)}, expected {T} x {width}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} is not contiguous")
        device = device or t.device
        if t.device != device:
            raise ValueError(f"{where}: {name} is on {t.device}, others on {device}")
    if not isinstance(layer, MoeWeightsC):
        for name, _ in MoeWeightsC._fields_:
            t = layer.get(name)
            if t is None:
                continue
            if not t.is_contiguous():
                raise ValueError(f"{where}: {name} is not contiguous")
            device = device or t.device
            if t.device != device:
                raise ValueError(f"{where}: {name} is on {t.device}, others on {device}")
    _ws_check(where, ws, device)
    if device is not None and device.type != "cuda":
        raise ValueError(f"{where}: tensors on {device}, expected a GPU")
    if device is not None and device.index != torch.cuda.current_device():
        raise ValueError(f"{where}: tensors on {device}, not the current device")


def moe_forward_few(cfg, layer, x, token_ids, T: int, y, ws, stream=None):
    """moe_forward for T <= MOE_FEW_MAX_TOKENS tokens.  A decode loop may build
    the C structs once and pass them: cfg a MoEConfig or config_c of it, layer
    the weights' dict or weights_c of it.  ws: alloc_few_workspace."""
    c = cfg if isinstance(cfg, MoeConfigC) else config_c(cfg)
    if 0 < T <= MOE_FEW_MAX_TOKENS:
        _few_check(c, layer, x, token_ids, T, y, ws)
    w = layer if isinstance(layer, MoeWeightsC) else weights_c(layer)
    _check(_lib.moe_forward_few(ctypes.byref(c), ctypes.byref(w), _ptr(x), _ptr(token_ids), T,
                                _ptr(y), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                _stream(stream)),
           "moe_forward_few")


_LINEAR_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _linear_config(cfg: LinearConfig, x, y, residual=None) -> MoeLinearConfigC:
    """cfg with the row strides of x, y (or dy) and the residual.  One row has
    none to speak of, whatever its tensor says."""
    return MoeLinearConfigC(
        cfg.rows, cfg.in_dim, cfg.out_dim, DTYPE[cfg.dtype], ACTIVATION[cfg.activation], cfg.limit,
        *(0 if t is None or cfg.rows < 2 else t.stride(0) for t in (x, y, residual)))


def _linear_check(cfg: LinearConfig, where, launches, matrices, contiguous, ws):
    """Types, shapes, strides and devices of a call's tensors (None: not given):
    the library sees addresses only.  launches: whether the call writes anything
    (an empty batch's gradients are written, with zeros)."""
    dt, device = _LINEAR_DTYPE[cfg.dtype], None
    for name, t, shape in matrices:
        if t is None:
            continue
        if t.dtype is not dt or t.shape != shape:
            raise ValueError(f"{where}: {name} is {tuple(t.shape)} {t.dtype}, "
                             f"expected {shape} {dt}")
        if not t.is_contiguous() and t.numel() and (
                t.stride(1) != 1 and shape[1] > 1 or t.stride(0) < shape[1] and shape[0] > 1):
            raise ValueError(f"{where}: {name}'s rows are not contiguous or overlap")
        device = device or t.device
        if t.device != device:
            raise ValueError(f"{where}: {name} is on {t.device}, others on {device}")
    for name, t, shape in contiguous:
        if t is None:
            continue
        if t.dtype is not dt or t.shape != shape:
            raise ValueError(f"{where}: {name} is {tuple(t.shape)} {t.dtype}, "
                             f"expected {shape} {dt}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} is not contiguous")
        device = device or t.device
        if t.device != device:
            raise ValueError(f"{where}: {name} is on {t.device}, others on {device}")
    if not launches:
        return
    _ws_check(where, ws, device)
    if device is None or device.type != "cuda":
        raise ValueError(f"{where}: tensors on {device}, expected a GPU")
    if device.index != torch.cuda.current_device():
        raise ValueError(f"{where}: tensors on {device}, not the current device")


def _raw(t):
    return None if t is None else t.data_ptr()


MOE_LINEAR_MAX_LD = 1 << 20


def moe_linear_workspace_size(cfg: LinearConfig, backward=False, ld_x=0, ld_y=0,
                              ld_residual=0) -> int:
    """Bytes for calls whose tensors have these row strides (0: contiguous)."""
    c = MoeLinearConfigC(cfg.rows, cfg.in_dim, cfg.out_dim, DTYPE[cfg.dtype],
                         ACTIVATION[cfg.activation], cfg.limit, ld_x, ld_y, ld_residual)
    return _lib.moe_linear_workspace_size(ctypes.byref(c), int(bool(backward)))


LINEAR_PRODUCT = {"forward": 0, "dx": 1, "dw": 2}
LINEAR_PATH = ("tiled", "few", "small")


def moe_linear_path(cfg: LinearConfig, product="forward", ld_x=0, ld_y=0) -> tuple:
    """(path, tile rows, tile columns, parts) of a product of calls whose tensors
    have these row strides (0: contiguous)."""
    c = MoeLinearConfigC(cfg.rows, cfg.in_dim, cfg.out_dim, DTYPE[cfg.dtype],
                         ACTIVATION[cfg.activation], cfg.limit, ld_x, ld_y, 0)
    info = MoeLinearPathC()
    _check(_lib.moe_linear_path(ctypes.byref(c), LINEAR_PRODUCT[product], ctypes.byref(info)),
           "moe_linear_path")
    return LINEAR_PATH[info.path], info.tile_rows, info.tile_cols, info.parts


def moe_linear(cfg: LinearConfig, x, w, y, *, bias=None, residual=None, w_up=None, bias_up=None,
               z=None, z_up=None, ws=None, stream=None):
    """y = act(x w^T + bias) + residual; z (and z_up) receive the
    pre-activations that moe_linear_backward takes.  x, y and residual may be
    rows of wider buffers.  ws: alloc_linear_workspace."""
    M, K, N = cfg.rows, cfg.in_dim, cfg.out_dim
    _linear_check(cfg, "moe_linear", cfg.rows > 0,
                  [("x", x, (M, K)), ("y", y, (M, N)), ("residual", residual, (M, N))],
                  [("w", w, (N, K)), ("w_up", w_up, (N, K)), ("bias", bias, (N,)),
                   ("bias_up", bias_up, (N,)), ("z", z, (M, N)), ("z_up", z_up, (M, N))], ws)
    weights = MoeLinearWeightsC(_raw(w), _raw(w_up), _raw(bias), _raw(bias_up))
    _check(_lib.moe_linear(ctypes.byref(_linear_config(cfg, x, y, residual)),
                           ctypes.byref(weights), _raw(x), _raw(residual), _raw(y), _raw(z),
                           _raw(z_up), _raw(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                           _stream(stream)), "moe_linear")


def moe_linear_backward(cfg: LinearConfig, dy, x, w, *, w_up=None, z=None, z_up=None, dx=None,
                        dw=None, dw_up=None, dbias=None, dbias_up=None, ws=None, stream=None):
    """Gradients of moe_linear for dy, into the tensors given (the residual's
    is dy itself)."""
    M, K, N = cfg.rows, cfg.in_dim, cfg.out_dim
    _linear_check(cfg, "moe_linear_backward", True,
                  [("dy", dy, (M, N)), ("x", x, (M, K)), ("dx", dx, (M, K))],
                  [("w", w, (N, K)), ("w_up", w_up, (N, K)), ("z", z, (M, N)),
                   ("z_up", z_up, (M, N)), ("dw", dw, (N, K)), ("dw_up", dw_up, (N, K)),
                   ("dbias", dbias, (N,)), ("dbias_up", dbias_up, (N,))], ws)
    weights = MoeLinearWeightsC(_raw(w), _raw(w_up), None, None)
    grads = MoeLinearGradsC(_raw(dx), _raw(dw), _raw(dw_up), _raw(dbias), _raw(dbias_up),
                            0 if dx is None or M < 2 else dx.stride(0))
    _check(_lib.moe_linear_backward(
        ctypes.byref(_linear_config(cfg, x, dy)), ctypes.byref(weights),
        _raw(x), _raw(dy), _raw(z), _raw(z_up), ctypes.byref(grads), _raw(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
        "moe_linear_backward")


def _tensors_check(where, tensors, ws=None, launches=True):
    """Types, shapes, contiguity and devices of a call's tensors, (name, tensor,
    shape, dtype) each (None: not given, which the library refuses where it needs
    one): it sees addresses only.  ws and the current device, where it launches."""
    device = None
    for name, t, shape, dtype in tensors:
        if t is None:
            continue
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{where}: {name} is {tuple(t.shape)} {t.dtype}, "
                             f"expected {shape} {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} is not contiguous")
        device = device or t.device
        if t.device != device:
            raise ValueError(f"{where}: {name} is on {t.device}, others on {device}")
    if launches:
        _device_check(where, device, ws)


def _device_check(where, device, ws=None):
    _ws_check(where, ws, device)
    if device is None or device.type != "cuda":
        raise ValueError(f"{where}: tensors on {device}, expected a GPU")
    if device.index != torch.cuda.current_device():
        raise ValueError(f"{where}: tensors on {device}, not the current device")


def _as_config_c(cfg):
    return cfg if isinstance(cfg, MoeConfigC) else config_c(cfg)


def _act_dtype(c: MoeConfigC):
    return torch.float32 if c.act_dtype == DTYPE["f32"] else torch.bfloat16


def _sorted_rows(rows):
    return 0 if rows is None else rows.shape[0]


def moe_dispatch(cfg, x, inverse, T: int, rows, stream=None):
    """rows[inverse[t, j]] = x[t] for the T tokens; inverse [T, k] as moe_permute
    writes it.  cfg, here and below: a MoEConfig or config_c of one."""
    c, R = _as_config_c(cfg), _sorted_rows(rows)
    dt, d = _act_dtype(c), c.dim
    _tensors_check("moe_dispatch", (("x", x, (T, d), dt), ("rows", rows, (R, d), dt), (
        "inverse", inverse, (T, c.n_activated_experts), torch.int32)), launches=T > 0 and R > 0)
    _check(_lib.moe_dispatch(ctypes.byref(c), _raw(x), _raw(inverse), T, R, _raw(rows),
                             _stream(stream)), "moe_dispatch")


def moe_dispatch_backward(cfg, drows, inverse, T: int, dx, stream=None):
    """dx[t] = sum over j of drows[inverse[t, j]]."""
    c, R = _as_config_c(cfg), _sorted_rows(drows)
    dt, d = _act_dtype(c), c.dim
    _tensors_check("moe_dispatch_backward", (
        ("drows", drows, (R, d), dt), ("dx", dx, (T, d), dt),
        ("inverse", inverse, (T, c.n_activated_experts), torch.int32)), launches=T > 0)
    _check(_lib.moe_dispatch_backward(ctypes.byref(c), _raw(drows), _raw(inverse), T, R, _raw(dx),
                                      _stream(stream)), "moe_dispatch_backward")


def moe_combine(cfg, rows, inverse, weights, T: int, y, add=None, stream=None):
    """y[t] = sum over j of weights[t, j] rows[inverse[t, j]], + add[t]."""
    c, R = _as_config_c(cfg), _sorted_rows(rows)
    dt, d, pairs = _act_dtype(c), c.dim, (T, c.n_activated_experts)
    _tensors_check("moe_combine", (
        ("rows", rows, (R, d), dt), ("y", y, (T, d), dt), ("add", add, (T, d), dt),
        ("inverse", inverse, pairs, torch.int32), ("weights", weights, pairs, torch.float32)),
        launches=T > 0)
    _check(_lib.moe_combine(ctypes.byref(c), _raw(rows), _raw(inverse), _raw(weights), _raw(add), T,
                            R, _raw(y), _stream(stream)), "moe_combine")


def moe_combine_backward(cfg, dy, rows, inverse, weights, T: int, drows=None, dweights=None,
                         stream=None):
    """Gradients of moe_combine for dy, into the tensors given (add's is dy)."""
    c = _as_config_c(cfg)
    R = _sorted_rows(drows if rows is None else rows)
    dt, d, pairs = _act_dtype(c), c.dim, (T, c.n_activated_experts)
    _tensors_check("moe_combine_backward", (
        ("dy", dy, (T, d), dt), ("rows", rows, (R, d), dt), ("drows", drows, (R, d), dt),
        ("inverse", inverse, pairs, torch.int32), ("weights", weights, pairs, torch.float32),
        ("dweights", dweights, pairs, torch.float32)), launches=T > 0)
    _check(_lib.moe_combine_backward(ctypes.byref(c), _raw(dy), _raw(rows), _raw(inverse),
                                     _raw(weights), T, R, _raw(drows), _raw(dweights),
                                     _stream(stream)), "moe_combine_backward")


_CHECKPOINT_DTYPE = {torch.float32: DTYPE["f32"], torch.bfloat16: DTYPE["bf16"]}


def _checkpoint_check(where, name, m, codes, scales):
    """(rows, cols, row stride) of the matrix and checks of its codes."""
    if m.dtype not in _CHECKPOINT_DTYPE or m.dim() != 2:
        raise ValueError(f"{where}: {name} is {tuple(m.shape)} {m.dtype}, "
                         f"expected a matrix in float32 or bfloat16")
    rows, cols = m.shape
    ld, device = 0, m.device
    if not m.is_contiguous():
        ld, step = m.stride()
        if step != 1 and cols > 1 or ld < cols and rows > 1:
            raise ValueError(f"{where}: {name}'s rows are not contiguous or overlap")
        ld = 0 if rows < 2 else ld
    for other, t, shape in (("codes", codes, (rows, cols)), ("scales", scales, (rows, -(-cols // 32)))):
        if t.dtype is not torch.uint8 or t.shape != shape:
            raise ValueError(f"{where}: {other} is {tuple(t.shape)} {t.dtype}, "
                             f"expected {shape} {torch.uint8}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {other} is not contiguous")
        if t.device != device:
            raise ValueError(f"{where}: {other} is on {t.device}, others on {device}")
    if rows:
        _device_check(where, device)
    return rows, cols, ld


def moe_checkpoint_save(src, codes, scales, limit: float = 0.0, stream=None):
    """The rows of src (which may stand in a wider buffer) in 8 bits: codes [rows,
    cols] and scales [rows, ceil(cols / 32)], uint8."""
    rows, cols, ld = _checkpoint_check("moe_checkpoint_save", "src", src, codes, scales)
    _check(_lib.moe_checkpoint_save(_raw(src), _CHECKPOINT_DTYPE[src.dtype], rows, cols, ld, limit,
                                    _raw(codes), _raw(scales), _stream(stream)),
           "moe_checkpoint_save")


def moe_checkpoint_load(codes, scales, dst, stream=None):
    """The values that moe_checkpoint_save kept, into dst."""
    rows, cols, ld = _checkpoint_check("moe_checkpoint_load", "dst", dst, codes, scales)
    _check(_lib.moe_checkpoint_load(_raw(codes), _raw(scales), _CHECKPOINT_DTYPE[dst.dtype], rows,
                                    cols, ld, _raw(dst), _stream(stream)), "moe_checkpoint_load")


SAVE = {"none": 0, "full": 1, "mxfp8": 2}


def _experts_check(where, c: MoeConfigC, layer, offsets, rows, saved, row_tensors, weight_grads, ws,
                   launches=True):
    dt, E, d, I = _act_dtype(c), c.n_routed_experts, c.dim, c.moe_inter_dim
    tensors = [(n, t, (rows, d), dt) for n, t in row_tensors]
    tensors.append(("offsets", offsets, (E + 1,), torch.int32))
    shapes = {"w_gate": (E, I, d), "w_up": (E, I, d), "w_down": (E, d, I)}
    if not isinstance(layer, MoeWeightsC):     # of weights_c's addresses nothing is known
        tensors += [(n, layer.get(n), s, dt) for n, s in shapes.items()]
    tensors += [(n, t, shapes[n[1:]], dt) for n, t in weight_grads]
    if saved is not None and saved["kind"] != "none":
        mx = saved["kind"] == "mxfp8"
        tensors += [(n, saved[n], (rows, I), torch.uint8 if mx else torch.float32)
                    for n in ("gate", "up")]
        if mx:
            tensors += [(n, saved[n], (rows, I // 32), torch.uint8)
                        for n in ("gate_scales", "up_scales")]
    _tensors_check(where, tensors, ws, launches)


def _saved_c(saved):
    if saved is None:
        return None
    return ctypes.byref(MoeExpertsSavedC(SAVE[saved["kind"]], *(
        _raw(saved.get(n)) for n in ("gate", "up", "gate_scales", "up_scales"))))


def moe_experts_workspace_size(cfg, rows: int, backward=False) -> int:
    return _lib.moe_experts_workspace_size(_config_ref(cfg), rows, int(bool(backward)))


EXPERTS_PRODUCT = {"up": 0, "down": 1, "dh": 2, "dx": 3, "dw_down": 4, "dw": 5}


def moe_experts_path(cfg, rows: int, product: str) -> tuple:
    """(most tile rows, tile columns, whether the weights are streamed) of a product."""
    info = MoeExpertsPathC()
    _check(_lib.moe_experts_path(_config_ref(cfg), rows, EXPERTS_PRODUCT[product],
                                 ctypes.byref(info)), "moe_experts_path")
    return info.tile_rows, info.tile_cols, bool(info.streamed)


def moe_experts(cfg, layer, x, offsets, y, ws, saved=None, stream=None):
    """y = the routed experts' output of the sorted rows x, without gate values.
    offsets [E + 1] int32; saved: alloc_experts_saved, for moe_experts_backward;
    ws: alloc_experts_workspace.  A training loop may build the C structs once and
    pass them: cfg config_c of a MoEConfig, layer weights_c of the dict."""
    c, rows = _as_config_c(cfg), x.shape[0]
    _experts_check("moe_experts", c, layer, offsets, rows, saved, (("x", x), ("y", y)), (), ws,
                   rows > 0)
    w = layer if isinstance(layer, MoeWeightsC) else weights_c(layer)
    _check(_lib.moe_experts(ctypes.byref(c), ctypes.byref(w), _raw(x), _raw(offsets), rows, _raw(y),
                            _saved_c(saved), _raw(ws),
                            0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "moe_experts")


def moe_experts_backward(cfg, layer, x, offsets, dy, saved, grads, ws, stream=None):
    """Gradients of moe_experts for dy, into the tensors of grads (dx, dw_gate,
    dw_up, dw_down; those not there are not wanted)."""
    c, rows = _as_config_c(cfg), dy.shape[0]
    names = [n for n, _ in MoeExpertsGradsC._fields_]
    if not set(grads) <= set(names):
        raise ValueError(f"moe_experts_backward: grads has {sorted(set(grads) - set(names))}")
    _experts_check("moe_experts_backward", c, layer, offsets, rows, saved,
                   (("x", x), ("dy", dy), ("dx", grads.get("dx"))),
                   [(n, grads.get(n)) for n in names[1:]], ws)
    w = layer if isinstance(layer, MoeWeightsC) else weights_c(layer)
    g = MoeExpertsGradsC(*(_raw(grads.get(n)) for n in names))
    _check(_lib.moe_experts_backward(ctypes.byref(c), ctypes.byref(w), _raw(x), _raw(offsets), rows,
                                     _raw(dy), _saved_c(saved), ctypes.byref(g), _raw(ws),
                                     0 if ws is None else ws.numel() * ws.element_size(),
                                     _stream(stream)), "moe_experts_backward")


class HipEvents:
    """Raw HIP timing events from the HIP runtime torch already loaded."""

    def __init__(self, n):
        self.hip = ctypes.CDLL("libamdhip64.so.7")
        self.hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                                 ctypes.c_void_p]
        self.handles = []
        for _ in range(n):
            h = ctypes.c_void_p()
            if self.hip.hipEventCreate(ctypes.byref(h)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self.handles.append(h.value)

    def elapsed_ms(self, a, b):
        ms = ctypes.c_float()
        if self.hip.hipEventElapsedTime(ctypes.byref(ms), ctypes.c_void_p(self.handles[a]),
                                        ctypes.c_void_p(self.handles[b])) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return ms.value

    def close(self):
        for h in self.handles:
            self.hip.hipEventDestroy(ctypes.c_void_p(h))
        self.handles = []


# ---------------------------------------------------------------------------
# Convenience views of a forward workspace (no computation).

def alloc_workspace(cfg: MoEConfig, T: int, device="cuda"):
    size = moe_workspace_size(cfg, T)
    if size == 0:
        raise MoEError(moe_validate_config(cfg), "moe_workspace_size")
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(size, dtype=torch.uint8, device=device)


def workspace_views(cfg: MoEConfig, T: int, ws):
    """Typed views of the routing, permutation and intermediate buffers."""
    lay = moe_workspace_layout(cfg, T)
    k, E = cfg.n_activated_experts, cfg.n_routed_experts
    rows = T * k + T * cfg.n_shared_experts
    edt = torch.float32 if cfg.act_dtype == "f32" else torch.bfloat16

    def view(off, n, dtype):
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return ws[off:off + nbytes].view(dtype)

    out = {
        "route_weights": view(lay["route_weights"], T * k, torch.float32).view(T, k),
        "route_indices": view(lay["route_indices"], T * k, torch.int32).view(T, k),
        "counts": view(lay["counts"], E, torch.int32),
        "offsets": view(lay["offsets"], E + 1, torch.int32),
        "sorted_tok": view(lay["sorted_tok"], T * k + T, torch.int32),
        "sorted_slot": view(lay["sorted_slot"], T * k, torch.int32),
        "sorted_weight": view(lay["sorted_weight"], T * k, torch.float32),
        "inverse": view(lay["inverse"], T * k, torch.int32).view(T, k),
        "tiles": view(lay["tiles"], 4 * lay["max_tiles"], torch.int32).view(-1, 4),
        "tile_count": view(lay["tile_count"], 1, torch.int32),
        "flags": view(lay["flags"], 4, torch.int32),
        "perm_hist": view(lay["perm_hist"], (-(-T * k // 256) + 1) * E, torch.int32),
        "h": view(lay["h"], rows * cfg.moe_inter_dim, edt).view(rows, cfg.moe_inter_dim),
        "yrows": view(lay["yrows"], rows * cfg.dim, edt).view(rows, cfg.dim),
        "layout": lay,
    }
    if cfg.act_quant == "mxfp8":
        I = cfg.moe_inter_dim
        out["xq"] = view(lay["xq"], T * cfg.dim, torch.uint8).view(T, cfg.dim)
        out["xq_scales"] = view(lay["xq_scales"], T * cfg.dim // 32, torch.uint8).view(T, -1)
        out["hq"] = view(lay["hq"], T * k * I, torch.uint8).view(T * k, I)
        out["hq_scales"] = view(lay["hq_scales"], T * k * I // 32, torch.uint8).view(T * k, -1)
    return out


def alloc_few_workspace(cfg, T: int, device="cuda"):
    """Workspace of moe_forward_few for up to T tokens of this configuration."""
    lay = moe_few_workspace_layout(cfg, T)
    return torch.empty(max(lay["total_bytes"], 1), dtype=torch.uint8, device=device)


def few_views(cfg: MoEConfig, T: int, ws):
    """Routing and flags a moe_forward_few call left in its workspace."""
    lay = moe_few_workspace_layout(cfg, T)
    k = cfg.n_activated_experts

    def view(off, n, dtype):
        return ws[off:off + 4 * n].view(dtype)

    return {
        "route_weights": view(lay["route_weights"], T * k, torch.float32).view(T, k),
        "route_indices": view(lay["route_indices"], T * k, torch.int32).view(T, k),
        "flags": view(lay["flags"], 4, torch.int32),
        "layout": lay,
    }


def alloc_linear_workspace(cfg: LinearConfig, backward=False, device="cuda", **strides):
    """Workspace of moe_linear, or with `backward` one that serves both it and
    moe_linear_backward.  strides: ld_x, ld_y, ld_residual; without them it is
    large enough for tensors of any strides."""
    ways = [strides]
    if not strides:
        # what a call needs goes by which of its row strides are odd
        ways = [{"ld_x": cfg.in_dim + i, "ld_y": cfg.out_dim + j} for i in (0, 1) for j in (0, 1)
                if max(cfg.in_dim + i, cfg.out_dim + j) <= MOE_LINEAR_MAX_LD]
    sizes = [moe_linear_workspace_size(cfg, k, **w) for k in {False, bool(backward)} for w in ways]
    if not sizes:
        raise MoEError(MOE_ERR_UNSUPPORTED, "moe_linear_workspace_size")
    if 0 in sizes:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_linear_workspace_size")
    return torch.empty(max(sizes), dtype=torch.uint8, device=device)


def alloc_experts_workspace(cfg, rows: int, backward=False, device="cuda"):
    """Workspace of moe_experts for up to `rows` sorted rows, or with `backward` one
    that serves both it and moe_experts_backward."""
    size = moe_experts_workspace_size(cfg, rows, backward)
    if size == 0:
        raise MoEError(MOE_ERR_UNSUPPORTED, "moe_experts_workspace_size")
    return torch.empty(size, dtype=torch.uint8, device=device)


def alloc_experts_saved(cfg, rows: int, kind="mxfp8", device="cuda") -> dict:
    """Where moe_experts saves the pre-activations of `rows` sorted rows: kind "full"
    in fp32, "mxfp8" in 8 bits with a scale per 32."""
    I, dt = _as_config_c(cfg).moe_inter_dim, torch.uint8 if kind == "mxfp8" else torch.float32
    saved = {"kind": kind}
    if kind != "none":
        saved.update({n: torch.empty((rows, I), dtype=dt, device=device) for n in ("gate", "up")})
    if kind == "mxfp8":
        saved.update({n: torch.empty((rows, I // 32), dtype=torch.uint8, device=device)
                      for n in ("gate_scales", "up_scales")})
    elif kind not in SAVE:
        raise ValueError(f"alloc_experts_saved: kind {kind!r}, expected one of {sorted(SAVE)}")
    return saved
