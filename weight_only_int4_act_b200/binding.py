"""Python binding of the C ABI in include/awq.h (ctypes; argument marshalling only).

Every computation runs in the CUDA library; PyTorch only provides device
memory and the current stream. If the library is missing the calls raise:
there is no fallback.

Two builds of the library exist (see _build.py): "release" and "check", the
debug build with index checks. The environment variable AWQ_B200_LIB
(release | check) picks the one loaded at first use; select_library()
switches later calls to the other.
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import POINTER, c_char_p, c_float, c_int32, c_int64, c_size_t, c_void_p

from ._build import VARIANTS, calls_path, lib_path

AWQ_OK = 0
STATUS_NAMES = {
    0: "AWQ_OK", 1: "AWQ_ERR_INVALID_ARG", 2: "AWQ_ERR_SHAPE", 3: "AWQ_ERR_WORKSPACE",
    4: "AWQ_ERR_NONFINITE", 5: "AWQ_ERR_CUDA", 6: "AWQ_ERR_DEVICE", 7: "AWQ_ERR_UNSUPPORTED",
    8: "AWQ_ERR_BOUNDS",
}
AWQ_ERR_BOUNDS = 8
BOUNDS_SITE_SELFTEST = 0x7F
FORMS = {"auto": 0, "direct": 1, "gram": 2}
AWQ_DTYPE_BF16, AWQ_DTYPE_F16 = 0, 1

# every symbol include/awq.h declares
EXPORTED = (
    "awq_status_str", "awq_stats_workspace_size", "awq_act_stats", "awq_search_workspace_size",
    "awq_search_scales", "awq_search_form", "awq_workspace_error", "awq_quantize_pack",
    "awq_step_scales", "awq_step_fake_quant", "awq_step_gram", "awq_step_contract", "awq_step_reduce",
    "awq_debug_copy_dw", "awq_act_stats_noalloc", "awq_search_scales_segmented", "awq_search_candidates",
    "awq_quantize_pack_clipped", "awq_group_clip_workspace_size", "awq_search_group_clip",
    "awq_quantize_pack_group_clip", "awq_fold_inv_scales", "awq_w4a16_workspace_size", "awq_w4a16_gemm",
    "awq_pack_workspace_size", "awq_quantize_pack_ws", "awq_selftest_bounded_wait",
    "awq_bounds_checks_enabled", "awq_bounds_error", "awq_selftest_bounds",
    "awq_quantize_int8", "awq_w8a8_workspace_size", "awq_w8a8_gemm", "awq_kv4_page_bytes", "awq_kv4_append",
    "awq_kv4_gather", "awq_kv4_attention_workspace_size", "awq_kv4_attention", "awq_device_error",
)


class AwqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")


class QCfg(ctypes.Structure):
    _fields_ = [
        ("bits", c_int32), ("group", c_int32), ("symmetric", c_int32), ("n_alpha", c_int32),
        ("form", c_int32), ("eps_a", c_float), ("alphas", POINTER(c_float)),
    ]


def make_cfg(bits=4, group=128, symmetric=False, n_alpha=20, form="auto", eps_a=1e-4, alphas=None) -> QCfg:
    cfg = QCfg(int(bits), int(group), int(bool(symmetric)), int(n_alpha), FORMS[form], float(eps_a), None)
    if alphas is not None:
        arr = (c_float * len(alphas))(*[float(x) for x in alphas])
        cfg.alphas = ctypes.cast(arr, POINTER(c_float))
        cfg._keep = arr  # keep the host array alive with the struct
    return cfg


class Kv4Cfg(ctypes.Structure):
    """Shape of a 4-bit key/value cache (awq_kv4cfg)."""
    _fields_ = [("n_kv_heads", c_int32), ("head_dim", c_int32), ("page_size", c_int32), ("group", c_int32)]


def make_kv4(n_kv_heads, head_dim, page_size=64, group=None) -> Kv4Cfg:
    """group=None: the widest one that divides head_dim."""
    if group is None:
        group = next((g for g in (128, 64, 32) if head_dim % g == 0), 0)
    return Kv4Cfg(int(n_kv_heads), int(head_dim), int(page_size), int(group))


_libs = {}
_active = os.environ.get("AWQ_B200_LIB", "release")


def select_library(variant: str) -> str:
    """Route later calls to the given build ("release" or "check"); returns
    the previous choice."""
    global _active
    if variant not in VARIANTS:
        raise ValueError(f"unknown library build {variant!r}; one of {sorted(VARIANTS)}")
    prev, _active = _active, variant
    return prev


def lib() -> ctypes.CDLL:
    """The selected build of the CUDA library (raises if it has not been built)."""
    if _active in _libs:
        return _libs[_active]
    if _active not in VARIANTS:
        raise ValueError(f"AWQ_B200_LIB={_active!r}; one of {sorted(VARIANTS)}")
    if _active not in _libs:
        path = lib_path(_active)
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing; build it with __graft_entry__.build()")
        L = ctypes.CDLL(path)
        cfgp = POINTER(QCfg)
        sig = {
            "awq_status_str": (c_char_p, [c_int32]),
            "awq_stats_workspace_size": (c_size_t, [c_int64, c_int64]),
            "awq_act_stats": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_size_t, c_void_p]),
            "awq_act_stats_noalloc": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p]),
            "awq_search_workspace_size": (c_size_t, [c_int64, c_int64, c_int64, cfgp]),
            "awq_search_form": (c_int32, [c_int64, c_int64, c_int64, cfgp]),
            "awq_search_scales": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int64, cfgp,
                                            c_void_p, c_size_t, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
            "awq_search_scales_segmented": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int64, cfgp,
                                                      c_int32, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p,
                                                      c_void_p, c_void_p, c_void_p]),
            "awq_search_candidates": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int64,
                                                cfgp, c_void_p, c_size_t, c_void_p, c_void_p, c_void_p, c_void_p,
                                                c_void_p]),
            "awq_quantize_pack_clipped": (c_int32, [c_void_p, c_void_p, c_int64, c_int64, cfgp, c_float, c_void_p,
                                                    c_void_p, c_void_p, c_void_p]),
            "awq_group_clip_workspace_size": (c_size_t, [c_int64, c_int64, c_int64, cfgp]),
            "awq_search_group_clip": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int64,
                                                cfgp, c_void_p, c_size_t, c_void_p, c_void_p, c_void_p]),
            "awq_quantize_pack_group_clip": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_int64,
                                                       c_int64, cfgp, c_void_p, c_void_p, c_void_p, c_void_p]),
            "awq_fold_inv_scales": (c_int32, [c_void_p, c_int64, c_void_p, c_int32, c_int64, c_void_p]),
            "awq_w4a16_workspace_size": (c_size_t, [c_int64, c_int64, c_int64, cfgp]),
            "awq_w4a16_gemm": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int64,
                                         cfgp, c_void_p, c_void_p, c_size_t, c_void_p]),
            "awq_pack_workspace_size": (c_size_t, [c_int64, c_int64, cfgp]),
            "awq_quantize_pack_ws": (c_int32, [c_void_p, c_void_p, c_int64, c_int64, cfgp, c_float, c_void_p,
                                               c_size_t, c_void_p, c_void_p, c_void_p, c_void_p]),
            "awq_selftest_bounded_wait": (c_int32, [c_void_p, c_void_p]),
            "awq_bounds_checks_enabled": (c_int32, []),
            "awq_bounds_error": (c_int32, [POINTER(c_int32), c_void_p]),
            "awq_selftest_bounds": (c_int32, [c_void_p, c_size_t, c_void_p]),
            "awq_workspace_error": (c_int32, [c_void_p, c_void_p]),
            "awq_quantize_pack": (c_int32, [c_void_p, c_void_p, c_int64, c_int64, cfgp, c_void_p, c_void_p,
                                            c_void_p, c_void_p]),
            "awq_step_scales": (c_int32, [c_void_p, c_int64, c_int64, c_int64, cfgp, c_void_p, c_size_t, c_void_p]),
            "awq_step_fake_quant": (c_int32, [c_void_p, c_int64, c_int64, c_int64, cfgp, c_void_p, c_size_t,
                                              c_void_p]),
            "awq_step_gram": (c_int32, [c_void_p, c_int64, c_int64, c_int64, cfgp, c_void_p, c_size_t, c_void_p]),
            "awq_step_contract": (c_int32, [c_void_p, c_int64, c_int64, c_int64, cfgp, c_void_p, c_size_t,
                                            c_void_p]),
            "awq_step_reduce": (c_int32, [c_int64, c_int64, c_int64, cfgp, c_void_p, c_size_t, c_void_p, c_void_p,
                                          c_void_p, c_void_p, c_void_p]),
            "awq_debug_copy_dw": (c_int32, [c_void_p, c_int64, c_int64, c_int64, cfgp, c_int32, c_void_p,
                                            c_void_p]),
        }
        kvp = POINTER(Kv4Cfg)
        sig |= {
            "awq_quantize_int8": (c_int32, [c_void_p, c_int32, c_int64, c_void_p, c_int32, c_int64, c_int64, c_void_p,
                                            c_void_p, c_void_p]),
            "awq_device_error": (c_int32, [c_void_p]),
            "awq_w8a8_workspace_size": (c_size_t, [c_int64, c_int64, c_int64]),
            "awq_w8a8_gemm": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int64, c_int64,
                                        c_int64, c_void_p, c_void_p, c_size_t, c_void_p]),
            "awq_kv4_page_bytes": (c_size_t, [kvp]),
            "awq_kv4_append": (c_int32, [c_void_p, c_void_p, c_int32, c_int64, c_int64, c_int64, c_int64, c_int64,
                                         c_void_p, c_void_p, c_int64, kvp, c_void_p]),
            "awq_kv4_gather": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, kvp, c_void_p, c_void_p, c_int32,
                                         c_void_p]),
            "awq_kv4_attention_workspace_size": (c_size_t, [c_int64, c_int64, c_int64, kvp]),
            "awq_kv4_attention": (c_int32, [c_void_p, c_int32, c_int64, c_int64, c_int64, c_int64, c_void_p, c_int64,
                                            c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_float, kvp,
                                            c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _libs[_active] = L
    return _libs[_active]


def status_str(status: int) -> str:
    return lib().awq_status_str(status).decode()


def _check(status: int, what: str):
    if status != AWQ_OK:
        raise AwqError(status, what)


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _stream():
    return c_void_p(_torch().cuda.current_stream().cuda_stream)


def _req(t, dtype, shape, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ptr(t):
    return c_void_p(t.data_ptr()) if t is not None else None


# --------------------------------------------------------------------------- sizes
def stats_workspace_size(N: int, d_in: int) -> int:
    return int(lib().awq_stats_workspace_size(N, d_in))


def search_workspace_size(d_out: int, d_in: int, N: int, cfg: QCfg) -> int:
    return int(lib().awq_search_workspace_size(d_out, d_in, N, ctypes.byref(cfg)))


def search_form(d_out: int, d_in: int, N: int, cfg: QCfg) -> str:
    f = int(lib().awq_search_form(d_out, d_in, N, ctypes.byref(cfg)))
    return {1: "direct", 2: "gram"}.get(f, "invalid")


def workspace(nbytes: int):
    torch = _torch()
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------- a1
def act_stats(X, ws=None, out=None):
    """a[i] = mean_t |X[t, i]| for bf16 X [N, d_in] (float32 [d_in])."""
    torch = _torch()
    _req(X, torch.bfloat16, None, "X")
    N, d_in = X.shape
    if ws is None:
        ws = workspace(stats_workspace_size(N, d_in))
    a = out if out is not None else torch.empty(d_in, dtype=torch.float32, device=X.device)
    _check(lib().awq_act_stats(_ptr(X), N, d_in, _ptr(a), _ptr(ws), ws.numel(), _stream()), "awq_act_stats")
    return a


# --------------------------------------------------------------------------- a2-a6
def search_scales(W, X, a, cfg: QCfg, ws=None, row_losses=False, outputs=None):
    """Loss of every alpha, the chosen index and its scales (device tensors).

    Returns dict(losses float32[n_alpha], best int32[1], s_best float32[d_in],
    row_losses float32[n_alpha, d_out] or None, ws)."""
    torch = _torch()
    _req(W, torch.bfloat16, None, "W")
    d_out, d_in = W.shape
    _req(X, torch.bfloat16, None, "X")
    N = X.shape[0]
    if X.shape[1] != d_in:
        raise ValueError("X must have d_in columns")
    _req(a, torch.float32, (d_in,), "a")
    if ws is None:
        ws = workspace(search_workspace_size(d_out, d_in, N, cfg))
    if outputs is None:
        outputs = dict(
            losses=torch.empty(cfg.n_alpha, dtype=torch.float32, device=W.device),
            best=torch.empty(1, dtype=torch.int32, device=W.device),
            s_best=torch.empty(d_in, dtype=torch.float32, device=W.device),
            row_losses=torch.empty((cfg.n_alpha, d_out), dtype=torch.float32, device=W.device) if row_losses else None,
        )
    o = outputs
    _check(lib().awq_search_scales(_ptr(W), _ptr(X), _ptr(a), d_out, d_in, N, ctypes.byref(cfg), _ptr(ws),
                                   ws.numel(), _ptr(o["losses"]), _ptr(o["best"]), _ptr(o["s_best"]),
                                   _ptr(o["row_losses"]), _stream()), "awq_search_scales")
    return dict(o, ws=ws)


def search_scales_segmented(W, X, a, cfg: QCfg, seg_rows, ws=None, row_losses=False):
    """Per-layer search for layers sharing X; W is their row concatenation and
    seg_rows the row count of each layer. Returns dict(losses float32[n_seg,
    n_alpha], best int32[n_seg], s_best float32[n_seg, d_in], row_losses, ws)."""
    torch = _torch()
    _req(W, torch.bfloat16, None, "W")
    d_out, d_in = W.shape
    _req(X, torch.bfloat16, None, "X")
    N = X.shape[0]
    if X.shape[1] != d_in:
        raise ValueError("X must have d_in columns")
    _req(a, torch.float32, (d_in,), "a")
    n_seg = len(seg_rows)
    rows = (ctypes.c_int64 * max(n_seg, 1))(*[int(r) for r in seg_rows])
    if ws is None:
        ws = workspace(search_workspace_size(d_out, d_in, N, cfg))
    o = dict(losses=torch.empty((n_seg, cfg.n_alpha), dtype=torch.float32, device=W.device),
             best=torch.empty(n_seg, dtype=torch.int32, device=W.device),
             s_best=torch.empty((n_seg, d_in), dtype=torch.float32, device=W.device),
             row_losses=torch.empty((cfg.n_alpha, d_out), dtype=torch.float32, device=W.device) if row_losses else None)
    _check(lib().awq_search_scales_segmented(_ptr(W), _ptr(X), _ptr(a), d_out, d_in, N, ctypes.byref(cfg), n_seg,
                                             ctypes.cast(rows, c_void_p), _ptr(ws), ws.numel(), _ptr(o["losses"]),
                                             _ptr(o["best"]), _ptr(o["s_best"]), _ptr(o["row_losses"]), _stream()),
           "awq_search_scales_segmented")
    return dict(o, ws=ws)


def search_candidates(W, X, s_cand, cfg: QCfg, clips=None, ws=None, row_losses=False):
    """Losses of explicit candidates: scale vectors s_cand float32 [n, d_in] (CUDA)
    and optional clip ratios (host sequence of n floats in (0, 1]); n must equal
    cfg.n_alpha. Returns dict(losses, best, s_best, row_losses, ws)."""
    torch = _torch()
    _req(W, torch.bfloat16, None, "W")
    d_out, d_in = W.shape
    _req(X, torch.bfloat16, None, "X")
    N = X.shape[0]
    _req(s_cand, torch.float32, (cfg.n_alpha, d_in), "s_cand")
    carr = None
    if clips is not None:
        if len(clips) != cfg.n_alpha:
            raise ValueError("need one clip ratio per candidate")
        carr = (c_float * len(clips))(*[float(c) for c in clips])
    if ws is None:
        ws = workspace(search_workspace_size(d_out, d_in, N, cfg))
    o = dict(losses=torch.empty(cfg.n_alpha, dtype=torch.float32, device=W.device),
             best=torch.empty(1, dtype=torch.int32, device=W.device),
             s_best=torch.empty(d_in, dtype=torch.float32, device=W.device),
             row_losses=torch.empty((cfg.n_alpha, d_out), dtype=torch.float32, device=W.device) if row_losses else None)
    _check(lib().awq_search_candidates(_ptr(W), _ptr(X), _ptr(s_cand), ctypes.cast(carr, c_void_p) if carr else None,
                                       d_out, d_in, N, ctypes.byref(cfg), _ptr(ws), ws.numel(), _ptr(o["losses"]),
                                       _ptr(o["best"]), _ptr(o["s_best"]), _ptr(o["row_losses"]), _stream()),
           "awq_search_candidates")
    return dict(o, ws=ws)


def group_clip_workspace_size(d_out, d_in, N, cfg: QCfg) -> int:
    return int(lib().awq_group_clip_workspace_size(d_out, d_in, N, ctypes.byref(cfg)))


def _clip_array(clips, n):
    if len(clips) != n:
        raise ValueError("need one clip ratio per candidate")
    return (c_float * n)(*[float(c) for c in clips])


def search_group_clip(W, X, s, clips, cfg: QCfg, ws=None, group_err=False):
    """Per-(row, group) clip choice with the scales s fixed: clips is a host
    sequence of cfg.n_alpha ratios. Returns dict(best_clip uint8 [d_out, d_in/g],
    group_err float32 [n, d_out, d_in/g] or None, ws)."""
    torch = _torch()
    _req(W, torch.bfloat16, None, "W")
    d_out, d_in = W.shape
    _req(X, torch.bfloat16, None, "X")
    N = X.shape[0]
    _req(s, torch.float32, (d_in,), "s")
    carr = _clip_array(clips, cfg.n_alpha)
    if ws is None:
        ws = workspace(group_clip_workspace_size(d_out, d_in, N, cfg))
    ng = d_in // cfg.group if cfg.group > 0 else 0
    o = dict(best_clip=torch.empty((d_out, ng), dtype=torch.uint8, device=W.device),
             group_err=torch.empty((cfg.n_alpha, d_out, ng), dtype=torch.float32, device=W.device)
             if group_err else None)
    _check(lib().awq_search_group_clip(_ptr(W), _ptr(X), _ptr(s), ctypes.cast(carr, c_void_p), d_out, d_in, N,
                                       ctypes.byref(cfg), _ptr(ws), ws.numel(), _ptr(o["best_clip"]),
                                       _ptr(o["group_err"]), _stream()), "awq_search_group_clip")
    return dict(o, ws=ws)


def quantize_pack_group_clip(W, s, clips, best_clip, cfg: QCfg, outputs=None):
    """quantize_pack with group j of row r clipped at clips[best_clip[r, j]]."""
    torch = _torch()
    _req(W, torch.bfloat16, None, "W")
    d_out, d_in = W.shape
    _req(s, torch.float32, (d_in,), "s")
    ng = d_in // cfg.group if cfg.group > 0 else 0
    _req(best_clip, torch.uint8, (d_out, ng), "best_clip")
    carr = _clip_array(clips, len(clips))
    if outputs is None:
        outputs = (torch.empty((d_out, d_in // 8), dtype=torch.int32, device=W.device),
                   torch.empty((d_out, ng), dtype=torch.float16, device=W.device),
                   torch.empty((d_out, ng), dtype=torch.float16, device=W.device))
    q, sc, zr = outputs
    _check(lib().awq_quantize_pack_group_clip(_ptr(W), _ptr(s), ctypes.cast(carr, c_void_p), len(clips),
                                              _ptr(best_clip), d_out, d_in, ctypes.byref(cfg), _ptr(q), _ptr(sc),
                                              _ptr(zr), _stream()), "awq_quantize_pack_group_clip")
    return q, sc, zr


# --------------------------------------------------------------------------- inference side
def _dtype_code(t, name):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return AWQ_DTYPE_BF16
    if t.dtype == torch.float16:
        return AWQ_DTYPE_F16
    raise ValueError(f"{name} must be bfloat16 or float16, got {t.dtype}")


def fold_inv_scales(s, p):
    """In place: row i of p (bf16 or fp16 [d_in] or [d_in, inner], CUDA) becomes p / s_i."""
    torch = _torch()
    _req(s, torch.float32, None, "s")
    dt = _dtype_code(p, "p")
    _req(p, p.dtype, None, "p")
    d_in = s.numel()
    if p.shape[0] != d_in:
        raise ValueError("p must have the channel (length of s) on its first axis")
    inner = p.numel() // d_in if d_in else 0
    _check(lib().awq_fold_inv_scales(_ptr(s), d_in, _ptr(p), dt, inner, _stream()), "awq_fold_inv_scales")
    return p


def w4a16_workspace_size(N, d_out, d_in, cfg: QCfg) -> int:
    return int(lib().awq_w4a16_workspace_size(N, d_out, d_in, ctypes.byref(cfg)))


def w4a16_gemm(Xp, qweight, scales, zeros, cfg: QCfg, ws=None, out=None):
    """Y [N, d_out] = X' ([N, d_in], fp16 or bf16) times the dequantised packed
    weights, in the activations' type."""
    torch = _torch()
    dt = _dtype_code(Xp, "X")
    _req(Xp, Xp.dtype, None, "X")
    N, d_in = Xp.shape
    _req(qweight, torch.int32, None, "qweight")
    d_out = qweight.shape[0]
    if qweight.shape != (d_out, d_in // 8):
        raise ValueError("qweight must be [d_out, d_in/8]")
    ng = d_in // cfg.group if cfg.group > 0 else 0
    _req(scales, torch.float16, (d_out, ng), "scales")
    _req(zeros, torch.float16, (d_out, ng), "zeros")
    if ws is None:
        ws = workspace(max(w4a16_workspace_size(N, d_out, d_in, cfg), 256))
    if out is None:
        out = torch.empty((N, d_out), dtype=Xp.dtype, device=Xp.device)
    _req(out, Xp.dtype, (N, d_out), "out")
    _check(lib().awq_w4a16_gemm(_ptr(Xp), dt, _ptr(qweight), _ptr(scales), _ptr(zeros), N, d_out, d_in,
                                ctypes.byref(cfg), _ptr(out), _ptr(ws), ws.numel(), _stream()), "awq_w4a16_gemm")
    return out


# The calls below are made once a layer and token, so their checks are short:
# one expression for a good argument, the full checks only to name what is wrong.
@functools.lru_cache(maxsize=None)
def _torch_names():
    """(Tensor, current_device, raw stream of a device, 16-bit types by code) of torch."""
    torch = _torch()
    torch.cuda.init()
    return (torch.Tensor, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream,
            {torch.bfloat16: AWQ_DTYPE_BF16, torch.float16: AWQ_DTYPE_F16})


def _here(t, name):
    """(current device, its current stream, ...): t must be a CUDA tensor of that device."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    _, current, stream, codes = _torch_names()
    dev = current()
    _same_device(t, dev, name)
    return dev, stream(dev), codes


def _same_device(t, dev, name):
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")


def _req_here(t, dtype, shape, dev, name):
    """A contiguous tensor of device dev (calls run on its current stream)."""
    if isinstance(t, _torch_names()[0]) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and (
            shape is None or t.shape == shape):
        return
    _req(t, dtype, shape, name)
    _same_device(t, dev, name)


def _req_rows(t, dtype, shape, dev, name):
    """A tensor of device dev whose last axis is contiguous; the others may be strided."""
    if not (isinstance(t, _torch_names()[0]) and t.dtype is dtype and t.get_device() == dev and t.shape == shape):
        if not isinstance(t, _torch_names()[0]):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
            raise ValueError(
                f"{name} must have shape {tuple('*' if n is None else n for n in shape)}, got {tuple(t.shape)}")
        _same_device(t, dev, name)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")


def _pitch(t, axis):
    """Elements from one entry of an axis to the next (the stride of a single entry means nothing)."""
    return t.stride(axis) if t.shape[axis] > 1 else 0


def _code(dtype, codes, name):
    code = codes.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float16, got {dtype}")
    return code


def _scratch(like, nbytes):
    return like.new_empty(max(nbytes, 256), dtype=_torch().uint8)


@functools.lru_cache(maxsize=None)
def _calls(variant):
    """The serving calls of csrc/torch_calls.cpp on a build of the library. Each
    returns its results, a status, or None for arguments that the functions
    below have to look at."""
    import importlib.machinery
    import importlib.util
    import types
    _torch()  # whose libraries the module needs
    path = calls_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing; build it with __graft_entry__.build()")
    loader = importlib.machinery.ExtensionFileLoader("awq_calls", path)
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("awq_calls", loader))
    loader.exec_module(m)
    L = lib()
    at = lambda name: ctypes.cast(getattr(L, name), c_void_p).value  # noqa: E731
    p = functools.partial
    return types.SimpleNamespace(
        quantize_int8=p(m.quantize_int8, at("awq_quantize_int8")), w8a8_gemm=p(m.w8a8_gemm, at("awq_w8a8_gemm")),
        kv4_append=p(m.kv4_append, at("awq_kv4_append")), kv4_gather=p(m.kv4_gather, at("awq_kv4_gather")),
        kv4_attention=p(m.kv4_attention, at("awq_kv4_attention"), at("awq_kv4_attention_workspace_size")))


@functools.lru_cache(maxsize=None)
def _unread(dev):
    """An error word for calls that have no workspace of their own, where the workspace is nothing else: device_error()
    tells what goes wrong in them."""
    return _torch().empty(1024, dtype=_torch().uint8, device=f"cuda:{dev}")


# --------------------------------------------------------------------------- 8-bit integer linear layer
def quantize_int8(X, s=None, inverse=False, outputs=None):
    """Codes int8 [rows, d_in] and steps float32 [rows] of the symmetric 8-bit
    quantiser, one step per row, of X (bf16 or fp16 [rows, d_in]; rows may be
    strided, and none is no work). s (float32 [d_in]): the channels are
    multiplied by it first (a weight: W S) or, with inverse=True, by 1 / s
    (activations: X S^-1); without it X is taken as it is."""
    if outputs is None:
        r = _calls(_active).quantize_int8(X, s, 2 if inverse else 1)
        if r.__class__ is tuple:
            return r
        _check(r or AWQ_OK, "awq_quantize_int8")
    torch = _torch()
    dev, stream, codes = _here(X, "X")
    dt = _code(X.dtype, codes, "X")
    rows, d_in = X.shape if X.dim() == 2 else (None, None)
    _req_rows(X, X.dtype, (rows, d_in), dev, "X")
    mode = 0
    if s is not None:
        _req_here(s, torch.float32, (d_in,), dev, "s")
        mode = 2 if inverse else 1
    if outputs is None:
        q = torch.empty_strided((rows, d_in), (d_in, 1), dtype=torch.int8, device=X.device)
        step = X.new_empty(rows, dtype=torch.float32)
    else:
        q, step = outputs
        _req_here(q, torch.int8, (rows, d_in), dev, "q")
        _req_here(step, torch.float32, (rows,), dev, "step")
    if rows == 0 and w8a8_workspace_size(1, 1, d_in):  # (a d_in that the library takes)
        return q, step
    st = lib().awq_quantize_int8(X.data_ptr(), dt, X.stride(0) if rows > 1 else max(d_in, 8),
                                 None if s is None else s.data_ptr(), mode, rows, d_in, q.data_ptr(), step.data_ptr(),
                                 stream)
    _check(st, "awq_quantize_int8")
    return q, step


@functools.lru_cache(maxsize=4096)
def w8a8_workspace_size(N, d_out, d_in) -> int:
    return int(lib().awq_w8a8_workspace_size(N, d_out, d_in))


def w8a8_gemm(xq, x_step, wq, w_step, dtype=None, bias=None, ws=None, out=None):
    """Y [N, d_out] (dtype bf16 by default, or fp16) = (xq wq^T) * x_step[:, None]
    * w_step (+ bias, float32 [d_out]), the integer sum exact; xq int8 [N, d_in]
    (no tokens: no work) and wq int8 [d_out, d_in] with their steps from quantize_int8. What the device
    finds wrong is in device_error(), and in workspace_error(ws) for a call with
    a workspace of its own."""
    torch = _torch()
    if out is None and ws is None and dtype in (None, torch.bfloat16, torch.float16):
        r = _calls(_active).w8a8_gemm(xq, x_step, wq, w_step, bias, dtype is torch.float16,
                                      _unread(_torch_names()[1]()) if isinstance(xq, torch.Tensor) and xq.is_cuda else None)
        if isinstance(r, torch.Tensor):
            return r
        _check(r or AWQ_OK, "awq_w8a8_gemm")
    dev, stream, codes = _here(xq, "xq")
    _req_here(xq, torch.int8, None, dev, "xq")
    _req_here(wq, torch.int8, None, dev, "wq")
    if xq.dim() != 2 or wq.dim() != 2 or xq.shape[1] != wq.shape[1]:
        raise ValueError("xq must be [N, d_in] and wq [d_out, d_in]")
    N, d_in = xq.shape
    d_out = wq.shape[0]
    _req_here(x_step, torch.float32, (N,), dev, "x_step")
    _req_here(w_step, torch.float32, (d_out,), dev, "w_step")
    if bias is not None:
        _req_here(bias, torch.float32, (d_out,), dev, "bias")
    if out is None:
        dt = _code(dtype or torch.bfloat16, codes, "out")
        out = torch.empty_strided((N, d_out), (d_out, 1), dtype=dtype or torch.bfloat16, device=xq.device)
    else:
        _req_here(out, dtype or out.dtype, (N, d_out), dev, "out")
        dt = _code(out.dtype, codes, "out")
    if ws is None:
        ws = _unread(dev)
    else:
        _same_device(ws, dev, "ws")
    if N == 0 and w8a8_workspace_size(1, d_out, d_in):
        return out
    st = lib().awq_w8a8_gemm(xq.data_ptr(), x_step.data_ptr(), wq.data_ptr(), w_step.data_ptr(),
                             None if bias is None else bias.data_ptr(), dt, N, d_out, d_in, out.data_ptr(),
                             ws.data_ptr(), ws.numel() * ws.element_size(), stream)
    _check(st, "awq_w8a8_gemm")
    return out


# --------------------------------------------------------------------------- 4-bit key/value cache
def kv4_page_bytes(cfg: Kv4Cfg) -> int:
    """Bytes of one (page, kv head) of a cache (0: invalid cfg)."""
    return _kv4_page_bytes(cfg.n_kv_heads, cfg.head_dim, cfg.page_size, cfg.group)


@functools.lru_cache(maxsize=256)
def _kv4_page_bytes(*cfg) -> int:
    return int(lib().awq_kv4_page_bytes(ctypes.byref(Kv4Cfg(*cfg))))


def kv4_new_cache(n_pages, cfg: Kv4Cfg):
    """An empty cache: int32 zeros [n_pages, n_kv_heads, page words]."""
    nbytes = kv4_page_bytes(cfg)
    if not nbytes:
        raise AwqError(1, "kv4_new_cache")
    return _torch().zeros((n_pages, cfg.n_kv_heads, nbytes // 4), dtype=_torch().int32, device="cuda")


def _req_cache(cache, cfg, dev):
    _req_here(cache, _torch().int32, None, dev, "cache")
    words = kv4_page_bytes(cfg) // 4
    if cache.dim() != 3 or (words and cache.shape[1:] != (cfg.n_kv_heads, words)):
        raise ValueError(f"cache must be [n_pages, {cfg.n_kv_heads}, {words}], got {tuple(cache.shape)}")


def kv4_append(k, v, slots, cache, cfg: Kv4Cfg):
    """Write the keys and values k, v (bf16 or fp16 [T, n_kv_heads, head_dim],
    tokens and heads may be strided) of T tokens to their slots (int32 [T]: page
    * page_size + position; outside the cache: skipped) of the cache, in place."""
    if cfg.__class__ is Kv4Cfg:
        r = _calls(_active).kv4_append(k, v, slots, cache, ctypes.addressof(cfg))
        if r is not None:
            _check(r, "awq_kv4_append")
            return cache
    dev, stream, codes = _here(k, "k")
    dt = _code(k.dtype, codes, "k")
    T = k.shape[0] if k.dim() else 0
    shape = (T, cfg.n_kv_heads, cfg.head_dim)
    _req_rows(k, k.dtype, shape, dev, "k")
    if isinstance(v, _torch().Tensor) and v.dtype is not k.dtype:
        raise ValueError("k and v must have one dtype")
    _req_rows(v, k.dtype, shape, dev, "v")
    _req_here(slots, _torch().int32, (T,), dev, "slots")
    _req_cache(cache, cfg, dev)
    st = lib().awq_kv4_append(k.data_ptr(), v.data_ptr(), dt, T, _pitch(k, 0), _pitch(k, 1), _pitch(v, 0), _pitch(v, 1),
                              slots.data_ptr(), cache.data_ptr(), cache.shape[0], ctypes.byref(cfg), stream)
    _check(st, "awq_kv4_append")
    return cache


def kv4_gather(cache, slots, cfg: Kv4Cfg, dtype=None, outputs=None):
    """Keys and values [T, n_kv_heads, head_dim] (bf16 by default, or fp16) that
    the cache holds for the T slots; a slot outside the cache reads as zeros."""
    if outputs is None and cfg.__class__ is Kv4Cfg and dtype in (None, _torch().bfloat16, _torch().float16):
        r = _calls(_active).kv4_gather(cache, slots, ctypes.addressof(cfg), dtype is _torch().float16)
        if r.__class__ is tuple:
            return r
        _check(r or AWQ_OK, "awq_kv4_gather")
    dev, stream, codes = _here(cache, "cache")
    _req_cache(cache, cfg, dev)
    _req_here(slots, _torch().int32, None, dev, "slots")
    if slots.dim() != 1:
        raise ValueError("slots must be [T]")
    shape = (slots.shape[0], cfg.n_kv_heads, cfg.head_dim)
    if outputs is None:
        dtype = dtype or _torch().bfloat16
        dt = _code(dtype, codes, "k")
        strides = (shape[1] * shape[2], shape[2], 1)
        k, v = (_torch().empty_strided(shape, strides, dtype=dtype, device=cache.device) for _ in range(2))
    else:
        k, v = outputs
        dt = _code(dtype or k.dtype, codes, "k")
        for t, name in ((k, "k"), (v, "v")):
            _req_here(t, dtype or k.dtype, shape, dev, name)
    st = lib().awq_kv4_gather(cache.data_ptr(), cache.shape[0], slots.data_ptr(), shape[0], ctypes.byref(cfg),
                              k.data_ptr(), v.data_ptr(), dt, stream)
    _check(st, "awq_kv4_gather")
    return k, v


def kv4_attention_workspace_size(batch, n_q_heads, max_q, cfg: Kv4Cfg) -> int:
    return _kv4_attention_workspace_size(batch, n_q_heads, max_q, cfg.n_kv_heads, cfg.head_dim, cfg.page_size, cfg.group)


@functools.lru_cache(maxsize=4096)
def _kv4_attention_workspace_size(batch, n_q_heads, max_q, *cfg) -> int:
    return int(lib().awq_kv4_attention_workspace_size(batch, n_q_heads, max_q, ctypes.byref(Kv4Cfg(*cfg))))


def kv4_attention(q, cache, table, lens, cfg: Kv4Cfg, q_start=None, max_q=None, scale=None, lse=False, ws=None,
                  out=None):
    """Attention of q (bf16 or fp16 [T, n_q_heads, head_dim], tokens and heads
    may be strided) over the cache: sequence b's context is lens[b] tokens
    (int32 [batch]) in the pages table[b] (int32 [batch, table_pages]), its
    queries the rows q_start[b] .. q_start[b+1] - 1 (int32 [batch + 1], with
    max_q at least the longest; default: one row a sequence), the last tokens of
    that context. scale: default 1 / sqrt(head_dim). Returns out [T, n_q_heads,
    head_dim], or (out, lse float32 [T, n_q_heads]) with lse=True (no rows: no
    work). Many rows a sequence (more than 64 tokens times query heads of a kv
    head) are fast for head_dim up to 128, in fp16 with group = head_dim, and in
    batches that fill the GPU (include/awq.h has the rule). Rows of no
    sequence are left as they were (unset in a fresh output). Pages outside the
    cache, lengths past the table and rows past max_q are left out without an
    exception: device_error() tells of them, and workspace_error(ws) for a call
    with a workspace of its own. A workspace given serves one call at a time, and
    one given to a captured call must live as long as its graph."""
    torch = _torch()
    if ws is None and out is None and cfg.__class__ is Kv4Cfg:
        r = _calls(_active).kv4_attention(q, cache, table, lens, ctypes.addressof(cfg), q_start, max_q, scale, bool(lse))
        if r.__class__ is tuple or isinstance(r, torch.Tensor):
            return r
        _check(r or AWQ_OK, "awq_kv4_attention")
    dev, stream, codes = _here(q, "q")
    dt = _code(q.dtype, codes, "q")
    T, n_q_heads, D = q.shape if q.dim() == 3 else (None, None, None)
    _req_rows(q, q.dtype, (T, n_q_heads, cfg.head_dim), dev, "q")
    _req_cache(cache, cfg, dev)
    _req_here(lens, torch.int32, None, dev, "lens")
    _req_here(table, torch.int32, None, dev, "table")
    batch = lens.shape[0] if lens.dim() == 1 else -1
    if batch < 0 or table.dim() != 2 or table.shape[0] != batch:
        raise ValueError("lens must be [batch] and table [batch, table_pages]")
    if q_start is not None:
        _req_here(q_start, torch.int32, (batch + 1,), dev, "q_start")
        if max_q is None:
            raise ValueError("q_start needs max_q, the most rows of a sequence")
    elif T != batch:
        raise ValueError("without q_start, q must have one row a sequence")
    max_q = 1 if max_q is None else int(max_q)
    if out is None:
        out = torch.empty_strided((T, n_q_heads, D), (n_q_heads * D, D, 1), dtype=q.dtype, device=q.device)
    else:
        _req_here(out, q.dtype, (T, n_q_heads, D), dev, "out")
    lse_t = q.new_empty((T, n_q_heads), dtype=torch.float32) if lse else None
    if T == 0 and kv4_attention_workspace_size(max(batch, 1), n_q_heads, max_q, cfg):
        return (out, lse_t) if lse else out
    if ws is None:
        ws = _scratch(q, kv4_attention_workspace_size(batch, n_q_heads, max_q, cfg))
    else:
        _same_device(ws, dev, "ws")
    st = lib().awq_kv4_attention(q.data_ptr(), dt, _pitch(q, 0), _pitch(q, 1), T, n_q_heads,
                                 None if q_start is None else q_start.data_ptr(), max_q, cache.data_ptr(),
                                 cache.shape[0], table.data_ptr(), table.shape[1], lens.data_ptr(), batch,
                                 D ** -0.5 if scale is None else float(scale), ctypes.byref(cfg), out.data_ptr(),
                                 lse_t.data_ptr() if lse else None, ws.data_ptr(), ws.numel() * ws.element_size(), stream)
    _check(st, "awq_kv4_attention")
    return (out, lse_t) if lse else out


def selftest_bounded_wait(ws):
    """Launch the bounded-wait failure path (see include/awq.h); the error lands in ws."""
    _check(lib().awq_selftest_bounded_wait(_ptr(ws), _stream()), "awq_selftest_bounded_wait")


def bounds_checks_enabled() -> bool:
    """True if the selected build carries the index checks."""
    return bool(lib().awq_bounds_checks_enabled())


def bounds_error():
    """(status, site) of the index checks since the last call; reading clears
    the device word (synchronises). Always (AWQ_OK, 0) in the release build."""
    site = c_int32(0)
    st = int(lib().awq_bounds_error(ctypes.byref(site), _stream()))
    if st not in (AWQ_OK, AWQ_ERR_BOUNDS):
        raise AwqError(st, "awq_bounds_error")
    return st, int(site.value)


def selftest_bounds(ws):
    """Launch the index checks' failure path (see include/awq.h)."""
    _check(lib().awq_selftest_bounds(_ptr(ws), ws.numel() * ws.element_size(), _stream()), "awq_selftest_bounds")


def device_error():
    """Raise AwqError if the device found something wrong in w8a8_gemm or kv4_attention (a page outside the cache, a length
    past the table, rows past max_q, a wait that gave up) since the last time this was called for the current device;
    waits for the current stream. One error is kept, whichever call it came from."""
    _check(lib().awq_device_error(_stream()), "device")


def workspace_error(ws):
    """Raise AwqError if a kernel recorded an error in the workspace (synchronises)."""
    _check(lib().awq_workspace_error(_ptr(ws), _stream()), "device")


def step(name: str, *args):
    """Call one awq_step_* entry point with already-marshalled arguments."""
    fn = getattr(lib(), "awq_step_" + name)
    _check(fn(*args), "awq_step_" + name)


def debug_dw(ws, d_out, d_in, N, cfg, k):
    """bf16 [d_out, d_in] copy of the candidate dW for grid index k."""
    torch = _torch()
    dst = torch.empty((d_out, d_in), dtype=torch.bfloat16, device="cuda")
    _check(lib().awq_debug_copy_dw(_ptr(ws), d_out, d_in, N, ctypes.byref(cfg), k, _ptr(dst), _stream()),
           "awq_debug_copy_dw")
    return dst


# --------------------------------------------------------------------------- a7
def pack_workspace_size(d_out, d_in, cfg: QCfg) -> int:
    return int(lib().awq_pack_workspace_size(d_out, d_in, ctypes.byref(cfg)))


def quantize_pack(W, s, cfg: QCfg, outputs=None, clip=1.0, ws=None):
    """(qweight int32 view of uint32 [d_out, d_in/8], scales fp16 [d_out, d_in/g], zeros fp16 [d_out, d_in/g]);
    per tensor (cfg.group == 0): scales and zeros are [1, 1] and a workspace is used."""
    torch = _torch()
    _req(W, torch.bfloat16, None, "W")
    d_out, d_in = W.shape
    _req(s, torch.float32, (d_in,), "s")
    if outputs is None:
        shape = (d_out, d_in // cfg.group) if cfg.group > 0 else (1, 1)
        outputs = (torch.empty((d_out, d_in // 8), dtype=torch.int32, device=W.device),
                   torch.empty(shape, dtype=torch.float16, device=W.device),
                   torch.empty(shape, dtype=torch.float16, device=W.device))
    q, sc, zr = outputs
    if cfg.group == 0 or ws is not None:
        if ws is None:
            ws = workspace(pack_workspace_size(d_out, d_in, cfg))
        _check(lib().awq_quantize_pack_ws(_ptr(W), _ptr(s), d_out, d_in, ctypes.byref(cfg), float(clip), _ptr(ws),
                                          ws.numel(), _ptr(q), _ptr(sc), _ptr(zr), _stream()), "awq_quantize_pack_ws")
    elif clip == 1.0:
        _check(lib().awq_quantize_pack(_ptr(W), _ptr(s), d_out, d_in, ctypes.byref(cfg), _ptr(q), _ptr(sc), _ptr(zr),
                                       _stream()), "awq_quantize_pack")
    else:
        _check(lib().awq_quantize_pack_clipped(_ptr(W), _ptr(s), d_out, d_in, ctypes.byref(cfg), float(clip), _ptr(q),
                                               _ptr(sc), _ptr(zr), _stream()), "awq_quantize_pack_clipped")
    return q, sc, zr
