"""S2O sparse prefill attention for B200: thin Python binding of libs2o.so.

The functions below only marshal arguments (torch tensors -> device pointers,
the current CUDA stream) into the C ABI declared in include/s2o.h; every step
of the method runs in the library's CUDA kernels.  There is no CPU fallback:
if the compiled library is missing, importing the binding's entry points
raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "libs2o.so")
HEADER = os.path.join(ROOT, "include", "s2o.h")

OUT_BF16, OUT_F32 = 0, 1

STATUS = {
    0: "S2O_OK", 1: "S2O_ERR_INVALID_ARG", 2: "S2O_ERR_UNSUPPORTED_SHAPE",
    3: "S2O_ERR_WORKSPACE_TOO_SMALL", 4: "S2O_ERR_CUDA", 5: "S2O_ERR_DEVICE_TIMEOUT",
    6: "S2O_ERR_NONFINITE", 7: "S2O_ERR_BAD_PLAN", 8: "S2O_ERR_BAD_CACHE",
}

BF16, FP16 = 0, 1  # element types of the serving calls
OUT_SAME = 0       # attention_paged: O in the cache's type (or OUT_F32)


class S2OError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("N", ctypes.c_int32), ("d", ctypes.c_int32), ("Lq", ctypes.c_int32),
                ("Bk", ctypes.c_int32), ("n_sink", ctypes.c_int32), ("window_prev", ctypes.c_int32),
                ("tau", ctypes.c_double)]


def make_config(B, Hq, Hkv, N, d=128, tau=1e-3, Lq=128, Bk=64, n_sink=64, window_prev=128) -> Config:
    return Config(B, Hq, Hkv, N, d, Lq, Bk, n_sink, window_prev, float(tau))


class RotaryConfig(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("naxes", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("inv_freq", ctypes.c_double * 64), ("axis", ctypes.c_uint8 * 64)]


class View(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


_pack_view = struct.Struct("@Pqqq").pack  # a View's bytes


class CacheConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("Hq", "Hkv", "d", "page_size", "num_pages", "nseq", "max_pages", "Tq",
                                              "max_q", "prefix_len", "dtype")]


def make_rotary(rot_dim: int = 128, theta: float = 10000.0, sections=None, interleaved: bool = False,
                inv_freq=None) -> RotaryConfig:
    """Rotation of the first rot_dim elements of a head.  sections: how many of
    the rot_dim/2 frequencies, in order, go by each position axis (None: one
    axis); inv_freq: the frequencies themselves, in place of
    theta^(-2 i / rot_dim)."""
    if rot_dim < 0 or rot_dim > 128 or rot_dim % 2:
        raise S2OError(2, "make_rotary: rot_dim")
    F = rot_dim // 2
    sections = (F,) if sections is None else tuple(int(n) for n in sections)
    if not 1 <= len(sections) <= 3 or any(n < 0 for n in sections) or sum(sections) != F:
        raise S2OError(1, "make_rotary: sections must be 1 to 3 counts that add up to rot_dim / 2")
    freq = [theta ** (-2.0 * i / rot_dim) for i in range(F)] if inv_freq is None else [float(x) for x in inv_freq]
    if len(freq) != F:
        raise S2OError(1, "make_rotary: inv_freq needs rot_dim / 2 values")
    r = RotaryConfig(rot_dim, int(interleaved), len(sections), 0)
    r.inv_freq[:F] = freq
    r.axis[:F] = [a for a, n in enumerate(sections) for _ in range(n)]
    return r


def make_cache(Hq, Hkv, page_size, num_pages, nseq, max_pages, Tq, max_q=1, prefix_len=0, dtype=BF16,
               d=128) -> CacheConfig:
    """The paged cache of a batch, as include/s2o.h describes it."""
    return CacheConfig(Hq, Hkv, d, page_size, num_pages, nseq, max_pages, Tq, max_q, prefix_len, dtype)


_lib = None
_P = ctypes.c_void_p
_CFG = ctypes.POINTER(Config)


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (built in-tree by score_keys_pooled_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run `python -m score_keys_pooled_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.s2o_num_segments.argtypes = [_CFG]
        L.s2o_num_segments.restype = ctypes.c_int32
        L.s2o_num_candidates.argtypes = [_CFG]
        L.s2o_num_candidates.restype = ctypes.c_int64
        L.s2o_candidate_offset.argtypes = [_CFG, ctypes.c_int32]
        L.s2o_candidate_offset.restype = ctypes.c_int64
        L.s2o_plan_workspace_size.argtypes = [_CFG, ctypes.POINTER(ctypes.c_size_t)]
        L.s2o_plan.argtypes = [_CFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.s2o_plan_filtered.argtypes = [_CFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.s2o_plan_noalloc.argtypes = [_CFG, _P, _P, _P, _P, _P, _P, _P]
        L.s2o_plan_contiguous.argtypes = [_CFG, _P, _P, _P, _P, _P]
        L.s2o_attention.argtypes = [_CFG, _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P]
        L.s2o_attention_bounded.argtypes = [_CFG, _P, _P, _P, _P, _P, _P, ctypes.c_int32, ctypes.c_uint32, _P]
        L.s2o_attention_online.argtypes = [_CFG, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P]
        L.s2o_block_truth_workspace_size.argtypes = [_CFG, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
        L.s2o_plan_qperm_workspace_size.argtypes = [_CFG, ctypes.POINTER(ctypes.c_size_t)]
        L.s2o_plan_qperm.argtypes = [_CFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.s2o_attention_qperm.argtypes = [_CFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P]
        L.s2o_block_truth.argtypes = [_CFG, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]
        L.s2o_prefill_arena_size.argtypes = [_CFG, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
        L.s2o_prefill_host.argtypes = [_CFG, _P, _P, _P, _P, ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]
        L.s2o_status_string.argtypes = [ctypes.c_int]
        L.s2o_status_string.restype = ctypes.c_char_p
        L.s2o_last_device_error.argtypes = [_P]
        L.s2o_last_launch_count.restype = ctypes.c_int32
        L.s2o_stage_timing.argtypes = [ctypes.c_int32]
        L.s2o_stage_timing.restype = ctypes.c_int
        L.s2o_last_stage_times.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_char_p),
                                           ctypes.c_int32]
        L.s2o_last_stage_times.restype = ctypes.c_int32
        # views go in as packed bytes (a View made for each costs more than the rest of the call)
        _R, _V, _C = ctypes.POINTER(RotaryConfig), _P, ctypes.POINTER(CacheConfig)
        i32 = ctypes.c_int32
        L.s2o_rotary.argtypes = [_R, i32, i32, i32, i32, i32, _V, _V, _P, _V, _V, i32, _P]
        L.s2o_cache_append.argtypes = [_C, _R, _V, _V, _V, _P, _P, _P, _P, _P, _P, _V, _P]
        L.s2o_attention_paged_workspace_size.argtypes = [_C, ctypes.POINTER(ctypes.c_size_t)]
        L.s2o_attention_paged.argtypes = [_C, _P, _P, _P, _P, _P, _P, _P, _P, i32, _P, _P, ctypes.c_size_t, _P]
        for name in ("s2o_rotary", "s2o_cache_append", "s2o_attention_paged_workspace_size", "s2o_attention_paged"):
            getattr(L, name).restype = ctypes.c_int
        for name in ("s2o_plan_workspace_size", "s2o_plan", "s2o_plan_filtered", "s2o_plan_noalloc", "s2o_plan_contiguous", "s2o_attention", "s2o_attention_bounded", "s2o_attention_online",
                     "s2o_block_truth_workspace_size", "s2o_block_truth", "s2o_plan_qperm_workspace_size",
                     "s2o_plan_qperm", "s2o_attention_qperm",
                     "s2o_prefill_arena_size", "s2o_prefill_host", "s2o_last_device_error"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/s2o.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(s2o_[a-z_0-9]+)\s*\(", text)))


def _check(code: int, what: str):
    if code != 0:
        raise S2OError(code, what)


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def num_segments(cfg: Config) -> int:
    return lib().s2o_num_segments(ctypes.byref(cfg))


def num_candidates(cfg: Config) -> int:
    return lib().s2o_num_candidates(ctypes.byref(cfg))


def candidate_offset(cfg: Config, s: int) -> int:
    return lib().s2o_candidate_offset(ctypes.byref(cfg), s)


def plan_workspace_size(cfg: Config) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().s2o_plan_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "s2o_plan_workspace_size")
    return n.value


def prefill_arena_size(cfg: Config, out_dtype: int = OUT_BF16) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().s2o_prefill_arena_size(ctypes.byref(cfg), out_dtype, ctypes.byref(n)), "s2o_prefill_arena_size")
    return n.value


def alloc_plan(cfg: Config, device="cuda", workspace=True):
    """Device buffers for one s2o_plan call (allocated by torch)."""
    import torch
    BH = cfg.B * cfg.Hkv
    S, T = num_segments(cfg), num_candidates(cfg)
    out = dict(
        scores=torch.empty(BH * T + 4, dtype=torch.float32, device=device),
        perm=torch.empty(BH * T + 4, dtype=torch.int32, device=device),
        nblocks=torch.empty(BH * S, dtype=torch.int32, device=device),
        seg_stats=torch.empty(BH * S * 2, dtype=torch.float32, device=device),
    )
    if workspace:
        out["workspace"] = torch.empty(plan_workspace_size(cfg), dtype=torch.uint8, device=device)
    return out


def plan(cfg: Config, Q, K, bufs=None, stream=None, filtered: bool = False):
    """Run s2o_plan (or s2o_plan_filtered); returns the buffer dict (scores,
    perm, nblocks, seg_stats)."""
    bufs = alloc_plan(cfg, Q.device) if bufs is None else bufs
    ws = bufs["workspace"]
    fn, name = (lib().s2o_plan_filtered, "s2o_plan_filtered") if filtered else (lib().s2o_plan, "s2o_plan")
    _check(fn(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(bufs["scores"]), _ptr(bufs["perm"]),
              _ptr(bufs["nblocks"]), _ptr(bufs.get("seg_stats")), _ptr(ws), ws.numel(), _stream(stream)), name)
    return bufs


def plan_noalloc(cfg: Config, Q, K, bufs, stream=None):
    """s2o_plan_noalloc: the plan with the library's static scratch; `bufs`
    holds the output buffers (no workspace is needed or used)."""
    _check(lib().s2o_plan_noalloc(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(bufs["scores"]), _ptr(bufs["perm"]),
                                  _ptr(bufs["nblocks"]), _ptr(bufs.get("seg_stats")), _stream(stream)),
           "s2o_plan_noalloc")
    return bufs


def plan_contiguous(cfg: Config, scores, seg_stats, nblocks_match, perm_out, stream=None):
    _check(lib().s2o_plan_contiguous(ctypes.byref(cfg), _ptr(scores), _ptr(seg_stats), _ptr(nblocks_match),
                                     _ptr(perm_out), _stream(stream)), "s2o_plan_contiguous")
    return perm_out


def attention(cfg: Config, Q, K, V, perm, nblocks, O=None, out_dtype: int = OUT_BF16, stream=None):
    import torch
    if O is None:
        O = torch.empty(Q.shape, dtype=torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32,
                        device=Q.device)
    _check(lib().s2o_attention(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(perm), _ptr(nblocks),
                               _ptr(O), out_dtype, _stream(stream)), "s2o_attention")
    return O


def attention_bounded(cfg: Config, Q, K, V, perm, nblocks, max_polls: int, O=None, out_dtype: int = OUT_BF16,
                      stream=None):
    """s2o_attention with every pipeline wait limited to max_polls polls (tests of the timeout path)."""
    import torch
    if O is None:
        O = torch.empty(Q.shape, dtype=torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32,
                        device=Q.device)
    _check(lib().s2o_attention_bounded(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(perm), _ptr(nblocks),
                                       _ptr(O), out_dtype, max_polls, _stream(stream)), "s2o_attention_bounded")
    return O


def attention_online(cfg: Config, Q, K, V, perm, O=None, nblocks_out=None, out_dtype: int = OUT_BF16, stream=None):
    """s2o_attention_online: the run-time stop; returns (O, nblocks_out [B*Hq*S])."""
    import torch
    if O is None:
        O = torch.empty(Q.shape, dtype=torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32,
                        device=Q.device)
    if nblocks_out is None:
        nblocks_out = torch.empty(cfg.B * cfg.Hq * num_segments(cfg), dtype=torch.int32, device=Q.device)
    _check(lib().s2o_attention_online(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(perm), _ptr(O), out_dtype,
                                      _ptr(nblocks_out), _stream(stream)), "s2o_attention_online")
    return O, nblocks_out


def plan_qperm(cfg: Config, Q, K, stream=None):
    """s2o_plan_qperm; returns dict(scores [2*B*Hkv*T], perm, nblocks [2*B*Hkv*S], rowsub [B*Hkv*S*128])."""
    import torch
    BH = cfg.B * cfg.Hkv
    S, T = num_segments(cfg), num_candidates(cfg)
    dev = Q.device
    out = dict(scores=torch.empty(2 * BH * T + 4, dtype=torch.float32, device=dev),
               perm=torch.empty(2 * BH * T + 4, dtype=torch.int32, device=dev),
               nblocks=torch.empty(2 * BH * S, dtype=torch.int32, device=dev),
               rowsub=torch.empty(BH * S * 128, dtype=torch.uint8, device=dev))
    n = ctypes.c_size_t(0)
    _check(lib().s2o_plan_qperm_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "s2o_plan_qperm_workspace_size")
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    _check(lib().s2o_plan_qperm(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(out["scores"]), _ptr(out["perm"]),
                                _ptr(out["nblocks"]), _ptr(out["rowsub"]), _ptr(ws), ws.numel(), _stream(stream)),
           "s2o_plan_qperm")
    return out


def attention_qperm(cfg: Config, Q, K, V, qp, O=None, out_dtype: int = OUT_BF16, stream=None):
    import torch
    if O is None:
        O = torch.empty(Q.shape, dtype=torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32,
                        device=Q.device)
    _check(lib().s2o_attention_qperm(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(qp["perm"]),
                                     _ptr(qp["nblocks"]), _ptr(qp["rowsub"]), _ptr(O), out_dtype, _stream(stream)),
           "s2o_attention_qperm")
    return O


def block_truth(cfg: Config, Q, K, perm, nblocks, segments, with_mass: bool = True, stream=None):
    """s2o_block_truth on the listed segments; returns (stats [n, B*Hkv, 5],
    mass [n, B*Hkv, nbmax] or None) as device tensors."""
    import numpy as np
    import torch
    segs = np.ascontiguousarray(np.asarray(segments, dtype=np.int32))
    n = len(segs)
    BH = cfg.B * cfg.Hkv
    nbmax = max(0, 128 * (num_segments(cfg) - 1) - 192) // 64
    stats = torch.empty(n * BH * 5, dtype=torch.float32, device=Q.device)
    mass = torch.empty(max(1, n * BH * nbmax), dtype=torch.float32, device=Q.device) if with_mass else None
    nbytes = ctypes.c_size_t(0)
    _check(lib().s2o_block_truth_workspace_size(ctypes.byref(cfg), n, ctypes.byref(nbytes)),
           "s2o_block_truth_workspace_size")
    ws = torch.empty(nbytes.value, dtype=torch.uint8, device=Q.device)
    _check(lib().s2o_block_truth(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(perm), _ptr(nblocks),
                                 segs.ctypes.data, n, _ptr(stats), _ptr(mass), _ptr(ws), ws.numel(),
                                 _stream(stream)), "s2o_block_truth")
    return stats.view(n, BH, 5), (mass[:n * BH * nbmax].view(n, BH, nbmax) if with_mass else None)


def prefill_host(cfg: Config, Q_host, K_host, V_host, O_host, arena, nblocks_host=None,
                 out_dtype: int = OUT_BF16, stream=None):
    """Whole path from host tensors (pinned for speed) through the C ABI."""
    _check(lib().s2o_prefill_host(ctypes.byref(cfg), _ptr(Q_host), _ptr(K_host), _ptr(V_host), _ptr(O_host),
                                  out_dtype, _ptr(nblocks_host), _ptr(arena), arena.numel(), _stream(stream)),
           "s2o_prefill_host")
    return O_host


# --- serving: rotary positions, the paged cache and attention over it -----------
# These calls check what only the tensors know (type, shape, layout, device);
# sizes and pointers are checked by the library.


def _torch_type(dtype: int):
    import torch
    return torch.float16 if dtype == FP16 else torch.bfloat16


def _refuse(what: str):
    raise S2OError(1, what)


def _wrong(t, what, shape, dtype, device, layout):
    _refuse(f"{what}: want a {dtype} {list(shape)} tensor with {layout} on {device}, "
            f"got {t.dtype} {list(t.shape)} strides {t.stride()} on {t.device}")


def _view3(t, what, shape, dtype, device):
    """[T, H, 128] with contiguous rows, as a packed s2o_view."""
    if t.dtype is not dtype or t.device != device or t.shape != shape:
        _wrong(t, what, shape, dtype, device, "contiguous rows")
    st, sh, one = t.stride()
    if one != 1 and t.numel():
        _wrong(t, what, shape, dtype, device, "contiguous rows")
    return _pack_view(t.data_ptr(), 0, st, sh)


def _view4(t, what, shape, dtype, device):
    """[B, N, H, 128] with contiguous rows, as a packed s2o_view."""
    if t.dtype is not dtype or t.device != device or t.shape != shape:
        _wrong(t, what, shape, dtype, device, "contiguous rows")
    sb, st, sh, one = t.stride()
    if one != 1 and t.numel():
        _wrong(t, what, shape, dtype, device, "contiguous rows")
    return _pack_view(t.data_ptr(), sb, st, sh)


def _plain(t, what, shape, dtype, device):
    """A contiguous tensor of this shape."""
    if t.dtype is not dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        _wrong(t, what, shape, dtype, device, "no gaps")
    return t.data_ptr()


def _empty(shape, dtype, device, stream, strides=None):
    """Memory that belongs to the stream it is used on."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return _empty(shape, dtype, device, None, strides)
    if strides is not None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _call_on(device, stream, fn, name, *args):
    """fn(*args, stream) with the tensors' device current."""
    import torch
    if device.type != "cuda":
        _refuse(f"{name}: the tensors are on {device}, not on a CUDA device")
    at = device.index
    if at != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _call_on(device, stream, fn, name, *args)
    # the raw handle: a Stream object costs 2 us, as much as the launch
    code = fn(*args, torch._C._cuda_getCurrentRawStream(at) if stream is None else stream.cuda_stream)
    if code:
        raise S2OError(code, name)


def rotary(r: RotaryConfig, q, k, positions, q_out=None, k_out=None, inverse: bool = False, stream=None):
    """s2o_rotary: q [B, N, Hq, 128] and k [B, N, Hkv, 128] (any strides; either
    may be None) turned at positions int32 [naxes, B, N]; returns (q_out, k_out)
    of the same shapes.  Outputs that are not given are allocated head-major
    (q_out.transpose(1, 2) is contiguous: what plan and attention read), or
    token-major for the inverse, which takes head-major gradients back."""
    import torch
    x = q if q is not None else k
    if x is None or x.dim() != 4:
        _refuse("rotary: q or k must be a [B, N, H, 128] tensor")
    B, N, dev, t = x.shape[0], x.shape[1], x.device, x.dtype
    if t is not torch.bfloat16 and t is not torch.float16:
        _refuse(f"rotary: {t} is neither bfloat16 nor float16")
    Hq, qi, qo, q_out = _turned("rotary: q", q, q_out, B, N, t, dev, inverse, stream)
    Hkv, ki, ko, k_out = _turned("rotary: k", k, k_out, B, N, t, dev, inverse, stream)
    if positions is None:
        _refuse("rotary: positions")
    pos = _plain(positions, "rotary: positions", (r.naxes, B, N), torch.int32, dev)
    _call_on(dev, stream, lib().s2o_rotary, "s2o_rotary", r, FP16 if t is torch.float16 else BF16, B, N, Hq, Hkv, qi,
             ki, pos, qo, ko, int(inverse))
    return q_out, k_out


def _turned(name, src, dst, B, N, t, dev, inverse, stream):
    """(heads, input view, output view, output) of one side of a rotation."""
    if src is None:
        return 0, None, None, None
    if src.dim() != 4:
        _refuse(f"{name} must be a [B, N, H, 128] tensor")
    H = src.shape[2]
    shape = (B, N, H, 128)
    vin = _view4(src, name, shape, t, dev)
    if dst is None:
        strides = (H * N * 128, H * 128, 128, 1) if inverse else (H * N * 128, 128, N * 128, 1)
        dst = _empty(shape, t, dev, stream, strides)
        return H, vin, _pack_view(dst.data_ptr(), *strides[:3]), dst
    return H, vin, _view4(dst, name + "_out", shape, t, dev), dst


def alloc_cache(cfg: CacheConfig, device="cuda"):
    """(k_cache, v_cache) of the config, zeroed."""
    import torch
    shape = (cfg.num_pages, cfg.Hkv, cfg.page_size, cfg.d)
    return tuple(torch.zeros(shape, dtype=_torch_type(cfg.dtype), device=device) for _ in range(2))


def _cache_args(cfg, k_cache, v_cache, page_table, q_start, kv_len, dev, t):
    import torch
    shape = (cfg.num_pages, cfg.Hkv, cfg.page_size, cfg.d)
    return (_plain(k_cache, "k_cache", shape, t, dev), _plain(v_cache, "v_cache", shape, t, dev),
            _plain(page_table, "page_table", (cfg.nseq, cfg.max_pages), torch.int32, dev),
            _plain(q_start, "q_start", (cfg.nseq + 1,), torch.int32, dev),
            _plain(kv_len, "kv_len", (cfg.nseq,), torch.int32, dev))


def cache_append(cfg: CacheConfig, q, k, v, k_cache, v_cache, page_table, q_start, kv_len, rotary=None,
                 positions=None, q_out=None, stream=None):
    """s2o_cache_append: k and v [Tq, Hkv, 128] (any strides) into the caches, k
    turned by `rotary` (None: as it is); q [Tq, Hq, 128] (or None) turned into
    q_out (allocated when not given).  positions int32 [naxes, Tq], or None:
    prefix_len + the token's place in its sequence.  Returns q_out."""
    import torch
    dev, t, T = k.device, _torch_type(cfg.dtype), cfg.Tq
    qv = qo = None
    if q is not None:
        shape = (T, cfg.Hq, 128)
        qv = _view3(q, "cache_append: q", shape, t, dev)
        if q_out is None:
            q_out = _empty(shape, t, dev, stream)
        qo = _view3(q_out, "cache_append: q_out", shape, t, dev)
    elif q_out is not None:
        _refuse("cache_append: q_out without q")
    shape = (T, cfg.Hkv, 128)
    kv = _view3(k, "cache_append: k", shape, t, dev)
    vv = _view3(v, "cache_append: v", shape, t, dev)
    kc, vc, table, qs, kl = _cache_args(cfg, k_cache, v_cache, page_table, q_start, kv_len, dev, t)
    pos = None
    if positions is not None:
        if rotary is None:
            _refuse("cache_append: positions without a rotation")
        pos = _plain(positions, "cache_append: positions", (rotary.naxes, T), torch.int32, dev)
    _call_on(dev, stream, lib().s2o_cache_append, "s2o_cache_append", cfg, rotary, qv, kv, vv, pos, table, qs, kl, kc,
             vc, qo)
    return q_out


def attention_paged_workspace_size(cfg: CacheConfig) -> int:
    """Bytes for the current device."""
    n = ctypes.c_size_t(0)
    _check(lib().s2o_attention_paged_workspace_size(cfg, n), "s2o_attention_paged_workspace_size")
    return n.value


def alloc_attention_paged(cfg: CacheConfig, device="cuda"):
    """A workspace for attention_paged calls of this config on `device` (one per
    stream or captured graph whose work may overlap another's).  Smaller batches may
    need more (see include/s2o.h): calls of several configs share the largest one."""
    import torch
    with torch.cuda.device(device):
        return torch.empty(attention_paged_workspace_size(cfg), dtype=torch.uint8, device=device)


def attention_paged(cfg: CacheConfig, q, k_cache, v_cache, page_table, q_start, kv_len, prefix_pages=None, O=None,
                    lse=None, workspace=None, out_dtype: int = OUT_SAME, stream=None):
    """s2o_attention_paged: q [Tq, Hq, 128] over the caches; returns (O, lse).
    O, lse (float32 [Tq, Hq]) and the workspace are allocated when not given;
    rows behind q_start[nseq] are left as they were.  OUT_F32 leaves out O's own
    rounding; the probabilities are of the cache's type in either form."""
    import torch
    dev, t, T = q.device, _torch_type(cfg.dtype), cfg.Tq
    qp = _plain(q, "attention_paged: q", (T, cfg.Hq, 128), t, dev)
    kc, vc, table, qs, kl = _cache_args(cfg, k_cache, v_cache, page_table, q_start, kv_len, dev, t)
    pre = None
    if cfg.prefix_len > 0:
        if prefix_pages is None:
            _refuse("attention_paged: prefix_len without prefix_pages")
        pre = _plain(prefix_pages, "attention_paged: prefix_pages", (-(-cfg.prefix_len // max(1, cfg.page_size)),),
                     torch.int32, dev)
    to = torch.float32 if out_dtype == OUT_F32 else t
    if O is None:
        O = _empty((T, cfg.Hq, 128), to, dev, stream)
    if lse is None:
        lse = _empty((T, cfg.Hq), torch.float32, dev, stream)
    if workspace is None:
        if dev.type != "cuda":
            _refuse(f"attention_paged: the tensors are on {dev}, not on a CUDA device")
        with torch.cuda.device(dev):
            workspace = _empty((attention_paged_workspace_size(cfg),), torch.uint8, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        _refuse("attention_paged: workspace")
    _call_on(dev, stream, lib().s2o_attention_paged, "s2o_attention_paged", cfg, qp, kc, vc, pre, table, qs, kl,
             _plain(O, "attention_paged: O", (T, cfg.Hq, 128), to, dev), out_dtype,
             _plain(lse, "attention_paged: lse", (T, cfg.Hq), torch.float32, dev), workspace.data_ptr(),
             workspace.numel() * workspace.element_size())
    return O, lse


def last_device_error(stream=None) -> int:
    return lib().s2o_last_device_error(_stream(stream))


def last_launch_count() -> int:
    return lib().s2o_last_launch_count()


def stage_timing(enable: bool):
    """Turn per-kernel event timing of the plan calls on or off (this thread)."""
    _check(lib().s2o_stage_timing(1 if enable else 0), "s2o_stage_timing")


def last_stage_times() -> list[tuple[str, float]]:
    """(kernel name, device ms) of each kernel of the last plan call on this thread."""
    ms = (ctypes.c_float * 16)()
    names = (ctypes.c_char_p * 16)()
    n = lib().s2o_last_stage_times(ms, names, 16)
    if n < 0:
        raise S2OError(4, "s2o_last_stage_times")
    return [(names[i].decode(), float(ms[i])) for i in range(n)]


def status_string(code: int) -> str:
    return lib().s2o_status_string(code).decode()
