"""Python binding of libbpt (include/bpt.h): argument marshalling only.

Every step of the layer runs in the CUDA library; this module turns torch
tensors into the pointers and structs the C ABI takes.  PyTorch supplies
device memory and streams.  There is no fallback: if the library is missing
or fails to load, importing the binding's entry points raises.

Entry points keep the C names: bpt_layer_fwd, bpt_layer_bwd,
bpt_attn_headchunk, bpt_attention_fwd, bpt_attention_bwd, bpt_attention_bwd_noalloc,
bpt_lm_loss_fwd, bpt_lm_loss_bwd, bpt_lm_workspace_bytes,
bpt_attention_mod_fwd, bpt_attention_mod_bwd, bpt_attention_mod_bwd_workspace_bytes,
bpt_qk_norm_rope_fwd, bpt_qk_norm_rope_bwd, bpt_qk_norm_rope_workspace_bytes,
bpt_clip_grads, bpt_clip_workspace_bytes,
bpt_workspace_bytes, bpt_saved_bytes, bpt_attention_bwd_workspace_bytes,
bpt_status_string, bpt_last_device_error, bpt_check_device_range, bpt_watchdog_selftest,
bpt_profile_enable, bpt_profile_collect, bpt_profile_list.  The layer stack
with a checkpoint every k layers is in :mod:`.stack` (a scheduler over
bpt_layer_fwd / bpt_layer_bwd).
"""
from __future__ import annotations

import ctypes
import os
from array import array
from dataclasses import dataclass

from .presets import PRESETS, LayerConfig  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbpt.so")

BPT_OK, BPT_EINVAL, BPT_ENOSPC, BPT_ECUDA, BPT_ETIMEOUT, BPT_EUNSUPPORTED = range(6)
BPT_PASS_FWD, BPT_PASS_BWD, BPT_PASS_HEADCHUNK = 0, 1, 2
BPT_STAGE_CONTIGUOUS, BPT_STAGE_INTERLEAVED = 0, 1
BPT_SAVE_NOTHING, BPT_SAVE_PROJECTIONS, BPT_SAVE_ATTN_OUT = 0, 1, 2
BPT_FLAG_ACCUM_GRADS = 1
BPT_FLAG_ONE_STREAM = 2
BPT_FLAG_DETERMINISTIC = 4
BPT_FLAG_DEBUG_CHECKS = 8
BPT_DTYPE_F32, BPT_DTYPE_BF16 = 0, 1

WEIGHT_FIELDS = ("ln1_w", "ln1_b", "wq", "bq", "wk", "bk", "wv", "bv", "wo", "bo",
                 "ln2_w", "ln2_b", "w1", "b1", "w2", "b2", "w3")


class BptConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "b", "s", "h", "n_heads", "n_kv_heads", "head_dim", "ffn_dim",
        "q_block", "kv_block", "ffn_block", "head_chunk", "causal", "norm", "act", "has_bias")] + \
        [("norm_eps", ctypes.c_float), ("flags", ctypes.c_int32), ("rope_base", ctypes.c_float),
         ("stage_order", ctypes.c_int32), ("save_policy", ctypes.c_int32)]


class BptWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_FIELDS]


class BptGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_FIELDS]


class BptLmConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "h", "vocab", "vocab_block", "flags")]


class BptScoreMod(ctypes.Structure):
    _fields_ = [("row_begin", ctypes.c_void_p), ("row_end", ctypes.c_void_p), ("slopes", ctypes.c_void_p),
                ("softcap", ctypes.c_float)]


class BptClipTensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class BptError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bpt_status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libbpt.so (raises if it is missing: build it first with
    ``python -m blockwise_attention_ffn_gb300.build`` or __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libbpt.so not built ({LIB_PATH} missing)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        cfgp = ctypes.POINTER(BptConfig)
        L.bpt_workspace_bytes.argtypes = [cfgp, i32]
        L.bpt_workspace_bytes.restype = sz
        L.bpt_saved_bytes.argtypes = [cfgp]
        L.bpt_saved_bytes.restype = sz
        L.bpt_layer_fwd.argtypes = [cfgp, ctypes.POINTER(BptWeights), vp, vp, vp, vp, sz, vp]
        L.bpt_layer_fwd.restype = i32
        L.bpt_layer_bwd.argtypes = [cfgp, ctypes.POINTER(BptWeights), vp, vp, vp, vp,
                                    ctypes.POINTER(BptGrads), vp, sz, vp]
        L.bpt_layer_bwd.restype = i32
        L.bpt_attn_headchunk.argtypes = [cfgp, ctypes.POINTER(BptWeights), vp, vp, vp, vp, sz, vp]
        L.bpt_attn_headchunk.restype = i32
        L.bpt_attention_fwd.argtypes = [cfgp, vp, vp, vp, vp]
        L.bpt_attention_fwd.restype = i32
        L.bpt_attention_bwd_workspace_bytes.argtypes = [cfgp]
        L.bpt_attention_bwd_workspace_bytes.restype = sz
        L.bpt_attention_bwd.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.bpt_attention_bwd.restype = i32
        L.bpt_attention_bwd_noalloc.argtypes = [cfgp, vp, vp, vp, vp, vp, vp]
        L.bpt_attention_bwd_noalloc.restype = i32
        L.bpt_status_string.argtypes = [i32]
        L.bpt_status_string.restype = ctypes.c_char_p
        L.bpt_last_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
        L.bpt_last_device_error.restype = i32
        lmp = ctypes.POINTER(BptLmConfig)
        L.bpt_lm_workspace_bytes.argtypes = [lmp, i32]
        L.bpt_lm_workspace_bytes.restype = sz
        L.bpt_lm_loss_fwd.argtypes = [lmp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.bpt_lm_loss_fwd.restype = i32
        L.bpt_lm_loss_bwd.argtypes = [lmp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, sz, vp]
        L.bpt_lm_loss_bwd.restype = i32
        modp = ctypes.POINTER(BptScoreMod)
        L.bpt_attention_mod_fwd.argtypes = [cfgp, modp, vp, vp, vp, vp]
        L.bpt_attention_mod_fwd.restype = i32
        L.bpt_attention_mod_bwd_workspace_bytes.argtypes = [cfgp]
        L.bpt_attention_mod_bwd_workspace_bytes.restype = sz
        L.bpt_attention_mod_bwd.argtypes = [cfgp, modp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.bpt_attention_mod_bwd.restype = i32
        L.bpt_qk_norm_rope_workspace_bytes.argtypes = [cfgp]
        L.bpt_qk_norm_rope_workspace_bytes.restype = sz
        L.bpt_qk_norm_rope_fwd.argtypes = [cfgp, vp, vp, vp, vp, vp, vp]
        L.bpt_qk_norm_rope_fwd.restype = i32
        L.bpt_qk_norm_rope_bwd.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.bpt_qk_norm_rope_bwd.restype = i32
        L.bpt_clip_workspace_bytes.argtypes = []
        L.bpt_clip_workspace_bytes.restype = sz
        L.bpt_clip_grads.argtypes = [i32, vp, ctypes.c_float, i32, vp, vp, sz, vp]
        L.bpt_clip_grads.restype = i32
        L.bpt_check_device_range.argtypes = [vp, sz]
        L.bpt_check_device_range.restype = i32
        L.bpt_watchdog_selftest.argtypes = [vp]
        L.bpt_watchdog_selftest.restype = i32
        L.bpt_profile_enable.argtypes = [i32]
        L.bpt_profile_enable.restype = i32
        dp = ctypes.POINTER(ctypes.c_double)
        L.bpt_profile_collect.argtypes = [i32, dp, dp, dp, ctypes.POINTER(ctypes.c_int)]
        L.bpt_profile_collect.restype = i32
        L.bpt_profile_list.argtypes = [i32, ctypes.POINTER(ctypes.c_int), dp, dp, dp]
        L.bpt_profile_list.restype = i32
        _lib = L
    return _lib


# ------------------------------------------------------------------ marshalling

def make_config(c) -> BptConfig:
    """BptConfig from a LayerConfig (or any object with the same fields)."""
    return BptConfig(c.b, c.s, c.h, c.n_heads, c.n_kv_heads, c.head_dim, c.ffn_dim, c.q_block,
                     c.kv_block, c.ffn_block, c.head_chunk, c.causal, c.norm, c.act, c.has_bias,
                     c.norm_eps, c.flags, float(getattr(c, "rope_base", 0.0)),
                     int(getattr(c, "stage_order", 0)), int(getattr(c, "save_policy", 0)))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def make_weights(w: dict) -> BptWeights:
    return BptWeights(*[(None if w.get(n) is None else w[n].data_ptr()) for n in WEIGHT_FIELDS])


def make_grads(g: dict) -> BptGrads:
    return BptGrads(*[(None if g.get(n) is None else g[n].data_ptr()) for n in WEIGHT_FIELDS])


def _stream(stream):
    if stream is None:
        import torch
        if torch.cuda.is_initialized():  # the current stream's handle, without building a Stream object
            return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc, where):
    if rc != BPT_OK:
        raise BptError(rc, where)


def bpt_status_string(status: int) -> str:
    return lib().bpt_status_string(int(status)).decode()


def bpt_workspace_bytes(cfg, pass_: int) -> int:
    return int(lib().bpt_workspace_bytes(ctypes.byref(make_config(cfg)), int(pass_)))


def bpt_saved_bytes(cfg) -> int:
    return int(lib().bpt_saved_bytes(ctypes.byref(make_config(cfg))))


def bpt_attention_bwd_workspace_bytes(cfg) -> int:
    return int(lib().bpt_attention_bwd_workspace_bytes(ctypes.byref(make_config(cfg))))


def bpt_layer_fwd(cfg, weights: dict, x, y, saved, ws, stream=None) -> None:
    c = make_config(cfg)
    w = make_weights(weights)
    rc = lib().bpt_layer_fwd(ctypes.byref(c), ctypes.byref(w), _ptr(x), _ptr(y), _ptr(saved),
                             _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "bpt_layer_fwd")


def bpt_layer_bwd(cfg, weights: dict, x, saved, dy, dx, grads: dict, ws, stream=None) -> None:
    c = make_config(cfg)
    w = make_weights(weights)
    g = make_grads(grads)
    rc = lib().bpt_layer_bwd(ctypes.byref(c), ctypes.byref(w), _ptr(x), _ptr(saved), _ptr(dy),
                             _ptr(dx), ctypes.byref(g), _ptr(ws), ws.numel() * ws.element_size(),
                             _stream(stream))
    _check(rc, "bpt_layer_bwd")


def bpt_attn_headchunk(cfg, weights: dict, xn, o, lse, ws, stream=None) -> None:
    c = make_config(cfg)
    w = make_weights(weights)
    rc = lib().bpt_attn_headchunk(ctypes.byref(c), ctypes.byref(w), _ptr(xn), _ptr(o), _ptr(lse),
                                  _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "bpt_attn_headchunk")


def bpt_attention_fwd(cfg, qkv, o, lse, stream=None) -> None:
    c = make_config(cfg)
    rc = lib().bpt_attention_fwd(ctypes.byref(c), _ptr(qkv), _ptr(o), _ptr(lse), _stream(stream))
    _check(rc, "bpt_attention_fwd")


def bpt_attention_bwd(cfg, qkv, o, lse, dout, dqkv, ws, stream=None) -> None:
    c = make_config(cfg)
    rc = lib().bpt_attention_bwd(ctypes.byref(c), _ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout),
                                 _ptr(dqkv), _ptr(ws), ws.numel() * ws.element_size(),
                                 _stream(stream))
    _check(rc, "bpt_attention_bwd")


def make_lm_config(c) -> BptLmConfig:
    """BptLmConfig from an LmConfig (or any object with n, h, vocab,
    vocab_block and flags)."""
    return BptLmConfig(c.n, c.h, c.vocab, c.vocab_block, c.flags)


def bpt_lm_workspace_bytes(cfg, pass_: int) -> int:
    return int(lib().bpt_lm_workspace_bytes(ctypes.byref(make_lm_config(cfg)), int(pass_)))


def bpt_lm_loss_fwd(cfg, x, w, targets, loss, lse, ws, stream=None) -> None:
    """Mean token cross-entropy of x [n, h] through w [V, h] against int32
    targets [n]: writes loss (one fp32 element) and lse [n] (optional)."""
    c = make_lm_config(cfg)
    rc = lib().bpt_lm_loss_fwd(ctypes.byref(c), _ptr(x), _ptr(w), _ptr(targets), _ptr(loss), _ptr(lse),
                               _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "bpt_lm_loss_fwd")


def bpt_lm_loss_bwd(cfg, x, w, targets, lse, dloss, dx, dw, ws, stream=None) -> None:
    """Gradients of dloss * loss: dx [n, h] bf16 and dw [V, h] fp32."""
    c = make_lm_config(cfg)
    rc = lib().bpt_lm_loss_bwd(ctypes.byref(c), _ptr(x), _ptr(w), _ptr(targets), _ptr(lse), float(dloss),
                               _ptr(dx), _ptr(dw), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "bpt_lm_loss_bwd")


def _want(where, what, t, dtype, numel, dev):
    """The address of t.  Refuses (BPT_EINVAL) a tensor the library would read
    past or misread: not on the current CUDA device `dev`, not contiguous, of
    another type or with fewer elements than the call touches."""
    if t is None:
        raise BptError(BPT_EINVAL, f"{where}: {what} is missing")
    if t.dtype is dtype and t.get_device() == dev and t.numel() >= numel and t.is_contiguous():
        return t.data_ptr()
    raise BptError(BPT_EINVAL, f"{where}: {what} must be a contiguous {dtype} tensor of at least {numel} elements on "
                               f"the current device, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _may(where, what, t, dtype, numel, dev):
    return None if t is None else _want(where, what, t, dtype, numel, dev)


def _packed_numel(c):
    return c.b * c.s * (c.n_heads + 2 * c.n_kv_heads) * c.head_dim


@dataclass(frozen=True)
class ScoreMod:
    """What bpt_attention_mod_fwd/bwd change about the attention: the keys
    [row_begin, row_end) that each query row sees ([b*s] int32 tensors, None:
    from 0, to s), the per-head slopes of a bias -slope * |i - j| ([H] fp32),
    and the cap of softcap * tanh(score / softcap) (0: none)."""
    row_begin: object = None
    row_end: object = None
    slopes: object = None
    softcap: float = 0.0


def _score_mod(where, cfg, mod, dev):
    import torch
    rows = cfg.b * cfg.s
    return BptScoreMod(_may(where, "row_begin", mod.row_begin, torch.int32, rows, dev),
                       _may(where, "row_end", mod.row_end, torch.int32, rows, dev),
                       _may(where, "slopes", mod.slopes, torch.float32, cfg.n_heads, dev), mod.softcap)


def bpt_attention_mod_fwd(cfg, mod, qkv, o, lse, stream=None) -> None:
    """Attention of the packed qkv [b*s, (H + 2 H_kv) d] with the scores
    modified by mod (a ScoreMod): o [b*s, H d] bf16 and lse [b, H, s_pad] fp32
    (None: not wanted)."""
    import torch
    where, dev = "bpt_attention_mod_fwd", torch.cuda.current_device()
    hd = cfg.b * cfg.s * cfg.n_heads * cfg.head_dim
    c, m = make_config(cfg), _score_mod(where, cfg, mod, dev)
    _check(lib().bpt_attention_mod_fwd(
        c, m, _want(where, "qkv", qkv, torch.bfloat16, _packed_numel(cfg), dev),
        _want(where, "o", o, torch.bfloat16, hd, dev),
        _may(where, "lse", lse, torch.float32, cfg.b * cfg.n_heads * s_pad(cfg), dev), _stream(stream)), where)


def bpt_attention_mod_bwd_workspace_bytes(cfg) -> int:
    return int(lib().bpt_attention_mod_bwd_workspace_bytes(ctypes.byref(make_config(cfg))))


def bpt_attention_mod_bwd(cfg, mod, qkv, o, lse, dout, dqkv, ws, stream=None) -> None:
    """Gradients of bpt_attention_mod_fwd with respect to qkv, given dout
    [b*s, H d] and what the forward wrote; dqkv like qkv, a buffer of its own."""
    import torch
    where, dev = "bpt_attention_mod_bwd", torch.cuda.current_device()
    n, hd = _packed_numel(cfg), cfg.b * cfg.s * cfg.n_heads * cfg.head_dim
    c, m = make_config(cfg), _score_mod(where, cfg, mod, dev)
    _check(lib().bpt_attention_mod_bwd(
        c, m, _want(where, "qkv", qkv, torch.bfloat16, n, dev), _want(where, "o", o, torch.bfloat16, hd, dev),
        _want(where, "lse", lse, torch.float32, cfg.b * cfg.n_heads * s_pad(cfg), dev),
        _want(where, "dout", dout, torch.bfloat16, hd, dev), _want(where, "dqkv", dqkv, torch.bfloat16, n, dev),
        _want(where, "ws", ws, torch.uint8, 0, dev), ws.numel(), _stream(stream)), where)


def bpt_qk_norm_rope_workspace_bytes(cfg) -> int:
    return int(lib().bpt_qk_norm_rope_workspace_bytes(ctypes.byref(make_config(cfg))))


def bpt_qk_norm_rope_fwd(cfg, qkv, wq, wk, positions, out, stream=None) -> None:
    """Head norm (weights wq, wk [d]; both None: none) and rotation (base
    cfg.rope_base; 0: none) of the query and key heads of qkv [b*s, (H +
    2 H_kv) d] at `positions` [b*s] int32 (None: the row's index in its
    sequence), into out (qkv itself: in place)."""
    import torch
    n, where, dev = _packed_numel(cfg), "bpt_qk_norm_rope_fwd", torch.cuda.current_device()
    bf16, d = torch.bfloat16, cfg.head_dim
    _check(lib().bpt_qk_norm_rope_fwd(
        make_config(cfg), _want(where, "qkv", qkv, bf16, n, dev), _may(where, "wq", wq, bf16, d, dev),
        _may(where, "wk", wk, bf16, d, dev), _may(where, "positions", positions, torch.int32, cfg.b * cfg.s, dev),
        _want(where, "out", out, bf16, n, dev), _stream(stream)), where)


def bpt_qk_norm_rope_bwd(cfg, qkv, wq, wk, positions, dout, dqkv, dwq, dwk, ws, stream=None) -> None:
    """Gradients of bpt_qk_norm_rope_fwd: dqkv (dout itself: in place) and
    the weights' dwq, dwk [d] fp32.  qkv is the forward's input, before the
    norm.  Without weights qkv, dwq, dwk and ws may be None."""
    import torch
    n, where, dev = _packed_numel(cfg), "bpt_qk_norm_rope_bwd", torch.cuda.current_device()
    bf16, f32, d = torch.bfloat16, torch.float32, cfg.head_dim
    need = _may if wq is None and wk is None else _want  # without weights these may be missing
    _check(lib().bpt_qk_norm_rope_bwd(
        make_config(cfg), need(where, "qkv", qkv, bf16, n, dev), _may(where, "wq", wq, bf16, d, dev),
        _may(where, "wk", wk, bf16, d, dev), _may(where, "positions", positions, torch.int32, cfg.b * cfg.s, dev),
        _want(where, "dout", dout, bf16, n, dev), _want(where, "dqkv", dqkv, bf16, n, dev),
        need(where, "dwq", dwq, f32, d, dev), need(where, "dwk", dwk, f32, d, dev),
        need(where, "ws", ws, torch.uint8, 0, dev), 0 if ws is None else ws.numel(), _stream(stream)), where)


def bpt_clip_workspace_bytes() -> int:
    return int(lib().bpt_clip_workspace_bytes())


def bpt_clip_grads(grads, max_norm, norm, ws, out=None, flags=0, stream=None) -> None:
    """Global norm of the tensors `grads` (fp32 or bf16, contiguous) into
    norm (one fp32 element), and grads * min(1, max_norm / (norm + 1e-6)) into
    the tensors `out` (None: in place)."""
    import torch
    where, dev = "bpt_clip_grads", torch.cuda.current_device()
    out = grads if out is None else out
    if len(out) != len(grads):
        raise BptError(BPT_EINVAL, f"{where}: {len(grads)} gradients, {len(out)} outputs")
    f32, bf16 = torch.float32, torch.bfloat16
    rows = []  # BptClipTensor records as 64-bit words (the dtype in the low half of its last)
    for g, o in zip(grads, out):
        n, kind = g.numel(), g.dtype
        if not ((kind is f32 or kind is bf16) and o.dtype is kind and o.numel() == n and g.get_device() == dev
                and o.get_device() == dev and g.is_contiguous() and o.is_contiguous()):
            raise BptError(BPT_EINVAL, f"{where}: gradients and outputs must be contiguous fp32 or bf16 tensors of "
                                       f"equal type and size on the current device")
        rows += (g.data_ptr(), o.data_ptr(), n, BPT_DTYPE_F32 if kind is f32 else BPT_DTYPE_BF16)
    table = array("q", rows)
    _check(lib().bpt_clip_grads(len(grads), table.buffer_info()[0], max_norm, flags,
                                _want(where, "norm", norm, f32, 1, dev), _want(where, "ws", ws, torch.uint8, 0, dev),
                                ws.numel(), _stream(stream)), where)


BPT_LM_BAD_TARGET_SITE = 950
NOALLOC_SCRATCH_BYTES = 192 * 1024 * 1024


def bpt_attention_bwd_noalloc(cfg, qkv, o, lse, dout, dqkv, stream=None) -> None:
    """bpt_attention_bwd for callers that cannot allocate device memory at
    call time: the scratch (bpt_attention_bwd_workspace_bytes(cfg) =
    24*b*H*s_pad bytes: the fp32 dO.O sums and -LSE*log2(e), and a 16-byte
    bf16 row of both per query) is a fixed array inside the library (at most
    NOALLOC_SCRATCH_BYTES; larger problems raise BptError with BPT_ENOSPC).
    Calls that overlap on the GPU share that array and race: serialise them."""
    c = make_config(cfg)
    rc = lib().bpt_attention_bwd_noalloc(ctypes.byref(c), _ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout),
                                         _ptr(dqkv), _stream(stream))
    _check(rc, "bpt_attention_bwd_noalloc")


def bpt_check_device_range(ptr: int, nbytes: int) -> int:
    """BPT_OK if [ptr, ptr + nbytes) lies inside one device allocation of the
    current device, else BPT_EINVAL (launches nothing)."""
    return int(lib().bpt_check_device_range(ctypes.c_void_p(ptr), int(nbytes)))


def bpt_last_device_error(stream=None):
    """(status, detail) after synchronising the stream; clears the word."""
    d = ctypes.c_int(0)
    rc = lib().bpt_last_device_error(_stream(stream), ctypes.byref(d))
    return int(rc), int(d.value)


BPT_WATCHDOG_SELFTEST_SITE = 900


def bpt_watchdog_selftest(stream=None) -> None:
    """Launch the watchdog self-test: a wait on a barrier nothing signals runs
    out after about 2 s and is recorded as (BPT_ETIMEOUT,
    BPT_WATCHDOG_SELFTEST_SITE), which bpt_last_device_error() then reads."""
    _check(lib().bpt_watchdog_selftest(_stream(stream)), "bpt_watchdog_selftest")


PROF_KINDS = ("gemm", "attn_fwd", "attn_bwd", "norm", "misc")


def bpt_profile_enable(on: bool) -> None:
    _check(lib().bpt_profile_enable(1 if on else 0), "bpt_profile_enable")


def bpt_profile_collect() -> dict:
    """{kind: dict(ms=..., flops=..., bytes=..., launches=...)} since the
    last collect (synchronises on the recorded events)."""
    n = len(PROF_KINDS)
    ms, fl, by = (ctypes.c_double * n)(), (ctypes.c_double * n)(), (ctypes.c_double * n)()
    la = (ctypes.c_int * n)()
    _check(lib().bpt_profile_collect(n, ms, fl, by, la), "bpt_profile_collect")
    return {k: dict(ms=ms[i], flops=fl[i], bytes=by[i], launches=la[i])
            for i, k in enumerate(PROF_KINDS)}


def bpt_profile_list(max_launches: int = 4096) -> list:
    """[(kind, flops, bytes, ms)] of every launch recorded since the last
    collect, in launch order (does not clear the record)."""
    n = max_launches
    kd = (ctypes.c_int * n)()
    fl, by, ms = (ctypes.c_double * n)(), (ctypes.c_double * n)(), (ctypes.c_double * n)()
    got = lib().bpt_profile_list(n, kd, fl, by, ms)
    if got < 0:
        _check(-got, "bpt_profile_list")
    return [(PROF_KINDS[kd[i]], fl[i], by[i], ms[i]) for i in range(got)]


# ------------------------------------------------------------------ helpers

def s_pad(cfg) -> int:
    return (cfg.s + 127) // 128 * 128


def alloc_bytes(n: int, device="cuda"):
    """A 256-byte aligned uint8 device buffer of at least n bytes."""
    import torch
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device=device)


def alloc_grads(weights: dict, device="cuda") -> dict:
    import torch
    return {k: (None if v is None else torch.empty(v.shape, dtype=torch.float32, device=device))
            for k, v in weights.items()}
