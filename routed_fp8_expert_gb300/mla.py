"""Latent attention: the binding of the mla_* calls of include/moe_fp8.h.

Argument marshalling only, as in _lib: tensors on the CUDA device, bf16 or fp16, the
innermost dimension contiguous; any other stride goes to the kernels as it is (views
of wider projections and of multi-layer caches need no copy). Outputs are allocated
when not given; the current stream of the inputs' device is used.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from ._lib import MOE_ERR_ARG, RMS_NORM_EPS, MoeError, _check, _cuda, _p, _stream, load

MLA_LATENT, MLA_ROPE, MLA_NOPE, MLA_V = 512, 64, 128, 128
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_LAYOUTS = {"interleaved": 0, "half": 1}


def _bad(msg):
    raise MoeError(MOE_ERR_ARG, msg)


def _dtype(*named):
    """The dtype code shared by the given (name, tensor) pairs."""
    first = named[0][1].dtype
    if first not in _DTYPES:
        _bad(f"{named[0][0]} must be bf16 or fp16, not {first}")
    for name, t in named:
        if t.dtype != first:
            _bad(f"{name} is {t.dtype}, {named[0][0]} is {first}")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            _bad(f"the innermost dimension of {name} must be contiguous")
    return _DTYPES[first]


def _device(*ts):
    """All tensors on one CUDA device."""
    _cuda(*ts)
    devs = {t.device for t in ts if t is not None}
    if len(devs) > 1:
        _bad(f"tensors on several devices: {sorted(map(str, devs))}")


def _shape(name, t, *want):
    if t.dim() != len(want) or any(w is not None and s != w for s, w in zip(t.shape, want)):
        _bad(f"{name} has shape {tuple(t.shape)}, expected {tuple('*' if w is None else w for w in want)}")


def _int32(name, t, *want):
    _shape(name, t, *want)
    if t.dtype != torch.int32:
        _bad(f"{name} must be int32, not {t.dtype}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        _bad(f"the innermost dimension of {name} must be contiguous")


def _st(t, dim, width=0):
    """Stride of a dimension; a dimension of one has any stride, so it gets a legal one."""
    return t.stride(dim) if t.shape[dim] > 1 else max(8, (width + 7) // 8 * 8)


def _th(t):
    """Token and head strides of [T, H, width]."""
    return _st(t, 0, t.shape[1] * t.shape[2] if t.shape[1] == 1 else max(t.shape[2], t.stride(1))), _st(t, 1, t.shape[2])


@dataclass
class RopePlan:
    """Rotary frequencies on the device and what goes with them (rope_plan)."""
    freq: torch.Tensor        # int64 [dim / 2]: 2^-64 turns per position
    dim: int
    layout: int               # 0 interleaved, 1 half
    amplitude: float          # factor of the rotated values
    softmax_factor: float     # multiply the softmax scale 1 / sqrt(width) by this


def rope_plan(dim: int = MLA_ROPE, base: float = 10000.0, factor: float = 1.0, original_ctx: int = 4096,
              beta_fast: float = 32.0, beta_slow: float = 1.0, mscale: float = 1.0, mscale_all_dim: float = 0.0,
              layout: str = "interleaved", device="cuda") -> RopePlan:
    """Rotary positions for mla_rope_append, stretched by `factor` for long contexts (YaRN).

    With g(m) = 1 + 0.1 m ln(factor): the rotated values are multiplied by
    g(mscale) / g(mscale_all_dim), and the softmax scale is to be multiplied by
    g(mscale_all_dim)^2 ("Kimi K2 · Architecture", Sources: YaRN rotary embedding)."""
    if layout not in _LAYOUTS:
        _bad(f"layout {layout!r} must be one of {sorted(_LAYOUTS)}")
    host = torch.empty(max(1, dim // 2), dtype=torch.int64)
    _check(load().mla_rope_freqs(dim, float(base), float(factor), int(original_ctx), float(beta_fast),
                                 float(beta_slow), _p(host)))
    g = lambda m: 1.0 + 0.1 * m * math.log(factor)  # noqa: E731
    return RopePlan(host.to(device), dim, _LAYOUTS[layout], g(mscale) / g(mscale_all_dim), g(mscale_all_dim) ** 2)


def mla_rope_append(q_pe, kv, positions, plan: RopePlan, gamma=None, eps: float = RMS_NORM_EPS, cache=None, slots=None,
                    q_out=None, kv_out=None):
    """Rotate the queries' rotary part q_pe [T, H, dim] and append kv [T, latent + dim]
    (RMSNorm of the latent by gamma, rotated key) to the cache [pages, page, latent + dim]
    at `slots` [T] (negative: not cached). positions, slots int32. q_pe or kv may be None.
    kv_out [T, latent + dim] receives the rows too; without a cache it is allocated.
    Returns (q_out, kv_out)."""
    ref = q_pe if q_pe is not None else kv
    if ref is None:
        _bad("q_pe and kv are both None")
    _device(q_pe, kv, positions, plan.freq, gamma, cache, slots, q_out, kv_out)
    T, dim = ref.shape[0], plan.dim
    H, latent = 1, 0
    if q_pe is not None:
        _shape("q_pe", q_pe, T, None, dim)
        H = q_pe.shape[1]
        q_out = torch.empty((T, H, dim), dtype=q_pe.dtype, device=q_pe.device) if q_out is None else q_out
        _shape("q_out", q_out, T, H, dim)
    elif q_out is not None:
        _bad("q_out is given without q_pe")
    if kv is not None:
        _shape("kv", kv, T, None)
        latent = kv.shape[1] - dim
        if cache is None and kv_out is None:
            kv_out = torch.empty((T, latent + dim), dtype=kv.dtype, device=kv.device)
        if kv_out is not None:
            _shape("kv_out", kv_out, T, latent + dim)
        if gamma is not None:
            _shape("gamma", gamma, latent)
        if cache is not None:
            _shape("cache", cache, None, None, latent + dim)
            if slots is None:
                _bad("cache is given without slots")
            _int32("slots", slots, T)
    elif cache is not None or kv_out is not None:
        _bad("cache or kv_out is given without kv")
    _int32("positions", positions, T)
    dt = _dtype(*[(n, t) for n, t in (("q_pe", q_pe), ("kv", kv), ("q_out", q_out), ("kv_out", kv_out),
                                      ("gamma", gamma), ("cache", cache)) if t is not None])
    q_s, qo_s = (_th(q_pe), _th(q_out)) if q_pe is not None else ((0, 0), (0, 0))
    w = latent + dim
    _check(load().mla_rope_append(
        _p(q_pe), *q_s, _p(q_out), *qo_s, _p(kv), _st(kv, 0, w) if kv is not None else 0, _p(gamma), float(eps),
        _p(kv_out), _st(kv_out, 0, w) if kv_out is not None else 0,
        _p(cache), _st(cache, 0, w) if cache is not None else 0, _st(cache, 1, w) if cache is not None else 0,
        cache.shape[0] if cache is not None else 0, cache.shape[1] if cache is not None else 1, _p(slots),
        _p(positions), _p(plan.freq), plan.amplitude, plan.layout, T, H, dim, latent, dt, _stream(ref.device)))
    return q_out, kv_out


def mla_paged_workspace(device=None) -> torch.Tensor:
    """Workspace of mla_attn_paged: one size for every call on the device."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = load().mla_paged_workspace_bytes()
        return torch.empty(n, dtype=torch.uint8, device="cuda")


def mla_attn_paged(q, cache, block_table, ctx_lens, scale: float, cu_q=None, out=None, want_lse: bool = False, ws=None):
    """Absorbed attention of q [Tq, H, 576] over the paged latent cache [pages, page, 576].

    block_table [B, max_pages], ctx_lens [B] (tokens in the cache, the new ones included)
    and cu_q [B + 1] are int32; cu_q None: one query per sequence. Causal: each query sees
    the keys up to its own. Returns out [Tq, H, 512] (and lse [Tq, H] fp32)."""
    _device(q, cache, block_table, ctx_lens, cu_q, out, ws)
    _shape("q", q, None, None, MLA_LATENT + MLA_ROPE)
    _shape("cache", cache, None, None, MLA_LATENT + MLA_ROPE)
    _int32("block_table", block_table, None, None)
    B, max_pages = block_table.shape
    _int32("ctx_lens", ctx_lens, B)
    if cu_q is not None:
        _int32("cu_q", cu_q, B + 1)
    Tq, H = q.shape[0], q.shape[1]
    dev = q.device
    out = torch.empty((Tq, H, MLA_LATENT), dtype=q.dtype, device=dev) if out is None else out
    _shape("out", out, Tq, H, MLA_LATENT)
    dt = _dtype(("q", q), ("cache", cache), ("out", out))
    lse = torch.empty((Tq, H), dtype=torch.float32, device=dev) if want_lse else None
    ws = mla_paged_workspace(dev) if ws is None else ws
    w = MLA_LATENT + MLA_ROPE
    _check(load().mla_attn_paged(
        _p(q), *_th(q), Tq, _p(cache), _st(cache, 0, w), _st(cache, 1, w), cache.shape[0], cache.shape[1],
        _p(block_table), block_table.stride(0) if B > 1 else max_pages, max_pages, _p(ctx_lens), _p(cu_q), B, H,
        float(scale), dt, _p(out), *_th(out), _p(lse), _p(ws), ws.numel() * ws.element_size(), _stream(dev)))
    return (out, lse) if want_lse else out


def mla_attn_ragged(q, k_nope, k_pe, v, cu_q, cu_k, max_q: int, scale: float, causal: bool = True, out=None,
                    want_lse: bool = False):
    """Expanded attention of a ragged batch: q [Tq, H, 192], k_nope and v [Tk, H, 128]
    (views of one tensor, if so), k_pe [Tk, 64] shared by the heads, cu_q and cu_k
    [B + 1] int32 row offsets, max_q at least the longest query run. Causal masks align
    the last query with the last key. Returns out [Tq, H, 128] (and lse [Tq, H] fp32)."""
    _device(q, k_nope, k_pe, v, cu_q, cu_k, out)
    _shape("q", q, None, None, MLA_NOPE + MLA_ROPE)
    Tq, H = q.shape[0], q.shape[1]
    _shape("k_nope", k_nope, None, H, MLA_NOPE)
    Tk = k_nope.shape[0]
    _shape("k_pe", k_pe, Tk, MLA_ROPE)
    _shape("v", v, Tk, H, MLA_V)
    _int32("cu_q", cu_q, None)
    _int32("cu_k", cu_k, cu_q.shape[0])
    B = cu_q.shape[0] - 1
    if B < 0:
        _bad("cu_q is empty")
    dev = q.device
    out = torch.empty((Tq, H, MLA_V), dtype=q.dtype, device=dev) if out is None else out
    _shape("out", out, Tq, H, MLA_V)
    dt = _dtype(("q", q), ("k_nope", k_nope), ("k_pe", k_pe), ("v", v), ("out", out))
    lse = torch.empty((Tq, H), dtype=torch.float32, device=dev) if want_lse else None
    _check(load().mla_attn_ragged(
        _p(q), *_th(q), Tq, _p(k_nope), *_th(k_nope), _p(k_pe), _st(k_pe, 0, MLA_ROPE), _p(v), *_th(v), Tk, _p(cu_q),
        _p(cu_k), B, int(max_q), H, float(scale), int(causal), dt, _p(out), *_th(out), _p(lse), _stream(dev)))
    return (out, lse) if want_lse else out


def mla_head_proj(x, w, w_kn: bool = False, out=None):
    """out[t, h] = x[t, h] W_h with x [T, H, K] (or [T, 1, K], the same for every head) and
    w [H, N, K], or [H, K, N] with w_kn. Returns out [T, H, N]."""
    _device(x, w, out)
    _shape("w", w, None, None, None)
    H = w.shape[0]
    K, N = (w.shape[1], w.shape[2]) if w_kn else (w.shape[2], w.shape[1])
    _shape("x", x, None, None, K)
    shared = x.shape[1] == 1
    if not shared and x.shape[1] != H:
        _bad(f"x has {x.shape[1]} heads, w has {H}")
    T = x.shape[0]
    out = torch.empty((T, H, N), dtype=x.dtype, device=x.device) if out is None else out
    _shape("out", out, T, H, N)
    dt = _dtype(("x", x), ("w", w), ("out", out))
    x_st, x_sh = _th(x)
    o_st, o_sh = _th(out)
    _check(load().mla_head_proj(_p(x), x_st, x_sh, int(shared), _p(w), _st(w, 0, w.shape[1] * w.shape[2]),
                                _st(w, 1, w.shape[2]), int(w_kn), T, H, K, N, dt, _p(out), o_st, o_sh,
                                _stream(x.device)))
    return out
