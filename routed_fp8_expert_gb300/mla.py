"""Latent attention: the binding of the mla_* calls of include/moe_fp8.h (forward only).

Argument marshalling only, as in _lib: tensors on the CUDA device, bf16 or fp16, the
innermost dimension contiguous; any other stride goes to the kernels as it is (views
of wider projections and of multi-layer caches need no copy). Outputs are allocated
when not given; a call runs on the inputs' device, on its current stream.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from ._lib import MOE_ERR_ARG, RMS_NORM_EPS, MoeError, _check, _p, load

MLA_LATENT, MLA_ROPE, MLA_NOPE, MLA_V = 512, 64, 128, 128
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_LAYOUTS = {"interleaved": 0, "half": 1}


# the raw handle: building a torch.cuda.Stream object costs more than a small launch
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _enqueue(dev, fn, *args):
    """Make the C call on device `dev`: the library asks the current device for its SMs, its
    error word and its launch, which has to be the device of the tensors and the stream."""
    if _current_device() == dev:
        _check(fn(*args))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args))


def _bad(msg):
    raise MoeError(MOE_ERR_ARG, msg)


def _index(t):
    """CUDA device index of the tensor that names a call's device."""
    i = t.get_device()
    if i < 0:
        raise ValueError("tensors must be on a CUDA device")
    return i


def _refuse(name, t, shape, dtype, index):
    """Say what is wrong with a tensor of another shape, type, device or innermost stride."""
    if t.get_device() < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    if tuple(t.shape) != shape:
        _bad(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype != dtype:
        _bad(f"{name} is {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        _bad(f"{name} is on device {t.get_device()}, the call on {index}")
    _bad(f"the innermost dimension of {name} must be contiguous")


# The argument forms: address (and outer strides) of a tensor that has to have the given
# shape, type and device and a contiguous innermost dimension. A dimension of one may
# carry any stride, so it gets a legal one.
def _vec(name, t, n, dtype, index):
    if t.shape != (n,) or t.dtype is not dtype or t.get_device() != index or (n > 1 and t.stride(0) != 1):
        _refuse(name, t, (n,), dtype, index)
    return t.data_ptr()


def _mat(name, t, n0, n1, dtype, index):
    s0, s1 = t.stride() if t.dim() == 2 else (0, 0)
    if t.shape != (n0, n1) or t.dtype is not dtype or t.get_device() != index or (s1 != 1 and n1 > 1):
        _refuse(name, t, (n0, n1), dtype, index)
    return t.data_ptr(), s0 if n0 > 1 else _pad8(n1)


def _ten(name, t, n0, n1, n2, dtype, index):
    s0, s1, s2 = t.stride() if t.dim() == 3 else (0, 0, 0)
    if t.shape != (n0, n1, n2) or t.dtype is not dtype or t.get_device() != index or (s2 != 1 and n2 > 1):
        _refuse(name, t, (n0, n1, n2), dtype, index)
    if n1 <= 1:
        s1 = _pad8(n2)
    if n0 <= 1:
        s0 = _pad8(max(n2, s1))
    return t.data_ptr(), s0, s1


def _code(name, t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        _bad(f"{name} must be bf16 or fp16, not {t.dtype}")
    return code


def _dims(name, t, n):
    if t.dim() != n:
        _bad(f"{name} has shape {tuple(t.shape)}, expected {n} dimensions")
    return t.shape


def _pad8(n):
    return max(8, (n + 7) & ~7)


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
    dev, ty, dim, T = _index(ref), ref.dtype, plan.dim, ref.shape[0]
    code = _code("q_pe" if q_pe is not None else "kv", ref)
    H, page, latent, pages, gp, sp = 1, 1, 0, 0, None, None
    qa = qo = (None, 0, 0)
    ka = ko = (None, 0)
    ca = (None, 0, 0)
    if q_pe is not None:
        H = _dims("q_pe", q_pe, 3)[1]
        qa = _ten("q_pe", q_pe, T, H, dim, ty, dev)
        if q_out is None:
            q_out = torch.empty((T, H, dim), dtype=ty, device=ref.device)
        qo = _ten("q_out", q_out, T, H, dim, ty, dev)
    elif q_out is not None:
        _bad("q_out is given without q_pe")
    if kv is not None:
        width = _dims("kv", kv, 2)[1]
        latent = width - dim
        ka = _mat("kv", kv, T, width, ty, dev)
        if kv_out is None and cache is None:
            kv_out = torch.empty((T, width), dtype=ty, device=ref.device)
        if kv_out is not None:
            ko = _mat("kv_out", kv_out, T, width, ty, dev)
        if gamma is not None:
            gp = _vec("gamma", gamma, latent, ty, dev)
        if cache is not None:
            if slots is None:
                _bad("cache is given without slots")
            pages, page, _ = _dims("cache", cache, 3)
            ca = _ten("cache", cache, pages, page, width, ty, dev)
            if pages == 0:   # no address, which would mean no cache: any will do, since no slot lies in it
                ca = (kv.data_ptr(), *ca[1:])
            sp = _vec("slots", slots, T, torch.int32, dev)
    elif cache is not None or kv_out is not None:
        _bad("cache or kv_out is given without kv")
    pp = _vec("positions", positions, T, torch.int32, dev)
    fp = _vec("plan.freq", plan.freq, dim // 2, torch.int64, dev)
    _enqueue(dev, load().mla_rope_append, *qa, *qo, *ka, gp, eps, *ko, *ca, pages, page, sp, pp, fp, plan.amplitude,
             plan.layout, T, H, dim, latent, code, _raw_stream(dev))
    return q_out, kv_out


def mla_paged_workspace(device=None) -> torch.Tensor:
    """Workspace of mla_attn_paged: one size for every call on the device. Calls that
    may overlap (on several streams) need one each."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = load().mla_paged_workspace_bytes()
        return torch.empty(n, dtype=torch.uint8, device="cuda")


def mla_attn_paged(q, cache, block_table, ctx_lens, scale: float, cu_q=None, out=None, want_lse: bool = False, ws=None):
    """Absorbed attention of q [Tq, H, 576] over the paged latent cache [pages, page, 576].

    block_table [B, max_pages], ctx_lens [B] (tokens in the cache, the new ones included)
    and cu_q [B + 1] are int32; cu_q None: one query per sequence. Causal: each query sees
    the keys up to its own. Returns out [Tq, H, 512] (and lse [Tq, H] fp32)."""
    dev, ty = _index(q), q.dtype
    code, width = _code("q", q), MLA_LATENT + MLA_ROPE
    Tq, H, _ = _dims("q", q, 3)
    pages, page, _ = _dims("cache", cache, 3)
    B, max_pages = _dims("block_table", block_table, 2)
    tp, t_st = _mat("block_table", block_table, B, max_pages, torch.int32, dev)
    if out is None:
        out = torch.empty((Tq, H, MLA_LATENT), dtype=ty, device=q.device)
    lse = torch.empty((Tq, H), dtype=torch.float32, device=q.device) if want_lse else None
    if ws is None:
        ws = mla_paged_workspace(q.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        _bad("ws must be contiguous and on the call's device")
    _enqueue(
        dev, load().mla_attn_paged, *_ten("q", q, Tq, H, width, ty, dev), Tq,
        *_ten("cache", cache, pages, page, width, ty, dev), pages, page, tp, t_st if B > 1 else max_pages, max_pages,
        _vec("ctx_lens", ctx_lens, B, torch.int32, dev),
        None if cu_q is None else _vec("cu_q", cu_q, B + 1, torch.int32, dev), B, H, scale, code,
        *_ten("out", out, Tq, H, MLA_LATENT, ty, dev), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes,
        _raw_stream(dev))
    return (out, lse) if want_lse else out


def mla_attn_ragged(q, k_nope, k_pe, v, cu_q, cu_k, max_q: int, scale: float, causal: bool = True, out=None,
                    want_lse: bool = False):
    """Expanded attention of a ragged batch: q [Tq, H, 192], k_nope and v [Tk, H, 128]
    (views of one tensor, if so), k_pe [Tk, 64] shared by the heads, cu_q and cu_k
    [B + 1] int32 row offsets, max_q at least the longest query run. Causal masks align
    the last query with the last key. Returns out [Tq, H, 128] (and lse [Tq, H] fp32)."""
    dev, ty, code = _index(q), q.dtype, _code("q", q)
    Tq, H, _ = _dims("q", q, 3)
    Tk = _dims("k_nope", k_nope, 3)[0]
    B = _dims("cu_q", cu_q, 1)[0] - 1
    if B < 0:
        _bad("cu_q is empty")
    if out is None:
        out = torch.empty((Tq, H, MLA_V), dtype=ty, device=q.device)
    lse = torch.empty((Tq, H), dtype=torch.float32, device=q.device) if want_lse else None
    _enqueue(
        dev, load().mla_attn_ragged, *_ten("q", q, Tq, H, MLA_NOPE + MLA_ROPE, ty, dev), Tq,
        *_ten("k_nope", k_nope, Tk, H, MLA_NOPE, ty, dev), *_mat("k_pe", k_pe, Tk, MLA_ROPE, ty, dev),
        *_ten("v", v, Tk, H, MLA_V, ty, dev), Tk, _vec("cu_q", cu_q, B + 1, torch.int32, dev),
        _vec("cu_k", cu_k, B + 1, torch.int32, dev), B, max_q, H, scale, 1 if causal else 0, code,
        *_ten("out", out, Tq, H, MLA_V, ty, dev), None if lse is None else lse.data_ptr(), _raw_stream(dev))
    return (out, lse) if want_lse else out


def mla_head_proj(x, w, w_kn: bool = False, out=None):
    """out[t, h] = x[t, h] W_h with x [T, H, K] (or [T, 1, K], the same for every head) and
    w [H, N, K], or [H, K, N] with w_kn. Returns out [T, H, N]."""
    dev, ty, code = _index(x), x.dtype, _code("x", x)
    H, N, K = _dims("w", w, 3)
    if w_kn:
        N, K = K, N
    T, xh, _ = _dims("x", x, 3)
    if xh != 1 and xh != H:
        _bad(f"x has {xh} heads, w has {H}")
    if out is None:
        out = torch.empty((T, H, N), dtype=ty, device=x.device)
    wa = _ten("w", w, H, K, N, ty, dev) if w_kn else _ten("w", w, H, N, K, ty, dev)
    _enqueue(dev, load().mla_head_proj, *_ten("x", x, T, xh, K, ty, dev), 1 if xh == 1 else 0, *wa, 1 if w_kn else 0, T,
             H, K, N, code, *_ten("out", out, T, H, N, ty, dev), _raw_stream(dev))
    return out
