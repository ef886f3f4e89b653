"""Latent attention on the host: rotary frequencies and the refusals of every call.
No GPU: bad arguments are turned away before anything is enqueued."""
import contextlib
import ctypes
import decimal
import math
import os
import re
import types

import pytest
import torch

import routed_fp8_expert_gb300 as moe
from _mla_ref import rope_frequencies
from routed_fp8_expert_gb300 import _lib, build, mla

P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("dim,base,kw", [
    (64, 10000.0, {}), (64, 50000.0, dict(factor=32.0)), (128, 500000.0, dict(factor=8.0, original_ctx=8192)),
    (2, 10000.0, {}), (64, 50000.0, dict(factor=32.0, beta_fast=1.0, beta_slow=1.0)), (256, 1.5, dict(factor=2.0)),
])
def test_rope_frequencies(lib, dim, base, kw):
    f = (ctypes.c_uint64 * (dim // 2))()
    assert lib.mla_rope_freqs(dim, base, kw.get("factor", 1.0), kw.get("original_ctx", 4096),
                              kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0), f) == _lib.MOE_OK
    want = rope_frequencies(dim, base, **kw) / (2 * math.pi)
    got = torch.tensor([v / 2.0 ** 64 for v in f], dtype=torch.float64)
    assert torch.allclose(got, want, rtol=1e-14, atol=2.0 ** -63)


@pytest.mark.parametrize("dim,base,factor", [(64, 10000.0, 1.0), (64, 50000.0, 32.0), (128, 500000.0, 8.0), (16, 1.5, 40.0)])
def test_rope_frequencies_to_50_bits(lib, dim, base, factor):
    # against 60 decimal digits: what the kernel's statement of the angle's error counts on
    D = decimal.Decimal
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        two_pi = 2 * D("3.14159265358979323846264338327950288419716939937510582097494459")
        f = (ctypes.c_uint64 * (dim // 2))()
        assert lib.mla_rope_freqs(dim, base, factor, 4096, 32.0, 1.0, f) == _lib.MOE_OK
        pair = lambda r: dim * (D(4096) / (two_pi * D(r))).ln() / (2 * D(base).ln())  # noqa: E731
        low, high = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), dim - 1)
        for i in range(dim // 2):
            want = (-D(2 * i) / D(dim) * D(base).ln()).exp() / two_pi
            if factor > 1:
                ramp = min(D(1), max(D(0), D(i - low) / max(D(high - low), D("0.001"))))
                want = want * (1 - ramp) + want / D(factor) * ramp
            assert abs(D(f[i]) - want * 2 ** 64) <= want * 2 ** 14 + 1


@pytest.mark.parametrize("args,code", [
    ((63, 1e4, 1.0, 4096, 32.0, 1.0), _lib.MOE_ERR_UNSUPPORTED), ((258, 1e4, 1.0, 4096, 32.0, 1.0), _lib.MOE_ERR_UNSUPPORTED),
    ((0, 1e4, 1.0, 4096, 32.0, 1.0), _lib.MOE_ERR_UNSUPPORTED), ((64, 1.0, 1.0, 4096, 32.0, 1.0), _lib.MOE_ERR_ARG),
    ((64, math.nan, 1.0, 4096, 32.0, 1.0), _lib.MOE_ERR_ARG), ((64, 1e4, 0.5, 4096, 32.0, 1.0), _lib.MOE_ERR_ARG),
    ((64, 1e4, 2.0, 0, 32.0, 1.0), _lib.MOE_ERR_ARG), ((64, 1e4, 2.0, 4096, 0.0, 1.0), _lib.MOE_ERR_ARG),
    ((64, 1e4, 2.0, 4096, 32.0, math.inf), _lib.MOE_ERR_ARG),
])
def test_rope_frequencies_refused(lib, args, code):
    assert lib.mla_rope_freqs(*args, (ctypes.c_uint64 * 256)()) == code
    assert lib.moe_last_error_string()


ROPE = dict(q=P, q_st=4096, q_sh=64, q_out=P, qo_st=4096, qo_sh=64, kv=P, kv_st=576, gamma=P, eps=1e-6, kv_out=P,
            kvo_st=576, cache=P, page_st=64 * 576, row_st=576, num_pages=4, page_size=64, slots=P, positions=P, freq=P,
            amplitude=1.0, layout=0, T=4, H=64, dim=64, latent=512, dtype=0, stream=None)
PAGED = dict(q=P, q_st=64 * 576, q_sh=576, Tq=4, cache=P, page_st=64 * 576, row_st=576, num_pages=9, page_size=64,
             table=P, table_st=8, max_pages=8, ctx=P, cu_q=None, B=4, H=64, scale=0.07, dtype=0, out=P, o_st=64 * 512,
             o_sh=512, lse=None, ws=P, ws_bytes=1 << 30, stream=None)
RAGGED = dict(q=P, q_st=64 * 192, q_sh=192, Tq=4, kn=P, kn_st=64 * 256, kn_sh=256, kp=P, kp_st=64, v=P, v_st=64 * 256,
              v_sh=256, Tk=4, cu_q=P, cu_k=P, B=1, max_q=4, H=64, scale=0.07, causal=1, dtype=0, out=P, o_st=64 * 128,
              o_sh=128, lse=None, stream=None)
PROJ = dict(x=P, x_st=64 * 128, x_sh=128, shared=0, w=P, w_sh=512 * 128, w_sr=128, w_kn=0, T=4, H=64, K=128, N=512,
            dtype=0, out=P, o_st=64 * 512, o_sh=512, stream=None)
ARG, UNS = _lib.MOE_ERR_ARG, _lib.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,base,change,code", [
    ("mla_rope_append", ROPE, dict(dtype=2), ARG), ("mla_rope_append", ROPE, dict(dim=24), UNS),
    ("mla_rope_append", ROPE, dict(dim=272), UNS), ("mla_rope_append", ROPE, dict(layout=2), ARG),
    ("mla_rope_append", ROPE, dict(q=None, kv=None), ARG), ("mla_rope_append", ROPE, dict(q=ODD), ARG),
    ("mla_rope_append", ROPE, dict(q_out=None), ARG), ("mla_rope_append", ROPE, dict(q_st=4097), ARG),
    ("mla_rope_append", ROPE, dict(qo_sh=32), ARG), ("mla_rope_append", ROPE, dict(latent=4), UNS),
    ("mla_rope_append", ROPE, dict(latent=2048), UNS), ("mla_rope_append", ROPE, dict(kv_out=None, cache=None), ARG),
    ("mla_rope_append", ROPE, dict(row_st=512), ARG), ("mla_rope_append", ROPE, dict(slots=None), ARG),
    ("mla_rope_append", ROPE, dict(page_size=0), UNS), ("mla_rope_append", ROPE, dict(eps=-1.0), ARG),
    ("mla_rope_append", ROPE, dict(positions=None), ARG), ("mla_rope_append", ROPE, dict(freq=None), ARG),
    ("mla_rope_append", ROPE, dict(T=-1), ARG), ("mla_rope_append", ROPE, dict(H=0), UNS),
    ("mla_rope_append", ROPE, dict(amplitude=math.inf), ARG), ("mla_rope_append", ROPE, dict(kv_st=0), ARG),
    ("mla_attn_paged", PAGED, dict(dtype=-1), ARG), ("mla_attn_paged", PAGED, dict(H=0), UNS),
    ("mla_attn_paged", PAGED, dict(H=129), UNS), ("mla_attn_paged", PAGED, dict(scale=0.0), ARG),
    ("mla_attn_paged", PAGED, dict(scale=math.nan), ARG), ("mla_attn_paged", PAGED, dict(B=-1), ARG),
    ("mla_attn_paged", PAGED, dict(B=8193, Tq=8193), UNS), ("mla_attn_paged", PAGED, dict(Tq=5), ARG),
    ("mla_attn_paged", PAGED, dict(page_size=12), UNS), ("mla_attn_paged", PAGED, dict(page_size=0), UNS),
    ("mla_attn_paged", PAGED, dict(num_pages=0), UNS), ("mla_attn_paged", PAGED, dict(q=None), ARG),
    ("mla_attn_paged", PAGED, dict(cache=ODD), ARG), ("mla_attn_paged", PAGED, dict(row_st=568), ARG),
    ("mla_attn_paged", PAGED, dict(row_st=580), ARG), ("mla_attn_paged", PAGED, dict(table=None), ARG),
    ("mla_attn_paged", PAGED, dict(table_st=7), ARG), ("mla_attn_paged", PAGED, dict(ctx=None), ARG),
    ("mla_attn_paged", PAGED, dict(out=None), ARG), ("mla_attn_paged", PAGED, dict(o_sh=500), ARG),
    ("mla_attn_paged", PAGED, dict(ws=None), ARG), ("mla_attn_paged", PAGED, dict(ws_bytes=1000), ARG),
    ("mla_attn_paged", PAGED, dict(max_pages=-1), UNS), ("mla_attn_paged", PAGED, dict(q_sh=-8), ARG),
    ("mla_attn_ragged", RAGGED, dict(dtype=3), ARG), ("mla_attn_ragged", RAGGED, dict(causal=2), ARG),
    ("mla_attn_ragged", RAGGED, dict(H=0), UNS), ("mla_attn_ragged", RAGGED, dict(H=1025), UNS),
    ("mla_attn_ragged", RAGGED, dict(B=65536), UNS), ("mla_attn_ragged", RAGGED, dict(Tk=-1), ARG),
    ("mla_attn_ragged", RAGGED, dict(max_q=-1), ARG), ("mla_attn_ragged", RAGGED, dict(kn=None), ARG),
    ("mla_attn_ragged", RAGGED, dict(v=ODD), ARG), ("mla_attn_ragged", RAGGED, dict(kp_st=60), ARG),
    ("mla_attn_ragged", RAGGED, dict(cu_k=None), ARG), ("mla_attn_ragged", RAGGED, dict(o_st=64), ARG),
    ("mla_attn_ragged", RAGGED, dict(scale=-1.0), ARG), ("mla_attn_ragged", RAGGED, dict(q_st=1 << 40), ARG),
    ("mla_attn_paged", PAGED, dict(B=0, cu_q=P), ARG), ("mla_attn_ragged", RAGGED, dict(B=0), ARG),   # rows, but no sequence
    ("mla_head_proj", PROJ, dict(dtype=9), ARG), ("mla_head_proj", PROJ, dict(shared=2), ARG),
    ("mla_head_proj", PROJ, dict(w_kn=-1), ARG), ("mla_head_proj", PROJ, dict(K=12), UNS),
    ("mla_head_proj", PROJ, dict(K=0), UNS), ("mla_head_proj", PROJ, dict(N=4), UNS),
    ("mla_head_proj", PROJ, dict(N=16384), UNS), ("mla_head_proj", PROJ, dict(H=0), UNS),
    ("mla_head_proj", PROJ, dict(T=-1), ARG), ("mla_head_proj", PROJ, dict(T=(1 << 20) + 1), UNS),
    ("mla_head_proj", PROJ, dict(x=None), ARG), ("mla_head_proj", PROJ, dict(w=ODD), ARG),
    ("mla_head_proj", PROJ, dict(w_sr=64), ARG), ("mla_head_proj", PROJ, dict(o_sh=256), ARG),
    ("mla_head_proj", PROJ, dict(x_st=12), ARG),
])
def test_refusals(lib, call, base, change, code):
    args = dict(base)
    args.update(change)
    assert getattr(lib, call)(*args.values()) == code
    assert lib.moe_last_error_string() and lib.moe_last_launch_count() == 0


@pytest.mark.parametrize("T,H,K,N,shared,form", [
    (4096, 64, 512, 256, 1, 1), (1500, 64, 512, 256, 1, 1), (2049, 10, 512, 264, 1, 1), (1281, 2, 1024, 1024, 0, 1),
    (4096, 64, 128, 512, 0, 0), (1, 64, 512, 256, 1, 0), (0, 64, 512, 256, 1, 0),
    (2000, 4, 1024, 1152, 0, 0), (3001, 9, 1024, 264, 1, 0),   # an odd number of weight blocks
    (-1, 4, 128, 128, 0, ARG), (4, 4, 128, 128, 2, ARG), (4, 0, 128, 128, 0, UNS), (4, 4, 12, 128, 0, UNS), (4, 4, 128, 8200, 1, UNS),
])
def test_head_proj_form(lib, T, H, K, N, shared, form):
    assert lib.mla_head_proj_form(T, H, K, N, shared) == form


def test_an_empty_page_table_needs_no_address(lib):
    assert lib.mla_attn_paged(*dict(PAGED, table=None, max_pages=0, ctx=None).values()) == ARG
    assert b"ctx is NULL" in lib.moe_last_error_string()     # the check after the table's
    assert lib.mla_attn_paged(*dict(PAGED, table=None, max_pages=1, ctx=None).values()) == ARG
    assert b"table is NULL" in lib.moe_last_error_string()


def test_nothing_to_do(lib):
    assert lib.mla_rope_append(*dict(ROPE, T=0, q=None, positions=None).values()) == _lib.MOE_OK
    assert lib.mla_attn_paged(*dict(PAGED, B=0, Tq=0, q=None, ctx=None).values()) == _lib.MOE_OK
    assert lib.mla_attn_ragged(*dict(RAGGED, Tq=0, q=None).values()) == _lib.MOE_OK
    assert lib.mla_head_proj(*dict(PROJ, T=0, x=None).values()) == _lib.MOE_OK
    assert lib.moe_last_launch_count() == 0
    assert lib.mla_paged_workspace_bytes() > 0


def test_binding_wants_cuda_tensors():
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.mla_head_proj(x, torch.zeros(4, 8, 128, dtype=torch.bfloat16))


class On:
    """A CPU tensor that says it lies on a CUDA device."""

    def __init__(self, device, t):
        self.t, self.index = t, device

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("dev", [0, 1])
def test_binding_calls_on_the_device_of_the_tensors(monkeypatch, dev):
    # current device 0: a fake library notes the device that is current when it is called
    current, seen = [0], []

    @contextlib.contextmanager
    def device(i):
        before, current[0] = current[0], i
        yield
        current[0] = before

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, current[0], a[-1])) or _lib.MOE_OK

    monkeypatch.setattr(mla, "load", Lib)
    monkeypatch.setattr(mla, "_raw_stream", lambda i: 100 + i)
    monkeypatch.setattr(mla, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)

    def z(*shape, dtype=torch.bfloat16):
        return On(dev, torch.zeros(*shape, dtype=dtype))

    i32 = torch.int32
    plan = types.SimpleNamespace(freq=z(32, dtype=torch.int64), dim=64, layout=0, amplitude=1.0)
    moe.mla_rope_append(z(4, 8, 64), z(4, 576), z(4, dtype=i32), plan, q_out=z(4, 8, 64), kv_out=z(4, 576))
    moe.mla_attn_paged(z(2, 8, 576), z(3, 8, 576), z(2, 1, dtype=i32), z(2, dtype=i32), 1.0, out=z(2, 8, 512),
                       ws=z(64, dtype=torch.uint8))
    moe.mla_attn_ragged(z(4, 8, 192), z(4, 8, 128), z(4, 64), z(4, 8, 128), z(2, dtype=i32), z(2, dtype=i32), 4, 1.0,
                        out=z(4, 8, 128))
    moe.mla_head_proj(z(4, 8, 128), z(8, 16, 128), out=z(4, 8, 16))
    names = ("mla_rope_append", "mla_attn_paged", "mla_attn_ragged", "mla_head_proj")
    assert seen == [(n, dev, 100 + dev) for n in names] and current == [0]
    monkeypatch.setattr(_lib, "load", Lib)
    monkeypatch.setattr(_lib, "_stream", lambda i: 100 + i)
    moe.check_device_error(dev)                              # the error word of that device
    assert seen[-1][:2] == ("moe_check_device_error", dev) and current == [0]


def test_paged_exchanges_of_a_single_tile_are_separated_by_barriers():
    # Two warps of a tile exchange values through shared arrays: each writes its [half] and
    # reads the other's. In a segment of one key tile (nothing behind `if (j > 0)` runs) the
    # next write of an array has to stand behind a barrier that follows its last read.
    with open(os.path.join(build.CSRC, "mla_paged.cu")) as f:
        src = f.read()
    body = src[src.index("softmax and results"):src.index("the segment's result")]
    out = src[src.index("the segment's result"):src.index("Joins the partial results")]
    first = re.search(r"if \(j > 0\) \{", body)
    depth, end = 1, first.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(body[end], 0)
        end += 1
    text = body[:first.start()] + body[end:] + out
    pending, writes = set(), 0                               # arrays read since the last barrier
    for m in re.finditer(r"(named_bar_(?:sync|or)\()|sh\.(\w+)\[half\]\[\w+\] = |sh\.(\w+)\[(?:half \^ 1|0|1)\]\[", text):
        if m[1]:
            pending.clear()
        elif m[2]:
            writes += 1
            assert m[2] not in pending, f"{m[2]} is written before its last values are read everywhere"
        else:
            pending.add(m[3])
    assert writes == 4                                       # both rows' maxima, both rows' sums
