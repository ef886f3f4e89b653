"""The latent-attention operators against plain 64-bit forms, at the sizes and masks
where they can go wrong."""
import ctypes
import math

import pytest
import torch

import routed_fp8_expert_gb300 as moe
from _mla_ref import attention, check, rope_frequencies, rotate, rounding
from routed_fp8_expert_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 192 ** -0.5
BF16, FP16 = torch.bfloat16, torch.float16


def randn(*shape, seed=0, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def error_word():
    detail = ctypes.c_uint32(0)
    st = moe.load().moe_check_device_error(ctypes.c_void_p(torch.cuda.current_stream(DEV).cuda_stream),
                                           ctypes.byref(detail))
    return st, detail.value


def added_up(n, mag):
    """What n products added in tensor memory may lose, by _mla_ref's model: 16 at a time, truncating
    fp32 adds. mag: the sum of their magnitudes. (_mla_ref.attention's 2^-18 holds it up to 384 keys.)"""
    return (n / 16 + 8) * 2.0 ** -23 * mag


# ------------------------------------------------------------------ projections

@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("T,H,K,N,shared", [
    (1, 1, 8, 8, False), (1, 64, 128, 512, False), (5, 3, 72, 40, False), (129, 5, 512, 128, False),
    (300, 4, 512, 256, True), (64, 2, 136, 264, True), (257, 7, 128, 512, False),
])
def test_head_proj(T, H, K, N, shared, w_kn, dtype):
    x = randn(T, 1 if shared else H, K, seed=T, dtype=dtype)
    w = randn(*((H, K, N) if w_kn else (H, N, K)), seed=K, dtype=dtype, std=K ** -0.5)
    y = moe.mla_head_proj(x.to(DEV), w.to(DEV), w_kn=w_kn)
    assert error_word() == (_lib.MOE_OK, 0)
    xd, wd = x.double().expand(T, H, K), w.double() if w_kn else w.double().transpose(1, 2)
    ref = torch.einsum("thk,hkn->thn", xd, wd)
    mag = torch.einsum("thk,hkn->thn", xd.abs(), wd.abs())
    check(y, ref, rounding(dtype, ref) + (K / 16 + 8) * 2.0 ** -23 * mag, "out")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("T,H,K,N,shared", [
    (1025, 3, 512, 256, False), (1100, 2, 128, 512, False), (2000, 5, 640, 240, False), (1153, 4, 512, 128, True),
    (1281, 3, 72, 128, True), (3001, 1, 8, 136, False),
])
def test_head_proj_of_long_inputs(T, H, K, N, shared, w_kn, dtype):
    # pairs of CTAs (an even number of weight blocks that read the same x), or the
    # 128-token tiles where the number is odd
    x = randn(T, 1 if shared else H, K, seed=T, dtype=dtype)
    w = randn(*((H, K, N) if w_kn else (H, N, K)), seed=K, dtype=dtype, std=K ** -0.5)
    buf = torch.full((T + 1, H, N + 8), 3.0, dtype=dtype, device=DEV)
    y = moe.mla_head_proj(x.to(DEV), w.to(DEV), w_kn=w_kn, out=buf[:T, :, :N])
    assert error_word() == (_lib.MOE_OK, 0)
    xd, wd = x.double().expand(T, H, K), w.double() if w_kn else w.double().transpose(1, 2)
    ref = torch.einsum("thk,hkn->thn", xd, wd)
    mag = torch.einsum("thk,hkn->thn", xd.abs(), wd.abs())
    check(y, ref, rounding(dtype, ref) + (K / 16 + 8) * 2.0 ** -23 * mag, "out")
    assert (buf[T] == 3.0).all() and (buf[:, :, N:] == 3.0).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("T,H,K,N,shared", [
    (1281, 2, 1024, 1024, False),                            # weights through the ring; one row in the last tile
    (3001, 2, 776, 1000, False),                             # partial chunks, token tiles and weight blocks
    (2049, 10, 512, 264, True),                              # three weight blocks a head: pairs span two heads
    (1500, 24, 512, 256, True), (1100, 24, 640, 136, True),
])
def test_head_proj_of_cta_pairs(T, H, K, N, shared, w_kn, dtype):
    assert moe.load().mla_head_proj_form(T, H, K, N, int(shared)) == 1
    x = randn(T, 1 if shared else H, K + 8, seed=T, dtype=dtype)[..., :K]
    w = randn(*((H, K, N) if w_kn else (H, N, K)), seed=K, dtype=dtype, std=K ** -0.5)
    buf = torch.full((T + 1, H, N + 8), 3.0, dtype=dtype, device=DEV)
    y = moe.mla_head_proj(x.to(DEV), w.to(DEV), w_kn=w_kn, out=buf[:T, :, :N])
    assert error_word() == (_lib.MOE_OK, 0)
    xd, wd = x.double().expand(T, H, K).transpose(0, 1), w.double() if w_kn else w.double().transpose(1, 2)
    ref = torch.bmm(xd, wd).transpose(0, 1)
    mag = torch.bmm(xd.abs(), wd.abs()).transpose(0, 1)
    check(y, ref, rounding(dtype, ref) + (K / 16 + 8) * 2.0 ** -23 * mag, "out")
    assert (buf[T] == 3.0).all() and (buf[:, :, N:] == 3.0).all()
    assert torch.equal(y, moe.mla_head_proj(x.to(DEV), w.to(DEV), w_kn=w_kn))


def test_head_proj_reads_views_in_place():
    # one up-projection weight [H, 256, 512] holds the key and the value halves of each
    # head; the absorb product reads the key half with K contiguous rows swapped
    H, T = 6, 19
    w = randn(H, 256, 512, seed=1, std=0.05)
    q = randn(T, H, 192, seed=2)
    wd, qd = w.to(DEV), q.to(DEV)
    out = torch.full((T, H, 576), 7.0, dtype=BF16, device=DEV)
    moe.mla_head_proj(qd[..., :128], wd[:, :128], w_kn=True, out=out[..., :512])
    ref = torch.einsum("thk,hkn->thn", q[..., :128].double(), w[:, :128].double())
    mag = torch.einsum("thk,hkn->thn", q[..., :128].double().abs(), w[:, :128].double().abs())
    check(out[..., :512], ref, rounding(BF16, ref) + 16 * 2.0 ** -23 * mag, "absorbed")
    assert (out[..., 512:] == 7.0).all()                     # nothing written past the view
    o = randn(T, H, 512, seed=3)
    y = moe.mla_head_proj(o.to(DEV), wd[:, 128:])
    ref = torch.einsum("thk,hnk->thn", o.double(), w[:, 128:].double())
    mag = torch.einsum("thk,hnk->thn", o.double().abs(), w[:, 128:].double().abs())
    check(y, ref, rounding(BF16, ref) + 40 * 2.0 ** -23 * mag, "value")


# ------------------------------------------------------------------------ rope

@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,H,dim,latent,page,factor", [
    (1, 1, 64, 512, 64, 1.0), (37, 64, 64, 512, 16, 32.0), (5, 3, 128, 256, 8, 4.0), (9, 20, 16, 8, 1, 1.0),
    (3, 2, 256, 1792, 24, 40.0),
])
def test_rope_append(T, H, dim, latent, page, factor, layout, dtype):
    g = torch.Generator().manual_seed(T)
    plan = moe.rope_plan(dim, 50000.0, factor, mscale=1.0, mscale_all_dim=0.7, layout=layout, device=DEV)
    amp = (1 + 0.1 * math.log(factor)) / (1 + 0.07 * math.log(factor))
    assert abs(plan.amplitude - amp) < 1e-12
    q = randn(T, H, 40 + dim, seed=T, dtype=dtype)           # the rotary part of wider heads
    kv = randn(T, latent + dim, seed=T + 1, dtype=dtype, std=2.0)
    gamma = (1 + 0.1 * torch.randn(latent, generator=g)).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 0
    pages = (T + page - 1) // page + 2
    cache = randn(pages, page, latent + dim, seed=5, dtype=dtype)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 2:
        slots[1] = -1                                        # a padding token
    cd = cache.to(DEV)
    q_out, kv_out = moe.mla_rope_append(q.to(DEV)[..., 40:], kv.to(DEV), pos.to(DEV), plan, gamma=gamma.to(DEV),
                                        cache=cd, slots=slots.to(DEV),
                                        kv_out=torch.empty(T, latent + dim, dtype=dtype, device=DEV))
    assert error_word() == (_lib.MOE_OK, 0)
    freq = rope_frequencies(dim, 50000.0, factor)
    ref, mag = rotate(q[..., 40:], pos, freq, layout, amp)
    check(q_out, ref, rounding(dtype, ref) + 2.0 ** -20 * mag, "q")
    c = kv[:, :latent].double()
    c = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6) * gamma.double()
    kr, kmag = rotate(kv[:, latent:], pos, freq, layout, amp)
    row = torch.cat((c, kr), 1)
    bound = rounding(dtype, row) + 2.0 ** -18 * torch.cat((c.abs(), kmag), 1)
    check(kv_out, row, bound, "kv_out")
    want = cache.clone()                                     # the cache holds kv_out's bits, and nothing else changed
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // page, s % page] = kv_out[t].cpu()
    assert torch.equal(cd.cpu(), want)


def test_rope_in_place_and_alone():
    T, H = 7, 4
    plan = moe.rope_plan(64, device=DEV)
    q, pos = randn(T, H, 192, seed=1).to(DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    want, _ = moe.mla_rope_append(q[..., 128:], None, pos, plan)
    before = q.clone()
    moe.mla_rope_append(q[..., 128:], None, pos, plan, q_out=q[..., 128:])
    assert torch.equal(q[..., 128:], want) and torch.equal(q[..., :128], before[..., :128])
    kv = randn(T, 576, seed=2).to(DEV)
    _, out = moe.mla_rope_append(None, kv, pos, plan)        # no gamma: the latent is copied
    assert torch.equal(out[:, :512], kv[:, :512])
    none, _ = moe.mla_rope_append(q[:0, :, 128:], None, pos[:0], plan)
    assert none.shape == (0, H, 64)


def test_rope_bad_slot_is_skipped_and_reported():
    plan = moe.rope_plan(64, device=DEV)
    kv, cache = randn(3, 576, seed=1).to(DEV), torch.zeros(2, 8, 576, dtype=BF16, device=DEV)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    slots = torch.tensor([3, 16, -5], dtype=torch.int32, device=DEV)
    moe.mla_rope_append(None, kv, pos, plan, cache=cache, slots=slots)
    assert error_word() == (_lib.MOE_ERR_INDEX, 0x80)
    assert error_word() == (_lib.MOE_OK, 0)
    flat = cache.view(16, 576)
    assert (flat[3] != 0).any() and flat.abs().sum() == flat[3].abs().sum()


def test_rope_with_a_cache_of_no_pages():
    # no slot lies in it: tokens that are not cached are fine, any other is reported
    plan = moe.rope_plan(64, device=DEV)
    kv, cache = randn(3, 576, seed=1).to(DEV), torch.zeros(0, 8, 576, dtype=BF16, device=DEV)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    _, want = moe.mla_rope_append(None, kv, pos, plan)
    before = kv.clone()
    for slots, word in (([-1, -1, -1], (_lib.MOE_OK, 0)), ([-1, 0, -1], (_lib.MOE_ERR_INDEX, 0x80))):
        slots = torch.tensor(slots, dtype=torch.int32, device=DEV)
        _, rows = moe.mla_rope_append(None, kv, pos, plan, cache=cache, slots=slots, kv_out=torch.empty_like(kv))
        assert error_word() == word
        assert torch.equal(rows, want) and torch.equal(kv, before)
        moe.mla_rope_append(None, kv, pos, plan, cache=cache, slots=slots)
        assert error_word() == word and torch.equal(kv, before)


def test_rope_of_a_strided_multi_layer_cache():
    layers, page = 3, 16
    plan = moe.rope_plan(64, device=DEV)
    big = torch.zeros(4, layers, page, 576, dtype=BF16, device=DEV)
    kv, pos = randn(20, 576, seed=4).to(DEV), torch.arange(20, dtype=torch.int32, device=DEV)
    _, rows = moe.mla_rope_append(None, kv, pos, plan)
    moe.mla_rope_append(None, kv, pos, plan, cache=big[:, 1], slots=pos + 7)
    flat = big[:, 1].reshape(-1, 576)
    assert torch.equal(flat[7:27], rows)
    assert (big[:, 0] == 0).all() and (big[:, 2] == 0).all() and (flat[:7] == 0).all() and (flat[27:] == 0).all()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("H,latent", [(1, 512), (16, 512), (32, 1024), (5, 1032), (0, 512)])
def test_rope_long_calls_equal_short_ones(H, latent, layout):
    # many tokens of few heads are launched in another shape: the same bits token by token
    T = 3001
    plan = moe.rope_plan(64, 50000.0, 32.0, layout=layout, device=DEV)
    q, kv = randn(T, H, 64, seed=1).to(DEV) if H else None, randn(T, latent + 64, seed=2).to(DEV)
    gamma = randn(latent, seed=3).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 41
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    cache = torch.zeros(2, 47, 64, latent + 64, dtype=BF16, device=DEV)
    rows = torch.zeros(2, T, latent + 64, dtype=BF16, device=DEV)
    whole, _ = moe.mla_rope_append(q, kv, pos, plan, gamma=gamma, cache=cache[0], slots=slots, kv_out=rows[0])
    for i in range(0, T, 500):
        c = slice(i, min(T, i + 500))
        part, _ = moe.mla_rope_append(q[c] if H else None, kv[c], pos[c], plan, gamma=gamma, cache=cache[1],
                                      slots=slots[c], kv_out=rows[1, c])
        assert not H or torch.equal(whole[c], part)
    assert torch.equal(cache[0], cache[1]) and torch.equal(rows[0], rows[1]) and (rows[0] != 0).any(1).all()
    assert error_word() == (_lib.MOE_OK, 0)


# ----------------------------------------------------------------------- paged

def paged_inputs(ctx, n, H, page, seed=0, dtype=BF16, std=1.0, junk=None, extra_cols=3):
    """A cache whose pages are shuffled; page rows past a sequence's end (and unused
    pages) hold `junk`."""
    g = torch.Generator().manual_seed(seed)
    need = [(c + page - 1) // page for c in ctx]
    total = sum(need) + 2
    perm = torch.randperm(total, generator=g)
    cache = randn(total, page, 576, seed=seed, dtype=dtype, std=std)
    table = torch.full((len(ctx), max(need + [1]) + extra_cols), 2 ** 30, dtype=torch.int32)   # unused entries: not a page
    at, used = 0, torch.zeros(total, page, dtype=torch.bool)
    for b, (c, k) in enumerate(zip(ctx, need)):
        pages = perm[at:at + k]
        table[b, :k] = pages.to(torch.int32)
        at += k
        for i in range(k):
            used[pages[i], :min(page, c - i * page)] = True
    if junk is not None:
        cache[~used] = junk
    q = randn(sum(n), H, 576, seed=seed + 1, dtype=dtype)
    return q, cache, table, torch.tensor(ctx, dtype=torch.int32)


def paged_ref(q, cache, table, ctx, n, dtype, scale=SCALE):
    outs, at = [], 0
    page, H = cache.shape[1], q.shape[1]
    for b, c in enumerate(ctx.tolist()):
        keys = torch.cat([cache[p] for p in table[b, :(c + page - 1) // page].tolist()] + [cache[:0, 0]])[:c]
        rows = q[at:at + n[b]].reshape(-1, 576)
        vis = [max(0, c - n[b] + i + 1) for i in range(n[b]) for _ in range(H)]
        outs.append(attention(rows, keys, keys[:, :512], vis, scale, dtype))
        at += n[b]
    o, lse, ob, lb = (torch.cat(x) for x in zip(*outs))
    return o.view(at, H, 512), lse.view(at, H), ob.view(at, H, 512), lb.view(at, H)


def run_paged(q, cache, table, ctx, n, **kw):
    cu = None
    if any(x != 1 for x in n):
        cu = torch.tensor([0] + n, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)
    return moe.mla_attn_paged(q.to(DEV), cache.to(DEV), table.to(DEV), ctx.to(DEV), SCALE, cu_q=cu, want_lse=True, **kw)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("ctx,n,H,page", [
    ([1], [1], 64, 64), ([64], [1], 64, 64), ([65], [1], 16, 64), ([0], [1], 64, 64),
    ([130, 0, 1, 63, 1000], [1] * 5, 64, 64), ([257, 700], [1, 1], 128, 32), ([5, 77, 300], [1] * 3, 1, 8),
    ([333, 90], [1, 1], 20, 24), ([40, 129, 128], [4, 4, 1], 16, 16), ([3, 200], [5, 70], 20, 128),
    ([100, 10], [100, 10], 7, 64), ([1500], [3], 64, 192), ([50, 60], [0, 2], 64, 64),
])
def test_paged(ctx, n, H, page, dtype):
    q, cache, table, ctx_t = paged_inputs(ctx, n, H, page, seed=sum(ctx) + H, dtype=dtype, junk=math.nan)
    o, lse = run_paged(q, cache, table, ctx_t, n)
    assert error_word() == (_lib.MOE_OK, 0)
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, n, dtype)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")


@pytest.mark.parametrize("junk", [math.inf, -math.inf, torch.finfo(BF16).max])
def test_paged_stale_rows_do_not_count(junk):
    ctx, n = [70, 1, 128, 190], [1] * 4
    q, cache, table, ctx_t = paged_inputs(ctx, n, 64, 64, seed=3, junk=junk)
    o, lse = run_paged(q, cache, table, ctx_t, n)
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, n, BF16)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")


def test_paged_rising_scores_move_the_reference_maximum():
    # scores that grow along the keys: the running maximum rises by far more than the
    # lag in every tile; then scores of the lowest magnitude
    L = 900
    q, cache, table, ctx_t = paged_inputs([L], [1], 64, 64, seed=8)
    page = 64
    for i, p in enumerate(table[0, :(L + 63) // 64].tolist()):
        cache[p] = cache[p] * 0.1
        cache[p, :, 0] = (torch.arange(page) + i * page).to(BF16)
    q[..., 0] = 4.0
    o, lse = run_paged(q, cache, table, ctx_t, [1])
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, [1], BF16)
    check(o, ro, ob, "rising out")
    check(lse, rl, lb, "rising lse")
    q[..., 0] = -4.0
    o, lse = run_paged(q, cache, table, ctx_t, [1])
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, [1], BF16)
    check(o, ro, ob, "falling out")
    check(lse, rl, lb, "falling lse")


@pytest.mark.parametrize("gap", [1.2, 16.0, 17.0, 17.5])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_paged_lse_of_many_small_weights(dtype, gap):
    # 131,072 keys at weights near e^-gap of the first one's, in one running sum: as many
    # sequences as processors, so that no item is split
    n, page, B = 131072, 64, torch.cuda.get_device_properties(0).multi_processor_count
    cache = randn(n // page, page, 576, seed=1, dtype=dtype, std=0.1)
    q = torch.zeros(1, 2, 576, dtype=dtype)
    q[..., 513:] = randn(1, 2, 63, seed=2, dtype=dtype, std=0.1)
    q[..., 512], cache[..., 512] = 16.0, 0.0
    cache[0, 0, 512] = gap / (16 * SCALE)
    table, ctx = torch.arange(n // page, dtype=torch.int32), torch.full((B,), n, dtype=torch.int32)
    _, lse = run_paged(q.expand(B, 2, 576).contiguous(), cache, table.expand(B, n // page).contiguous(), ctx, [1] * B)
    assert error_word() == (_lib.MOE_OK, 0)
    _, rl, _, lb = paged_ref(q, cache, table[None], ctx[:1], [1], dtype)
    check(lse, rl.expand(B, 2), lb.expand(B, 2), "lse")


@pytest.mark.parametrize("gap", [17.0, 17.5, 20.0])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_paged_one_key_far_above_many(dtype, gap):
    # 131,072 keys of weights near e^-gap of the first one's: each is next to nothing, together
    # they are not (e^-17.33 is 2^-25, where a weight below one vanishes in fp16). As many
    # sequences as processors, so that no item is split.
    n, page, B = 131072, 64, torch.cuda.get_device_properties(0).multi_processor_count
    cache = randn(n // page, page, 576, seed=1, dtype=dtype, std=0.1)
    cache[..., :512] += 1.0
    cache[0, 0, :512] = -0.05
    q = torch.zeros(1, 2, 576, dtype=dtype)
    q[..., 513:] = randn(1, 2, 63, seed=2, dtype=dtype)
    q[..., 512], cache[..., 512] = 16.0, 0.0
    cache[0, 0, 512] = gap / (16 * SCALE)
    table, ctx = torch.arange(n // page, dtype=torch.int32), torch.full((B,), n, dtype=torch.int32)
    o, lse = run_paged(q.expand(B, 2, 576).contiguous(), cache, table.expand(B, n // page).contiguous(), ctx, [1] * B)
    assert error_word() == (_lib.MOE_OK, 0)
    ro, rl, ob, lb = paged_ref(q, cache, table[None], ctx[:1], [1], dtype)
    keys = cache.view(n, 576)
    ob = ob + added_up(n, attention(q[0], keys, keys[:, :512].abs(), [n, n], SCALE, dtype)[0])
    check(o, ro.expand(B, 2, 512), ob.expand(B, 2, 512), "out")
    check(lse, rl.expand(B, 2), lb.expand(B, 2), "lse")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("L", [900, 30000])
def test_paged_rising_scores_in_both_types(L, dtype):
    # the reference maximum moves in every tile, up to weights near the largest that fit the
    # type; the long one is split and joined
    q, cache, table, ctx_t = paged_inputs([L], [1], 64, 64, seed=8, dtype=dtype)
    for step in (0.02, 0.6, 4.0):
        for i, p in enumerate(table[0, :(L + 63) // 64].tolist()):
            cache[p] = cache[p].clamp(-1, 1)
            cache[p, :, 0] = ((torch.arange(64) + i * 64) * (900 / L)).to(dtype)
        q[..., 0] = step
        o, lse = run_paged(q, cache, table, ctx_t, [1])
        ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, [1], dtype)
        check(o, ro, ob, "out")
        check(lse, rl, lb, "lse")


def test_paged_long_context_is_split_and_joined():
    ctx, n = [20000, 3, 9000], [1, 1, 2]
    q, cache, table, ctx_t = paged_inputs(ctx, n, 16, 64, seed=9)
    o, lse = run_paged(q, cache, table, ctx_t, n)
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, n, BF16)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")
    o2, lse2 = run_paged(q, cache, table, ctx_t, n)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)     # the same bits again


@pytest.mark.parametrize("H", [16, 40, 64, 100])
@pytest.mark.parametrize("ctx", [
    [64] * 7, [65 + 9 * i for i in range(7)], [1 + 11 * i for i in range(20)], [190, 191, 192], [100] * 5 + [700],
    [3] * 160 + [130], [40] * 90, [0] * 3 + [70, 0, 200],
])
def test_paged_short_batches(ctx, H):
    # one key tile each, two each, mixed, more sequences than processors: every way of cutting
    n = [1] * len(ctx)
    q, cache, table, ctx_t = paged_inputs(ctx, n, H, 32, seed=len(ctx) + H, junk=math.nan)
    o, lse = run_paged(q, cache, table, ctx_t, n)
    assert error_word() == (_lib.MOE_OK, 0)
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, n, BF16)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")


@pytest.mark.parametrize("ctx,H", [([64] * 150, 64), ([9 + i % 50 for i in range(151)], 33), ([64 * 151], 64), ([64 * 37 - 5] * 4, 64)])
def test_paged_single_tile_segments_repeat(ctx, H):
    # every CTA has one key tile: the exchange of the two halves' maxima, then at once of their sums
    n = [1] * len(ctx)
    q, cache, table, ctx_t = paged_inputs(ctx, n, H, 64, seed=len(ctx) + H, junk=math.nan)
    args = [x.to(DEV) for x in (q, cache, table, ctx_t)]
    ws = moe.mla_paged_workspace(DEV)
    o, lse = moe.mla_attn_paged(*args, SCALE, want_lse=True, ws=ws)
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, n, BF16)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")
    again = [moe.mla_attn_paged(*args, SCALE, want_lse=True, ws=ws) for _ in range(200)]
    assert all(torch.equal(o, x) and torch.equal(lse, y) for x, y in again)
    assert error_word() == (_lib.MOE_OK, 0)


@pytest.mark.parametrize("H,n,ctx,joins", [
    (128, 1, [129], [[0, 2], [3, 5]]),                       # two items of three tiles: one tile a CTA
    (128, 1, [256], [[0, 1], [2, 3]]),                       # of four: two
    (64, 1, [129, 60], [[0, 2]]), (64, 1, [128, 256], [[1, 2]]), (16, 4, [65], []), (64, 2, [130], [[0, 2], [3, 5]]),
])
def test_paged_cuts_items_of_odd_tiles_singly(H, n, ctx, joins):
    # the list of shared items that the first kernel leaves to the join: (first, last) CTA of each
    q, cache, table, ctx_t = paged_inputs(ctx, [n] * len(ctx), H, 64, seed=H)
    ws = moe.mla_paged_workspace(DEV)
    o, lse = run_paged(q, cache, table, ctx_t, [n] * len(ctx), ws=ws)
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, [n] * len(ctx), BF16)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    entries = ws[-16 * ctas:].view(torch.int32).view(ctas, 4).tolist()
    assert [[c, e[3]] for c, e in enumerate(entries) if e[2] > 0] == joins


def test_paged_views_and_strides():
    ctx, n, H = [150, 90], [1, 1], 8
    q, cache, table, ctx_t = paged_inputs(ctx, n, H, 32, seed=11)
    base, lse0 = run_paged(q, cache, table, ctx_t, n)
    wide_q = torch.zeros(2, H, 640, dtype=BF16)
    wide_q[..., 32:608] = q
    big = torch.full((cache.shape[0], 2, 32, 584), math.nan, dtype=BF16)
    big[:, 1, :, :576] = cache
    out = torch.full((H, 2, 520), 5.0, dtype=BF16, device=DEV)
    got, lse = moe.mla_attn_paged(wide_q.to(DEV)[..., 32:608], big.to(DEV)[:, 1, :, :576], table.to(DEV), ctx_t.to(DEV),
                                  SCALE, out=out.transpose(0, 1)[..., :512], want_lse=True)
    assert torch.equal(got, base) and torch.equal(lse, lse0) and (out[..., 512:] == 5.0).all()


def check_paged_sample(q, cache, table, ctx, n, o, lse, rows, dtype=BF16):
    """The given (sequence, query) rows of a call against their 64-bit form: q [Tq, H, 576]."""
    page, start = cache.shape[1], [0]
    for x in n:
        start.append(start[-1] + x)
    for b, i in rows:
        c = int(ctx[b])
        keys = torch.cat([cache[p] for p in table[b, :(c + page - 1) // page].tolist()])[:c]
        t, H = start[b] + i, q.shape[1]
        ro, rl, ob, lb = attention(q[t], keys, keys[:, :512], [max(0, c - n[b] + i + 1)] * H, SCALE, dtype)
        check(o[t], ro, ob, f"out of query {i} of sequence {b}")
        check(lse[t], rl, lb, f"lse of query {i} of sequence {b}")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("H,ctx,n", [
    (64, [700, 6001, 300, 9000, 33, 4100], [300, 1, 257, 1, 1, 4]),      # prompts' chunks beside single tokens
    (16, [513, 20000, 2000, 1, 77], [513, 1, 70, 1, 5]),
    (128, [9000, 513, 64], [1, 200, 1]), (100, [3000, 800], [2, 333]),
])
def test_paged_chunks_beside_single_tokens(H, ctx, n, dtype):
    q, cache, table, ctx_t = paged_inputs(ctx, n, H, 64, seed=sum(n) + H, dtype=dtype, junk=math.nan)
    o, lse = run_paged(q, cache, table, ctx_t, n)
    assert error_word() == (_lib.MOE_OK, 0)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    rows = sorted({(b, i) for b, x in enumerate(n) for i in (0, 1, x // 2, x - 2, x - 1) if 0 <= i < x})
    check_paged_sample(q, cache, table, ctx_t, n, o, lse, rows, dtype)
    o2, lse2 = run_paged(q, cache, table, ctx_t, n)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)     # the same bits again


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("H,n,ctx", [
    (128, 1, [12000, 700, 9001, 64, 3000]), (128, 1, [4000 + 61 * i for i in range(40)]), (96, 3, [8000, 5000, 7001]),
    (64, 4, [6000 + 77 * i for i in range(12)]), (128, 2, [20000]),
])
def test_paged_many_row_tiles_over_long_contexts(H, n, ctx, dtype):
    q, cache, table, ctx_t = paged_inputs(ctx, [n] * len(ctx), H, 32, seed=len(ctx) + H, dtype=dtype, junk=math.inf)
    o, lse = run_paged(q, cache, table, ctx_t, [n] * len(ctx))
    assert error_word() == (_lib.MOE_OK, 0)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    check_paged_sample(q, cache, table, ctx_t, [n] * len(ctx), o, lse,
                       sorted({(b, i) for b in (0, len(ctx) // 2, len(ctx) - 1) for i in (0, n - 1)}), dtype)


def test_offsets_past_32_bits():
    # pages whose element offsets pass 2^32: appended to, then read
    page, pages = 64, 120_000
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 9 GB for the cache")
    cache = torch.empty(pages, page, 576, dtype=BF16, device=DEV)
    assert cache.numel() > 2 ** 32
    n, last = 200, pages - 1
    kv, pos = randn(n, 576, seed=1).to(DEV), torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.tensor([[last, 0, last - 7, last - 1]], dtype=torch.int32)
    slots = torch.cat([torch.arange(p * page, (p + 1) * page) for p in table[0].tolist()])[:n].to(torch.int32)
    plan = moe.rope_plan(64, device=DEV)
    _, rows = moe.mla_rope_append(None, kv, pos, plan, cache=cache, slots=slots.to(DEV),
                                  kv_out=torch.empty(n, 576, dtype=BF16, device=DEV))
    q = randn(1, 64, 576, seed=2)
    o, lse = moe.mla_attn_paged(q.to(DEV), cache, table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV), SCALE,
                                want_lse=True)
    assert error_word() == (_lib.MOE_OK, 0)
    keys = rows.cpu()
    ro, rl, ob, lb = attention(q[0], keys, keys[:, :512], [n] * 64, SCALE, BF16)
    check(o[0], ro, ob, "out")
    check(lse[0], rl, lb, "lse")


def test_paged_many_sequences():
    # more sequences than the start-up scan takes at once
    ctx = [(37 * i) % 150 for i in range(500)]
    n = [1] * 500
    q, cache, table, ctx_t = paged_inputs(ctx, n, 4, 16, seed=2)
    o, lse = run_paged(q, cache, table, ctx_t, n)
    ro, rl, ob, lb = paged_ref(q, cache, table, ctx_t, n, BF16)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")


def test_paged_bad_indices_are_reported_and_skipped():
    q, cache, table, ctx_t = paged_inputs([100, 100], [1, 1], 64, 64, seed=5)
    good, _ = run_paged(q, cache, table, ctx_t, [1, 1])
    bad = table.clone()
    bad[1, 1] = cache.shape[0]                               # a page past the cache
    o, _ = run_paged(q, cache, bad, ctx_t, [1, 1])
    assert error_word() == (_lib.MOE_ERR_INDEX, 0x80)
    assert torch.equal(o[0], good[0])
    long = ctx_t.clone()
    long[1] = table.shape[1] * 64 + 1                        # more tokens than its table holds
    out = torch.full_like(good, 3.0)
    moe.mla_attn_paged(q.to(DEV), cache.to(DEV), table.to(DEV), long.to(DEV), SCALE, out=out)
    assert error_word() == (_lib.MOE_ERR_INDEX, 0x80)
    assert torch.equal(out[0], good[0]) and (out[1] == 3.0).all()
    cu = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)   # past the two rows of q
    out = torch.full_like(good, 3.0)
    moe.mla_attn_paged(q.to(DEV), cache.to(DEV), table.to(DEV), ctx_t.to(DEV), SCALE, cu_q=cu, out=out)
    assert error_word() == (_lib.MOE_ERR_INDEX, 0x80)
    assert torch.equal(out[0], good[0]) and (out[1] == 3.0).all()
    assert error_word() == (_lib.MOE_OK, 0)


def test_paged_without_any_page():
    q, cache = randn(3, 5, 576, seed=1).to(DEV), randn(2, 16, 576, seed=2).to(DEV)
    table, ctx = torch.zeros(3, 0, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    out = torch.full((3, 5, 512), 4.0, dtype=BF16, device=DEV)
    o, lse = moe.mla_attn_paged(q, cache, table, ctx, SCALE, out=out, want_lse=True)
    assert error_word() == (_lib.MOE_OK, 0) and (o == 0).all() and (lse == -math.inf).all()
    ctx[1] = 1                                               # a key, but no page
    moe.mla_attn_paged(q, cache, table, ctx, SCALE)
    assert error_word() == (_lib.MOE_ERR_INDEX, 0x80)


@pytest.mark.parametrize("entry", [9, 0])
@pytest.mark.parametrize("page", [-(2 ** 31), -1, 2 ** 31 - 1])
def test_paged_extreme_page_entries_are_reported(entry, page):
    q, cache, table, ctx_t = paged_inputs([100, 100], [1, 1], 64, 8, seed=5)
    good, _ = run_paged(q, cache, table, ctx_t, [1, 1])
    table[1, entry] = page
    o, _ = run_paged(q, cache, table, ctx_t, [1, 1])
    assert error_word() == (_lib.MOE_ERR_INDEX, 0x80)
    assert torch.equal(o[0], good[0])


def test_paged_in_a_graph_follows_new_lengths():
    ctx, n = [90, 700], [1, 1]
    q, cache, table, ctx_t = paged_inputs([200, 800], n, 64, 64, seed=6)
    qd, cd, td, ld = q.to(DEV), cache.to(DEV), table.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV)
    ws, out = moe.mla_paged_workspace(DEV), torch.empty(2, 64, 512, dtype=BF16, device=DEV)
    moe.mla_attn_paged(qd, cd, td, ld, SCALE, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.mla_attn_paged(qd, cd, td, ld, SCALE, out=out, ws=ws)
    for lens in ([90, 700], [200, 0], [1, 800]):
        ld.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, moe.mla_attn_paged(qd, cd, td, ld, SCALE, ws=ws))


# ---------------------------------------------------------------------- ragged

def ragged_ref(q, kn, kp, v, nq, nk, causal, dtype):
    outs, qa, ka = [], 0, 0
    H = q.shape[1]
    for n, c in zip(nq, nk):
        per = []
        for h in range(H):
            k = torch.cat((kn[ka:ka + c, h], kp[ka:ka + c]), 1)
            vis = [max(0, c - n + i + 1) if causal else c for i in range(n)]
            per.append(attention(q[qa:qa + n, h], k, v[ka:ka + c, h], vis, SCALE, dtype))
        outs.append([torch.stack(x, 1) for x in zip(*per)])
        qa, ka = qa + n, ka + c
    return [torch.cat(x) for x in zip(*outs)]


def offsets(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("nq,nk,H", [
    ([1], [1], 1), ([128], [128], 2), ([129], [129], 1), ([300], [300], 2), ([1, 0, 260, 17], [1, 5, 260, 400], 3),
    ([64, 3], [0, 2], 2), ([40], [700], 2), ([513], [200], 1), ([5, 5, 5], [130, 128, 127], 8),
])
def test_ragged(nq, nk, H, causal, dtype):
    s = sum(nq) + 7 * H
    q = randn(sum(nq), H, 192, seed=s, dtype=dtype)
    kv = randn(sum(nk) + 3, H, 256, seed=s + 1, dtype=dtype)
    kp = randn(sum(nk) + 3, 64, seed=s + 2, dtype=dtype)
    kv[sum(nk):], kp[sum(nk):] = math.nan, math.nan          # rows past every sequence
    kvd = kv.to(DEV)
    o, lse = moe.mla_attn_ragged(q.to(DEV), kvd[..., :128], kp.to(DEV), kvd[..., 128:], offsets(nq), offsets(nk),
                                 max(nq), SCALE, causal=causal, want_lse=True)
    assert error_word() == (_lib.MOE_OK, 0)
    ro, rl, ob, lb = ragged_ref(q, kv[..., :128], kp, kv[..., 128:], nq, nk, causal, dtype)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")


def test_ragged_neighbours_do_not_leak():
    # the sequence between two of NaN and infinity
    nq = nk = [70, 200, 90]
    H = 2
    q, kv, kp = randn(360, H, 192, seed=1), randn(360, H, 256, seed=2), randn(360, 64, seed=3)
    clean = [x.clone() for x in (q, kv, kp)]
    for x, bad in ((q, math.nan), (kv, math.inf), (kp, math.nan)):
        x[:70], x[270:] = bad, bad
    kvd = kv.to(DEV)
    o, lse = moe.mla_attn_ragged(q.to(DEV), kvd[..., :128], kp.to(DEV), kvd[..., 128:], offsets(nq), offsets(nk), 200,
                                 SCALE, want_lse=True)
    ro, rl, ob, lb = ragged_ref(clean[0], clean[1][..., :128], clean[2], clean[1][..., 128:], nq, nk, True, BF16)
    check(o[70:270], ro[70:270], ob[70:270], "out")
    check(lse[70:270], rl[70:270], lb[70:270], "lse")


def test_ragged_rising_scores_move_the_reference_maximum():
    n = 640
    q, kv, kp = randn(n, 1, 192, seed=1) * 0.1, randn(n, 1, 256, seed=2), randn(n, 64, seed=3) * 0.1
    kp[:, 0], q[..., 128] = torch.arange(n).to(BF16), 4.0
    for sign in (1, -1):
        kvd = kv.to(DEV)
        o, lse = moe.mla_attn_ragged((q * sign).to(DEV), kvd[..., :128], kp.to(DEV), kvd[..., 128:], offsets([n]),
                                     offsets([n]), n, SCALE, want_lse=True)
        ro, rl, ob, lb = ragged_ref(q * sign, kv[..., :128], kp, kv[..., 128:], [n], [n], True, BF16)
        check(o, ro, ob, "out")
        check(lse, rl, lb, "lse")


@pytest.mark.parametrize("gap", [1.2, 16.0, 17.0, 17.5])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_ragged_lse_of_many_small_weights(dtype, gap):
    n, nq = 131072, 3
    q, kv, kp = torch.zeros(nq, 1, 192, dtype=dtype), randn(n, 1, 256, seed=1, dtype=dtype, std=0.1), randn(n, 64, seed=2, dtype=dtype, std=0.1)
    q[..., 128:] = randn(nq, 1, 64, seed=3, dtype=dtype, std=0.1)
    q[..., 0], kv[..., 0], kv[0, :, 0] = 16.0, 0.0, gap / (16 * SCALE)
    kvd = kv.to(DEV)
    _, lse = moe.mla_attn_ragged(q.to(DEV), kvd[..., :128], kp.to(DEV), kvd[..., 128:], offsets([nq]), offsets([n]), nq,
                                 SCALE, causal=False, want_lse=True)
    assert error_word() == (_lib.MOE_OK, 0)
    _, rl, _, lb = ragged_ref(q, kv[..., :128], kp, kv[..., 128:], [nq], [n], False, dtype)
    check(lse, rl, lb, "lse")


@pytest.mark.parametrize("gap", [17.0, 17.5, 20.0])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_ragged_one_key_far_above_many(dtype, gap):
    # 131,072 keys of weights near e^-gap of the first one's: each is next to nothing, together
    # they are not (e^-17.33 is 2^-25, where a weight below one vanishes in fp16)
    n, nq = 131072, 3
    q, kv, kp = torch.zeros(nq, 1, 192, dtype=dtype), randn(n, 1, 256, seed=1, dtype=dtype, std=0.1), randn(n, 64, seed=2, dtype=dtype, std=0.1)
    kv[..., 128:] += 1.0
    kv[0, :, 128:] = -0.05
    q[..., 128:] = randn(nq, 1, 64, seed=3, dtype=dtype)
    q[..., 0], kv[..., 0], kv[0, :, 0] = 16.0, 0.0, gap / (16 * SCALE)
    kvd = kv.to(DEV)
    o, lse = moe.mla_attn_ragged(q.to(DEV), kvd[..., :128], kp.to(DEV), kvd[..., 128:], offsets([nq]), offsets([n]), nq,
                                 SCALE, causal=False, want_lse=True)
    assert error_word() == (_lib.MOE_OK, 0)
    ro, rl, ob, lb = ragged_ref(q, kv[..., :128], kp, kv[..., 128:], [nq], [n], False, dtype)
    ob = ob + added_up(n, ragged_ref(q, kv[..., :128], kp, kv[..., 128:].abs(), [nq], [n], False, dtype)[0])
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_ragged_rising_scores_in_both_types(dtype):
    # the reference maximum moves in every tile, up to weights near the largest that fit the type
    n = 640
    q, kv, kp = randn(n, 1, 192, seed=1, dtype=dtype) * 0.1, randn(n, 1, 256, seed=2, dtype=dtype), randn(n, 64, seed=3, dtype=dtype) * 0.1
    for step in (0.02, 0.6, 4.0):
        kp[:, 0], q[..., 128] = torch.arange(n).to(dtype), step
        kvd = kv.to(DEV)
        o, lse = moe.mla_attn_ragged(q.to(DEV), kvd[..., :128], kp.to(DEV), kvd[..., 128:], offsets([n]), offsets([n]), n,
                                     SCALE, want_lse=True)
        ro, rl, ob, lb = ragged_ref(q, kv[..., :128], kp, kv[..., 128:], [n], [n], True, dtype)
        check(o, ro, ob, "out")
        check(lse, rl, lb, "lse")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_ragged_long_uneven_sequences(dtype, causal):
    # long, short, after a prefix, queries that see nothing, more queries than keys
    nq, nk, H = [1900, 3, 700, 0, 513, 1], [1900, 2500, 1217, 300, 100, 4097], 2
    q = randn(sum(nq), H, 192, seed=1, dtype=dtype)
    kv, kp = randn(sum(nk), H, 256, seed=2, dtype=dtype), randn(sum(nk), 64, seed=3, dtype=dtype)
    kvd = kv.to(DEV)
    o, lse = moe.mla_attn_ragged(q.to(DEV), kvd[..., :128], kp.to(DEV), kvd[..., 128:], offsets(nq), offsets(nk), max(nq),
                                 SCALE, causal=causal, want_lse=True)
    assert error_word() == (_lib.MOE_OK, 0)
    ro, rl, ob, lb = ragged_ref(q, kv[..., :128], kp, kv[..., 128:], nq, nk, causal, dtype)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")


def test_ragged_strides_and_output_view():
    n, H = 140, 4
    q, kv, kp = randn(n, H, 192, seed=4).to(DEV), randn(n, H, 256, seed=5).to(DEV), randn(n, 64, seed=6).to(DEV)
    cu = offsets([100, 40])
    base = moe.mla_attn_ragged(q, kv[..., :128], kp, kv[..., 128:], cu, cu, 100, SCALE)
    qh = q.transpose(0, 1).contiguous().transpose(0, 1)      # heads outermost
    kh = kv[..., :128].transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros(n, 96, dtype=BF16, device=DEV)
    wide[:, 16:80] = kp
    out = torch.full((H, n, 136), 9.0, dtype=BF16, device=DEV)
    got = moe.mla_attn_ragged(qh, kh, wide[:, 16:80], kv[..., 128:], cu, cu, 100, SCALE,
                              out=out.transpose(0, 1)[..., :128])
    assert torch.equal(got, base) and (out[..., 128:] == 9.0).all()


def test_ragged_bad_offsets_are_reported_and_skipped():
    q, kv, kp = randn(20, 1, 192).to(DEV), randn(20, 1, 256).to(DEV), randn(20, 64).to(DEV)
    for cu, max_q in (([0, 21], 30), ([0, 20], 10), ([-1, 20], 30), ([5, 2], 30)):
        cu_t = torch.tensor(cu, dtype=torch.int32, device=DEV)
        out = torch.full((20, 1, 128), 3.0, dtype=BF16, device=DEV)
        moe.mla_attn_ragged(q, kv[..., :128], kp, kv[..., 128:], cu_t, cu_t, max_q, SCALE, out=out)
        assert error_word() == (_lib.MOE_ERR_INDEX, 0x80)
        assert (out == 3.0).all()


def test_ragged_bound_of_zero_reports_queries():
    q, kv, kp = randn(20, 3, 192).to(DEV), randn(20, 3, 256).to(DEV), randn(20, 64).to(DEV)
    for lens, word in (([0, 20, 0], (_lib.MOE_ERR_INDEX, 0x80)), ([0, 0, 0], (_lib.MOE_OK, 0))):
        out = torch.full((20, 3, 128), 3.0, dtype=BF16, device=DEV)
        moe.mla_attn_ragged(q, kv[..., :128], kp, kv[..., 128:], offsets(lens), offsets(lens), 0, SCALE, out=out)
        assert error_word() == word
        assert (out == 3.0).all()
    with pytest.raises(moe.MoeError, match="B=0"):
        moe.mla_attn_ragged(q, kv[..., :128], kp, kv[..., 128:], offsets([]), offsets([]), 20, SCALE)


@pytest.mark.parametrize("nq", [
    [9], [700, 3, 0, 256, 512, 1, 257], [255, 1, 0, 0, 300] * 8, [i % 4 for i in range(1100)], [0] * 40 + [513] + [0] * 40,
])
def test_ragged_long_bound_on_the_queries(nq):
    # far more room than queries: the grid follows the rows, the results do not change
    n, H = sum(nq), 2
    q, kv, kp = randn(n, H, 192, seed=n).to(DEV), randn(n, H, 256, seed=n + 1).to(DEV), randn(n, 64, seed=n + 2).to(DEV)
    cu = offsets(nq)
    args = (q, kv[..., :128], kp, kv[..., 128:], cu, cu)
    o, lse = moe.mla_attn_ragged(*args, 100_000, SCALE, want_lse=True)
    assert error_word() == (_lib.MOE_OK, 0)
    ro, rl, ob, lb = ragged_ref(q.cpu(), kv[..., :128].cpu(), kp.cpu(), kv[..., 128:].cpu(), nq, nq, True, BF16)
    check(o, ro, ob, "out")
    check(lse, rl, lb, "lse")
    o1, lse1 = moe.mla_attn_ragged(*args, max(nq), SCALE, want_lse=True)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)


@pytest.mark.parametrize("bad", [[0, 10, 21], [0, 15, 10], [-3, 10, 20], [0, 300, 20]])
def test_ragged_bad_offsets_with_a_long_bound(bad):
    q, kv, kp = randn(20, 1, 192).to(DEV), randn(20, 1, 256).to(DEV), randn(20, 64).to(DEV)
    cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
    moe.mla_attn_ragged(q, kv[..., :128], kp, kv[..., 128:], cu, offsets([10, 10]), 100_000, SCALE)
    assert error_word() == (_lib.MOE_ERR_INDEX, 0x80)
    assert error_word() == (_lib.MOE_OK, 0)


# ------------------------------------------------------------- streams, both forms

def test_absorbed_and_expanded_forms_agree():
    # one prompt through both forms: c -> W_ukv -> expanded attention, and W_uk^T q ->
    # absorbed attention over the cache -> W_uv; differently rounded, the same attention
    n, H, page = 150, 8, 64
    w = randn(H, 256, 512, seed=1, std=512 ** -0.5).to(DEV)
    q, kv = randn(n, H, 192, seed=2).to(DEV), randn(n, 576, seed=3, std=2.0).to(DEV)
    gamma = (1 + 0.1 * randn(512, seed=4).float()).to(BF16).to(DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    plan = moe.rope_plan(64, 50000.0, 32.0, mscale_all_dim=1.0, device=DEV)
    scale = SCALE * plan.softmax_factor
    cache = torch.zeros(4, page, 576, dtype=BF16, device=DEV)
    q_abs, row = torch.empty(n, H, 576, dtype=BF16, device=DEV), torch.empty(n, 576, dtype=BF16, device=DEV)
    q_rot = q.clone()
    moe.mla_rope_append(q[..., 128:], kv, pos, plan, gamma=gamma, cache=cache, slots=pos + 64,
                        q_out=q_abs[..., 512:], kv_out=row)
    q_rot[..., 128:] = q_abs[..., 512:]
    kvx = moe.mla_head_proj(row[:, None, :512], w)
    cu = offsets([n])
    expanded = moe.mla_attn_ragged(q_rot, kvx[..., :128], row[:, 512:], kvx[..., 128:], cu, cu, n, scale)
    moe.mla_head_proj(q[..., :128], w[:, :128], w_kn=True, out=q_abs[..., :512])
    table = torch.tensor([[1, 2, 3]], dtype=torch.int32, device=DEV)
    o = moe.mla_attn_paged(q_abs, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale, cu_q=cu)
    absorbed = moe.mla_head_proj(o, w[:, 128:])
    # the 64-bit form of the same roundings-free attention, from the shared inputs
    c, kp = row[:, :512].double().cpu(), row[:, 512:].double().cpu()
    wd, qd = w.double().cpu(), q_rot.double().cpu()
    k = torch.einsum("sc,hnc->shn", c, wd)
    u = 2.0 ** -8
    for h in range(H):
        s = (qd[:, h, :128] @ k[:, h, :128].T + qd[:, h, 128:] @ kp.T) * scale
        s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -math.inf)
        p = torch.softmax(s, 1)
        ref, mag = p @ k[:, h, 128:], p @ k[:, h, 128:].abs()
        # one rounding of every factor of a score (q', or k), of a weight, of a value and of
        # a result: the scores' error reaches every weight
        e = 2 * u * scale * (qd[:, h].abs() @ torch.cat((k[:, h, :128], kp), 1).abs().T).max(1).values[:, None]
        big = torch.einsum("tc,cn->tn", (p.abs() @ c.abs()), wd[h, 128:].abs().T)   # sums of the absorbed form's terms
        check(expanded[:, h], ref, 4 * u * mag + 2 * e * mag, "expanded")
        q_lat = qd[:, h, :128].abs() @ wd[h, :128].abs()
        e_abs = 2 * u * scale * ((q_lat @ c.abs().T) + qd[:, h, 128:].abs() @ kp.abs().T).max(1).values[:, None]
        check(absorbed[:, h], ref, 4 * u * big + 2 * e_abs * mag, "absorbed")


def test_two_streams_with_a_workspace_each():
    q, cache, table, ctx_t = paged_inputs([5000, 40, 900], [1] * 3, 64, 64, seed=21)
    args = [x.to(DEV) for x in (q, cache, table, ctx_t)]
    want = moe.mla_attn_paged(*args, SCALE)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    ws = [moe.mla_paged_workspace(DEV) for _ in streams]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(moe.mla_attn_paged(*args, SCALE, ws=ws[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs[0] + outs[1])

def test_on_another_stream():
    q, kv, kp = randn(50, 2, 192).to(DEV), randn(50, 2, 256).to(DEV), randn(50, 64).to(DEV)
    cu = offsets([50])
    want = moe.mla_attn_ragged(q, kv[..., :128], kp, kv[..., 128:], cu, cu, 50, SCALE)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    with torch.cuda.stream(s):
        late = q * 0
        late += q                                            # q is produced on this stream
        got = moe.mla_attn_ragged(late, kv[..., :128], kp, kv[..., 128:], cu, cu, 50, SCALE)
    s.synchronize()
    assert torch.equal(got, want)
