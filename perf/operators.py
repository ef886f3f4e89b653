"""The latent-attention operators at the sizes that are measured.

The attention half of the block whose FFN half this package computes: 64 heads,
latents of 512 with a shared rotary key of 64, head dimensions 128 + 64 (query and
key) and 128 (value), YaRN rotary positions of a 4,096-token model stretched 32x.

    rope    rotary positions on the queries' rotary part and the shared key, RMSNorm
            of the latent, both appended to the paged cache
    paged   absorbed attention over the paged latent cache (single tokens, chunks)
    ragged  expanded attention of a ragged batch of prompts
    proj    the per-head projections between the two forms

`run` is the plain form (elementary torch operations in fp32) unless `own` is set;
then it makes the calls of the package's operators.
"""
import math

import torch

own = False

DEV = "cuda"
LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
THETA, FACTOR, ORIG_CTX, BETA_FAST, BETA_SLOW, MSCALE = 50000.0, 32.0, 4096, 32.0, 1.0, 1.0
EPS = 1e-6
SCALE = (NOPE + ROPE) ** -0.5 * (0.1 * MSCALE * math.log(FACTOR) + 1.0) ** 2

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # the new tokens of one small decode step: latency
        {"name": "rope-decode-16", "op": "rope", "T": 16, "H": 64, "layout": "interleaved", "dtype": "bf16", "page": 64,
         "pos_hi": 131072},
        # the tokens of one prefill batch: bandwidth
        {"name": "rope-prefill-8192", "op": "rope", "T": 8192, "H": 64, "layout": "half", "dtype": "bf16", "page": 64,
         "pos_hi": 131072},
        # one user's next token
        {"name": "paged-b1-c8000", "op": "paged", "B": 1, "lo": 8000, "hi": 8000, "n": 1, "H": 64, "page": 64,
         "dtype": "bf16", "lse": False},
        # the decode batch of the benchmark's size, contexts from short to long
        {"name": "paged-b256-c4096", "op": "paged", "B": 256, "lo": 300, "hi": 8192, "n": 1, "H": 64, "page": 64,
         "dtype": "bf16", "lse": False},
        # few users with long contexts: the keys' axis is split
        {"name": "paged-b4-c131072", "op": "paged", "B": 4, "lo": 98304, "hi": 131072, "n": 1, "H": 64, "page": 64,
         "dtype": "bf16", "lse": True},
        # a GPU's quarter of the heads, small pages, four tokens to verify per sequence
        {"name": "paged-b33-h16-n4", "op": "paged", "B": 33, "lo": 5, "hi": 6000, "n": 4, "H": 16, "page": 16,
         "dtype": "fp16", "lse": True},
        # a chunk of a long prompt over what the cache holds of it
        {"name": "paged-chunk-512", "op": "paged", "B": 2, "lo": 6001, "hi": 8192, "n": 512, "H": 64, "page": 64,
         "dtype": "bf16", "lse": False},
        # a short question
        {"name": "ragged-b1-200", "op": "ragged", "B": 1, "lo": 200, "hi": 200, "past": 0, "H": 64, "dtype": "bf16",
         "lse": False},
        # one long prompt
        {"name": "ragged-b1-8192", "op": "ragged", "B": 1, "lo": 8192, "hi": 8192, "past": 0, "H": 64, "dtype": "bf16",
         "lse": False},
        # a batch of uneven prompts, each after a cached prefix
        {"name": "ragged-b9-prefix", "op": "ragged", "B": 9, "lo": 3, "hi": 1900, "past": 517, "H": 64,
         "dtype": "fp16", "lse": True},
        # decode: queries into the latent space
        {"name": "proj-absorb-256", "op": "proj", "T": 256, "H": 64, "K": 128, "N": 512, "kn": True, "shared": False,
         "dtype": "bf16"},
        # prefill: every head's keys and values from the shared latents
        {"name": "proj-expand-4096", "op": "proj", "T": 4096, "H": 64, "K": 512, "N": 256, "kn": False, "shared": True,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _within(case):
    """No more work than the largest listed cases of its kind."""
    w = work(case)
    return w["bytes"] <= 1.25e9 and w["flops"] <= (9e11 if case["op"] == "paged" else 1.3e12)


def draw(rng):
    op = rng.choice(["rope", "paged", "paged", "ragged", "proj"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, 8192), "H": rng.choice([1, 8, 16, 40, 64]),
                "layout": rng.choice(["interleaved", "half"]), "dtype": dtype, "page": rng.choice([16, 32, 64, 128]),
                "pos_hi": _log(rng, 4096, 1 << 20)}
    if op == "paged":
        B, H = _log(rng, 1, 256), rng.choice([8, 16, 20, 64, 64, 128])
        hi = min(_log(rng, 1, 131072), 1000000 // B)
        n = 1 if rng.random() < 0.6 else min(_log(rng, 2, 512), hi)
        case = {"op": op, "B": B, "lo": max(n, _log(rng, 1, hi)), "hi": hi, "n": n, "H": H,
                "page": rng.choice([8, 16, 32, 64, 128]), "dtype": dtype, "lse": rng.random() < 0.3}
        while not _within(case):
            case["n"] = max(1, case["n"] // 2)
            case["B"] = max(1, case["B"] * 3 // 4)
        return case
    if op == "ragged":
        B, H = _log(rng, 1, 32), rng.choice([8, 16, 20, 64])
        hi = min(_log(rng, 1, 8192), 16384 // B)
        case = {"op": op, "B": B, "lo": _log(rng, 1, hi), "hi": hi,
                "past": 0 if rng.random() < 0.5 else _log(rng, 1, min(2048, 8192 // B)), "H": H, "dtype": dtype,
                "lse": rng.random() < 0.3}
        while not _within(case):
            case["B"] = max(1, case["B"] * 3 // 4)
            case["past"] = case["past"] // 2
            case["hi"] = max(case["lo"], case["hi"] * 7 // 8)
        return case
    K, N, kn, shared = rng.choice([(128, 512, True, False), (512, 128, False, False), (512, 256, False, True)])
    return {"op": op, "T": _log(rng, 1, 4096), "H": rng.choice([8, 16, 20, 64]), "K": K, "N": N, "kn": kn,
            "shared": shared, "dtype": dtype}


def _lengths(B, lo, hi):
    """B lengths over [lo, hi], spread evenly and out of order."""
    if B == 1:
        return [hi]
    return [lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.5) % 1.0) + 0.5) for i in range(B)]


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------------ the inputs

def _randn(shape, gen, dtype, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = _DT[case["dtype"]]
    st = {"case": case}
    op = case["op"]
    if op == "rope":
        T, H, page = case["T"], case["H"], case["page"]
        # the query projection's output holds 128 + 64 columns a head; the key-value
        # down-projection's 512 + 64
        st["q"] = _randn((T, H, NOPE + ROPE), gen, dt)
        st["kv"] = _randn((T, LATENT + ROPE), gen, dt, 2.0)
        st["gamma"] = (1.0 + 0.1 * torch.randn(LATENT, generator=gen, device=DEV)).to(dt)
        st["pos"] = torch.randint(0, case["pos_hi"], (T,), generator=gen, device=DEV).to(torch.int32)
        pages = 2 * ((T + page - 1) // page)
        st["cache"] = _randn((pages, page, LATENT + ROPE), gen, dt)
        st["slots"] = torch.randperm(pages * page, generator=gen, device=DEV)[:T].to(torch.int32)
        # the absorbed query [latent | rotary]: its rotary columns are this call's output
        st["q_abs"] = torch.zeros((T, H, LATENT + ROPE), device=DEV, dtype=dt)
        if own:
            import routed_fp8_expert_gb300 as moe
            st["plan"] = moe.rope_plan(ROPE, THETA, FACTOR, ORIG_CTX, BETA_FAST, BETA_SLOW, MSCALE, MSCALE,
                                       layout=case["layout"], device=DEV)
    elif op == "paged":
        B, n, H, page = case["B"], case["n"], case["H"], case["page"]
        ctx = _lengths(B, case["lo"], case["hi"])
        need = [(c + page - 1) // page for c in ctx]
        total = sum(need)
        st["cache"] = _randn((total, page, LATENT + ROPE), gen, dt)
        perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
        first = torch.tensor(_starts(need)[:-1], device=DEV)[:, None]
        col = torch.arange(max(need), device=DEV)[None]
        st["table"] = torch.where(col < torch.tensor(need, device=DEV)[:, None],
                                  perm[(first + col).clamp(max=total - 1)], 0).to(torch.int32)
        st["ctx_host"] = ctx
        st["ctx"] = torch.tensor(ctx, device=DEV, dtype=torch.int32)
        st["cu_q"] = torch.arange(0, B * n + 1, n, device=DEV, dtype=torch.int32)
        st["q"] = _randn((B * n, H, LATENT + ROPE), gen, dt)
        if own:
            import routed_fp8_expert_gb300 as moe
            st["ws"] = moe.mla_paged_workspace(DEV)
    elif op == "ragged":
        B, H, past = case["B"], case["H"], case["past"]
        lens = _lengths(B, case["lo"], case["hi"])
        st["cq_host"], st["ck_host"] = _starts(lens), _starts([n + past for n in lens])
        Tq, Tk = st["cq_host"][-1], st["ck_host"][-1]
        st["cu_q"] = torch.tensor(st["cq_host"], device=DEV, dtype=torch.int32)
        st["cu_k"] = torch.tensor(st["ck_host"], device=DEV, dtype=torch.int32)
        st["max_q"] = max(lens)
        st["q"] = _randn((Tq, H, NOPE + ROPE), gen, dt)
        # the up-projection's output: every head's keys and values side by side
        st["kv"] = _randn((Tk, H, NOPE + VDIM), gen, dt)
        st["k_pe"] = _randn((Tk, ROPE), gen, dt)
    else:
        T, H, K, N = case["T"], case["H"], case["K"], case["N"]
        st["x"] = _randn((T, 1 if case["shared"] else H, K), gen, dt)
        st["w"] = _randn((H, K, N) if case["kn"] else (H, N, K), gen, dt, K ** -0.5)
    return st


# -------------------------------------------------------------- the plain forms

def _frequencies():
    """YaRN's rotary frequencies (radians a position) of the ROPE / 2 pairs, in 64 bits."""
    def pair_of(turns):
        return ROPE * math.log(ORIG_CTX / (turns * 2 * math.pi)) / (2 * math.log(THETA))
    low = max(math.floor(pair_of(BETA_FAST)), 0)
    high = min(math.ceil(pair_of(BETA_SLOW)), ROPE - 1)
    out = []
    for i in range(ROPE // 2):
        f = THETA ** (-2.0 * i / ROPE)
        ramp = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
        out.append(f / FACTOR * ramp + f * (1.0 - ramp))
    return out


def _rotate(x, cos, sin, layout):
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)


def _plain_rope(st):
    case = st["case"]
    freq = torch.tensor(_frequencies(), device=DEV, dtype=torch.float64)
    angle = st["pos"].double()[:, None] * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    dt = st["q"].dtype
    q_abs, cache = st["q_abs"], st["cache"]
    q_abs[..., LATENT:] = _rotate(st["q"][..., NOPE:].float(), cos[:, None], sin[:, None], case["layout"]).to(dt)
    kv = st["kv"].float()
    c = kv[:, :LATENT]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * st["gamma"].float()
    row = torch.cat((c, _rotate(kv[:, LATENT:], cos, sin, case["layout"])), dim=-1)
    cache.view(-1, LATENT + ROPE)[st["slots"].long()] = row.to(dt)
    return q_abs, cache


def _softmax_rows(s, values):
    """softmax(s) @ values over the last axis and its log-sum-exp; -inf marks a masked score."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    return (p @ values) / l, (m + torch.log(l)).squeeze(-1)


def _plain_paged(st):
    case = st["case"]
    B, n, H, page = case["B"], case["n"], case["H"], case["page"]
    out = torch.empty((B * n, H, LATENT), device=DEV, dtype=st["q"].dtype)
    lse = torch.empty((B * n, H), device=DEV, dtype=torch.float32)
    for b, c in enumerate(st["ctx_host"]):
        pages = st["table"][b, :(c + page - 1) // page].long()
        keys = st["cache"][pages].flatten(0, 1)[:c].float()
        step = max(1, (1 << 28) // (H * c))
        for i in range(0, n, step):
            q = st["q"][b * n + i:b * n + min(n, i + step)].float()
            s = (q.flatten(0, 1) @ keys.t()).view(q.shape[0], H, c) * SCALE
            if n > 1:
                last = c - n + i + torch.arange(q.shape[0], device=DEV)
                s = s.masked_fill(torch.arange(c, device=DEV) > last[:, None, None], -math.inf)
            o, e = _softmax_rows(s, keys[:, :LATENT])
            out[b * n + i:b * n + i + q.shape[0]] = o.to(out.dtype)
            lse[b * n + i:b * n + i + q.shape[0]] = e
    return (out, lse) if case["lse"] else out


def _plain_ragged(st):
    case = st["case"]
    H = case["H"]
    cq, ck = st["cq_host"], st["ck_host"]
    out = torch.empty((cq[-1], H, VDIM), device=DEV, dtype=st["q"].dtype)
    lse = torch.empty((cq[-1], H), device=DEV, dtype=torch.float32)
    for b in range(case["B"]):
        n, c = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        mask = torch.arange(c, device=DEV) > (c - n + torch.arange(n, device=DEV))[:, None]
        step = max(1, (1 << 29) // (n * c))
        kpe = st["k_pe"][ck[b]:ck[b + 1]].float()
        for h in range(0, H, step):
            q = st["q"][cq[b]:cq[b + 1], h:h + step].float().transpose(0, 1)
            kv = st["kv"][ck[b]:ck[b + 1], h:h + step].float().transpose(0, 1)
            s = (q[..., :NOPE] @ kv[..., :NOPE].transpose(1, 2) + q[..., NOPE:] @ kpe.t()) * SCALE
            o, e = _softmax_rows(s.masked_fill_(mask, -math.inf), kv[..., NOPE:])
            out[cq[b]:cq[b + 1], h:h + step] = o.transpose(0, 1).to(out.dtype)
            lse[cq[b]:cq[b + 1], h:h + step] = e.t()
    return (out, lse) if case["lse"] else out


def _plain_proj(st):
    x, w = st["x"].float().transpose(0, 1), st["w"].float()
    y = x @ (w if st["case"]["kn"] else w.transpose(1, 2))
    return y.transpose(0, 1).to(st["x"].dtype).contiguous()


# ------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "paged": _plain_paged, "ragged": _plain_ragged, "proj": _plain_proj}[op](state)
    import routed_fp8_expert_gb300 as moe
    if op == "rope":
        moe.mla_rope_append(state["q"][..., NOPE:], state["kv"], state["pos"], state["plan"], gamma=state["gamma"],
                            eps=EPS, cache=state["cache"], slots=state["slots"],
                            q_out=state["q_abs"][..., LATENT:])
        return state["q_abs"], state["cache"]
    if op == "paged":
        return moe.mla_attn_paged(state["q"], state["cache"], state["table"], state["ctx"], SCALE,
                                  cu_q=state["cu_q"] if case["n"] > 1 else None, want_lse=case["lse"],
                                  ws=state["ws"])
    if op == "ragged":
        return moe.mla_attn_ragged(state["q"], state["kv"][..., :NOPE], state["k_pe"], state["kv"][..., NOPE:],
                                   state["cu_q"], state["cu_k"], state["max_q"], SCALE, want_lse=case["lse"])
    return moe.mla_head_proj(state["x"], state["w"], w_kn=case["kn"])


# ------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "rope":
        T, H = case["T"], case["H"]
        return {"bytes": 2 * T * (H * ROPE + LATENT + ROPE) * 2 + 8 * T + 2 * LATENT,
                "flops": T * (3 * H * ROPE + 4 * LATENT + 3 * ROPE)}
    if op == "paged":
        B, n, H = case["B"], case["n"], case["H"]
        ctx = _lengths(B, case["lo"], case["hi"])
        pairs = H * sum(n * c - n * (n - 1) // 2 for c in ctx)
        return {"bytes": 2 * sum(ctx) * (LATENT + ROPE) + 2 * B * n * H * (2 * LATENT + ROPE)
                + (4 * B * n * H if case["lse"] else 0),
                "flops": 2 * pairs * (2 * LATENT + ROPE)}
    if op == "ragged":
        B, H, past = case["B"], case["H"], case["past"]
        lens = _lengths(B, case["lo"], case["hi"])
        pairs = H * sum(n * past + n * (n + 1) // 2 for n in lens)
        Tq, Tk = sum(lens), sum(lens) + B * past
        return {"bytes": 2 * Tq * H * (NOPE + ROPE + VDIM) + 2 * Tk * (H * (NOPE + VDIM) + ROPE)
                + (4 * Tq * H if case["lse"] else 0),
                "flops": 2 * pairs * (NOPE + ROPE + VDIM)}
    T, H, K, N = case["T"], case["H"], case["K"], case["N"]
    return {"bytes": 2 * (T * K * (1 if case["shared"] else H) + H * K * N + T * H * N), "flops": 2 * T * H * K * N}


# ------------------------------------------------------------ the definition in 64 bits

def _exact_rotation(x, pos, layout):
    """Each pair as a complex number times exp(i * angle)."""
    def corr(turns):
        return ROPE / 2 * math.log(ORIG_CTX / (2 * math.pi * turns)) / math.log(THETA)
    first, last = max(math.floor(corr(BETA_FAST)), 0), min(math.ceil(corr(BETA_SLOW)), ROPE - 1)
    i = torch.arange(ROPE // 2, device=DEV, dtype=torch.float64)
    own_share = 1.0 - ((i - first) / (last - first)).clamp(0.0, 1.0)
    freq = torch.exp(-2.0 * i / ROPE * math.log(THETA)) * (own_share + (1.0 - own_share) / FACTOR)
    angle = pos.to(torch.float64).unsqueeze(-1) * freq
    turn = torch.complex(torch.cos(angle), torch.sin(angle))
    while turn.dim() < x.dim():
        turn = turn.unsqueeze(1)
    x = x.double()
    if layout == "interleaved":
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], ROPE // 2, 2).contiguous()) * turn
        return torch.view_as_real(z).reshape(x.shape)
    z = torch.complex(x[..., :ROPE // 2].contiguous(), x[..., ROPE // 2:].contiguous()) * turn
    return torch.cat((z.real, z.imag), -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        q_abs, cache = st["q_abs"].double(), st["cache"].double()
        q_abs[..., LATENT:] = _exact_rotation(st["q"][..., NOPE:], st["pos"], case["layout"])
        c = st["kv"][:, :LATENT].double()
        norm = torch.sqrt(c.square().sum(-1, keepdim=True) / LATENT + EPS)
        flat = cache.view(-1, LATENT + ROPE)
        flat[st["slots"].long(), :LATENT] = c / norm * st["gamma"].double()
        flat[st["slots"].long(), LATENT:] = _exact_rotation(st["kv"][:, LATENT:], st["pos"], case["layout"])
        return q_abs, cache
    if case["op"] == "paged":
        n, H, page = case["n"], case["H"], case["page"]
        outs, lses = [], []
        for b, c in enumerate(st["ctx_host"]):
            j = torch.arange(c, device=DEV)
            rows = st["cache"].view(-1, LATENT + ROPE)[st["table"][b].long()[j // page] * page + j % page].double()
            for t0 in range(0, n, 32):
                q = st["q"][b * n + t0:b * n + min(t0 + 32, n)].double()
                s = torch.einsum("thd,jd->thj", q, rows) * SCALE
                limit = c - n + t0 + torch.arange(q.shape[0], device=DEV)
                s = torch.where(j[None, None] <= limit[:, None, None], s, -math.inf)
                e = torch.logsumexp(s, -1)
                outs.append(torch.einsum("thj,jd->thd", torch.exp(s - e[..., None]), rows[:, :LATENT]))
                lses.append(e)
        return (torch.cat(outs), torch.cat(lses)) if case["lse"] else torch.cat(outs)
    if case["op"] == "ragged":
        cq, ck = st["cq_host"], st["ck_host"]
        outs, lses = [], []
        for b in range(case["B"]):
            n, c = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
            seen = torch.ones((n, c), device=DEV, dtype=torch.bool).tril(c - n)
            kpe = st["k_pe"][ck[b]:ck[b + 1]].double()
            os_, es = [], []
            for h in range(case["H"]):
                q = st["q"][cq[b]:cq[b + 1], h].double()
                k = torch.cat((st["kv"][ck[b]:ck[b + 1], h, :NOPE].double(), kpe), 1)
                s = torch.where(seen, (q @ k.t()) * SCALE, -math.inf)
                e = torch.logsumexp(s, 1)
                os_.append(torch.exp(s - e[:, None]) @ st["kv"][ck[b]:ck[b + 1], h, NOPE:].double())
                es.append(e)
            outs.append(torch.stack(os_, 1))
            lses.append(torch.stack(es, 1))
        return (torch.cat(outs), torch.cat(lses)) if case["lse"] else torch.cat(outs)
    w = st["w"].double()
    x = st["x"].double().expand(-1, case["H"], -1)
    return torch.einsum("thk,hkn->thn" if case["kn"] else "thk,hnk->thn", x, w)
