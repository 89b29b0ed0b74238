"""Timed cases of the paged-attention operators: the page plan, the per-head
norm with rotation (forward, backward, and appending to the paged cache) and
the decode attention over the pages.

``run`` computes a pass in plain torch operations, or, where ``own`` is true,
through the package's entry points; ``exact`` computes the same in 64 bits from
the definitions.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
THETA = 10000.0
EPS = 1e-6


# --------------------------------------------------------------------------- cases
def listed():
    attn = dict(D=128, page=64, Hk=8, G=8)
    return [
        # one decode step of a 64-request server: every request gets one token
        dict(name="plan_step_64", op="plan", N=64, page=64, cached_lo=0, cached_hi=16384,
             new_lo=1, new_hi=1, lens_seed=1),
        # prompts of a packed batch of about 32768 tokens, some with a cached prefix
        dict(name="plan_packed_32768", op="plan", N=16, page=64, cached_lo=0, cached_hi=4096,
             new_lo=1, new_hi=4096, lens_seed=4),
        # a short training sequence that crosses two chunk boundaries
        dict(name="rope_129_bf16", op="rope", T=129, Hq=64, Hk=8, D=128, rot=128,
             interleaved=False, start=0, rope_scale=1.0, dtype="bf16"),
        # a piece far into a long context with a scaled table: half of the head
        # rotated, neighbouring channels paired, FP32
        dict(name="rope_2048_f32_far", op="rope", T=2048, Hq=64, Hk=64, D=128, rot=64,
             interleaved=True, start=1000003, rope_scale=1.2, dtype="f32"),
        # backward of a long training sequence
        dict(name="rope_bwd_16384_bf16", op="rope_bwd", T=16384, Hq=64, Hk=8, D=128, rot=128,
             interleaved=False, start=0, rope_scale=1.0, dtype="bf16"),
        # backward in FP32 with heads of 64 channels, partly rotated
        dict(name="rope_bwd_2048_f32", op="rope_bwd", T=2048, Hq=16, Hk=16, D=64, rot=32,
             interleaved=True, start=17, rope_scale=1.0, dtype="f32"),
        # the new tokens of a decode step, written to their pages
        dict(name="append_step_64", op="append", N=64, cached_lo=0, cached_hi=4096, new_lo=1,
             new_hi=1, lens_seed=5, rot=128, interleaved=False, rope_scale=1.0, dtype="bf16",
             **attn),
        # prompts of a packed batch of about 32768 tokens, written to their pages
        dict(name="append_packed_32768", op="append", N=16, cached_lo=0, cached_hi=0, new_lo=1,
             new_hi=4096, lens_seed=4, rot=128, interleaved=False, rope_scale=1.0, dtype="bf16",
             **attn),
        # one request shortly after its prompt: latency only
        dict(name="decode_1x129_bf16", op="decode", N=1, lo=129, hi=129, lens_seed=6,
             dtype="bf16", **attn),
        # a server's batch of requests of very different lengths
        dict(name="decode_64_ragged_bf16", op="decode", N=64, lo=0, hi=16384, lens_seed=7,
             dtype="bf16", **attn),
        # two very long contexts: the work has to be split over the length
        dict(name="decode_2_long_bf16", op="decode", N=2, lo=131072, hi=262144, lens_seed=8,
             dtype="bf16", **dict(attn, page=128)),
        # every head with its own keys, heads of 64 channels, FP32, small pages
        dict(name="decode_16_f32", op="decode", N=16, lo=1, hi=4096, lens_seed=9, dtype="f32",
             D=64, page=16, Hk=16, G=1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_bwd", "append", "decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    D = rng.choice([64, 128, 128])
    rope = dict(rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= D]),
                interleaved=rng.random() < 0.5, rope_scale=rng.choice([1.0, 1.0, 1.2]))
    heads = dict(Hk=rng.choice([1, 2, 4, 8, 16]), G=rng.choice([1, 2, 3, 4, 5, 8, 8, 16]))
    page = rng.choice([16, 32, 64, 128])
    lens_seed = rng.randrange(1 << 20)
    if op == "plan":
        if rng.random() < 0.5:
            return dict(op=op, N=_log_int(rng, 1, 1024), page=page, cached_lo=0,
                        cached_hi=_log_int(rng, 16, 16384), new_lo=rng.choice([0, 1]), new_hi=1,
                        lens_seed=lens_seed)
        N = _log_int(rng, 1, 64)
        return dict(op=op, N=N, page=page, cached_lo=0, cached_hi=_log_int(rng, 16, 16384),
                    new_lo=1, new_hi=_log_int(rng, 2, min(4096, 65536 // N)),
                    lens_seed=lens_seed)
    if op in ("rope", "rope_bwd"):
        Hk, Hq = heads["Hk"], heads["Hk"] * heads["G"]
        most = 16384 * 72 * 128 * 2 // ((Hq + Hk) * D * size)
        return dict(op=op, T=_log_int(rng, 1, min(32768, most)), Hq=Hq, Hk=Hk, D=D,
                    start=rng.choice([0, 0, rng.randrange(1 << 20)]), dtype=dtype, **rope)
    if op == "append":
        most = 32768 * 72 * 128 * 2 // ((heads["Hk"] * (heads["G"] + 2)) * D * size)
        N = _log_int(rng, 1, 128)
        if rng.random() < 0.5:
            return dict(op=op, N=N, cached_lo=0, cached_hi=_log_int(rng, 16, 4096), new_lo=1,
                        new_hi=1, lens_seed=lens_seed, dtype=dtype, D=D, page=page, **heads,
                        **rope)
        return dict(op=op, N=N, cached_lo=0, cached_hi=0, new_lo=1,
                    new_hi=_log_int(rng, 2, max(2, min(4096, most // N))), lens_seed=lens_seed,
                    dtype=dtype, D=D, page=page, **heads, **rope)
    N = _log_int(rng, 1, 128)
    most = (1 << 31) // (N * heads["Hk"] * D * size * 2)
    hi = _log_int(rng, 2, max(2, min(262144, most)))
    return dict(op=op, N=N, lo=rng.choice([0, 1, hi // 2]), hi=hi, lens_seed=lens_seed,
                dtype=dtype, D=D, page=page, **heads)


def _lengths(case):
    """(tokens cached, new tokens) of each request; for decode, (lengths, ones)."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "decode":
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["N"])], [1] * case["N"]
    cached = [r.randint(case["cached_lo"], case["cached_hi"]) for _ in range(case["N"])]
    return cached, [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["N"])]


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------- inputs
def _randn(gen, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=dtype)
    return x if scale == 1.0 else x * scale


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _offsets(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _pages(gen, counts, spare):
    """A shuffled pool's ids dealt to requests of counts[n] pages: (table [N, M]
    with -1 where a request has no page, the ids that are left, the pool's size)."""
    total = sum(counts) + spare
    ids = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    M = max(1, max(counts, default=0))
    at = _ints(_offsets(counts)[:-1], torch.int64)[:, None] + torch.arange(M, device=DEV)
    held = torch.arange(M, device=DEV) < _ints(counts)[:, None]
    table = torch.where(held, ids[at.clamp(max=total - 1)], -1).to(torch.int32).contiguous()
    return table, ids[sum(counts):].contiguous(), total


def _inv_freq(case):
    """Frequencies of a rotation of case['rot'] channels; a table stretched by 8
    (positions interpolated) where the case scales its rotation."""
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64)
    f = THETA ** (-i / case["rot"])
    return (f / 8 if case["rope_scale"] != 1.0 else f).to(torch.float32).to(DEV)


def _weights(gen, D):
    return 0.5 + torch.rand(D, generator=gen, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "plan":
        cached, new = _lengths(case)
        P = case["page"]
        have = [_ceil(c, P) for c in cached]
        want = [_ceil(c + n, P) for c, n in zip(cached, new)]
        need = sum(want) - sum(have)
        table, free, _ = _pages(gen, have, need + 8)
        M = max(1, max(want))
        bt = torch.full((case["N"], M), -1, dtype=torch.int32, device=DEV)
        bt[:, :min(M, table.shape[1])] = table[:, :M]
        T = sum(new)
        s.update(T=T, cached=_ints(cached), cu=_ints(_offsets(new)), table=bt, free=free,
                 seq_lens=torch.empty(case["N"], dtype=torch.int32, device=DEV),
                 positions=torch.empty(T, dtype=torch.int32, device=DEV),
                 slots=torch.empty(T, dtype=torch.int64, device=DEV),
                 free_end=torch.empty(1, dtype=torch.int32, device=DEV))
        return s
    D, dt = case["D"], TYPES[case["dtype"]]
    if op in ("rope", "rope_bwd"):
        T, Hq, Hk = case["T"], case["Hq"], case["Hk"]
        s.update(q=_randn(gen, (T, Hq, D), dt), k=_randn(gen, (T, Hk, D), dt),
                 positions=torch.arange(T, dtype=torch.int32, device=DEV) + case["start"],
                 inv_freq=_inv_freq(case), q_weight=_weights(gen, D), k_weight=_weights(gen, D))
        if op == "rope_bwd":
            s.update(dq=_randn(gen, (T, Hq, D), dt), dk=_randn(gen, (T, Hk, D), dt),
                     q_grad=torch.empty(T, Hq, D, dtype=dt, device=DEV),
                     k_grad=torch.empty(T, Hk, D, dtype=dt, device=DEV))
        else:
            s.update(q_out=torch.empty_like(s["q"]), k_out=torch.empty_like(s["k"]))
        return s
    Hk, Hq, P = case["Hk"], case["Hk"] * case["G"], case["page"]
    cached, new = _lengths(case)
    if op == "decode":
        table, _, total = _pages(gen, [_ceil(c, P) for c in cached], 1)
        # normed keys and queries, as the append leaves them: unit mean square
        s.update(q=_randn(gen, (case["N"], Hq, D), dt), k_cache=_randn(gen, (total, Hk, P, D), dt),
                 v_cache=_randn(gen, (total, Hk, P, D), dt), table=table,
                 seq_lens=_ints(cached), scale=D ** -0.5,
                 out=torch.empty(case["N"], Hq, D, dtype=dt, device=DEV),
                 lse=torch.empty(case["N"], Hq, dtype=torch.float32, device=DEV))
        return s
    T = sum(new)
    table, _, total = _pages(gen, [_ceil(c + n, P) for c, n in zip(cached, new)], 1)
    req = torch.repeat_interleave(torch.arange(case["N"], device=DEV), _ints(new, torch.int64))
    at = _ints(_offsets(new)[:-1], torch.int64)
    pos = _ints(cached, torch.int64)[req] + torch.arange(T, device=DEV) - at[req]
    # q, k and v side by side, as one projection writes them
    qkv = _randn(gen, (T, Hq + 2 * Hk, D), dt)
    s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:],
             positions=pos.to(torch.int32), slots=table.long()[req, pos // P] * P + pos % P,
             k_cache=_randn(gen, (total, Hk, P, D), dt), v_cache=_randn(gen, (total, Hk, P, D), dt),
             inv_freq=_inv_freq(case), q_weight=_weights(gen, D), k_weight=_weights(gen, D),
             q_out=torch.empty(T, Hq, D, dtype=dt, device=DEV))
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plain_plan, "rope": _plain_rope, "rope_bwd": _plain_rope_bwd,
            "append": _plain_append, "decode": _plain_decode}[s["op"]](s)


def _run_own(s):
    import kimi_delta_attention_10_gb300 as kda
    c, op = s["case"], s["op"]
    if op == "plan":
        kda.kda_page_plan(s["cached"], s["cu"], s["table"], s["free"], c["page"], s["T"],
                          seq_lens=s["seq_lens"], positions=s["positions"], slots=s["slots"],
                          free_end=s["free_end"])
        return {"table": s["table"], "seq_lens": s["seq_lens"], "positions": s["positions"],
                "slots": s["slots"], "free_end": s["free_end"]}
    if op == "decode":
        kda.kda_paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                             s["scale"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    rope = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                interleaved=c["interleaved"], rope_scale=c["rope_scale"])
    if op == "rope":
        kda.kda_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_out=s["q_out"],
                             k_out=s["k_out"], **rope)
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        kda.kda_qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                    s["k_cache"], s["v_cache"], s["inv_freq"], q_out=s["q_out"],
                                    **rope)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    dq, dk, dwq, dwk = kda.kda_qk_norm_rope_bwd(
        s["q"], s["k"], s["dq"], s["dk"], s["positions"], s["inv_freq"], q_grad=s["q_grad"],
        k_grad=s["k_grad"], **rope)
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def _plain_plan(s):
    c, cu, bt, free, P = s["cached"].long(), s["cu"].long(), s["table"], s["free"], s["case"]["page"]
    T, (N, M), F = s["T"], bt.shape, free.numel()
    new = cu[1:] - cu[:-1]
    have, want = (c + P - 1) // P, (c + new + P - 1) // P
    fits = want <= M
    need = torch.where(fits, want - have, 0)
    end = need.cumsum(0)
    ok = fits & ((need == 0) | (end <= F))
    j = torch.arange(M, device=bt.device)
    fresh = (j >= have[:, None]) & (j < want[:, None]) & ok[:, None]
    at = (end - need - have)[:, None] + j
    bt.copy_(torch.where(fresh, free[at.clamp(0, max(0, F - 1))], bt))
    t = torch.arange(T, device=bt.device)
    req = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = c[req] + t - cu[req]
    page = bt.long()[req, (pos // P).clamp(max=M - 1)]
    slots = torch.where(ok[req], page * P + pos % P, -1)
    return {"table": bt, "seq_lens": torch.where(ok, c + new, c).to(torch.int32),
            "positions": pos.to(torch.int32), "slots": slots,
            "free_end": torch.where(ok, need, 0).sum().to(torch.int32).reshape(1)}


def _cos_sin(s):
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    m = s["case"]["rope_scale"]
    return (torch.cos(a) * m).float()[:, None], (torch.sin(a) * m).float()[:, None]


def _pairs(x, case):
    """(first, second) channel of each rotated pair, and the channels left alone."""
    rot = case["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        return r[..., 0::2], r[..., 1::2], rest
    return r[..., :rot // 2], r[..., rot // 2:], rest


def _joined(a, b, rest, case):
    r = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _norm_rope(x, w, cos, sin, case):
    x = x.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    a, b, rest = _pairs(n, case)
    return _joined(a * cos - b * sin, a * sin + b * cos, rest, case)


def _plain_rope(s):
    cos, sin = _cos_sin(s)
    c = s["case"]
    return {"q": _norm_rope(s["q"], s["q_weight"], cos, sin, c).to(s["q"].dtype),
            "k": _norm_rope(s["k"], s["k_weight"], cos, sin, c).to(s["k"].dtype)}


def _plain_append(s):
    cos, sin = _cos_sin(s)
    c, P = s["case"], s["case"]["page"]
    q = _norm_rope(s["q"], s["q_weight"], cos, sin, c).to(s["q"].dtype)
    k = _norm_rope(s["k"], s["k_weight"], cos, sin, c).to(s["k_cache"].dtype)
    page, row = s["slots"] // P, s["slots"] % P
    s["k_cache"][page, :, row] = k
    s["v_cache"][page, :, row] = s["v"].to(s["v_cache"].dtype)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _norm_rope_grad(x, dy, w, cos, sin, case):
    x = x.float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * rstd
    a, b, rest = _pairs(dy.float(), case)
    d = _joined(a * cos + b * sin, b * cos - a * sin, rest, case)
    h = d * w
    return rstd * (h - n * (h * n).mean(-1, keepdim=True)), (d * n).sum((0, 1))


def _plain_rope_bwd(s):
    cos, sin = _cos_sin(s)
    c = s["case"]
    dq, dwq = _norm_rope_grad(s["q"], s["dq"], s["q_weight"], cos, sin, c)
    dk, dwk = _norm_rope_grad(s["k"], s["dk"], s["k_weight"], cos, sin, c)
    return {"dq": dq.to(s["q"].dtype), "dk": dk.to(s["k"].dtype), "dq_weight": dwq,
            "dk_weight": dwk}


def _plain_decode(s):
    q, bt, L = s["q"].float(), s["table"].clamp(min=0).long(), s["seq_lens"]
    N, Hq, D = q.shape
    Hk, P = s["k_cache"].shape[1:3]
    M = bt.shape[1]
    k = s["k_cache"][bt].float().transpose(1, 2).reshape(N, Hk, M * P, D)
    x = torch.einsum("nhgd,nhtd->nhgt", q.view(N, Hk, Hq // Hk, D), k) * s["scale"]
    del k
    live = (torch.arange(M * P, device=q.device) < L[:, None])[:, None, None]
    x = torch.where(live, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    del x
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][bt].float().transpose(1, 2).reshape(N, Hk, M * P, D)
    v = torch.where(live.transpose(-1, -2), v, 0.0)
    o = torch.einsum("nhgt,nhtd->nhgd", p, v) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).view(N, Hq)
    return {"out": o.reshape(N, Hq, D).to(s["q"].dtype), "lse": lse}


# --------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _lengths(case)
        P, T = case["page"], sum(new)
        need = sum(_ceil(c + n, P) - _ceil(c, P) for c, n in zip(cached, new))
        partial = sum(1 for c, n in zip(cached, new) if c % P and n)
        # lengths, offsets, taken ids, started pages; table entries, lengths, positions, slots
        return {"bytes": 4 * (2 * case["N"] + 1 + need + partial) + 4 * (need + case["N"] + 1)
                + 12 * T, "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    D = case["D"]
    if op in ("rope", "rope_bwd"):
        values = case["T"] * (case["Hq"] + case["Hk"]) * D
        n = 2 if op == "rope" else 3
        return {"bytes": n * values * size + 4 * case["T"] + 2 * case["rot"]
                + (8 * D if op == "rope" else 16 * D), "flops": (8 if op == "rope" else 16) * values}
    Hk, Hq = case["Hk"], case["Hk"] * case["G"]
    a, new = _lengths(case)
    if op == "append":
        values = sum(new) * (Hq + 2 * Hk) * D
        return {"bytes": 2 * values * size + 12 * sum(new) + 2 * case["rot"] + 8 * D,
                "flops": 8 * sum(new) * (Hq + Hk) * D}
    L, pages = sum(a), sum(_ceil(x, case["page"]) for x in a)
    return {"bytes": 2 * L * Hk * D * size + 2 * case["N"] * Hq * D * size + 4 * case["N"] * (Hq + 1)
            + 4 * pages, "flops": 4 * L * Hq * D}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(s)
    if op == "decode":
        return _exact_decode(s)
    f = s["inv_freq"].double()
    angle = s["positions"].double()[:, None, None] * f
    # each pair of channels as a complex number, turned by its angle
    turn = case["rope_scale"] * torch.polar(torch.ones_like(angle), angle)
    if op == "rope":
        return {"q": _exact_forward(s["q"], s["q_weight"], turn, case),
                "k": _exact_forward(s["k"], s["k_weight"], turn, case)}
    if op == "append":
        P = case["page"]
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        page, row = s["slots"] // P, s["slots"] % P
        kc[page, :, row] = _exact_forward(s["k"], s["k_weight"], turn, case)
        vc[page, :, row] = s["v"].double()
        return {"q": _exact_forward(s["q"], s["q_weight"], turn, case), "k_cache": kc,
                "v_cache": vc}
    out = {}
    for name in ("q", "k"):
        out["d" + name], out["d%s_weight" % name] = _exact_grad(
            s[name], s["d" + name], s[name + "_weight"], turn, case)
    return out


def _channels(case):
    """Index of the first and of the second channel of every pair."""
    i = torch.arange(case["rot"] // 2, device=DEV)
    return (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)


def _turned(x, turn, case):
    a, b = _channels(case)
    z = torch.complex(x[..., a], x[..., b]) * turn
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_forward(x, w, turn, case):
    x = x.double()
    n = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["D"] + EPS)
    return _turned(n * w.double(), turn, case)


def _exact_grad(x, dy, w, turn, case):
    x, w, D = x.double(), w.double(), case["D"]
    r2 = x.square().sum(-1, keepdim=True) / D + EPS
    d = _turned(dy.double(), turn.conj(), case)      # the transposed rotation
    dw = (d * x / torch.sqrt(r2)).sum(1).sum(0)
    h = d * w
    # y = x r2^(-1/2) w:  dx = h r2^(-1/2) - x r2^(-3/2) (h . x) / D
    dx = h * r2.pow(-0.5) - x * r2.pow(-1.5) * (h * x).sum(-1, keepdim=True) / D
    return dx, dw


def _exact_plan(s):
    c, cu, P = s["cached"].tolist(), s["cu"].tolist(), s["case"]["page"]
    bt, free = s["table"].tolist(), s["free"].tolist()
    at, positions, slots = 0, [], []
    for n in range(s["case"]["N"]):
        for t in range(cu[n + 1] - cu[n]):
            p = c[n] + t
            if p % P == 0:
                bt[n][p // P] = free[at]
                at += 1
            positions.append(p)
            slots.append(bt[n][p // P] * P + p % P)
    return {"table": _ints(bt), "seq_lens": _ints([c[n] + cu[n + 1] - cu[n] for n in range(len(c))]),
            "positions": _ints(positions), "slots": _ints(slots, torch.int64),
            "free_end": _ints([at])}


def _exact_decode(s):
    q, G = s["q"].double(), s["case"]["G"]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    P = s["case"]["page"]
    for n, L in enumerate(s["seq_lens"].tolist()):
        if not L:
            continue
        ids = s["table"][n, :_ceil(L, P)].long()
        for h in range(s["case"]["Hk"]):
            k = s["k_cache"][ids, h].reshape(-1, s["case"]["D"])[:L].double()
            v = s["v_cache"][ids, h].reshape(-1, s["case"]["D"])[:L].double()
            rows = slice(h * G, (h + 1) * G)
            x = (q[n, rows] @ k.T) * s["scale"]
            lse[n, rows] = torch.logsumexp(x, -1)
            out[n, rows] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}
