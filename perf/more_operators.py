"""Timed cases of attention for several tokens: packed causal attention (forward, and
forward with backward), prompts and pieces of prompts over the paged cache, and
decode of requests that share a prefix.

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
# a drawn case's operations and scores: at most those of the largest listed; keys that the
# plain form lays out for the requests, in elements
MOST_FLOPS = 4 * 64 * 128 * 16384 * 16385 // 2
MOST_SCORES = 64 * 16384 * 16384
MOST_KEYS = 1 << 31


# --------------------------------------------------------------------------- cases
def listed():
    attn = dict(D=128, Hk=8, G=8)
    return [
        # the tokens of a short prompt: latency
        dict(name="attn_129_bf16", op="attn", N=1, lo=129, hi=129, lens_seed=1, dtype="bf16",
             **attn),
        # one long prompt without a cache
        dict(name="attn_16384_bf16", op="attn", N=1, lo=16384, hi=16384, lens_seed=1,
             dtype="bf16", **attn),
        # FP32, heads of 64 channels, every head with its own keys
        dict(name="attn_2048_f32", op="attn", N=1, lo=2048, hi=2048, lens_seed=1, dtype="f32",
             D=64, Hk=16, G=1),
        # training on a packed batch of about 8192 tokens in sequences of very different lengths
        dict(name="train_packed_8192_bf16", op="train", N=8, lo=1, hi=2048, lens_seed=4,
             dtype="bf16", **attn),
        # training on one long sequence
        dict(name="train_8192_bf16", op="train", N=1, lo=8192, hi=8192, lens_seed=1,
             dtype="bf16", **attn),
        # many short sequences, 3 query heads a key head of 64 channels
        dict(name="train_short_d64_bf16", op="train", N=24, lo=1, hi=700, lens_seed=5,
             dtype="bf16", D=64, Hk=4, G=3),
        # training in FP32
        dict(name="train_1024_f32", op="train", N=1, lo=1024, hi=1024, lens_seed=1, dtype="f32",
             D=64, Hk=16, G=1),
        # pieces of prompts of up to 512 tokens over what is cached already
        dict(name="pieces_16_bf16", op="prompt", N=16, cached_lo=0, cached_hi=16384, new_lo=1,
             new_hi=512, lens_seed=6, dtype="bf16", page=64, **attn),
        # a server's step that checks four drafted tokens a request
        dict(name="drafts_64_bf16", op="prompt", N=64, cached_lo=0, cached_hi=16384, new_lo=4,
             new_hi=4, lens_seed=7, dtype="bf16", page=64, **attn),
        # FP32 prompts over small pages
        dict(name="prompts_4_f32", op="prompt", N=4, cached_lo=0, cached_hi=1000, new_lo=1,
             new_hi=300, lens_seed=8, dtype="f32", page=16, D=64, Hk=4, G=4),
        # 64 requests behind one long system prompt
        dict(name="shared_64_bf16", op="shared", groups=1, N=64, prefix_lo=16384, prefix_hi=16384,
             lo=0, hi=1024, lens_seed=9, dtype="bf16", page=64, **attn),
        # few requests in FP32 behind three prefixes
        dict(name="shared_9_f32", op="shared", groups=3, N=9, prefix_lo=500, prefix_hi=2048, lo=1,
             hi=256, lens_seed=10, dtype="f32", page=32, D=128, Hk=2, G=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _pads(case):
    """Scores that the plain form holds at once."""
    Hq = case["Hk"] * case["G"]
    if case["op"] in ("attn", "train"):
        return case["N"] * Hq * case["hi"] ** 2 * (2 if case["op"] == "train" else 1)
    if case["op"] == "prompt":
        return case["N"] * Hq * case["new_hi"] * (case["cached_hi"] + case["new_hi"])
    return case["N"] * Hq * (case["prefix_hi"] + case["hi"])


def _keys(case):
    """Elements of the keys that the plain form lays out."""
    longest = (case["hi"] if case["op"] in ("attn", "train") else case["cached_hi"] + case["new_hi"]
               if case["op"] == "prompt" else case["prefix_hi"] + case["hi"])
    return case["N"] * longest * case["Hk"] * case["D"]


def _drawn(rng):
    op = rng.choice(["attn", "train", "prompt", "shared"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    common = dict(op=op, dtype=dtype, D=rng.choice([64, 128, 128]), Hk=rng.choice([1, 2, 4, 8, 16]),
                  G=rng.choice([1, 2, 3, 4, 5, 8, 8, 16]), lens_seed=rng.randrange(1 << 20))
    if op in ("attn", "train"):
        # lengths, unlike sizes of plain matrices, cost their square
        hi = _log_int(rng, 1, 16384 if dtype == "bf16" else 4096)
        N = _log_int(rng, 1, 64)
        return dict(common, N=N, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi)
    common["page"] = rng.choice([16, 32, 64, 128])
    if op == "prompt":
        return dict(common, N=_log_int(rng, 1, 64), cached_lo=0,
                    cached_hi=rng.choice([0, _log_int(rng, 16, 16384)]), new_lo=rng.choice([0, 1]),
                    new_hi=_log_int(rng, 1, 4096))
    groups = rng.choice([1, 1, 1, 2, 5])
    return dict(common, groups=groups, N=max(groups, _log_int(rng, 1, 128)),
                prefix_lo=0, prefix_hi=_log_int(rng, 16, 32768), lo=rng.choice([0, 1]),
                hi=_log_int(rng, 1, 2048))


def draw(rng):
    while True:
        case = _drawn(rng)
        flops, most = work(case)["flops"], MOST_FLOPS // (16 if case["dtype"] == "f32" else 1)
        if 0 < flops <= most and _pads(case) <= MOST_SCORES and _keys(case) <= MOST_KEYS:
            return case


def _spread(case):
    """Per sequence (cached tokens, new tokens); of shared: (own tokens, 1)."""
    r = random.Random(case["lens_seed"])
    if case["op"] in ("attn", "train"):
        return [0] * case["N"], [r.randint(case["lo"], case["hi"]) for _ in range(case["N"])]
    if case["op"] == "shared":
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["N"])], [1] * case["N"]
    cached = [r.randint(case["cached_lo"], case["cached_hi"]) for _ in range(case["N"])]
    return cached, [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["N"])]


def _groups(case):
    """(requests of each group, its prefix's length)."""
    r = random.Random(case["lens_seed"] + 1)
    cuts = sorted(r.sample(range(1, case["N"]), case["groups"] - 1))
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [case["N"]])]
    return sizes, [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in sizes]


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------- inputs
def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _offsets(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _dealt(ids, counts):
    """Table [len(counts), most] of a shuffled pool's ids, -1 where a row has no page."""
    M = max(1, max(counts, default=0))
    at = _ints(_offsets(counts)[:-1], torch.int64)[:, None] + torch.arange(M, device=DEV)
    held = torch.arange(M, device=DEV) < _ints(counts)[:, None]
    return torch.where(held, ids[at.clamp(max=ids.numel() - 1)], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, D, dt = case["op"], case["D"], TYPES[case["dtype"]]
    Hk, Hq = case["Hk"], case["Hk"] * case["G"]
    cached, new = _spread(case)
    T = sum(new)
    s = {"case": case, "op": op, "scale": D ** -0.5, "cu": _ints(_offsets(new)), "T": T,
         "most_new": max(1, max(new)),
         "out": torch.empty(T, Hq, D, dtype=dt, device=DEV),
         "lse": torch.empty(T, Hq, dtype=torch.float32, device=DEV)}
    if op in ("attn", "train"):
        # q, k and v side by side, as one projection writes them, normed
        qkv = _randn(gen, (T, Hq + 2 * Hk, D), dt)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:])
        if op == "train":
            s.update(dout=_randn(gen, (T, Hq, D), dt),
                     q_grad=torch.empty(T, Hq, D, dtype=dt, device=DEV),
                     k_grad=torch.empty(T, Hk, D, dtype=dt, device=DEV),
                     v_grad=torch.empty(T, Hk, D, dtype=dt, device=DEV))
        return s
    P = case["page"]
    lens = cached if op == "shared" else [c + n for c, n in zip(cached, new)]
    pages = [_ceil(x, P) for x in lens]
    if op == "shared":
        sizes, prefix = _groups(case)
        prefix_pages = [_ceil(x, P) for x in prefix]
    else:
        prefix_pages = []
    total = sum(pages) + sum(prefix_pages) + 1
    ids = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    s.update(q=_randn(gen, (T, Hq, D), dt), k_cache=_randn(gen, (total, Hk, P, D), dt),
             v_cache=_randn(gen, (total, Hk, P, D), dt), table=_dealt(ids, pages),
             seq_lens=_ints(lens))
    if op == "shared":
        s.update(cu=_ints(_offsets(sizes)), prefix_table=_dealt(ids[sum(pages):], prefix_pages),
                 prefix_lens=_ints(prefix))
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"attn": _plain_attn, "train": _plain_train, "prompt": _plain_prompt,
            "shared": _plain_shared}[s["op"]](s)


def _run_own(s):
    import kimi_delta_attention_10_gb300 as kda
    op = s["op"]
    if op == "attn":
        kda.kda_attention_fwd(s["q"], s["k"], s["v"], s["cu"], s["scale"], out=s["out"],
                              lse=s["lse"])
    elif op == "train":
        kda.kda_attention_fwd(s["q"], s["k"], s["v"], s["cu"], s["scale"], out=s["out"],
                              lse=s["lse"])
        kda.kda_attention_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["cu"],
                              s["scale"], q_grad=s["q_grad"], k_grad=s["k_grad"],
                              v_grad=s["v_grad"])
        return {"out": s["out"], "q_grad": s["q_grad"], "k_grad": s["k_grad"],
                "v_grad": s["v_grad"]}
    elif op == "prompt":
        kda.kda_paged_prompt(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["cu"],
                             s["scale"], out=s["out"], lse=s["lse"])
    else:
        kda.kda_paged_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"],
                                    s["prefix_lens"], s["cu"], s["table"], s["seq_lens"],
                                    s["scale"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _where_packed(s):
    """(sequence, place in it) of every packed token, and the packed token of every place."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device=cu.device)
    n = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    place = torch.arange(s["most_new"], device=cu.device)
    at = cu[:-1, None] + place
    return n, t - cu[n], at.clamp(max=max(0, s["T"] - 1)), at < cu[1:, None]


def _heads_first(x, at, Hk):
    """Packed [T, H, D] as [N, Hk, H / Hk, L, D] in 32 bits."""
    x = x.float()[at]
    N, L, H, D = x.shape
    return x.view(N, L, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).contiguous()


def _packed(x, n, i):
    """[N, Hk, G, L, ...] back to [T, Hk * G, ...]."""
    return x.transpose(1, 3).transpose(2, 3)[n, i].flatten(1, 2)


def _weights(q, k, live, scale):
    """(e^(s - m), m, sums) of q [N, Hk, G, L, D] and k [N, Hk, S, D]."""
    N, Hk, G, L, D = q.shape
    x = torch.matmul(q.view(N, Hk, G * L, D) * scale, k.transpose(-1, -2)).view(N, Hk, G, L, -1)
    x.masked_fill_(~live, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x.sub_(m).exp_()
    return x, m, x.sum(-1, keepdim=True)


def _attend(q, k, v, live, scale):
    """(out [N, Hk, G, L, D], lse [N, Hk, G, L])."""
    p, m, total = _weights(q, k, live, scale)
    N, Hk, G, L, D = q.shape
    o = torch.matmul(p.view(N, Hk, G * L, -1), v).view(q.shape)
    return o / torch.where(total == 0, 1.0, total), (m + torch.log(total)).squeeze(-1)


def _causal(s, at_valid):
    i = torch.arange(s["most_new"], device=DEV)
    return ((i <= i[:, None]) & at_valid[:, None])[:, None, None]


def _plain_attn(s):
    Hk = s["case"]["Hk"]
    n, i, at, valid = _where_packed(s)
    q, k, v = (_heads_first(s[x], at, Hk) for x in "qkv")
    o, lse = _attend(q, k[:, :, 0], v[:, :, 0], _causal(s, valid), s["scale"])
    return {"out": _packed(o, n, i).to(s["q"].dtype), "lse": _packed(lse, n, i)}


def _plain_train(s):
    Hk, dt = s["case"]["Hk"], s["q"].dtype
    n, i, at, valid = _where_packed(s)
    q, k, v = (_heads_first(s[x], at, Hk) for x in "qkv")
    d = torch.where(valid[:, None, None, :, None], _heads_first(s["dout"], at, Hk), 0.0)
    k, v = k[:, :, 0], v[:, :, 0]
    N, _, G, L, D = q.shape
    p, _, total = _weights(q, k, _causal(s, valid), s["scale"])
    p.div_(torch.where(total == 0, 1.0, total))
    flat = (N, Hk, G * L, -1)
    o = torch.matmul(p.view(flat), v).view(q.shape)
    dv = torch.matmul(p.view(flat).transpose(-1, -2), d.view(flat))
    ds = torch.matmul(d.view(flat), v.transpose(-1, -2)).view(p.shape)
    ds.sub_((d * o).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds.view(flat), k).view(q.shape) * s["scale"]
    dk = torch.matmul(ds.view(flat).transpose(-1, -2), q.view(flat)) * s["scale"]
    return {"out": _packed(o, n, i).to(dt), "q_grad": _packed(dq, n, i).to(dt),
            "k_grad": _packed(dk[:, :, None], n, i).to(dt),
            "v_grad": _packed(dv[:, :, None], n, i).to(dt)}


def _from_pages(cache, table):
    """[N, Hk, most tokens, D] in 32 bits."""
    x = cache[table.clamp(min=0).long()].float().transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _plain_prompt(s):
    n, i, at, _ = _where_packed(s)
    q = _heads_first(s["q"], at, s["case"]["Hk"])
    k, v = _from_pages(s["k_cache"], s["table"]), _from_pages(s["v_cache"], s["table"])
    lens, cu = s["seq_lens"].long(), s["cu"].long()
    place = torch.arange(s["most_new"], device=DEV)
    last = (lens - (cu[1:] - cu[:-1]))[:, None] + place          # the last token that a query sees
    j = torch.arange(k.shape[2], device=DEV)
    live = (j <= last[..., None]) & (j < lens[:, None, None])
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    o, lse = _attend(q, k, v, live[:, None, None], s["scale"])
    return {"out": _packed(o, n, i).to(s["q"].dtype), "lse": _packed(lse, n, i)}


def _plain_shared(s):
    N, Hq, D = s["q"].shape
    Hk = s["case"]["Hk"]
    q = s["q"].float().view(N, Hk, Hq // Hk, 1, D)
    group = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(N, device=DEV,
                                                                      dtype=torch.int32), right=True)

    def pages(table, lens, rows):
        k, v = _from_pages(s["k_cache"], table), _from_pages(s["v_cache"], table)
        live = torch.arange(k.shape[2], device=DEV) < lens[:, None]
        v = torch.where(live[:, None, :, None], v, 0.0)
        return k[rows], v[rows], live[rows]

    k1, v1, l1 = pages(s["prefix_table"], s["prefix_lens"], group)
    k2, v2, l2 = pages(s["table"], s["seq_lens"], torch.arange(N, device=DEV))
    o, lse = _attend(q, torch.cat((k1, k2), 2), torch.cat((v1, v2), 2),
                     torch.cat((l1, l2), 1)[:, None, None, None], s["scale"])
    return {"out": o.reshape(N, Hq, D).to(s["q"].dtype), "lse": lse.reshape(N, Hq)}


# --------------------------------------------------------------------------- work
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    D, Hk, Hq = case["D"], case["Hk"], case["Hk"] * case["G"]
    cached, new = _spread(case)
    T = sum(new)
    if case["op"] == "shared":
        sizes, prefix = _groups(case)
        tokens = sum(cached) + sum(prefix)
        pairs = sum(cached) + sum(a * b for a, b in zip(sizes, prefix))
        return {"bytes": 2 * tokens * Hk * D * size + 2 * T * Hq * D * size + 4 * T * Hq,
                "flops": 4 * Hq * D * pairs}
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
    rows = sum(cached) + T                       # of keys and values
    if case["op"] == "train":
        # q, k, v, dout read; out and three gradients written
        return {"bytes": (4 * T * Hq + 4 * T * Hk) * D * size, "flops": 14 * Hq * D * pairs}
    return {"bytes": 2 * (T * Hq + rows * Hk) * D * size + 4 * T * Hq, "flops": 4 * Hq * D * pairs}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return {"attn": _exact_attn, "train": _exact_train, "prompt": _exact_prompt,
            "shared": _exact_shared}[case["op"]](s)


def _softmax_rows(q, k, v, scale, last):
    """One head's (out, lse): query i sees keys 0 .. last[i]."""
    x = (q @ k.T) * scale
    x = x.masked_fill(torch.arange(k.shape[0], device=DEV) > last[:, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.softmax(x, -1).nan_to_num(0.0) @ v, lse


def _spans(s):
    cu = s["cu"].tolist()
    return [slice(a, b) for a, b in zip(cu, cu[1:]) if b > a]


def _exact_attn(s):
    G, (T, Hq, D) = s["case"]["G"], s["q"].shape
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, Hq, dtype=torch.float64, device=DEV)
    for span in _spans(s):
        last = torch.arange(span.stop - span.start, device=DEV)
        for h in range(Hq):
            out[span, h], lse[span, h] = _softmax_rows(
                s["q"][span, h].double(), s["k"][span, h // G].double(),
                s["v"][span, h // G].double(), s["scale"], last)
    return {"out": out, "lse": lse}


def _exact_train(s):
    G = s["case"]["G"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    grads = [torch.zeros(s[x].shape, dtype=torch.float64, device=DEV) for x in "qkv"]
    for span in _spans(s):
        last = torch.arange(span.stop - span.start, device=DEV)
        for h in range(s["q"].shape[1]):
            x = [s[a][span, b].double().requires_grad_() for a, b in (("q", h), ("k", h // G),
                                                                      ("v", h // G))]
            with torch.enable_grad():
                o, _ = _softmax_rows(*x, s["scale"], last)
                d = torch.autograd.grad(o, x, s["dout"][span, h].double())
            out[span, h] = o.detach()
            grads[0][span, h] += d[0]
            grads[1][span, h // G] += d[1]
            grads[2][span, h // G] += d[2]
    return {"out": out, "q_grad": grads[0], "k_grad": grads[1], "v_grad": grads[2]}


def _page_rows(s, cache, ids, h, L):
    return s[cache][ids.long(), h].reshape(-1, s["case"]["D"])[:L].double()


def _exact_prompt(s):
    G, (T, Hq, D) = s["case"]["G"], s["q"].shape
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, Hq, dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist()
    for n, L in enumerate(s["seq_lens"].tolist()):
        span = slice(cu[n], cu[n + 1])
        m = cu[n + 1] - cu[n]
        ids = s["table"][n, :_ceil(L, s["case"]["page"])]
        for h in range(Hq if m else 0):
            out[span, h], lse[span, h] = _softmax_rows(
                s["q"][span, h].double(), _page_rows(s, "k_cache", ids, h // G, L),
                _page_rows(s, "v_cache", ids, h // G, L), s["scale"],
                L - m + torch.arange(m, device=DEV))
    return {"out": out, "lse": lse}


def _exact_shared(s):
    G, P, (N, Hq, D) = s["case"]["G"], s["case"]["page"], s["q"].shape
    out = torch.zeros(N, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64, device=DEV)
    cu, lens, prefix = s["cu"].tolist(), s["seq_lens"].tolist(), s["prefix_lens"].tolist()
    for g, first in enumerate(prefix):
        front = s["prefix_table"][g, :_ceil(first, P)]
        for n in range(cu[g], cu[g + 1]):
            back = s["table"][n, :_ceil(lens[n], P)]
            if first + lens[n] == 0:
                continue
            for h in range(s["case"]["Hk"]):
                rows = slice(h * G, (h + 1) * G)
                k, v = (torch.cat((_page_rows(s, c, front, h, first),
                                   _page_rows(s, c, back, h, lens[n])))
                        for c in ("k_cache", "v_cache"))
                x = (s["q"][n, rows].double() @ k.T) * s["scale"]
                lse[n, rows] = torch.logsumexp(x, -1)
                out[n, rows] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}
