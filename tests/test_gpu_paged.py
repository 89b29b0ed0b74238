"""GPU parity of the paged-attention operators against the FP64 oracle, at the
sizes, masks and layouts where they can go wrong.

Tolerances count roundings, u = 2^-24 for FP32 and 2^-8 for one rounding to BF16
(relative to the value):
  rotation   the norm's sum and root 9 u, its two products 2 u, cosine and sine 4 u
             (2 u of the angle's rounding, 2 of the function), the scale 1 u, the
             rotation's products and sum 3 u: 19 u, taken as 24 u, of |a| + |b| of
             the normed pair
  decode     a score: 12 u of scale * sum |q k| twice (numerator and sum), each
             e^s 8 u of its own, running sums of n tokens at most n u, of the
             weighted mean of |v|; the BF16 kernel adds 2^-15 for its weights in
             two BF16 parts and the tensor core's sums
"""
import numpy as np
import pytest
import torch

import kimi_delta_attention_10_gb300 as kda
from kimi_delta_attention_10_gb300.binding import KDA_ERR_DEVICE_ARG, KDA_ERR_NO_PAGES
from oracle import paged

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
ROUND = {F32: U, BF16: 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def randn(*shape, seed, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def status_word():
    return torch.zeros(4, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- plan
def run_plan(cached, new, page, M, free, start=None, cu=None, table=None):
    cu = np.concatenate([[0], np.cumsum(new)]) if cu is None else np.asarray(cu)
    T = int(sum(new))
    rng = np.random.default_rng(len(cached) + T)
    if table is None:
        table = rng.integers(0, 1 << 20, (len(cached), M))
    t, st = ints(table.tolist()).reshape(len(cached), M), status_word()
    out = kda.kda_page_plan(ints(cached), ints(cu.tolist()), t, ints(free), page, T,
                            free_start=None if start is None else ints([start]), status=st)
    torch.cuda.synchronize()
    ref = paged.page_plan(cached, cu, T, table, free, page, start or 0)
    for name, a, b in zip(("table", "seq_lens", "positions", "slots"), (t, *out), ref):
        assert np.array_equal(a.cpu().numpy(), b), name
    assert int(out[3]) == ref[4]
    assert int(st[0]) == {None: 0, "arg": KDA_ERR_DEVICE_ARG, "pages": KDA_ERR_NO_PAGES}[ref[5]]
    return out


@pytest.mark.parametrize("N,page,hi_c,hi_m,seed", [
    (1, 16, 0, 1, 0), (1, 64, 100, 1, 1), (3, 1, 9, 5, 2), (7, 7, 50, 30, 3), (64, 64, 5000, 1, 4),
    (257, 16, 300, 3, 5), (300, 8, 40, 0, 6), (1000, 128, 1000, 1, 7), (16, 64, 4096, 4096, 8),
    (2, 1024, 5000, 20000, 9), (1500, 4, 3, 2, 10)])
def test_plan_matches_oracle(N, page, hi_c, hi_m, seed):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, hi_c + 1, N).tolist()
    new = rng.integers(0, hi_m + 1, N).tolist()      # zero new tokens among them
    M = max(1, max(-(-(c + m) // page) for c, m in zip(cached, new)))
    need = sum(-(-(c + m) // page) + (-c // page) for c, m in zip(cached, new))
    free = rng.permutation(need + 5).tolist()
    run_plan(cached, new, page, M, free, start=3 if seed % 2 else None)


def test_plan_where_the_list_or_a_row_runs_out():
    free = list(range(100, 110))
    run_plan([0, 0, 0, 5, 0], [30, 60, 40, 0, 3], 8, 8, free)           # request 2 is cut off
    run_plan([0] * 400, [2] * 400, 2, 1, list(range(300)))              # cut in the second round
    run_plan([0, 0, 60], [30, 90, 5], 8, 8, free)                       # row 1, then row 2 too short
    run_plan([70, 0], [0, 3], 8, 8, free)                               # held more than its row
    run_plan([0, 3], [3, 3], 8, 2, free, start=10)                      # nothing left at all
    run_plan([1], [1], 8, 2, [])                                        # nothing needed


def test_plan_reports_bad_lengths():
    free = list(range(10))
    for cached, cu in [([-1, 0], [0, 2, 4]), ([0, 0], [0, 3, 2]), ([0, 0], [1, 2, 4]),
                       ([0, 0], [0, 2, 3]), ([0, 0], [0, 5, 4]), ([0, 2 ** 31 - 2], [0, 0, 4])]:
        run_plan(cached, [0, 4], 8, 4, free, cu=cu)


def test_plan_reports_bad_page_ids():
    # a held entry and a free entry below zero: their tokens get no slot
    st = status_word()
    table = ints([[-5, -1, -1]])
    out = kda.kda_page_plan(ints([6]), ints([0, 12]), table, ints([4, -2]), 8, 12, status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG
    assert out[2].tolist() == [-1, -1] + [32 + i for i in range(8)] + [-1, -1]


def test_plan_takes_slices():
    """Every array a slice that starts four (slots: eight) bytes into its buffer."""
    at = lambda x, dtype=torch.int32: ints([0, *x], dtype)[1:]
    out = [at([0, 0]), at([0] * 3), at([0] * 3, torch.int64), at([0])]
    table = at([4, -1, 6, -1]).view(2, 2)
    kda.kda_page_plan(at([3, 4]), at([0, 2, 3]), table, at([7, 8]), 4, 3, free_start=at([0]),
                      seq_lens=out[0], positions=out[1], slots=out[2], free_end=out[3])
    assert [o.tolist() for o in out] == [[5, 5], [3, 4, 4], [19, 28, 32], [2]]
    assert table.tolist() == [[4, 7], [6, 8]]


def test_plan_without_requests():
    out = run_plan([], [], 16, 2, [1, 2, 3], cu=[0], table=np.zeros((0, 2), int))
    assert out[0].numel() == 0 and out[1].numel() == 0


def test_plan_in_a_graph_follows_the_lengths():
    """Lengths change between replays; free_end feeds the next step's free_start."""
    cached, cu, start = ints([3, 15]), ints([0, 1, 2]), ints([0])
    table, free = ints([[9, -1], [8, -1]]), ints([5, 6, 7])
    out = kda.kda_page_plan(cached, cu, table, free, 16, 2, free_start=start)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_page_plan(cached, cu, table, free, 16, 2, free_start=start, seq_lens=out[0],
                          positions=out[1], slots=out[2], free_end=out[3])
        cached.copy_(out[0])
        start.copy_(out[3])
    seen = []
    for _ in range(14):
        g.replay()
        seen.append(out[2].tolist())
    assert [s[0] for s in seen] == [9 * 16 + p for p in range(3, 16)] + [6 * 16]
    assert [s[1] for s in seen] == [8 * 16 + 15] + [5 * 16 + p for p in range(13)]
    assert table.tolist() == [[9, 6], [8, 5]] and int(start) == 2


# ---------------------------------------------------------------- norm and rotation
def rope_case(T, Hq, Hk, D, rot, dtype, seed, weights=True, start=0, scale=1.0):
    g = np.random.default_rng(seed)
    # one projection's output: q, k and v side by side
    x = randn(T, Hq + 2 * Hk, D, seed=seed, dtype=dtype)
    f, m = kda.rope_inv_freq(rot, device="cuda") if rot else (None, 1.0)
    w = [torch.from_numpy(g.random(D) + 0.5).float().cuda() if weights else None for _ in range(2)]
    pos = ints((start + np.arange(T)).tolist())
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], pos, f, w, scale * m


def rope_ref(x, pos, f, w, eps, norm, inter, scale):
    f = np.zeros(0) if f is None else f64(f)
    w = np.ones(x.shape[2]) if w is None else f64(w)
    a = (f64(pos), f, w, eps, norm, inter, scale)
    y = paged.norm_rope(f64(x), *a)
    n = np.abs(paged.norm_rope(f64(x), f64(pos), f[:0], w, eps, norm, inter, scale))
    rot = 2 * len(f)
    r = n[..., :rot]
    if inter:
        pair = np.repeat(r[..., 0::2] + r[..., 1::2], 2, -1)
    else:
        pair = np.tile(r[..., :rot // 2] + r[..., rot // 2:], 2)
    n[..., :rot] = pair * abs(scale)
    return y, n


def close(y, ref, size, dtype):
    err, tol = np.abs(f64(y) - ref), 24 * U * size + ROUND[dtype] * np.abs(ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


ROPE_CASES = [
    # T, Hq, Hk, D, rot, interleaved, in, out, start
    (1, 1, 1, 128, 128, False, F32, F32, 0), (5, 4, 2, 64, 64, False, F32, F32, 7),
    (3, 3, 1, 128, 32, True, F32, F32, 1000003), (2, 5, 3, 64, 48, False, BF16, BF16, 100),
    (4, 8, 1, 128, 128, True, BF16, BF16, 0), (1, 7, 7, 128, 16, False, BF16, F32, 2 ** 30),
    (129, 9, 2, 128, 96, False, BF16, BF16, 0), (33, 2, 2, 64, 16, True, F32, BF16, 5),
    (6, 1, 9, 64, 0, False, BF16, BF16, 0), (700, 3, 2, 64, 64, True, BF16, BF16, 0)]


@pytest.mark.parametrize("case", ROPE_CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_rope_matches_oracle(case, norm):
    T, Hq, Hk, D, rot, inter, dt, odt, start = case
    q, k, _, pos, f, w, scale = rope_case(T, Hq, Hk, D, rot, dt, T + Hq, start=start, scale=1.1)
    yq, yk = kda.kda_qk_norm_rope(q, k, pos, f, *w, eps=1e-5, qk_norm=norm, interleaved=inter,
                                  rope_scale=scale, out_dtype=odt)
    assert yq.dtype == odt and yk.dtype == odt
    for x, wi, y in ((q, w[0], yq), (k, w[1], yk)):
        close(y, *rope_ref(x, pos, f, wi, 1e-5, norm, inter, scale), odt)


def test_rope_odd_positions_and_rows():
    """Negative, repeated and far positions; rows of zeros, without weights; in place."""
    q, k, _, _, f, _, _ = rope_case(8, 4, 2, 64, 64, F32, 3, weights=False)
    q, k = q.contiguous(), k.contiguous()
    q[2] = 0
    k[5, 1] = 0
    pos = ints([0, -1, -70000, 5, 5, 2 ** 31 - 1, -2 ** 31, 123456789])
    y = kda.kda_qk_norm_rope(q, k, pos, f)
    for x, a in zip((q, k), y):
        # at 2^31 the frequency's 53 bits leave 2^-22 turns: 1.5e-6 radians, 25 u
        ref, size = rope_ref(x, pos, f, None, 1e-6, True, False, 1.0)
        assert (np.abs(f64(a) - ref) <= 50 * U * size).all()
    assert torch.count_nonzero(y[0][2]) == 0 and torch.count_nonzero(y[1][5, 1]) == 0
    a, b = kda.kda_qk_norm_rope(q, k, pos, f, q_out=q, k_out=k)
    assert a is q and torch.equal(q, y[0]) and torch.equal(k, y[1])
    empty = torch.empty(0, 4, 64, device="cuda")
    assert kda.kda_qk_norm_rope(empty, empty, ints([]), f)[0].shape == (0, 4, 64)


@pytest.mark.parametrize("dt,cdt,D,page", [(BF16, BF16, 128, 64), (F32, F32, 64, 16),
                                           (BF16, F32, 128, 8), (F32, BF16, 64, 3)])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 4, 1), (37, 6, 3), (130, 16, 2)])
def test_append_writes_its_slots_and_nothing_else(dt, cdt, D, page, T, Hq, Hk):
    q, k, v, pos, f, w, scale = rope_case(T, Hq, Hk, D, 32, dt, T + page)
    pages = -(-T // page) + 3
    perm = np.random.default_rng(T).permutation(pages * page)[:T]
    perm[T // 2] = -1                                   # a token without a slot
    kc, vc = (torch.full((pages, Hk, page, D), float("nan"), dtype=cdt, device="cuda")
              for _ in range(2))
    st = status_word()
    y = kda.kda_qk_norm_rope_append(q, k, v, pos, ints(perm.tolist(), torch.int64), kc, vc, f, *w,
                                    rope_scale=scale, status=st)
    dense = kda.kda_qk_norm_rope(q, k, pos, f, *w, rope_scale=scale, out_dtype=cdt)
    assert torch.equal(y, dense[0]) and int(st[0]) == 0
    kw, vw = torch.full_like(kc, float("nan")), torch.full_like(vc, float("nan"))
    for t, s in enumerate(perm):
        if s >= 0:
            kw[s // page, :, s % page] = dense[1][t]
            vw[s // page, :, s % page] = v[t].to(cdt)
    assert torch.equal(kc.nan_to_num(9e9), kw.nan_to_num(9e9))
    assert torch.equal(vc.nan_to_num(9e9), vw.nan_to_num(9e9))


def test_append_reports_a_slot_past_the_cache():
    q, k, v, pos, f, w, _ = rope_case(3, 2, 1, 64, 64, BF16, 9)
    kc, vc = torch.zeros(2, 2, 1, 8, 64, dtype=BF16, device="cuda").unbind(0)
    st = status_word()
    kda.kda_qk_norm_rope_append(q, k, v, pos, ints([3, 16, 15], torch.int64), kc, vc, f, *w,
                                status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG
    rows = vc[:, 0].reshape(16, 64)
    assert torch.equal(rows[3], v[0, 0]) and torch.equal(rows[15], v[2, 0])
    assert torch.count_nonzero(rows.any(1)) == 2


@pytest.mark.parametrize("case", ROPE_CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_rope_bwd_matches_oracle(case, norm):
    T, Hq, Hk, D, rot, inter, dt, gdt, start = case
    q, k, _, pos, f, w, scale = rope_case(T, Hq, Hk, D, rot, dt, T + Hq, start=start, scale=0.9)
    dy = [randn(T, H, D, seed=H + 50, dtype=dt if T % 2 else gdt) for H in (Hq, Hk)]
    out = kda.kda_qk_norm_rope_bwd(q, k, *dy, pos, f, *w, eps=1e-5, qk_norm=norm,
                                   interleaved=inter, rope_scale=scale, grad_dtype=gdt)
    f_ = np.zeros(0) if f is None else f64(f)
    for i, (x, d, wi) in enumerate(zip((q, k), dy, w)):
        args = (f64(pos), f_, f64(wi), 1e-5, norm, inter, scale)
        dx, dw = paged.norm_rope_grad(f64(x), f64(d), *args)
        # d and h as the forward's rotation (24 u of |a| + |b|), then rstd (h - n m): the
        # mean of D products 14 u of mean |h n|, n 10 u, products 3 u, all within 64 u of
        # rstd (2 |d| w + |n| mean |d w n|)
        big = 2 * np.abs(f64(d)).max(-1, keepdims=True) * scale
        xs = f64(x)
        rstd = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-5) if norm else 1.0
        n = np.abs(xs * rstd)
        size = rstd * big * args[2].max() * (1 + n) if norm else big
        err = np.abs(f64(out[i]) - dx)
        assert (err <= 64 * U * size + ROUND[gdt] * np.abs(dx)).all(), "qk"[i]
        if norm:
            # T * H terms of 40 u each, summed in chains of at most T * H / 8 + 64 of them
            terms = (big * n).sum((0, 1))
            tol = (40 + min(T * x.shape[1], T * x.shape[1] / 8 + 64)) * U * terms
            assert (np.abs(f64(out[2 + i]) - dw) <= tol).all(), "qk"[i]
        else:
            assert out[2 + i] is None


def test_rope_bwd_repeats_bit_for_bit_and_in_place():
    q, k, _, pos, f, w, _ = rope_case(1000, 12, 4, 128, 128, BF16, 1)
    dy = [randn(1000, H, 128, seed=H, dtype=BF16) for H in (12, 4)]
    a = kda.kda_qk_norm_rope_bwd(q, k, *dy, pos, f, *w, grad_dtype=BF16)
    ws = torch.full((kda.qk_norm_rope_bwd_workspace_size(1000, 12, 4),), 255, dtype=torch.uint8,
                    device="cuda")
    b = kda.kda_qk_norm_rope_bwd(q, k, *dy, pos, f, *w, q_grad=dy[0], k_grad=dy[1], workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    e = torch.empty(0, 12, 128, device="cuda", dtype=BF16)
    out = kda.kda_qk_norm_rope_bwd(e, e, e, e, ints([]), f, *w)
    assert torch.count_nonzero(out[2]) == 0 and torch.count_nonzero(out[3]) == 0
    one = kda.kda_qk_norm_rope_bwd(q, k, *a[:2], pos, f, w[0], None)
    assert one[2] is not None and one[3] is None


def test_rope_bwd_against_differences():
    """The kernel's gradient against the kernel's own forward, one step along a direction."""
    q, k, _, pos, f, w, _ = rope_case(4, 2, 2, 64, 32, F32, 5)
    q, k = q.contiguous(), k.contiguous()
    dy = [randn(4, 2, 64, seed=s) for s in (1, 2)]
    val = lambda q, k, w: sum((f64(y) * f64(d)).sum() for y, d in zip(
        kda.kda_qk_norm_rope(q, k, pos, f, *w), dy))
    g = kda.kda_qk_norm_rope_bwd(q, k, *dy, pos, f, *w)
    v = [randn(4, 2, 64, seed=7), randn(4, 2, 64, seed=8), randn(64, seed=9), randn(64, seed=10)]
    h = 2.0 ** -7
    step = lambda s: val(q + s * h * v[0], k + s * h * v[1],
                         (w[0] + s * h * v[2], w[1] + s * h * v[3]))
    got = sum((f64(a) * f64(b)).sum() for a, b in zip(g, v))
    # Richardson of the central difference: error of h^4 times a fifth derivative of about
    # 1024 terms of order one, and 1024 roundings of u over h
    d1 = (step(1) - step(-1)) / (2 * h)
    d2 = (step(2) - step(-2)) / (4 * h)
    assert abs((4 * d1 - d2) / 3 - got) <= 1024 * (h ** 4 + 4 * U / h) + 0.01 * abs(d1 - d2)


@pytest.mark.parametrize("dt,D,Hq,Hk", [(BF16, 128, 4, 1), (BF16, 128, 3, 5), (BF16, 64, 3, 1),
                                        (BF16, 64, 6, 7), (F32, 64, 3, 1), (F32, 128, 2, 1)])
def test_rope_bwd_without_epsilon(dt, D, Hq, Hk):
    """eps = 0 with head counts that leave rows of a warp without a head: nothing of those
    reaches the weights' gradients.  Tolerances as in test_rope_bwd_matches_oracle."""
    T = 11
    q, k, _, pos, f, w, scale = rope_case(T, Hq, Hk, D, 32, dt, D + Hk)
    dy = [randn(T, H, D, seed=H + 50, dtype=dt) for H in (Hq, Hk)]
    out = kda.kda_qk_norm_rope_bwd(q, k, *dy, pos, f, *w, eps=0.0, rope_scale=scale)
    for i, (x, d, wi) in enumerate(zip((q, k), dy, w)):
        dx, dw = paged.norm_rope_grad(f64(x), f64(d), f64(pos), f64(f), f64(wi), 0.0, True, False, scale)
        xs, big = f64(x), 2 * np.abs(f64(d)).max(-1, keepdims=True) * scale
        rstd = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True))
        n = np.abs(xs * rstd)
        assert (np.abs(f64(out[i]) - dx) <= 64 * U * rstd * big * f64(wi).max() * (1 + n)
                + U * np.abs(dx)).all(), "qk"[i]
        tol = (40 + T * x.shape[1]) * U * (big * n).sum((0, 1))
        assert (np.abs(f64(out[2 + i]) - dw) <= tol).all(), "qk"[i]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 32), (128, 96)])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_leaves_other_channels_alone(dt, D, rot, inter):
    """Channels that are not rotated, without the norm: the very values, infinities and NaN
    among them, and nothing of theirs in their neighbours; forward, append and backward."""
    q, k, v, pos, f, _, _ = rope_case(6, 3, 2, D, rot, dt, D + rot, start=1)
    fine = kda.kda_qk_norm_rope(q, k, pos, f, qk_norm=False, interleaved=inter)
    for x in (q, k):
        x[0, 0, rot + 3], x[1, 1, D - 1], x[2, 0, rot + 8] = float("inf"), -float("inf"), float("nan")
    y = kda.kda_qk_norm_rope(q, k, pos, f, qk_norm=False, interleaved=inter)
    g = kda.kda_qk_norm_rope_bwd(q, k, q.contiguous(), k.contiguous(), pos, f, qk_norm=False,
                                 interleaved=inter, grad_dtype=dt)
    kc, vc = torch.zeros(2, 1, 2, 8, D, dtype=dt, device="cuda").unbind(0)
    a = kda.kda_qk_norm_rope_append(q, k, v, pos, ints(range(6), torch.int64), kc, vc, f,
                                    qk_norm=False, interleaved=inter)
    bits = lambda t: t.contiguous().view(torch.int16 if dt == BF16 else torch.int32)
    for x, out, grad, ref in ((q, y[0], g[0], fine[0]), (k, y[1], g[1], fine[1])):
        want = x[..., rot:].clone()
        nan = want.isnan()
        for got in (out, grad):
            assert torch.equal(got[..., rot:].isnan(), nan)
            assert torch.equal(bits(got[..., rot:])[~nan], bits(want)[~nan])
        assert torch.equal(out[..., :rot], ref[..., :rot])
    assert torch.equal(bits(a), bits(y[0]))
    assert torch.equal(bits(kc[0, :, :6].transpose(0, 1)), bits(y[1]))


# ---------------------------------------------------------------- decode
def decode_case(lens, Hq, Hk, D, page, dtype, seed, spare=2, extra=1):
    """Pages dealt from a shuffled pool; everything no request reaches is NaN, and so is
    every table entry past a request's pages out of range."""
    rng = np.random.default_rng(seed)
    need = [-(-L // page) for L in lens]
    total, M = sum(need) + spare, max(max(need), 1) + extra
    ids = rng.permutation(total)
    table = np.full((len(lens), M), -(2 ** 31), np.int64)
    table[:, 1::2] = 2 ** 31 - 1
    kc = torch.full((total, Hk, page, D), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    at = 0
    for n, L in enumerate(lens):
        table[n, :need[n]] = ids[at:at + need[n]]
        at += need[n]
        for j in range(need[n]):
            rows = min(page, L - j * page)
            kc[table[n, j], :, :rows] = randn(Hk, rows, D, seed=seed + 1000 * n + j, dtype=dtype)
            vc[table[n, j], :, :rows] = randn(Hk, rows, D, seed=seed + 1000 * n + j + 500, dtype=dtype)
    q = randn(len(lens), Hq, D, seed=seed + 77, dtype=dtype)
    return q, kc, vc, ints(table.tolist()), ints(lens)


def check_decode(case, scale=None, out_dtype=None):
    q, kc, vc, table, lens = case
    scale = q.shape[2] ** -0.5 if scale is None else scale
    st = status_word()
    out, lse = kda.kda_paged_decode(q, kc, vc, table, lens, scale, out_dtype=out_dtype,
                                    want_lse=True, status=st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    ref, ref_lse, mass, reach = paged.paged_decode(f64(q), f64(kc), f64(vc), table.cpu().numpy(),
                                                   lens.cpu().numpy(), scale)
    L = lens.cpu().numpy()[:, None].astype(float)
    score = 12 * U * reach
    rel = 2 * score + 16 * U + np.minimum(L, L / 8 + 64) * U
    if q.dtype == BF16:
        rel = rel + 2.0 ** -15
    err, tol = np.abs(f64(out) - ref), rel[..., None] * mass + ROUND[out.dtype] * np.abs(ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    live = np.broadcast_to(L > 0, ref_lse.shape)
    assert (f64(lse)[~live] == -np.inf).all() and (f64(out)[~live] == 0).all()
    e = np.abs(f64(lse) - ref_lse)[live]
    assert (e <= (rel + 8 * U * np.maximum(1, np.abs(np.where(live, ref_lse, 0))))[live]).all()
    return out, lse


EDGES = [1, 0, 7, 8, 9, 63, 64, 65, 127, 128, 129, 0, 255, 257, 700]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (128, 8), (64, 256), (128, 1024)])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 1), (6, 2), (4, 4)])
def test_decode_matches_oracle(dtype, D, page, Hq, Hk):
    check_decode(decode_case(EDGES, Hq, Hk, D, page, dtype, D + page + Hq))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("G", [2, 3, 5, 7, 9, 16, 17, 33, 64, 71, 130])
def test_decode_head_groups(dtype, G):
    check_decode(decode_case([300, 1, 130], G, 1, 128, 32, dtype, G))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [129], [20000], [5000, 0, 12345]])
def test_decode_few_rows_split_over_the_length(dtype, lens):
    for D, Hk in ((128, 2), (64, 1)):
        check_decode(decode_case(lens, 4 * Hk, Hk, D, 64, dtype, len(lens) + D))


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
def test_decode_many_tiles_a_block(dtype, D):
    """Each block goes through many tiles and several rows of very different lengths, and two
    rows are longer than a block's share; twice the same."""
    rng = np.random.default_rng(11)
    lens = rng.integers(1, 6000, 24).tolist() + [0, 30000, 1, 17000]
    a = check_decode(decode_case(lens, 16, 16, D, 64, dtype, 12))
    b = check_decode(decode_case(lens, 16, 16, D, 64, dtype, 12))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_many_rows(dtype):
    """More requests than threads in a block, most of them short or empty."""
    lens = (np.random.default_rng(3).integers(0, 40, 700) * (np.arange(700) % 3 > 0)).tolist()
    check_decode(decode_case(lens, 2, 1, 64, 8, dtype, 5))


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F32, BF16)])
def test_decode_output_types(dtype, out):
    y, _ = check_decode(decode_case([400, 3], 8, 2, 128, 64, dtype, 8), out_dtype=out)
    assert y.dtype == out


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_large_and_negative_scores(dtype):
    """Scores far from zero on both sides, and a maximum that grows along the row."""
    q, kc, vc, table, lens = decode_case([900, 200], 4, 2, 128, 64, dtype, 21)
    check_decode((q, kc, vc, table, lens), scale=4.0)
    check_decode((q, kc, vc, table, lens), scale=-4.0)
    q.fill_(1.0)
    for j in range(15):                                  # keys grow from page to page
        kc[int(table[0, j])] *= 0
        kc[int(table[0, j])] += j / 4
    kc = torch.where(torch.isnan(kc), torch.zeros_like(kc), kc)
    vc = torch.where(torch.isnan(vc), torch.zeros_like(vc), vc)
    check_decode((q, kc, vc, table, lens), scale=0.25)
    check_decode((q, kc, vc, table, lens), scale=-0.25)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_shared_pages(dtype):
    """Two requests that share the pages of a common prefix."""
    q, kc, vc, table, lens = decode_case([200, 330], 4, 2, 64, 32, dtype, 30)
    table[0, :6] = table[1, :6]
    kc[int(table[0, 6]), :, :8] = 1.0
    check_decode((q, kc, vc, table, lens))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_offsets_beyond_32_bits(dtype):
    """A cache of more than 2^32 bytes and 2^31 values; the request's pages at its end."""
    page, Hk, D = 1024, 8, 128
    total = 2 ** 31 // (page * Hk * D) + 3
    kc = torch.zeros(total, Hk, page, D, dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    ids = [total - 1, 0, total - 2]
    for i in ids:
        kc[i], vc[i] = randn(2, Hk, page, D, seed=i, dtype=dtype)
    q = randn(1, Hk, D, seed=3, dtype=dtype)
    small = decode_case([2500], Hk, Hk, D, page, dtype, 1)
    st = status_word()
    out, lse = kda.kda_paged_decode(q, kc, vc, ints([ids]), ints([2500]), want_lse=True, status=st)
    same = kda.kda_paged_decode(q, kc[ids].contiguous(), vc[ids].contiguous(), ints([[0, 1, 2]]),
                                ints([2500]), want_lse=True)
    assert int(st[0]) == 0 and torch.equal(out, same[0]) and torch.equal(lse, same[1])
    check_decode((q, kc[ids].contiguous(), vc[ids].contiguous(), ints([[0, 1, 2]]), ints([2500])))
    del small
    slots = ints([(total - 1) * page + 1023, 5], torch.int64)
    x = randn(2, Hk, D, seed=4, dtype=dtype)
    kda.kda_qk_norm_rope_append(x, x, x, ints([0, 1]), slots, kc, vc, None, qk_norm=False)
    assert torch.equal(kc[total - 1, :, 1023], x[0]) and torch.equal(vc[0, :, 5], x[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_reports_bad_lengths_and_pages(dtype):
    q, kc, vc, table, lens = decode_case([300, 100, 64], 4, 2, 64, 16, dtype, 40)
    good, _ = kda.kda_paged_decode(q, kc, vc, table, lens)
    for bad in (-3, 16 * table.shape[1] + 1):
        st, l2 = status_word(), lens.clone()
        l2[1] = bad
        out, lse = kda.kda_paged_decode(q, kc, vc, table, l2, want_lse=True, status=st)
        assert int(st[0]) == KDA_ERR_DEVICE_ARG
        assert torch.count_nonzero(out[1]) == 0 and bool((lse[1] == -float("inf")).all())
        assert torch.allclose(out[::2].float(), good[::2].float(), rtol=2 ** -7, atol=1e-6)
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        st, t2 = status_word(), table.clone()
        t2[0, 5] = bad
        out, _ = kda.kda_paged_decode(q, kc, vc, t2, lens, status=st)
        assert int(st[0]) == KDA_ERR_DEVICE_ARG
        assert torch.equal(out[1:], good[1:])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_repeats_bit_for_bit_and_in_a_graph(dtype):
    """Twice, on another stream with a dirty workspace, and replayed with new lengths."""
    q, kc, vc, table, lens = decode_case([3000, 17, 0, 900], 8, 2, 128, 64, dtype, 50)
    a, la = kda.kda_paged_decode(q, kc, vc, table, lens, want_lse=True)
    ws = torch.full((kda.paged_decode_workspace_size(4, 8, 2),), 255, dtype=torch.uint8,
                    device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(a), torch.empty_like(la)
    kda.kda_paged_decode(q, kc, vc, table, lens, out=out, lse=lse, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, a) and torch.equal(lse, la)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kda.kda_paged_decode(q, kc, vc, table, lens, out=out, lse=lse, workspace=ws)
    g.replay()
    assert torch.equal(out, a)
    lens.copy_(ints([5, 17, 0, 899]))
    g.replay()
    b, _ = kda.kda_paged_decode(q, kc, vc, table, lens)
    assert torch.equal(out, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,Hq", [(1, 4), (3, 20), (130, 8), (7000, 4)])
def test_decode_infinite_values(dtype, D, L, Hq):
    """An infinite value makes its channel infinite whatever its weight, both signs make it NaN,
    and no other channel notices."""
    q, kc, vc, table, lens = decode_case([L, 60], Hq, 1, D, 64, dtype, L + D)
    fine, lse = check_decode((q, kc, vc, table, lens))
    at = lambda t: (int(table[0, t // 64]), 0, t % 64)
    for t in {0, L // 2, L - 1}:
        vc[at(t)][3] = float("inf")
        vc[at(t)][D - 1] = -float("inf")
    vc[at(0)][10], vc[at(L - 1)][10] = float("inf"), float("inf") if L == 1 else -float("inf")
    vc[at(L // 2)][20] = float("nan")
    out, lse2 = kda.kda_paged_decode(q, kc, vc, table, lens, want_lse=True)
    assert torch.equal(lse2, lse) and torch.equal(out[1], fine[1])
    assert bool((out[0, :, 3] == float("inf")).all()) and bool((out[0, :, D - 1] == -float("inf")).all())
    assert bool((out[0, :, 10] == float("inf")).all() if L == 1 else out[0, :, 10].isnan().all())
    assert bool(out[0, :, 20].isnan().all())
    rest = [c for c in range(D) if c not in (3, 10, 20, D - 1)]
    assert torch.equal(out[0][:, rest], fine[0][:, rest])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 20)])
@pytest.mark.parametrize("lens", [[3, 60], [5000, 700, 1]])
def test_decode_scores_that_are_no_numbers(dtype, D, Hq, lens):
    """A query that holds NaN makes its head's output and log-sum-exp NaN, one whose scores are
    all -infinity sums nothing (lse -infinity, output 0 / 0); the other heads notice neither."""
    q, kc, vc, table, seq = decode_case(lens, Hq, 1, D, 64, dtype, 70 + D)
    kc[..., 5] = torch.where(kc[..., 5].isnan(), kc[..., 5], torch.ones_like(kc[..., 5]))
    fine, lse = check_decode((q, kc, vc, table, seq))
    q[:, 1, 0] = float("nan")
    q[:, 2, 5] = -float("inf")
    out, lse2 = kda.kda_paged_decode(q, kc, vc, table, seq, want_lse=True)
    assert bool(out[:, 1:3].isnan().all()) and bool(lse2[:, 1].isnan().all())
    assert bool((lse2[:, 2] == -float("inf")).all())
    rest = [h for h in range(Hq) if h not in (1, 2)]
    assert torch.equal(out[:, rest], fine[:, rest]) and torch.equal(lse2[:, rest], lse[:, rest])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("G", [9, 16, 17, 32, 33, 64, 71, 130])
def test_decode_head_groups_of_64_channels(dtype, G):
    check_decode(decode_case([300, 1, 130], G, 1, 64, 32, dtype, G))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,G", [(64, 8), (64, 16), (64, 32), (64, 64), (128, 16), (128, 32), (128, 64)])
def test_decode_head_groups_of_long_rows(dtype, D, G):
    """Rows long enough to go round the rings, to be split over blocks and to add up in several
    runs, with many short ones among them; first of even scores, then of scores that grow along
    a row, so that what is summed so far is rescaled again and again."""
    lens = [9000, 1, 0, 700, 20000] + [3, 129, 40, 260] * 20
    q, kc, vc, table, seq = decode_case(lens, 2 * G, 2, D, 64, dtype, D + G)
    check_decode((q, kc, vc, table, seq))
    q.abs_()
    for n in (0, 3, 4):
        for j in range(-(-lens[n] // 64)):
            kc[int(table[n, j])] += j / 8
    a = check_decode((q, kc, vc, table, seq))
    b = check_decode((q, kc, vc, table, seq))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- beside other kernels
def test_decode_behind_the_chunk_scan():
    """The scan lets the next kernel start early and takes tensor memory of its own: the two in
    turn, without a wait between them, give what each gives alone."""
    T, H = 2048, 8
    q, k, v, g = (randn(T, H, 128, seed=s) for s in range(4))
    g, beta, cu = -0.05 * g.abs(), torch.rand(T, H, device="cuda"), ints([0, T])
    ws = torch.empty(kda.chunk_workspace_size(1, T, H), dtype=torch.uint8, device="cuda")
    chunk = lambda: kda.kda_chunk_fwd(q.bfloat16(), k.bfloat16(), v.bfloat16(), g, beta, cu,
                                      cu_seqlens_host=[0, T], workspace=ws)[0]
    for D, G in ((128, 8), (64, 4)):
        case = decode_case([700, 3, 2000], 2 * G, 2, D, 64, BF16, 60)
        o, (y, _) = chunk(), check_decode(case)
        st = status_word()
        seen = []
        for _ in range(20):
            seen.append((chunk(), kda.kda_paged_decode(*case, status=st)[0]))
        torch.cuda.synchronize()
        assert int(st[0]) == 0
        assert all(torch.equal(a, o) and torch.equal(b, y) for a, b in seen)


# ---------------------------------------------------------------- long sums
@pytest.mark.parametrize("D", [128, 64])
def test_decode_long_rows_lose_nothing(D):
    """Rows of 262144 tokens, each whole in a block: a few pages over and over, so that the
    output is that of the pages once.  Values about one, which truncated sums would shrink.
    The tolerance in u = 2^-24 of |out|: a sum of 128 products' results in the tensor core, each
    truncated by up to 2 u of a partial sum that grows evenly, 128 u; 128 totals and the two parts
    added, 64 u + 2 u; a lane's sum of 2048 weights, 1024 u; a score's 12 u of reach twice, a
    weight's 2^-15 as above."""
    P, pages, L = 64, 16, 262144
    N = torch.cuda.get_device_properties(0).multi_processor_count * (2 if D == 64 else 1)
    kc = randn(pages, 1, P, D, seed=1, dtype=BF16)
    vc = (1 + 0.25 * randn(pages, 1, P, D, seed=2)).to(BF16)
    q = randn(N, 1, D, seed=3, dtype=BF16)
    table = ints([list(range(pages)) * (L // P // pages)]).expand(N, -1).contiguous()
    out, lse = kda.kda_paged_decode(q, kc, vc, table, ints([L] * N), out_dtype=F32, want_lse=True)
    once = np.arange(pages)[None].repeat(N, 0)
    ref, ref_lse, _, reach = paged.paged_decode(f64(q), f64(kc), f64(vc), once, [pages * P] * N, D ** -0.5)
    tol = (1218 * U + 24 * U * reach[..., None] + 2.0 ** -15) * np.abs(ref)
    err = np.abs(f64(out) - ref)
    assert (err <= tol).all(), float((err / tol).max())
    many = ref_lse + np.log(L / (pages * P))
    assert (np.abs(f64(lse) - many) <= 1024 * U + 12 * U * reach + 8 * U * np.abs(many)).all()


# ---------------------------------------------------------------- streams
def test_a_capture_on_the_given_stream_has_its_own_workspace():
    """The current stream is not the one that is captured: the graph must not hold the buffer
    that is kept for eager calls on that stream, which a larger call replaces."""
    case, big = decode_case([3000, 17, 900], 8, 2, 128, 64, BF16, 80), decode_case([4000], 64, 1, 128, 64, BF16, 81)
    want, lse = kda.kda_paged_decode(*case, want_lse=True)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    out, lse2 = torch.zeros_like(want), torch.zeros_like(lse)
    kda.kda_paged_decode(*case, out=out, lse=lse2, stream=side)          # a buffer is kept
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g.capture_begin()
    kda.kda_paged_decode(*case, out=out, lse=lse2, stream=side)
    with torch.cuda.stream(side):
        g.capture_end()
    kda.kda_paged_decode(*big, stream=side)                               # and replaced
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        taken = [torch.full((kda.paged_decode_workspace_size(3, 8, 2),), 255, dtype=torch.uint8, device="cuda")
                 for _ in range(4)]
    out.zero_()
    lse2.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse2, lse)
    assert all(bool((t == 255).all()) for t in taken)


def test_a_forked_stream_of_a_capture_has_its_workspace_there():
    """The current stream is captured, the call goes to a stream forked from it: its workspace
    belongs to that stream, not to the one whose next tensor would get the memory at once."""
    case = decode_case([3000, 17, 900], 8, 2, 128, 64, BF16, 80)
    want, lse = kda.kda_paged_decode(*case, want_lse=True)
    out, lse2, side = torch.zeros_like(want), torch.zeros_like(lse), torch.cuda.Stream()
    bytes_ = kda.paged_decode_workspace_size(3, 8, 2)
    mine = lambda: sum(s["total_size"] for s in torch.cuda.memory_snapshot()
                       if s["stream"] == side.cuda_stream)
    torch.cuda.synchronize()
    g, before = torch.cuda.CUDAGraph(), mine()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        kda.kda_paged_decode(*case, out=out, lse=lse2, stream=side)
        other = torch.full((bytes_,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
    assert mine() >= before + bytes_
    for _ in range(5):
        out.zero_()
        g.replay()
        assert torch.equal(out, want) and torch.equal(lse2, lse) and bool((other == 255).all())


def test_outputs_belong_to_the_call_s_stream():
    """What a call allocates is memory of the stream that writes it: neither a block whose
    kernels on the current stream are still to come, nor given to that stream's next tensor."""
    q, k, v, pos, f, w, _ = rope_case(40, 8, 2, 128, 64, BF16, 90)
    q, k = q.contiguous(), k.contiguous()
    kc, vc = torch.zeros(2, 8, 2, 16, 128, dtype=BF16, device="cuda").unbind(0)
    table, lens = ints([list(range(3))]), ints([40])
    none, cu, planned, free = ints([0]), ints([0, 40]), ints([[-1] * 3]), ints([2, 1, 0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def calls(**kw):
        plan = kda.kda_page_plan(none, cu, planned, free, 16, 40, **kw)
        return [*plan, *kda.kda_qk_norm_rope(q, k, pos, f, *w, **kw),
                kda.kda_qk_norm_rope_append(q, k, v, pos, plan[2], kc, vc, f, *w, **kw),
                *kda.kda_qk_norm_rope_bwd(q, k, q, k, pos, f, *w, **kw),
                *kda.kda_paged_decode(q[:1], kc, vc, table, lens, want_lse=True, **kw)]

    want = calls()
    torch.cuda.synchronize()
    got = calls(stream=side)
    torch.cuda.synchronize()
    assert len(got) == 13 and all(torch.equal(a, b) for a, b in zip(got, want))
    at = {b["address"]: seg["stream"] for seg in torch.cuda.memory_snapshot() for b in seg["blocks"]}
    assert [at[t.data_ptr()] for t in got] == [side.cuda_stream] * 13
    assert torch.cuda.current_stream() != side
