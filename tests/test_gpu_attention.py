"""GPU parity of attention for several tokens (packed causal attention and its backward,
prompts over pages, decode behind shared prefixes) against the FP64 oracle.

Tolerances count roundings, u = 2^-24 for FP32 and 2^-8 for one rounding to BF16
(relative to the value), per element and worst case:
  score      a sum of D <= 128 products in chains of at most 64, the chains' sum, the
             scaling: 70 u of scale * sum |q k| (its largest of a row: `reach`)
  output     scores twice (numerator and sum), e^s 8 u of its own twice, running sums of n
             keys n u twice, a join of up to 65 pieces 70 u, of the weighted mean of |v|;
             BF16 rounds each weight once more
  lse        a score, the sum n u, its logarithm and the reference 10 u and 4 u of itself
  p          (backward) two scores, e^s and the given lse: 2 scores + (20 + n) u + 4 u |lse|
  ds         p's share of |dp| + |delta|; dp 70 u of sum |dout v|; delta's 130 u of
             sum |dout out| and the output's own error; in BF16 one rounding of ds
  gradients  ds (p) times |k|, |q| (|dout|), with sums of n terms n u
"""
import math

import numpy as np
import pytest
import torch

import kimi_delta_attention_10_gb300 as kda
from kimi_delta_attention_10_gb300.binding import KDA_ERR_DEVICE_ARG
from oracle import attention

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
ROUND = {F32: U, BF16: 2.0 ** -8}
WEIGHT = {F32: 0.0, BF16: 2.0 ** -8}
NAN = float("nan")


def f64(t):
    return t.detach().cpu().double().numpy()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(*shape, seed, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def status_word():
    return torch.zeros(4, dtype=torch.int32, device="cuda")


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int).tolist()


def projected(T, Hq, Hk, D, dtype, seed):
    """q, k, v as slices of one projection's output."""
    x = randn(T, Hq + 2 * Hk, D, seed=seed, dtype=dtype)
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]


def out_tol(r, dtype):
    n = len(r.k)
    reach = r.reach.max(1, initial=0.0)[:, None]
    return (140 * U * reach + (90 + 2 * n) * U + WEIGHT[dtype]) * r.mass + ROUND[dtype] * np.abs(r.out)


def lse_tol(r):
    lse = np.where(np.isfinite(r.lse), r.lse, 0.0)
    return 70 * U * r.reach.max(1, initial=0.0) + (10 + len(r.k)) * U + 4 * U * np.abs(lse)


def within(got, ref, tol, what):
    with np.errstate(invalid="ignore"):
        err = np.where(got == ref, 0.0, np.abs(got - ref))
    assert (err <= tol).all(), (what, float(np.max(err / np.maximum(tol, 1e-300))))


def check_rows(out, lse, ref, spans, dtype):
    """spans[n]: the packed rows of sequence n."""
    out, lse = f64(out), f64(lse)
    for (n, h), r in ref.items():
        a, b = spans[n]
        within(out[a:b, h], r.out, out_tol(r, dtype), ("out", n, h))
        within(lse[a:b, h], r.lse, lse_tol(r), ("lse", n, h))


# ---------------------------------------------------------------- packed sequences
CASES = [
    # lengths, Hq, Hk, D
    ([1], 1, 1, 64), ([0, 5, 0, 1, 0], 4, 2, 128), ([63, 64, 65], 3, 1, 64),
    ([127, 128, 129], 4, 4, 128), ([300, 1, 17], 6, 2, 128), ([257], 16, 1, 128),
    ([255, 256], 1, 1, 64), ([70, 3, 130], 130, 1, 64), ([33] * 5, 5, 1, 128), ([600], 2, 1, 64),
    ([40] * 41, 1, 1, 64), ([129], 64, 8, 128), ([513], 2, 2, 128), ([9, 1, 30], 300, 2, 128),
    ([385, 2], 48, 1, 128),
    # few rows a sequence: the FP32 form's smaller tiles
    ([20], 1, 1, 64), ([9, 10], 6, 2, 128), ([20, 30], 2, 1, 128), ([50], 1, 1, 64),
    # many key tiles in a row for the tensor cores
    ([1300], 1, 1, 64), ([1030, 9], 9, 3, 128)]


def run_fwd(q, k, v, cu, **kw):
    st = status_word()
    out, lse = kda.kda_attention_fwd(q, k, v, ints(cu), want_lse=True, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    return out, lse


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES)
def test_forward_matches_oracle(case, dtype):
    lens, Hq, Hk, D = case
    cu = offsets(lens)
    q, k, v = projected(cu[-1], Hq, Hk, D, dtype, len(lens) + Hq)
    out, lse = run_fwd(q, k, v, cu, scale=0.11)
    assert out.dtype == dtype and lse.dtype == F32
    check_rows(out, lse, attention.packed(f64(q), f64(k), f64(v), cu, 0.11), attention.spans(cu), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,Hq,Hk,D", [(2100, 1, 1, 64), (1500, 4, 1, 128), (3333, 2, 2, 128)])
def test_forward_in_pieces(T, Hq, Hk, D, dtype):
    """Few rows over many keys: the keys' axis is cut and joined."""
    assert kda.attention_workspace_size(1, T, Hq, Hk, D) > 1024
    q, k, v = projected(T, Hq, Hk, D, dtype, T)
    out, lse = run_fwd(q, k, v, [0, T])
    check_rows(out, lse, attention.packed(f64(q), f64(k), f64(v), [0, T], D ** -0.5), [(0, T)], dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("falling", [False, True])
def test_forward_where_the_maximum_moves(dtype, falling):
    """Scores that grow (fall) from tile to tile by far more than the weights' range."""
    T, D = 700, 64
    q, k, v = projected(T, 2, 1, D, dtype, 3)
    ramp = torch.linspace(0, 30, T, device="cuda").flip(0) if falling else torch.linspace(0, 30, T, device="cuda")
    q, k = q.clone(), k.clone()
    q[..., 0] = 8.0
    k[..., 0] = ramp[:, None].to(dtype)
    out, lse = run_fwd(q, k, v, [0, T], scale=1.0)
    check_rows(out, lse, attention.packed(f64(q), f64(k), f64(v), [0, T], 1.0), [(0, T)], dtype)


def grad_tols(r, dout, dtype, out_t):
    """(dq, dk, dv) tolerances of one head's rows."""
    n, w = len(r.k) + len(r.q), WEIGHT[dtype]
    d, v, k, q = np.abs(dout), np.abs(r.v), np.abs(r.k), np.abs(r.q)
    lse = np.where(np.isfinite(r.lse), np.abs(r.lse), 0.0)[:, None]
    ep = 140 * U * r.reach.max(1, initial=0.0)[:, None] + (20 + n) * U + 4 * U * lse
    dp = dout @ r.v.T
    delta = (dout * r.out).sum(1, keepdims=True)
    delta_e = 130 * U * (d * np.abs(r.out)).sum(1, keepdims=True) + (d * out_t).sum(1, keepdims=True)
    ds = r.p * (dp - delta)
    ds_e = r.p * (ep * (np.abs(dp) + np.abs(delta)) + 70 * U * (d @ v.T) + delta_e) + (w + 4 * U) * np.abs(ds)
    ds_t = ds_e + n * U * np.abs(ds)
    s = abs(r.scale)
    return s * (ds_t @ k), s * (ds_t.T @ q), (r.p * (ep + w + n * U)).T @ d


def check_grads(q, k, v, dout, cu, scale, grads, dtype):
    G = q.shape[1] // k.shape[1]
    ref = attention.packed(f64(q), f64(k), f64(v), cu, scale)
    d = f64(dout)
    gq, gk, gv = (f64(g) for g in grads)
    sums = {}
    for (n, h), r in ref.items():
        a, b = attention.spans(cu)[n]
        dq, dk, dv, _ = r.grads(d[a:b, h])
        tq, tk, tv = grad_tols(r, d[a:b, h], dtype, out_tol(r, dtype))
        # 1.01: terms of second order
        within(gq[a:b, h], dq, 1.01 * tq + ROUND[dtype] * np.abs(dq), ("dq", n, h))
        part = sums.setdefault((n, h // G), [0.0, 0.0, 0.0, 0.0])
        for i, x in enumerate((dk, tk, dv, tv)):
            part[i] = part[i] + x
    for (n, h), (dk, tk, dv, tv) in sums.items():
        a, b = attention.spans(cu)[n]
        # the group's heads share the sums: G (m + n) terms instead of m + n
        more = G * U * (np.abs(dk).max(initial=0) + np.abs(dv).max(initial=0))
        within(gk[a:b, h], dk, 1.01 * tk + more + ROUND[dtype] * np.abs(dk), ("dk", n, h))
        within(gv[a:b, h], dv, 1.01 * tv + more + ROUND[dtype] * np.abs(dv), ("dv", n, h))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES)
def test_backward_matches_oracle(case, dtype):
    lens, Hq, Hk, D = case
    cu = offsets(lens)
    T = cu[-1]
    q, k, v = projected(T, Hq, Hk, D, dtype, len(lens) + Hq)
    dout = randn(T, Hq, D, seed=5, dtype=dtype)
    out, lse = run_fwd(q, k, v, cu, scale=0.11)
    st = status_word()
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu), 0.11, status=st)
    assert int(st[0]) == 0 and all(g.dtype == dtype for g in grads)
    check_grads(q, k, v, dout, cu, 0.11, grads, dtype)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_other_scales(scale):
    for dtype in (F32, BF16):
        q, k, v = projected(150, 2, 1, 64, dtype, 4)
        out, lse = run_fwd(q, k, v, [0, 150], scale=scale)
        check_rows(out, lse, attention.packed(f64(q), f64(k), f64(v), [0, 150], scale), [(0, 150)], dtype)
        dout = randn(150, 2, 64, seed=5, dtype=dtype)
        grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints([0, 150]), scale)
        check_grads(q, k, v, dout, [0, 150], scale, grads, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_thousands_of_short_sequences(dtype):
    """More sequences than a warp looks at at once, empty ones among them; forward, backward and
    the same tokens over pages, against one plain computation over padded rows in 64 bits."""
    lens = np.random.default_rng(3).integers(0, 6, 2500)
    cu = offsets(lens)
    T, Hq, Hk, D = cu[-1], 4, 2, 64
    q, k, v = (x.contiguous() for x in projected(T, Hq, Hk, D, dtype, 7))
    dout = randn(T, Hq, D, seed=8, dtype=dtype)
    out, lse = run_fwd(q, k, v, cu)
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu))
    q64, k64, v64 = (x.double().requires_grad_() for x in (q, k, v))
    c = torch.tensor(cu[:-1], device="cuda")[:, None] + torch.arange(5, device="cuda")
    held = torch.arange(5, device="cuda") < torch.tensor(lens, device="cuda")[:, None]
    c = c.clamp(max=T - 1)
    rep = lambda x: x[c].repeat_interleave(Hq // Hk, 2)
    s = torch.einsum("nihd,njhd->nhij", q64[c], rep(k64)) * D ** -0.5
    see = torch.ones(5, 5, device="cuda").tril().bool() & held[:, None, None, :]
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1).nan_to_num(0.0)
    o = torch.einsum("nhij,njhd->nihd", p, rep(v64))[held]
    want = torch.autograd.grad(o, (q64, k64, v64), dout.double())
    # five terms of a few units at most: 8 roundings to BF16 (60 of FP32) of values below 16
    tol = 8 * 2.0 ** -8 * 16 if dtype == BF16 else 600 * U * 16
    for a, b in zip((out, *grads), (o.detach(), *want)):
        assert (a.double() - b).abs().max() <= tol
    page = 8
    slots = torch.randperm(2500, generator=torch.Generator().manual_seed(1)).int().cuda()
    kc, vc = (torch.full((2500, Hk, page, D), NAN, dtype=dtype, device="cuda") for _ in range(2))
    n, i = held.nonzero(as_tuple=True)
    for cache, x in ((kc, k), (vc, v)):
        cache[slots[n].long(), :, i] = x
    paged, pl = kda.kda_paged_prompt(q, kc, vc, slots[:, None].contiguous(), ints(lens.tolist()), ints(cu),
                                     want_lse=True)
    assert (paged.double() - o.detach()).abs().max() <= tol and (pl - lse).abs().max() <= 600 * U * 16


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_hundreds_of_sequences_of_all_sizes(dtype):
    """Empty ones first, in the middle and last, long ones among short ones."""
    lens = [0] * 40 + [3, 500, 1] + [0] * 100 + [130, 0, 64] + [1, 0, 2] * 50 + [257] + [0] * 30
    assert len(lens) > 256
    cu = offsets(lens)
    q, k, v = projected(cu[-1], 4, 2, 64, dtype, 17)
    dout = randn(cu[-1], 4, 64, seed=18, dtype=dtype)
    out, lse = run_fwd(q, k, v, cu)
    check_rows(out, lse, attention.packed(f64(q), f64(k), f64(v), cu, 0.125), attention.spans(cu), dtype)
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu))
    check_grads(q, k, v, dout, cu, 0.125, grads, dtype)
    # bad offsets far from a tile's own
    for n, to in ((200, cu[199] - 1), (7, -1), (len(lens), cu[-1] + 1)):
        bad, st = list(cu), status_word()
        bad[n] = to
        g = [torch.full((cu[-1], h, 64), 7.0, dtype=dtype, device="cuda") for h in (4, 2, 2)]
        keep = g[0].clone()
        kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(bad), q_grad=g[0], k_grad=g[1], v_grad=g[2], status=st)
        assert int(st[0]) == KDA_ERR_DEVICE_ARG and all((x == 7).all() for x in g)
        st.zero_()
        kda.kda_attention_fwd(q, k, v, ints(bad), out=keep, status=st)
        assert int(st[0]) == KDA_ERR_DEVICE_ARG and (keep == 7).all()


def test_gradients_of_a_few_tokens():
    """The rounding of out and of the weights must not grow in sequences of 2 to 12 tokens: the
    gradients are what their own rounding leaves, 2^-9 a value on average at most, and a part more."""
    cu = offsets([2, 3, 4, 12, 7, 2])
    q, k, v = projected(cu[-1], 16, 4, 128, BF16, 19)
    dout = randn(cu[-1], 16, 128, seed=20, dtype=BF16)
    out, lse = run_fwd(q, k, v, cu)
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu))
    q64, k64, v64 = (x.double().requires_grad_() for x in (q, k, v))
    o = []
    for a, b in attention.spans(cu):
        s = torch.einsum("ihd,jhd->hij", q64[a:b], k64[a:b].repeat_interleave(4, 1)) * 128 ** -0.5
        p = torch.softmax(s.masked_fill(~torch.ones(b - a, b - a, device="cuda").tril().bool(), -math.inf), -1)
        o.append(torch.einsum("hij,jhd->ihd", p, v64[a:b].repeat_interleave(4, 1)))
    want = torch.autograd.grad(torch.cat(o), (q64, k64, v64), dout.double())
    for x, w in zip(grads[:2], want):
        assert (x.double() - w).norm() <= 2.0 ** -9 * w.norm()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_long(dtype):
    """Sequences that fill the GPU's tiles unevenly, with a group whose heads fill no tile."""
    cu = offsets([1100, 3, 700])
    q, k, v = projected(cu[-1], 6, 2, 128, dtype, 8)
    dout = randn(cu[-1], 6, 128, seed=9, dtype=dtype)
    out, lse = run_fwd(q, k, v, cu)
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu))
    check_grads(q, k, v, dout, cu, 128 ** -0.5, grads, dtype)


def test_backward_against_differences():
    """The FP32 gradient against the FP32 forward, one step along a direction."""
    cu = offsets([70, 5])
    q, k, v = (x.contiguous() for x in projected(75, 4, 2, 64, F32, 6))
    d = randn(75, 4, 64, seed=7)
    out, lse = run_fwd(q, k, v, cu)
    grads = kda.kda_attention_bwd(q, k, v, out, lse, d, ints(cu))
    w = [randn(*x.shape, seed=20 + i) for i, x in enumerate((q, k, v))]
    val = lambda t: (f64(run_fwd(q + t * w[0], k + t * w[1], v + t * w[2], cu)[0]) * f64(d)).sum()
    h = 2.0 ** -8
    got = sum((f64(a) * f64(b)).sum() for a, b in zip(grads, w))
    d1, d2 = (val(h) - val(-h)) / (2 * h), (val(2 * h) - val(-2 * h)) / (4 * h)
    # Richardson of the central difference: h^4 of a fifth derivative of 19200 terms of order
    # one, whose roundings (each 60 u) over h add up like their root
    assert abs((4 * d1 - d2) / 3 - got) <= 19200 * h ** 4 + math.sqrt(19200) * 60 * U / h + 0.01 * abs(d1 - d2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_same_bits_every_time(dtype):
    cu = offsets([400, 30, 900])
    q, k, v = projected(cu[-1], 12, 4, 128, dtype, 1)
    dout = randn(cu[-1], 12, 128, seed=2, dtype=dtype)
    out, lse = run_fwd(q, k, v, cu)
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu))
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in
          (kda.attention_workspace_size(3, cu[-1], 12, 4), kda.attention_bwd_workspace_size(3, cu[-1], 12, 4))]
    for _ in range(3):
        again = run_fwd(q, k, v, cu, workspace=ws[0])
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        more = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu), workspace=ws[1])
        assert all(torch.equal(a, b) for a, b in zip(grads, more))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nothing_of_other_sequences_or_of_rows_behind(dtype):
    """NaN in one sequence and in rows that belong to none: the others give the same bits,
    and rows behind the last sequence keep what they held."""
    T, cu = 400, [0, 90, 291, 350]
    q, k, v = (x.contiguous() for x in projected(T, 6, 2, 128, dtype, 2))
    dout = randn(T, 6, 128, seed=3, dtype=dtype)
    outs = lambda: [torch.full((T, h, 128), 7.0, dtype=dtype, device="cuda") for h in (6, 6, 2, 2)]

    def step():
        o = outs()
        lse = torch.full((T, 6), 7.0, device="cuda")
        kda.kda_attention_fwd(q, k, v, ints(cu), out=o[0], lse=lse)
        kda.kda_attention_bwd(q, k, v, o[0], lse, dout, ints(cu), q_grad=o[1], k_grad=o[2], v_grad=o[3])
        return [*o, lse]

    clean = step()
    for x in (q, k, v, dout):
        x[90:291] = NAN
        x[350:] = NAN
    dirty = step()
    for a, b in zip(clean, dirty):
        assert torch.equal(a[:90], b[:90]) and torch.equal(a[291:350], b[291:350])
        assert (a[350:] == 7).all() and (b[350:] == 7).all()
        assert b[90:291].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinities_and_nan_in_a_sequence(dtype):
    """A NaN key makes the rows that see it NaN and no other; a key whose scores are
    -infinity has no weight; a row with no other key gives zeros."""
    T = 300
    q, k, v = (x.contiguous() for x in projected(T, 2, 1, 64, dtype, 12))
    q[..., 0] = 1.0
    ref = run_fwd(q, k, v, [0, T])
    k2 = k.clone()
    k2[200] = NAN
    out, lse = run_fwd(q, k2, v, [0, T])
    assert torch.equal(out[:200], ref[0][:200]) and torch.equal(lse[:200], ref[1][:200])
    assert out[200:].isnan().all() and lse[200:].isnan().all()
    k3 = k.clone()
    k3[:5, :, 0] = -math.inf
    out, lse = run_fwd(q, k3, v, [0, T])
    assert (out[:5] == 0).all() and (lse[:5] == -math.inf).all()
    assert out[5:].isfinite().all() and lse[5:].isfinite().all()
    for h in range(2):
        rows = attention.Rows(f64(q[5:, h]), f64(k[5:, 0]), f64(v[5:, 0]), np.arange(T - 5) + 1, 0.125)
        within(f64(out[5:, h]), rows.out, out_tol(rows, dtype), h)
    grads = kda.kda_attention_bwd(q, k, v, *ref, randn(T, 2, 64, seed=1, dtype=dtype), ints([0, T]))
    assert all(g.isfinite().all() for g in grads)


@pytest.mark.parametrize("cu", [[0, 5, 3, 10], [1, 5, 7, 10], [0, 5, 7, 11], [0, -1, 7, 10]])
def test_bad_offsets_are_reported(cu):
    for dtype in (F32, BF16):
        q, k, v = projected(10, 4, 2, 64, dtype, 1)
        st = status_word()
        out = torch.full((10, 4, 64), 7.0, dtype=dtype, device="cuda")
        lse = torch.full((10, 4), 7.0, device="cuda")
        kda.kda_attention_fwd(q, k, v, ints(cu), out=out, lse=lse, status=st)
        assert int(st[0]) == KDA_ERR_DEVICE_ARG and (out == 7).all() and (lse == 7).all()
        st.zero_()
        g = [torch.full((10, h, 64), 7.0, dtype=dtype, device="cuda") for h in (4, 2, 2)]
        kda.kda_attention_bwd(q, k, v, out, lse, out.clone(), ints(cu), q_grad=g[0], k_grad=g[1], v_grad=g[2],
                              status=st)
        assert int(st[0]) == KDA_ERR_DEVICE_ARG and all((x == 7).all() for x in g)


def test_calls_without_tokens():
    for dtype in (F32, BF16):
        e = torch.empty(0, 4, 64, dtype=dtype, device="cuda")
        out, lse = kda.kda_attention_fwd(e, e, e, ints([0, 0, 0]), want_lse=True)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
        assert kda.kda_attention_bwd(e, e, e, out, lse, e, ints([0]))[0].shape == (0, 4, 64)
        q, k, v = projected(3, 4, 2, 64, dtype, 1)
        keep = torch.full((3, 4, 64), 7.0, dtype=dtype, device="cuda")
        kda.kda_attention_fwd(q, k, v, ints([0, 0, 0]), out=keep)
        assert (keep == 7).all()


# ---------------------------------------------------------------- prompts over pages
def paged_case(lens, Hk, D, page, dtype, seed, spare=2):
    """Caches whose every place that no request uses holds NaN; a table with room to spare."""
    r = np.random.default_rng(seed)
    want = [-(-n // page) for n in lens]
    total = sum(want) + spare
    ids, M = r.permutation(total), max(1, *want) + 1
    table = np.full((len(lens), M), -1)
    at = 0
    kc, vc = (torch.full((total, Hk, page, D), NAN) for _ in range(2))
    for n, (L, w) in enumerate(zip(lens, want)):
        table[n, :w] = ids[at:at + w]
        at += w
        for c in (kc, vc):
            x = torch.from_numpy(r.standard_normal((L, Hk, D))).float()
            for j in range(w):
                part = x[j * page:(j + 1) * page].transpose(0, 1)
                c[int(table[n, j]), :, :part.shape[1]] = part
    return kc.to(dtype).cuda(), vc.to(dtype).cuda(), table


PROMPTS = [
    # cached, new, Hq, Hk, D, page
    ([0], [1], 1, 1, 64, 8), ([0, 30, 5], [40, 1, 0], 4, 2, 128, 16), ([129, 0, 700], [4, 130, 1], 8, 1, 128, 64),
    ([5, 255, 256, 1000], [3, 3, 3, 3], 16, 2, 64, 128), ([63, 64, 65], [64, 64, 64], 3, 3, 64, 32),
    ([0] * 40, [3] * 40, 2, 1, 128, 8), ([900], [300], 5, 1, 128, 256), ([17, 3000], [200, 1], 48, 2, 64, 1024),
    ([10, 0], [2, 2], 200, 1, 128, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", PROMPTS)
def test_prompt_matches_oracle(case, dtype):
    cached, new, Hq, Hk, D, page = case
    lens, cu = [a + b for a, b in zip(cached, new)], offsets(new)
    kc, vc, table = paged_case(lens, Hk, D, page, dtype, sum(lens))
    q = randn(cu[-1], Hq + 1, D, seed=3, dtype=dtype)[:, :Hq]          # strided tokens
    st = status_word()
    out, lse = kda.kda_paged_prompt(q, kc, vc, ints(table.tolist()), ints(lens), ints(cu), want_lse=True,
                                    status=st)
    assert int(st[0]) == 0
    ref = attention.paged_prompt(f64(q), f64(kc), f64(vc), table, lens, cu, D ** -0.5)
    check_rows(out, lse, ref, attention.spans(cu), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_in_pieces_and_as_decode(dtype):
    """One token a request over long contexts: pieces, joined; what kda_paged_decode gives."""
    lens = [3000, 0, 1, 4097]
    kc, vc, table = paged_case(lens, 2, 128, 64, dtype, 5)
    q = randn(4, 8, 128, seed=4, dtype=dtype)
    out, lse = kda.kda_paged_prompt(q, kc, vc, ints(table.tolist()), ints(lens), ints([0, 1, 2, 3, 4]),
                                    want_lse=True)
    ref = attention.paged_prompt(f64(q), f64(kc), f64(vc), table, lens, [0, 1, 2, 3, 4], 128 ** -0.5)
    check_rows(out, lse, ref, attention.spans([0, 1, 2, 3, 4]), dtype)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    d, dl = kda.kda_paged_decode(q, kc, vc, ints(table.tolist()), ints(lens), want_lse=True)
    for (n, h), r in ref.items():
        within(f64(out[n, h]), f64(d[n, h]), 2 * out_tol(r, dtype)[0], n)
        within(f64(lse[n, h]), f64(dl[n, h]), 2 * lse_tol(r)[0], n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_of_few_among_hundreds_of_requests(dtype):
    """Most have no new token, the first neither; the others' keys are cut into pieces."""
    new, lens = [0] * 300, [1] * 300
    for n, m, L in ((30, 1, 2500), (150, 2, 900), (299, 1, 1)):
        new[n], lens[n] = m, L
    cu = offsets(new)
    kc, vc, table = paged_case(lens, 1, 64, 32, dtype, 6)
    q, st = randn(4, 2, 64, seed=6, dtype=dtype), status_word()
    out, lse = kda.kda_paged_prompt(q, kc, vc, ints(table.tolist()), ints(lens), ints(cu), want_lse=True, status=st)
    assert int(st[0]) == 0
    ref = attention.paged_prompt(f64(q), f64(kc), f64(vc), table, lens, cu, 0.125)
    check_rows(out, lse, ref, attention.spans(cu), dtype)
    lens[3] = -1                               # of a request without tokens
    kda.kda_paged_prompt(q, kc, vc, ints(table.tolist()), ints(lens), ints(cu), status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_tokens_before_the_first_key(dtype):
    """A request that holds fewer tokens than its queries: the first ones see none."""
    kc, vc, table = paged_case([3, 0], 1, 64, 8, dtype, 1)
    q = randn(10, 2, 64, seed=1, dtype=dtype)
    out, lse = kda.kda_paged_prompt(q, kc, vc, ints(table.tolist()), ints([3, 0]), ints([0, 7, 10]), want_lse=True)
    ref = attention.paged_prompt(f64(q), f64(kc), f64(vc), table, [3, 0], [0, 7, 10], 0.125)
    check_rows(out, lse, ref, [(0, 7), (7, 10)], dtype)
    assert (out[:4] == 0).all() and (lse[:4] == -math.inf).all() and (out[7:] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_reports_bad_lengths_and_pages(dtype):
    kc, vc, table = paged_case([20, 20, 20], 2, 64, 8, dtype, 1)
    q = randn(6, 4, 64, seed=1, dtype=dtype)
    good, _ = kda.kda_paged_prompt(q, kc, vc, ints(table.tolist()), ints([20, 20, 20]), ints([0, 2, 4, 6]))
    for lens, row in (([20, -1, 20], None), ([20, 33, 20], None), ([20, 20, 20], [0, 99, 1, -1]),
                      ([20, 20, 20], [0, -1, 1, -1])):
        st, t = status_word(), table.copy()
        if row is not None:
            t[1] = row
        out, _ = kda.kda_paged_prompt(q, kc, vc, ints(t.tolist()), ints(lens), ints([0, 2, 4, 6]), status=st)
        assert int(st[0]) == KDA_ERR_DEVICE_ARG
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
        if row is None:
            assert (out[2:4] == 0).all()
    st = status_word()
    none = kc[:0]
    out, _ = kda.kda_paged_prompt(q, none, none, ints(table.tolist()), ints([20, 0, 0]), ints([0, 2, 4, 6]), status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG and (out == 0).all()


# ---------------------------------------------------------------- shared prefixes
SHARED = [
    # prefixes, group sizes, own lengths, Hq, Hk, D, page
    ([40], [3], [1, 0, 9], 4, 2, 128, 16), ([0, 300], [2, 1], [5, 0, 130], 8, 1, 64, 64),
    ([2000, 1, 0], [5, 0, 3], [1, 2, 3, 300, 0, 7, 0, 64], 8, 2, 128, 32), ([128, 129], [1, 40], [3] * 41, 3, 1, 64, 128),
    ([5000], [20], list(range(20)), 16, 2, 128, 64), ([257], [4], [0] * 4, 130, 1, 128, 8)]


def run_shared(case, dtype, q, kc, vc, table, tail=0, **kw):
    prefixes, sizes, own = case[:3]
    g = len(prefixes)
    st = status_word()
    out = torch.full((len(own) + tail, *q.shape[1:]), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((len(own) + tail, q.shape[1]), 7.0, device="cuda")
    kda.kda_paged_decode_shared(q, kc, vc, ints(table[:g].tolist()), ints(prefixes), ints(offsets(sizes)),
                                ints(table[g:].tolist()), ints(own + [0] * tail), out=out, lse=lse, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    return out, lse


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", SHARED)
def test_shared_matches_oracle(case, dtype):
    prefixes, sizes, own, Hq, Hk, D, page = case
    kc, vc, table = paged_case(prefixes + own, Hk, D, page, dtype, sum(own))
    q = randn(len(own), Hq, D, seed=2, dtype=dtype)
    out, lse = run_shared(case, dtype, q, kc, vc, table)
    g = len(prefixes)
    ref = attention.decode_shared(f64(q), f64(kc), f64(vc), table[:g], prefixes, offsets(sizes), table[g:], own,
                                  D ** -0.5)
    check_rows(out, lse, ref, [(n, n + 1) for n in range(len(own))], dtype)
    ws = torch.full((kda.paged_decode_shared_workspace_size(len(own), g, Hq, Hk, D),), 255, dtype=torch.uint8,
                    device="cuda")
    again = run_shared(case, dtype, q, kc, vc, table, workspace=ws)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_shared_leaves_requests_behind_the_groups(dtype):
    case = ([50], [2], [3, 4], 4, 2, 128, 16)
    kc, vc, table = paged_case([50, 3, 4], 2, 128, 16, dtype, 3)
    table = np.concatenate([table, np.full((1, table.shape[1]), -1)])
    q = randn(3, 4, 128, seed=2, dtype=dtype)
    out, lse = run_shared(case, dtype, q, kc, vc, table, tail=1)
    assert (out[2] == 7).all() and (lse[2] == 7).all() and not (out[:2] == 7).all()
    st = status_word()
    kda.kda_paged_decode_shared(q, kc, vc, ints(table[:1].tolist()), ints([50]), ints([0, 4]),
                                ints(table[1:].tolist()), ints([3, 4, 0]), out=out, lse=lse, status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG


# ---------------------------------------------------------------- streams, graphs, together
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graphs_follow_the_lengths(dtype):
    """A captured forward and backward replayed with other offsets, beside eager calls."""
    T = 500
    q, k, v = projected(T, 4, 2, 64, dtype, 3)
    dout, cu = randn(T, 4, 64, seed=4, dtype=dtype), ints([0, 100, 500])
    out, lse = kda.kda_attention_fwd(q, k, v, cu, want_lse=True)
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = kda.kda_attention_fwd(q, k, v, cu, want_lse=True)
        d = kda.kda_attention_bwd(q, k, v, o, l, dout, cu)
    for lens in ([0, 100, 500], [0, 499, 500], [0, 0, 500], [0, 257, 257]):
        cu.copy_(ints(lens))
        g.replay()
        want, wl = kda.kda_attention_fwd(q, k, v, cu, want_lse=True)
        wd = kda.kda_attention_bwd(q, k, v, want, wl, dout, cu)
        n = lens[-1]
        assert torch.equal(o[:n], want[:n]) and torch.equal(l[:n], wl[:n])
        assert all(torch.equal(a[:n], b[:n]) for a, b in zip(d, wd))
    assert all(x.shape == y.shape for x, y in zip(grads, d))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_calls_on_two_streams(dtype):
    """Calls in pieces on two streams at once, each with its own kept workspace."""
    xs = [projected(2000, 2, 1, 128, dtype, s) for s in range(2)]
    cu = ints([0, 2000])
    want = [kda.kda_attention_fwd(*x, cu, want_lse=True) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [kda.kda_attention_fwd(*x, cu, want_lse=True, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_serving_together(dtype):
    """Prompts in two pieces, then tokens one by one, some behind a shared prefix: page plan,
    append, prompt attention and decode give what attention over the whole gives."""
    Hq, Hk, D, P, N = 8, 2, 128, 16, 3
    total = [70, 41, 90]
    x = [projected(L, Hq, Hk, D, dtype, 30 + n) for n, L in enumerate(total)]
    freq, m = kda.rope_inv_freq(D, device="cuda")
    w = [torch.rand(D, generator=torch.Generator().manual_seed(i)).cuda() + 0.5 for i in range(2)]
    kc, vc = (torch.full((40, Hk, P, D), NAN, dtype=dtype, device="cuda") for _ in range(2))
    table, lens, taken = torch.full((N, 8), -1, dtype=torch.int32, device="cuda"), ints([0] * N), ints([0])
    free = torch.randperm(40, generator=torch.Generator().manual_seed(1)).int().cuda()
    outs = [[] for _ in range(N)]
    at = [0] * N
    for new in ([40, 41, 1], [28, 0, 87], [1, 0, 1], [1, 0, 1]):
        cu = ints(offsets(new))
        pick = lambda i: torch.cat([x[n][i][at[n]:at[n] + new[n]] for n in range(N)])
        lens, pos, slots, taken = kda.kda_page_plan(lens, cu, table, free, P, sum(new), free_start=taken)
        q = kda.kda_qk_norm_rope_append(pick(0), pick(1), pick(2), pos, slots, kc, vc, freq, *w, rope_scale=m)
        o, _ = kda.kda_paged_prompt(q, kc, vc, table, lens, cu)
        for n in range(N):
            outs[n].append(o[int(cu[n]):int(cu[n + 1])])
            at[n] += new[n]
    assert at == total
    for n in range(N):
        pos = ints(list(range(total[n])))
        q, k = kda.kda_qk_norm_rope(x[n][0], x[n][1], pos, freq, *w, rope_scale=m)
        v = x[n][2]
        ref = attention.packed(f64(q), f64(k), f64(v), [0, total[n]], D ** -0.5)
        for h in range(Hq):
            r = ref[0, h]
            within(f64(torch.cat(outs[n])[:, h]), r.out, out_tol(r, dtype), (n, h))
        # the last token again, its first 32 tokens as a shared prefix of one
        last = q[-1:].contiguous()
        out, _ = kda.kda_paged_decode_shared(last, kc, vc, table[n:n + 1, :2].contiguous(), ints([32]), ints([0, 1]),
                                             table[n:n + 1, 2:].contiguous(), ints([total[n] - 32]))
        for h in range(Hq):
            within(f64(out[0, h]), ref[0, h].out[-1], out_tol(ref[0, h], dtype)[-1], (n, h))


def test_training_together():
    """norm and rotation, attention, and their backward as one chain, against differences."""
    T, Hq, Hk, D = 60, 4, 2, 64
    cu, pos = ints([0, 45, 60]), ints(list(range(45)) + list(range(15)))
    freq, _ = kda.rope_inv_freq(D, device="cuda")
    q, k, v = (x.contiguous() for x in projected(T, Hq, Hk, D, F32, 1))
    w = [torch.rand(D, generator=torch.Generator().manual_seed(i)).cuda() + 0.5 for i in range(2)]
    d = randn(T, Hq, D, seed=2)
    val = lambda q, k, v: (f64(kda.kda_attention_fwd(*kda.kda_qk_norm_rope(q, k, pos, freq, *w), v, cu)[0])
                           * f64(d)).sum()
    yq, yk = kda.kda_qk_norm_rope(q, k, pos, freq, *w)
    out, lse = kda.kda_attention_fwd(yq, yk, v, cu, want_lse=True)
    dq, dk, dv = kda.kda_attention_bwd(yq, yk, v, out, lse, d, cu)
    dq, dk, _, _ = kda.kda_qk_norm_rope_bwd(q, k, dq, dk, pos, freq, *w)
    z = [randn(*x.shape, seed=40 + i) for i, x in enumerate((q, k, v))]
    step = lambda t: val(q + t * z[0], k + t * z[1], v + t * z[2])
    got = sum((f64(a) * f64(b)).sum() for a, b in zip((dq, dk, dv), z))
    h = 2.0 ** -8
    d1, d2 = (step(h) - step(-h)) / (2 * h), (step(2 * h) - step(-2 * h)) / (4 * h)
    # as in test_backward_against_differences, with 15360 terms
    assert abs((4 * d1 - d2) / 3 - got) <= 15360 * h ** 4 + math.sqrt(15360) * 60 * U / h + 0.01 * abs(d1 - d2)
