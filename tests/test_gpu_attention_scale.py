"""Attention for several tokens at sizes past the other tests': training lengths, as many
sequences as a call may have, offsets past 32 bits.

References are plain computations in 64 bits on the device.  Bounds per element as in
test_gpu_attention (u = 2^-24, one rounding to BF16 2^-8), where a sum of n terms counts n u.  At
thousands of terms those are loose, so that long sequences are held to a bound in the L2 norm as
well: the result's rounding and the weights' (dS's), each uniform in up to 2^-8 of the value, are
2^-8 / sqrt(3) off, and as independent errors 0.82 * 2^-8 together; sums that the tensor core
truncates lose 6e-9 a term, 2^-12 at 32768.  FP32: the scores' rounding of up to 70 u * reach, here 2^-14."""
import math

import pytest
import torch

import kimi_delta_attention_10_gb300 as kda

from test_gpu_attention import BF16, F32, ROUND, U, WEIGHT, ints, offsets, projected, randn, run_fwd, status_word

pytestmark = pytest.mark.gpu


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (what, float((err / tol.clamp(min=1e-300)).max()))


def plain(q, k, v, dout, see, scale, dtype, two_parts):
    """Attention and its gradient of batches [.., tokens, D] in 64 bits, and bounds:
    ((out, its bound), lse, (dq, ..), (dk, ..), (dv, ..)).  see: which keys a row sees;
    two_parts: dS in two BF16 parts and delta from the weights."""
    q, k, v, dout = (x.double() for x in (q, k, v, dout))
    mT = lambda x: x.transpose(-1, -2)
    s = (scale * (q @ mT(k))).masked_fill(~see, -math.inf)
    reach = (scale * (q.abs() @ mT(k.abs()))).masked_fill(~see, 0.0).amax(-1, keepdim=True)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = (s - lse.nan_to_num(neginf=0.0)).exp()
    out = p @ v
    n = k.shape[-2]
    w = WEIGHT[dtype]
    out_e = (140 * U * reach + (90 + 2 * n) * U + w) * (p @ v.abs()) + ROUND[dtype] * out.abs()
    n += q.shape[-2]
    ep = 140 * U * reach + (20 + n) * U + 4 * U * lse.nan_to_num(neginf=0.0).abs()
    dp, dp_e = dout @ mT(v), 70 * U * (dout.abs() @ mT(v.abs()))
    delta = (p * dp).sum(-1, keepdim=True)
    if two_parts and dtype == BF16:
        delta_e = (p * (dp.abs() * (ep + n * U) + dp_e)).sum(-1, keepdim=True)
        w_ds = 2.0 ** -16
    else:
        delta_e = (130 * U * (dout * out).abs() + dout.abs() * out_e).sum(-1, keepdim=True)
        w_ds = w
    ds = p * (dp - delta)
    ds_e = p * (ep * (dp.abs() + delta.abs()) + dp_e + delta_e) + (w_ds + (4 + n) * U) * ds.abs()
    grads = [(scale * (ds @ k), scale * (ds_e @ k.abs())), (scale * (mT(ds) @ q), scale * (mT(ds_e) @ q.abs())),
             (mT(p) @ dout, mT(p * (ep + w + n * U)) @ dout.abs())]
    return (out, out_e), lse[..., 0], grads


def check(got, ref, bound, dtype, what):
    # 1.01: terms of second order
    within(got, ref, 1.01 * bound + ROUND[dtype] * ref.abs(), what)


def near(got, ref, dtype, what):
    e = float((got.double() - ref).norm() / ref.norm())
    assert e <= (2.0 ** -8 if dtype == BF16 else 2.0 ** -14), (what, e)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,Hq,Hk,D", [(8192, 2, 1, 128), (8191, 3, 1, 64), (16385, 1, 1, 64)])
def test_training_lengths(T, Hq, Hk, D, dtype):
    q, k, v = projected(T, Hq, Hk, D, dtype, T)
    dout = randn(T, Hq, D, seed=2, dtype=dtype)
    out, lse = run_fwd(q, k, v, [0, T])
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints([0, T]))
    see = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    want_k = want_v = bound_k = bound_v = 0.0
    wanted_q = []
    for h in range(Hq):
        (o, oe), l, g = plain(q[:, h], k[:, 0], v[:, 0], dout[:, h], see, D ** -0.5, dtype, False)
        within(out[:, h], o, oe, ("out", h))
        near(out[:, h], o, dtype, ("out", h))
        assert (lse[:, h] - l).abs().max() <= 2.0 ** -14
        check(grads[0][:, h], *g[0], dtype, ("dq", h))
        wanted_q.append(g[0][0])
        want_k, bound_k = want_k + g[1][0], bound_k + g[1][1]
        want_v, bound_v = want_v + g[2][0], bound_v + g[2][1]
        del g, o, oe
    near(grads[0], torch.stack(wanted_q, 1), dtype, "dq")
    for x, w, b, what in ((grads[1], want_k, bound_k, "dk"), (grads[2], want_v, bound_v, "dv")):
        more = Hq * U * w.abs().max()
        check(x[:, 0], w, b + more, dtype, what)
        near(x[:, 0], w, dtype, what)


def rows_of(lens, width):
    """[N, width] packed rows of sequences, and which places hold one."""
    c = torch.tensor(offsets(lens)[:-1], device="cuda")[:, None] + torch.arange(width, device="cuda")
    held = torch.arange(width, device="cuda") < torch.tensor(lens, device="cuda")[:, None]
    return c.clamp(max=max(0, sum(lens) - 1)), held


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,most,Hq,Hk,D", [(2500, 5, 4, 2, 64), (1 << 16, 2, 2, 1, 128), (300, 9, 3, 1, 128)])
def test_every_element_of_thousands_of_sequences(N, most, Hq, Hk, D, dtype):
    """Up to as many sequences as a call may have, each element against its own bound; the same
    tokens over pages."""
    g = torch.Generator().manual_seed(N)
    lens = torch.randint(0, most + 1, (N,), generator=g).tolist()
    cu, T, G = offsets(lens), sum(lens), Hq // Hk
    q, k, v = (x.contiguous() for x in projected(T, Hq, Hk, D, dtype, 7))
    dout = randn(T, Hq, D, seed=8, dtype=dtype)
    out, lse = run_fwd(q, k, v, cu)
    st = status_word()
    gq, gk, gv = kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu), status=st)
    assert int(st[0]) == 0
    at, held = rows_of(lens, most)
    see = torch.ones(most, most, dtype=torch.bool, device="cuda").tril() & held[:, None, None, :]
    pick = lambda x, H: (x[at] * held[..., None, None]).transpose(1, 2).repeat_interleave(Hq // H, 1)
    back = lambda x: x.transpose(1, 2)[held]
    (o, oe), l, grads = plain(pick(q, Hq), pick(k, Hk), pick(v, Hk), pick(dout, Hq), see, D ** -0.5, dtype, True)
    within(out, back(o), back(oe), "out")
    (dq, tq), (dk, tk), (dv, tv) = grads
    check(gq, back(dq), back(tq), dtype, "dq")
    group = lambda x: x.unflatten(1, (Hk, G)).sum(2)
    for x, w, t, what in ((gk, dk, tk, "dk"), (gv, dv, tv, "dv")):
        check(x, back(group(w)), back(group(t + G * U * w.abs())), dtype, what)
    for x, w in ((out, back(o)), (gq, back(dq)), (gk, back(group(dk))), (gv, back(group(dv)))):
        near(x, w, dtype, "all")
    # over pages of 16
    slots = torch.randperm(N, generator=g).int().cuda()
    kc, vc = (torch.full((N, Hk, 16, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    n, i = held.nonzero(as_tuple=True)
    for cache, x in ((kc, k), (vc, v)):
        cache[slots[n].long(), :, i] = x
    paged, pl = kda.kda_paged_prompt(q, kc, vc, slots[:, None].contiguous(), ints(lens), ints(cu), want_lse=True,
                                     status=st)
    assert int(st[0]) == 0
    within(paged, back(o), back(oe), "paged")
    assert (pl - lse).abs().max() <= 2.0 ** -14


def cuda_randn(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda", dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_packed_rows_past_2_to_the_31_elements(dtype):
    """The last sequences of a batch whose queries are more than 2^31 elements give the bits that
    they give alone."""
    L, Hq, Hk, D = 512, 64, 8, 128
    N = 2 ** 31 // (L * Hq * D) + 3
    T = N * L
    q, dout = (cuda_randn(T, Hq, D, seed=s, dtype=dtype) for s in (1, 2))
    k, v = (cuda_randn(T, Hk, D, seed=s, dtype=dtype) for s in (3, 4))
    assert q.numel() > 2 ** 31
    cu = ints([L * n for n in range(N + 1)])
    st = status_word()
    out, lse = kda.kda_attention_fwd(q, k, v, cu, want_lse=True, status=st)
    grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, cu, status=st)
    assert int(st[0]) == 0
    for first in (0, N - 4):
        rows, cut = slice(first * L, (first + 4) * L), ints([L * n for n in range(5)])
        a, al = kda.kda_attention_fwd(q[rows], k[rows], v[rows], cut, want_lse=True)
        ag = kda.kda_attention_bwd(q[rows], k[rows], v[rows], a, al, dout[rows], cut)
        assert torch.equal(a, out[rows]) and torch.equal(al, lse[rows])
        assert all(torch.equal(x, y[rows]) for x, y in zip(ag, grads))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pages_past_2_to_the_31_elements(dtype):
    """Pages at both ends of a cache of more than 2^31 elements give the bits of a small cache."""
    Hk, D, P, pages = 8, 128, 64, 33000
    small = [cuda_randn(16, Hk, P, D, seed=s, dtype=dtype) for s in (1, 2)]
    where = torch.tensor([*range(8), *range(pages - 8, pages)], device="cuda")
    large = [torch.empty(pages, Hk, P, D, dtype=dtype, device="cuda") for _ in range(2)]
    assert large[0].numel() > 2 ** 31
    for a, b in zip(small, large):
        b[where] = a
    table = torch.tensor([[0, 15, 9, 3], [14, 1, 8, 2], [10, 4, 11, 12]], dtype=torch.int32, device="cuda")
    far = where.int()[table.long()].contiguous()
    lens, cu = ints([256, 190, 77]), ints([0, 100, 101, 130])
    q = cuda_randn(130, 16, D, seed=3, dtype=dtype)
    st = status_word()
    a = kda.kda_paged_prompt(q, *small, table, lens, cu, want_lse=True, status=st)
    b = kda.kda_paged_prompt(q, *large, far, lens, cu, want_lse=True, status=st)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    shared = lambda caches, t: kda.kda_paged_decode_shared(
        q[:6], *caches, t, lens, ints([0, 3, 5, 6]), t[[0, 1, 2, 0, 1, 2]].contiguous(), ints([5, 0, 200, 64, 1, 9]),
        want_lse=True, status=st)
    a, b = shared(small, table), shared(large, far)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and int(st[0]) == 0
