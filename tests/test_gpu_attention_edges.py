"""Attention for several tokens at the edges of its documentation: offsets of any 32-bit
value, rows of padded batches, gradients through rows without weight, long sequences.
Tolerances and helpers are those of test_gpu_attention."""
import numpy as np
import numpy as np
import pytest
import torch

import kimi_delta_attention_10_gb300 as kda
from kimi_delta_attention_10_gb300.binding import KDA_ERR_DEVICE_ARG

from oracle import attention

from test_gpu_attention import (BF16, F32, ROUND, U, f64, grad_tols, ints, lse_tol, out_tol, paged_case, projected,
                                randn, run_fwd, status_word, within)

pytestmark = pytest.mark.gpu

LOWEST, HIGHEST = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cu", [
    [0, 5, LOWEST], [0, 1, LOWEST + 1], [0, 5, 10, LOWEST], [0, 10, 5, LOWEST], [0, 5, HIGHEST],
    [LOWEST, 5, 10], [0, LOWEST, 10], [0, HIGHEST, 10], [0, 5, HIGHEST, LOWEST],
    [0] * 200 + [5, LOWEST]])
def test_offsets_of_any_value_are_reported(cu, dtype):
    """A last offset so low that its sequence's length wraps to a positive number, and others
    far outside: the status, and no output of any entry point."""
    Hq, Hk, D, N = 4, 2, 64, len(cu) - 1
    q, k, v = projected(10, Hq, Hk, D, dtype, 1)
    full = lambda h: torch.full((10, h, D), 7.0, dtype=dtype, device="cuda")
    out, lse, st = full(Hq), torch.full((10, Hq), 7.0, device="cuda"), status_word()
    kda.kda_attention_fwd(q, k, v, ints(cu), out=out, lse=lse, status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG and (out == 7).all() and (lse == 7).all()
    st.zero_()
    g = [full(Hq), full(Hk), full(Hk)]
    kda.kda_attention_bwd(q, k, v, out, lse, full(Hq), ints(cu), q_grad=g[0], k_grad=g[1], v_grad=g[2],
                          status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG and all((x == 7).all() for x in g)
    st.zero_()
    kc, vc, table = paged_case([9] * N, Hk, D, 8, dtype, 1)
    kda.kda_paged_prompt(q, kc, vc, ints(table.tolist()), ints([9] * N), ints(cu), out=out, lse=lse, status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG and (out == 7).all() and (lse == 7).all()
    st.zero_()
    own = ints([[0, 1]] * 10)
    kda.kda_paged_decode_shared(q.contiguous(), kc, vc, ints(table.tolist()), ints([9] * N), ints(cu), own,
                                ints([9] * 10), out=out, lse=lse, status=st)
    assert int(st[0]) == KDA_ERR_DEVICE_ARG and (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("live,tail", [(3, 1), (3, 40), (3, 200), (140, 3), (0, 5)])
def test_shared_does_not_look_at_requests_behind_the_groups(live, tail, dtype):
    """A batch padded to a captured size: whatever the lengths and tables behind the last
    group hold, no status, the outputs there as they were, the others' bits the same."""
    Hq, Hk, D, P = 4, 2, 128, 16
    own = [7 * n % 50 for n in range(live)]
    kc, vc, table = paged_case([70] + own, Hk, D, P, dtype, 3)
    table = np.concatenate([table, np.full((tail, table.shape[1]), -1)])
    cu = [0, live // 2, live]
    q = randn(live + tail, Hq, D, seed=2, dtype=dtype)
    q[live:] = float("nan")
    results = []
    for behind in (0, 5, table.shape[1] * P, HIGHEST, LOWEST, -1):
        for entry in (-1, HIGHEST):
            t = table.copy()
            t[1 + live:] = entry
            st = status_word()
            out = torch.full((live + tail, Hq, D), 7.0, dtype=dtype, device="cuda")
            lse = torch.full((live + tail, Hq), 7.0, device="cuda")
            kda.kda_paged_decode_shared(q, kc, vc, ints(t[[0, 0]].tolist()), ints([70, 13]), ints(cu),
                                        ints(t[1:].tolist()), ints(own + [behind] * tail), out=out, lse=lse, status=st)
            assert int(st[0]) == 0 and (out[live:] == 7).all() and (lse[live:] == 7).all()
            results.append((out, lse))
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
    if live:
        alone, al = kda.kda_paged_decode_shared(
            q[:live].contiguous(), kc, vc, ints(table[[0, 0]].tolist()), ints([70, 13]), ints(cu),
            ints(table[1:1 + live].tolist()), ints(own), want_lse=True)
        # fewer requests may be split otherwise: the same values to their rounding
        torch.testing.assert_close(alone.float(), results[0][0][:live].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
        torch.testing.assert_close(al, results[0][1][:live], rtol=1e-5, atol=1e-5)
        # and a bad length of a request that has a group is reported
        st = status_word()
        kda.kda_paged_decode_shared(q, kc, vc, ints(table[[0, 0]].tolist()), ints([70, 13]), ints(cu),
                                    ints(table[1:].tolist()), ints(own[:-1] + [-1] + [0] * tail), status=st)
        assert int(st[0]) == KDA_ERR_DEVICE_ARG


def fine_tols(r, dout):
    """(ds, dq, dk) and tolerances of one head's rows whose dS goes in as two BF16 parts (2^-16 of
    it left) and whose delta is the sum of P dP: FP32 otherwise, roundings as in grad_tols."""
    n = len(r.k) + len(r.q)
    d, v = np.abs(dout), np.abs(r.v)
    lse = np.abs(np.where(np.isfinite(r.lse), r.lse, 0.0))[:, None]
    ep = 140 * U * r.reach.max(1, initial=0.0)[:, None] + (20 + n) * U + 4 * U * lse
    dp, dp_e = dout @ r.v.T, 70 * U * (d @ v.T)
    delta_e = (r.p * (np.abs(dp) * (ep + n * U) + dp_e)).sum(1, keepdims=True)
    dq, dk, _, ds = r.grads(dout)
    delta = (r.p * dp).sum(1, keepdims=True)
    ds_e = r.p * (ep * (np.abs(dp) + np.abs(delta)) + dp_e + delta_e) + (2.0 ** -16 + (4 + n) * U) * np.abs(ds)
    s = abs(r.scale)
    return (dq, s * (ds_e @ np.abs(r.k))), (dk, s * (ds_e.T @ np.abs(r.q)))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 16, 43])
@pytest.mark.parametrize("L", [1, 2, 43, 126, 127, 128])
def test_gradients_of_up_to_128_keys_lose_nothing_to_the_rounding_of_ds(L, G):
    """Heads with opposite queries and the same dout: dk is the small difference of their sums, so
    that one rounding of dS to BF16 would be a few per cent of it."""
    D, cu = 128, [0, L]
    _, k, v = projected(L, 1, 1, D, BF16, 5)
    x = randn(L, 1, D, seed=6, dtype=BF16) * 0.125
    q = torch.cat([x if h % 2 == 0 else -x for h in range(G)], 1).contiguous()
    dout = randn(L, 1, D, seed=7, dtype=BF16).expand(L, G, D).contiguous()
    out, lse = run_fwd(q, k, v, cu)
    st = status_word()
    gq, gk, _ = (f64(g) for g in kda.kda_attention_bwd(q, k, v, out, lse, dout, ints(cu), status=st))
    assert int(st[0]) == 0
    dk_sum, tol_sum = 0.0, 0.0
    for (_, h), r in attention.packed(f64(q), f64(k), f64(v), cu, D ** -0.5).items():
        (dq, tq), (dk, tk) = fine_tols(r, f64(dout[:, h]))
        # 1.01: terms of second order
        within(gq[:, h], dq, 1.01 * tq + ROUND[BF16] * np.abs(dq), ("dq", h))
        # the heads share the sums
        dk_sum, tol_sum = dk_sum + dk, tol_sum + tk + G * U * np.abs(dk)
    within(gk[:, 0], dk_sum, 1.01 * tol_sum + ROUND[BF16] * np.abs(dk_sum), "dk")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.125, -0.125])
@pytest.mark.parametrize("D", [64, 128])
def test_gradients_through_rows_without_weight(D, scale, dtype):
    """The first keys' scores are -infinity for every row, so that the first rows have no weight at
    all: they add nothing to dk and dv, and the other rows' gradients are those without these keys.
    The channel that holds the infinities is left out of dq (zero times infinity, in the formula too)."""
    T, H, bad = 300, 2, 5
    q, k, v = (x.contiguous() for x in projected(T, H, 1, D, dtype, 12))
    q[..., 0] = 1.0
    k[:bad, :, 0] = -np.inf if scale > 0 else np.inf
    dout = randn(T, H, D, seed=1, dtype=dtype)
    out, lse = run_fwd(q, k, v, [0, T], scale=scale)
    assert (out[:bad] == 0).all() and (lse[:bad] == -np.inf).all()
    gq, gk, gv = (f64(g) for g in kda.kda_attention_bwd(q, k, v, out, lse, dout, ints([0, T]), scale))
    assert (gq[:bad, :, 1:] == 0).all() and (gk[:bad] == 0).all() and (gv[:bad] == 0).all()
    d = f64(dout)[bad:]
    sums = [0.0] * 4
    for h in range(H):
        r = attention.Rows(f64(q[bad:, h]), f64(k[bad:, 0]), f64(v[bad:, 0]), np.arange(T - bad) + 1, scale)
        dq, dk, dv, _ = r.grads(d[:, h])
        tq, tk, tv = grad_tols(r, d[:, h], dtype, out_tol(r, dtype))
        # 1.01: terms of second order
        within(gq[bad:, h, 1:], dq[:, 1:], (1.01 * tq + ROUND[dtype] * np.abs(dq))[:, 1:], ("dq", h))
        sums = [a + b for a, b in zip(sums, (dk, tk, dv, tv))]
    dk, tk, dv, tv = sums
    more = H * U * (np.abs(dk).max() + np.abs(dv).max())
    within(gk[bad:, 0], dk, 1.01 * tk + more + ROUND[dtype] * np.abs(dk), "dk")
    within(gv[bad:, 0], dv, 1.01 * tv + more + ROUND[dtype] * np.abs(dv), "dv")


REACH = 255


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,at,Hq,Hk,D", [(900, 600, 4, 1, 64), (900, 513, 2, 2, 128), (700, 383, 3, 1, 64),
                                          (600, 300, 1, 1, 128)])
@pytest.mark.parametrize("what", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_how_far_one_token_reaches(what, bad, T, at, Hq, Hk, D, dtype):
    """NaN or an infinity in one token.  Everything that neither sees it nor is seen by it, and
    lies past the documented 255 tokens, keeps its bits; what the formula makes of it is no number."""
    q, k, v = (x.contiguous() for x in projected(T, Hq, Hk, D, dtype, 9))
    dout, cu = randn(T, Hq, D, seed=10, dtype=dtype), ints([0, T])
    x = dict(q=q, k=k, v=v, dout=dout)

    def step(out=None, lse=None):
        if out is None:
            out, lse = run_fwd(x["q"], x["k"], x["v"], [0, T])
        return [out, lse, *kda.kda_attention_bwd(x["q"], x["k"], x["v"], out, lse, x["dout"], cu)]

    clean = step()
    x[what] = x[what].clone()
    x[what][at] = bad
    dirty = step()
    # rows that see the token, or share its tile, may differ; queries up to 255 before it
    rows = slice(0, at - REACH) if what in "kv" else slice(0, at)
    for a, b in zip(clean[:3], dirty[:3]):
        assert torch.equal(a[rows], b[rows])
    if what in ("q", "dout"):
        for a, b in zip(clean[:3], dirty[:3]):
            assert torch.equal(a[at + 1:], b[at + 1:])
        # keys that the token does not see, past the reach
        for a, b in zip(clean[3:], dirty[3:]):
            assert torch.equal(a[at + REACH + 1:], b[at + REACH + 1:])
        assert not dirty[2][at].isfinite().any()
    elif np.isnan(bad):
        out, lse, dq = dirty[:3]
        assert out[at:].isnan().all() and dq[at:].isnan().all()
        assert lse[at:].isnan().all() if what == "k" else torch.equal(lse, clean[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("prefix,page", [([40, 300], 16), ([2000, 9], 64)])
def test_keys_without_weight_over_pages(prefix, page, dtype):
    """Scores of -infinity over a prefix, over a request's own tokens, over both: as if those keys
    were not there, zeros and lse -infinity where none is left.  A NaN reaches its group alone."""
    Hq, Hk, D, own, cu = 6, 2, 128, [9, 0, 130, 1], [0, 2, 4]
    scale = D ** -0.5
    kc, vc, table = paged_case(prefix + own, Hk, D, page, dtype, 4)
    q = randn(4, Hq, D, seed=5, dtype=dtype)
    q[..., 0] = 1.0
    pt, ot = ints(table[:2].tolist()), ints(table[2:].tolist())

    def pages_of(rows):
        ids = table[rows]
        return torch.tensor(ids[ids >= 0], device="cuda", dtype=torch.long)

    def shared(k):
        st = status_word()
        out, lse = kda.kda_paged_decode_shared(q, k, vc, pt, ints(prefix), ints(cu), ot, ints(own), want_lse=True,
                                               status=st)
        assert int(st[0]) == 0
        return out, lse

    def prompt(k, rows, lens):
        return kda.kda_paged_prompt(q, k, vc, ints(table[rows].tolist()), ints(lens), ints([0, 1, 2, 3, 4]),
                                    want_lse=True)

    clean = shared(kc)
    for rows, prefixes, owns in (([0], [0, prefix[1]], own), ([2, 3, 4, 5], prefix, [0] * 4),
                                 (list(range(6)), [0, 0], [0] * 4)):
        k = kc.clone()
        k[pages_of(rows), :, :, 0] = -np.inf
        out, lse = shared(k)
        ref = attention.decode_shared(f64(q), f64(kc), f64(vc), table[:2], prefixes, cu, table[2:], owns, scale)
        for (n, h), r in ref.items():
            within(f64(out[n, h]), r.out[0], out_tol(r, dtype)[0], (n, h))
            assert lse[n, h] == -np.inf if len(r.k) == 0 else abs(float(lse[n, h]) - r.lse[0]) <= lse_tol(r)[0]
        if owns == [0] * 4:
            # the same keys for prompts of one token
            po, pl = prompt(k, [2, 3, 4, 5], own)
            assert (po == 0).all() and (pl == -np.inf).all()
    k = kc.clone()
    k[int(table[0, 0]), :, 3] = np.nan
    out, lse = shared(k)
    assert out[:2].isnan().all() and lse[:2].isnan().all()
    assert torch.equal(out[2:], clean[0][2:]) and torch.equal(lse[2:], clean[1][2:])
