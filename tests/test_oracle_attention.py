"""What pins the FP64 oracle of attention for several tokens: closed forms, differences, and
the one-token oracle."""
import numpy as np

from oracle import attention, paged


def case(T, Hq, Hk, D, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((T, Hq, D)), r.standard_normal((T, Hk, D)), r.standard_normal((T, Hk, D))


def test_equal_scores_give_running_means():
    q, k, v = case(9, 2, 1, 4)
    got = attention.packed(np.zeros_like(q), k, v, [0, 4, 9], 0.5)
    for (n, h), r in got.items():
        a, b = ((0, 4), (4, 9))[n]
        want = np.cumsum(v[a:b, 0], 0) / np.arange(1, b - a + 1)[:, None]
        assert np.allclose(r.out, want, atol=1e-14)
        assert np.allclose(r.lse, np.log(np.arange(1, b - a + 1)), atol=1e-14)


def test_last_token_is_the_decode_oracle():
    q, k, v = case(13, 6, 2, 8)
    r = attention.packed(q, k, v, [0, 13], 0.3)
    cache = lambda x: x.transpose(1, 0, 2)[None]
    out, lse, _, _ = paged.paged_decode(q[12:], cache(k), cache(v), [[0]], [13], 0.3)
    for h in range(6):
        assert np.allclose(r[0, h].out[-1], out[0, h], atol=1e-14)
        assert np.isclose(r[0, h].lse[-1], lse[0, h], atol=1e-14)


def test_gradients_are_differences():
    q, k, v = (x[:, 0] for x in case(7, 1, 1, 5))
    r = np.random.default_rng(1)
    d = r.standard_normal((7, 5))
    seen = np.arange(7) + 1
    grads = attention.Rows(q, k, v, seen, 0.7).grads(d)
    for i, g in enumerate(grads[:3]):
        w = r.standard_normal(g.shape)
        val = lambda t: (attention.Rows(*(x + t * w if i == n else x for n, x in enumerate((q, k, v))),
                                        seen, 0.7).out * d).sum()
        h = 1e-5
        assert abs((val(h) - val(-h)) / (2 * h) - (g * w).sum()) < 1e-8


def test_rows_without_keys_and_pages():
    q, k, v = (x[:, 0] for x in case(3, 1, 1, 4))
    r = attention.Rows(q, k, v, [-1, 0, 2], 1.0)
    assert (r.out[:2] == 0).all() and (r.lse[:2] == -np.inf).all() and np.isfinite(r.lse[2])
    cache = np.arange(4 * 2 * 3 * 1.0).reshape(4, 2, 3, 1)
    assert attention.pages(cache, [2, 0], 4, 1).ravel().tolist() == [15, 16, 17, 3]
    assert attention.pages(cache, [-1], 0, 1).shape == (0, 1)
    # a prompt's pieces over pages are the same rows as the whole
    q, k, v = case(11, 4, 2, 8)
    whole = attention.packed(q, k, v, [0, 11], 0.4)
    kc, vc = (np.pad(x, ((0, 1), (0, 0), (0, 0))).reshape(3, 4, 2, 8).transpose(0, 2, 1, 3) for x in (k, v))
    part = attention.paged_prompt(q[6:], kc, vc, np.array([[0, 1, 2]]), [11], [0, 5], 0.4)
    for h in range(4):
        assert np.allclose(part[0, h].out, whole[0, h].out[6:], atol=1e-14)
    shared = attention.decode_shared(q[10:], kc, vc, np.array([[0]]), [4], [0, 1], np.array([[1, 2]]), [7], 0.4)
    for h in range(4):
        assert np.allclose(shared[0, h].out, whole[0, h].out[10:], atol=1e-14)
