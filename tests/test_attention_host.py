"""Host-side checks of the entry points of attention for several tokens (no GPU, no kernel
launched): refusals of bad arguments, sizes of workspaces."""
import ctypes

import pytest
import torch

import kimi_delta_attention_10_gb300 as kda
from kimi_delta_attention_10_gb300 import _build, binding

INVALID, UNSUPPORTED, ALIGNMENT = (binding.KDA_ERR_INVALID_ARG, binding.KDA_ERR_UNSUPPORTED,
                                   binding.KDA_ERR_ALIGNMENT)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load_library()


def P(i):
    """A fake, 16-byte-aligned device address of its own, never dereferenced."""
    return 0x100000 * (i + 1)


MIS = P(0) + 4
ODD = P(0) + 2        # integer arrays need four bytes only
BIG = 1 << 50


def call(fn, args, **kw):
    args = dict(args)
    for k in kw:
        assert k in args, k
    args.update(kw)
    return fn(*args.values())


FWD = dict(q=P(0), q_stride=8 * 128, k=P(1), k_stride=2 * 128, v=P(2), v_stride=2 * 128, dtype=1,
           cu=P(3), N=2, T=10, Hq=8, Hk=2, D=128, scale=0.1, out=P(4), lse=P(5), ws=P(6), ws_bytes=BIG,
           status=P(7), stream=None)
SIZES = [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID),
    (dict(D=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(Hk=3), UNSUPPORTED), (dict(T=1 << 28), UNSUPPORTED),
    (dict(N=2 ** 31 - 1), UNSUPPORTED), (dict(dtype=2), INVALID)]
PACKED = [
    (dict(q_stride=8 * 128 - 8), INVALID), (dict(k_stride=0), INVALID), (dict(v_stride=-256), INVALID),
    (dict(q_stride=8 * 128 + 4), ALIGNMENT), (dict(k_stride=1 << 31), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cu=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=8), INVALID), (dict(q=MIS), ALIGNMENT), (dict(v=MIS), ALIGNMENT), (dict(cu=ODD), ALIGNMENT),
    (dict(ws=MIS), ALIGNMENT), (dict(status=ODD), ALIGNMENT), (dict(lse=MIS), ALIGNMENT)]


@pytest.mark.parametrize("kw,expect", SIZES + PACKED + [
    (dict(out=None), INVALID), (dict(out=P(0)), INVALID), (dict(out=P(2)), INVALID), (dict(lse=P(4)), INVALID),
    (dict(ws=P(4)), INVALID), (dict(ws=P(3)), INVALID), (dict(out=MIS), ALIGNMENT)])
def test_forward_refuses(lib, kw, expect):
    assert call(lib.kda_attention_fwd, FWD, **kw) == expect


BWD = dict(q=P(0), q_stride=8 * 128, k=P(1), k_stride=2 * 128, v=P(2), v_stride=2 * 128, dtype=0,
           out=P(4), lse=P(5), dout=P(8), cu=P(3), N=2, T=10, Hq=8, Hk=2, D=128, scale=0.1, q_grad=P(9),
           k_grad=P(10), v_grad=P(11), ws=P(6), ws_bytes=BIG, status=P(7), stream=None)


@pytest.mark.parametrize("kw,expect", SIZES + [(k, e) for k, e in PACKED if k != dict(q_stride=8 * 128 + 4)] + [
    (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(dout=None), INVALID), (dict(q_grad=None), INVALID),
    (dict(k_grad=None), INVALID), (dict(v_grad=None), INVALID), (dict(dout=MIS), ALIGNMENT),
    (dict(v_grad=MIS), ALIGNMENT), (dict(q_grad=P(8)), INVALID), (dict(k_grad=P(11)), INVALID),
    (dict(v_grad=P(4)), INVALID), (dict(ws=P(9)), INVALID), (dict(q_stride=8 * 128 + 2), ALIGNMENT)])
def test_backward_refuses(lib, kw, expect):
    assert call(lib.kda_attention_bwd, BWD, **kw) == expect


CACHE = [
    (dict(num_pages=-1), INVALID), (dict(page=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(page=4), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=2048), UNSUPPORTED),
    (dict(num_pages=1 << 26), UNSUPPORTED), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(cu=None), INVALID), (dict(out=None), INVALID),
    (dict(q=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=8), INVALID), (dict(kc=MIS), ALIGNMENT),
    (dict(table=ODD), ALIGNMENT), (dict(lens=ODD), ALIGNMENT), (dict(cu=ODD), ALIGNMENT), (dict(out=P(1)), INVALID),
    (dict(lse=P(0)), INVALID), (dict(ws=P(3)), INVALID)]
PROMPT = dict(q=P(0), q_stride=8 * 128, kc=P(1), vc=P(2), dtype=1, table=P(3), lens=P(8), cu=P(9), N=2, T=10,
              Hq=8, Hk=2, D=128, num_pages=40, page=16, max_pages=8, scale=0.1, out=P(4), lse=P(5), ws=P(6),
              ws_bytes=BIG, status=P(7), stream=None)


@pytest.mark.parametrize("kw,expect", SIZES + CACHE + [
    (dict(q_stride=8 * 128 - 8), INVALID), (dict(q_stride=8 * 128 + 4), ALIGNMENT)])
def test_prompt_refuses(lib, kw, expect):
    assert call(lib.kda_paged_prompt, PROMPT, **kw) == expect


SHARED = dict(q=P(0), kc=P(1), vc=P(2), dtype=1, ptable=P(10), plens=P(11), cu=P(9), groups=2, max_prefix=8,
              table=P(3), lens=P(8), N=10, Hq=8, Hk=2, D=128, num_pages=40, page=16, max_pages=8, scale=0.1,
              out=P(4), lse=P(5), ws=P(6), ws_bytes=BIG, status=P(7), stream=None)


@pytest.mark.parametrize("kw,expect", CACHE + [
    (dict(N=-1), INVALID), (dict(Hq=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(Hk=3), UNSUPPORTED),
    (dict(groups=-1), INVALID), (dict(max_prefix=0), INVALID), (dict(ptable=None), INVALID),
    (dict(plens=None), INVALID), (dict(ptable=ODD), ALIGNMENT), (dict(plens=ODD), ALIGNMENT), (dict(dtype=7), INVALID),
    (dict(out=P(10)), INVALID), (dict(N=1 << 28), UNSUPPORTED)])
def test_shared_refuses(lib, kw, expect):
    assert call(lib.kda_paged_decode_shared, SHARED, **kw) == expect


def test_nothing_to_do_is_fine(lib):
    """Without tokens nothing is looked at."""
    none = dict(out=None, ws=None, ws_bytes=0)
    assert call(lib.kda_attention_fwd, FWD, T=0, **none) == 0
    assert call(lib.kda_attention_fwd, FWD, N=0, **none) == 0
    assert call(lib.kda_attention_bwd, BWD, T=0, **none) == 0
    assert call(lib.kda_paged_prompt, PROMPT, T=0, **none) == 0
    assert call(lib.kda_paged_decode_shared, SHARED, N=0, **none) == 0
    assert call(lib.kda_paged_decode_shared, SHARED, groups=0, **none) == 0


def test_integer_arrays_may_be_slices(lib):
    """Looked at before the sizes of the workspace, which then refuses."""
    for fn, args, names in ((lib.kda_attention_fwd, FWD, ["cu"]), (lib.kda_attention_bwd, BWD, ["cu"]),
                            (lib.kda_paged_prompt, PROMPT, ["cu", "table", "lens"]),
                            (lib.kda_paged_decode_shared, SHARED, ["cu", "table", "lens", "ptable", "plens"])):
        assert call(fn, args, ws_bytes=8, **{n: args[n] + 4 for n in names}) == INVALID


def test_workspace_sizes(lib):
    n = ctypes.c_int64()
    for name, args in (("kda_attention", (1, 100, 4, 2, 64)), ("kda_attention_bwd", (1, 100, 4, 2, 64)),
                       ("kda_paged_prompt", (3, 100, 4, 2, 128)), ("kda_paged_decode_shared", (3, 2, 4, 2, 128))):
        fn = getattr(lib, name + "_workspace_size")
        assert fn(*args, None) == INVALID
        assert fn(*args, ctypes.byref(n)) == 0 and n.value >= 16
        assert fn(*args[:-1], 80, ctypes.byref(n)) == UNSUPPORTED
    # many rows need no pieces
    assert kda.attention_workspace_size(1, 32768, 64, 8) <= 256
    with pytest.raises(kda.KDAError):
        kda.attention_workspace_size(1, 10, 3, 2)


@pytest.mark.parametrize("name", ["kda_attention", "kda_attention_bwd", "kda_paged_prompt",
                                  "kda_paged_decode_shared"])
@pytest.mark.parametrize("first,second", [(0, 0), (0, 5), (3, 0)])
def test_workspace_sizes_of_nothing(lib, name, first, second):
    """No sequences, or no tokens: a size all the same."""
    n = ctypes.c_int64()
    assert getattr(lib, name + "_workspace_size")(first, second, 4, 2, 64, ctypes.byref(n)) == 0
    assert n.value >= 16


MANY = (1 << 16) + 1


@pytest.mark.parametrize("fn,args,kw", [
    ("kda_attention_fwd", FWD, dict(N=MANY)), ("kda_attention_bwd", BWD, dict(N=MANY)),
    ("kda_paged_prompt", PROMPT, dict(N=MANY)), ("kda_paged_decode_shared", SHARED, dict(groups=MANY)),
    # rows of 2^31 elements
    ("kda_paged_prompt", PROMPT, dict(T=1, Hq=1 << 24, q_stride=(1 << 31) - 8)),
    ("kda_paged_decode_shared", SHARED, dict(N=1, Hq=1 << 24))])
def test_sizes_beyond_the_indices(lib, fn, args, kw):
    assert call(getattr(lib, fn), args, **kw) == UNSUPPORTED


def test_binding_refuses_by_name(lib):
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    cu = z(2, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="q must be a CUDA tensor"):
        kda.kda_attention_fwd(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64), cu)
    with pytest.raises(TypeError, match="k must be"):
        kda.kda_attention_fwd(z(4, 2, 64), z(4, 1, 64, dtype=torch.bfloat16), z(4, 1, 64), cu)
    with pytest.raises(ValueError, match="q must have shape"):
        kda.kda_attention_fwd(z(4, 64), z(4, 1, 64), z(4, 1, 64), cu)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        kda.kda_attention_bwd(None, z(4, 1, 64), z(4, 1, 64), z(1), z(1), z(1), cu)
    with pytest.raises(ValueError, match="k_cache must have shape"):
        kda.kda_paged_prompt(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64), cu, cu, cu)
    with pytest.raises(ValueError, match="v_cache must have the shape"):
        kda.kda_paged_decode_shared(z(4, 2, 64), z(4, 1, 8, 64), z(4, 1, 16, 64), cu, cu, cu, cu, cu)
