"""Host-side checks of the paged-attention entry points (no GPU, no kernel
launched): refusals of bad arguments, and the frequencies of a rotation."""
import ctypes
import math
import os

import numpy as np
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


def call(fn, args, **kw):
    args = dict(args)
    for k in kw:
        assert k in args, k
    args.update(kw)
    return fn(*args.values())


PLAN = dict(cached=P(0), cu=P(1), N=2, T=10, page=16, table=P(2), max_pages=4, free=P(3),
            num_free=8, free_start=None, seq_lens=P(4), positions=P(5), slots=P(6),
            free_end=P(7), status=None, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(page=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_free=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED),
    (dict(N=0), INVALID), (dict(cached=None), INVALID), (dict(cu=None), INVALID),
    (dict(table=None), INVALID), (dict(free=None), INVALID), (dict(seq_lens=None), INVALID),
    (dict(positions=None), INVALID), (dict(slots=None), INVALID), (dict(free_end=None), INVALID),
    (dict(cached=P(0) + 2), ALIGNMENT), (dict(free_start=P(0) + 1), ALIGNMENT),
    (dict(status=P(0) + 2), ALIGNMENT), (dict(slots=MIS), ALIGNMENT),
    (dict(seq_lens=P(0)), INVALID), (dict(free_start=P(7)), INVALID), (dict(slots=P(5)), INVALID),
])
def test_plan_refuses(lib, kw, expect):
    assert call(lib.kda_page_plan, PLAN, **kw) == expect


ROPE = dict(q=P(0), q_stride=4 * 128, k=P(1), k_stride=2 * 128, x_dtype=1, positions=P(2),
            inv_freq=P(3), rot=128, interleaved=0, rope_scale=1.0, q_weight=P(4), k_weight=P(5),
            eps=1e-6, norm=1, T=10, Hq=4, Hk=2, D=128, q_out=P(6), k_out=P(7), out_dtype=1,
            stream=None)
ROPE_BAD = [
    (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(D=0), INVALID),
    (dict(rot=-16), INVALID), (dict(x_dtype=2), INVALID), (dict(interleaved=2), INVALID),
    (dict(norm=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(rot=8), UNSUPPORTED),
    (dict(rot=144), UNSUPPORTED), (dict(q_stride=4 * 128 - 8), INVALID),
    (dict(k_stride=0), INVALID), (dict(q_stride=4 * 128 + 4), ALIGNMENT), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(positions=None), INVALID), (dict(inv_freq=None), INVALID),
    (dict(q=MIS), ALIGNMENT), (dict(q_weight=MIS), ALIGNMENT), (dict(positions=MIS), ALIGNMENT),
]


@pytest.mark.parametrize("kw,expect", ROPE_BAD + [
    (dict(out_dtype=5), INVALID), (dict(q_out=None), INVALID), (dict(k_out=None), INVALID),
    (dict(k_out=MIS), ALIGNMENT), (dict(k_out=P(6)), INVALID), (dict(q_out=P(1)), INVALID),
    (dict(k_out=P(0)), INVALID),
    (dict(q_out=P(0), out_dtype=0), INVALID),              # in place, other type
    (dict(q_out=P(0), q_stride=5 * 128), INVALID),         # in place, not dense
])
def test_rope_refuses(lib, kw, expect):
    assert call(lib.kda_qk_norm_rope, ROPE, **kw) == expect


APPEND = dict(q=P(0), q_stride=4 * 128, k=P(1), k_stride=2 * 128, v=P(2), v_stride=2 * 128,
              x_dtype=1, positions=P(3), slots=P(4), inv_freq=P(5), rot=128, interleaved=0,
              rope_scale=1.0, q_weight=P(6), k_weight=P(7), eps=1e-6, norm=1, T=10, Hq=4, Hk=2,
              D=128, q_out=P(8), k_cache=P(9), v_cache=P(10), dtype=1, num_pages=4, page=16,
              status=None, stream=None)


@pytest.mark.parametrize("kw,expect", ROPE_BAD + [
    (dict(dtype=7), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
    (dict(q_out=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(num_pages=-1), INVALID), (dict(page=0), INVALID), (dict(v_stride=8), INVALID),
    (dict(v_stride=2 * 128 + 1), ALIGNMENT), (dict(slots=MIS), ALIGNMENT),
    (dict(status=MIS), ALIGNMENT), (dict(v_cache=P(9)), INVALID), (dict(q_out=P(9)), INVALID),
    (dict(k_cache=P(1)), INVALID), (dict(v_cache=P(2)), INVALID), (dict(k_cache=P(0)), INVALID),
    (dict(q_out=P(0), dtype=0), INVALID),
])
def test_append_refuses(lib, kw, expect):
    assert call(lib.kda_qk_norm_rope_append, APPEND, **kw) == expect


def rope_bwd_args(lib):
    out = ctypes.c_int64(-1)
    assert lib.kda_qk_norm_rope_bwd_workspace_size(10, 4, 2, 128, ctypes.byref(out)) == 0
    return dict(q=P(0), q_stride=4 * 128, k=P(1), k_stride=2 * 128, x_dtype=1, dq=P(2), dk=P(3),
                dy_dtype=1, positions=P(4), inv_freq=P(5), rot=128, interleaved=0, rope_scale=1.0,
                q_weight=P(6), k_weight=P(7), eps=1e-6, norm=1, T=10, Hq=4, Hk=2, D=128,
                q_grad=P(8), k_grad=P(9), grad_dtype=1, q_wgrad=P(10), k_wgrad=P(11), ws=P(12),
                ws_bytes=out.value, stream=None)


@pytest.mark.parametrize("kw,expect", ROPE_BAD + [
    (dict(dy_dtype=3), INVALID), (dict(grad_dtype=3), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(q_grad=None), INVALID), (dict(k_grad=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=64), INVALID), (dict(ws=MIS), ALIGNMENT),
    (dict(q_wgrad=MIS), ALIGNMENT), (dict(q_grad=P(0)), INVALID), (dict(q_grad=P(9)), INVALID),
    (dict(q_grad=P(3)), INVALID), (dict(q_grad=P(2), grad_dtype=0), INVALID),
    (dict(q_wgrad=P(11)), INVALID), (dict(q_wgrad=P(6)), INVALID), (dict(ws=P(8)), INVALID),
])
def test_rope_bwd_refuses(lib, kw, expect):
    assert call(lib.kda_qk_norm_rope_bwd, rope_bwd_args(lib), **kw) == expect


def test_rope_bwd_workspace_size_refuses(lib):
    out = ctypes.c_int64(0)
    f = lambda *a: lib.kda_qk_norm_rope_bwd_workspace_size(*a, ctypes.byref(out))
    assert f(-1, 1, 1, 128) == INVALID and f(1, 0, 1, 128) == INVALID
    assert f(1, 1, 1, 80) == UNSUPPORTED and f(1 << 31, 1, 1, 64) == UNSUPPORTED
    assert lib.kda_qk_norm_rope_bwd_workspace_size(1, 1, 1, 64, None) == INVALID


def decode_args(lib):
    out = ctypes.c_int64(-1)
    assert lib.kda_paged_decode_workspace_size(3, 4, 2, 128, ctypes.byref(out)) == 0
    return dict(q=P(0), k=P(1), v=P(2), dtype=1, table=P(3), lens=P(4), N=3, Hq=4, Hk=2, D=128,
                num_pages=9, page=16, max_pages=4, scale=0.1, out=P(5), out_dtype=1, lse=P(6),
                ws=P(7), ws_bytes=out.value, status=None, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(D=-1), INVALID),
    (dict(D=80), UNSUPPORTED), (dict(Hq=5), UNSUPPORTED), (dict(Hq=1 << 30), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(out_dtype=2), INVALID), (dict(num_pages=-1), INVALID),
    (dict(page=0), INVALID), (dict(max_pages=0), INVALID), (dict(page=24), UNSUPPORTED),
    (dict(page=4), UNSUPPORTED), (dict(page=2048), UNSUPPORTED),
    (dict(num_pages=1 << 27), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=100), INVALID),
    (dict(q=MIS), ALIGNMENT), (dict(table=MIS), ALIGNMENT), (dict(lse=MIS), ALIGNMENT),
    (dict(ws=MIS), ALIGNMENT), (dict(out=P(0)), INVALID), (dict(lse=P(5)), INVALID),
    (dict(ws=P(2)), INVALID),
])
def test_decode_refuses(lib, kw, expect):
    assert call(lib.kda_paged_decode, decode_args(lib), **kw) == expect


def test_decode_workspace_size_refuses(lib):
    out = ctypes.c_int64(0)
    f = lambda *a: lib.kda_paged_decode_workspace_size(*a, ctypes.byref(out))
    assert f(-1, 1, 1, 128) == INVALID and f(1, 3, 2, 128) == UNSUPPORTED
    assert lib.kda_paged_decode_workspace_size(1, 1, 1, 64, None) == INVALID


def test_nothing_to_do_is_accepted(lib):
    assert call(lib.kda_qk_norm_rope, ROPE, T=0, q=None, k=None, positions=None, q_out=None,
                k_out=None) == 0
    assert call(lib.kda_qk_norm_rope_append, APPEND, T=0, q=None, k=None, v=None) == 0
    assert call(lib.kda_paged_decode, decode_args(lib), N=0, q=None) == 0


# ---------------------------------------------------------------- binding
def test_binding_refuses_cpu_tensors_and_wrong_types():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="CUDA"):
        kda.kda_page_plan(i32(2), i32(3), i32(2, 4), i32(5), 16, 0)
    with pytest.raises(TypeError, match="cached_lens"):
        kda.kda_page_plan(torch.zeros(2), i32(3), i32(2, 4), i32(5), 16, 0)
    with pytest.raises(ValueError, match="block_table"):
        kda.kda_page_plan(i32(2), i32(3), i32(3, 4), i32(5), 16, 0)
    x = torch.zeros(3, 2, 64)
    with pytest.raises(RuntimeError, match="CUDA"):
        kda.kda_qk_norm_rope(x, x, i32(3), None)
    with pytest.raises(TypeError, match="k must be"):
        kda.kda_qk_norm_rope(x, x.bfloat16(), i32(3), None)
    c = torch.zeros(2, 2, 16, 64)
    with pytest.raises(ValueError, match="k_cache"):
        kda.kda_qk_norm_rope_append(x, x, x, i32(3), i32(3), torch.zeros(2, 1, 16, 64), c, None)
    with pytest.raises(ValueError, match="v_cache"):
        kda.kda_paged_decode(x, c, c.bfloat16(), i32(3, 1), i32(3))
    with pytest.raises(ValueError, match="block_table"):
        kda.kda_paged_decode(x, c, c, i32(2, 1), i32(3))
    with pytest.raises(TypeError, match="q must be"):
        kda.kda_paged_decode(x, c.bfloat16(), c.bfloat16(), i32(3, 1), i32(3),
                             workspace=torch.zeros(16))


def test_binding_refuses_tensors_of_two_devices(lib):
    """Before anything is allocated or launched; the tensors have a device and no memory."""
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    with fake.FakeTensorMode():
        on = lambda d, *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=f"cuda:{d}")
        i32 = lambda d, *s: on(d, *s, dtype=torch.int32)
        x, c = on(1, 3, 2, 64), on(1, 2, 2, 16, 64)
        two = pytest.raises(ValueError, match="one device, not cuda:1 and cuda:0")
        with two:
            kda.kda_page_plan(i32(1, 2), i32(1, 3), i32(0, 2, 4), i32(1, 5), 16, 0)
        with two:
            kda.kda_qk_norm_rope(x, x, i32(1, 3), None, q_weight=on(0, 64))
        with two:
            kda.kda_qk_norm_rope_append(x, x, x, i32(1, 3), on(1, 3, dtype=torch.int64), c, on(0, 2, 2, 16, 64), None)
        with two:
            kda.kda_qk_norm_rope_bwd(x, x, x, on(0, 3, 2, 64), i32(1, 3), None)
        with two:
            kda.kda_paged_decode(x, c, c, i32(1, 3, 1), i32(1, 3), workspace=on(0, 1 << 20))


# ---------------------------------------------------------------- frequencies
HALF = 2.0 ** -24      # one rounding to FP32; the FP64 work before it adds far less


def near(a, b):
    b = np.asarray(b)
    return np.all(np.abs(a.double().numpy() - b) <= HALF * 1.001 * np.abs(b))


def test_rope_inv_freq_of_each_scaling():
    i = np.arange(64)
    f = 1e4 ** (-i / 64)
    a, m = kda.rope_inv_freq(128)
    assert near(a, f) and m == 1.0
    assert near(kda.rope_inv_freq(128, scaling="linear", factor=4.0)[0], f / 4)
    a, m = kda.rope_inv_freq(128, scaling="ntk", factor=4.0)
    assert near(a, (1e4 * 4 ** (128 / 126)) ** (-i / 64)) and m == 1.0
    # the slowest channel of the changed base is the interpolated one
    assert abs(a[63].item() / (f[63] / 4) - 1) < 1e-6
    a, m = kda.rope_inv_freq(128, scaling="yarn", factor=4.0, original_len=4096)
    assert abs(m - (0.1 * math.log(4) + 1)) < 1e-7
    turns = 4096 * f / (2 * math.pi)
    fast, slow = turns > 32 * 1.4, turns < 1 / 1.4     # beyond the rounded ends of the ramp
    assert near(a[torch.from_numpy(fast)], f[fast]) and near(a[torch.from_numpy(slow)], f[slow] / 4)
    mid = a.double().numpy()[~fast & ~slow] / f[~fast & ~slow]
    assert (np.diff(mid) <= 1e-7).all() and mid[0] <= 1 + 1e-7 and mid[-1] >= 0.25 - 1e-7
    # the same method without stretching is the plain rotation
    a, m = kda.rope_inv_freq(64, 5e5, "yarn", 1.0, 8192)
    assert near(a, 5e5 ** (-np.arange(32) / 32)) and m == 1.0


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1., 1., 32., 1.), (7, 1e4, 0, 1., 1., 32., 1.), (64, 1.0, 0, 1., 1., 32., 1.),
    (64, 1e4, 4, 1., 1., 32., 1.), (64, 1e4, 1, 0.5, 1., 32., 1.), (2, 1e4, 2, 2., 1., 32., 1.),
    (64, 1e4, 3, 2., 0., 32., 1.), (64, 1e4, 3, 2., 4096., 1., 1.), (64, 1e4, 3, 2., 4096., 1., 0.),
    (64, math.nan, 0, 1., 1., 32., 1.), (64, 1e4, 1, math.nan, 1., 32., 1.)])
def test_rope_inv_freq_refuses(lib, args):
    buf, m = (ctypes.c_float * 64)(), ctypes.c_float()
    assert lib.kda_rope_inv_freq(*args, ctypes.addressof(buf), ctypes.addressof(m)) == INVALID
    assert lib.kda_rope_inv_freq(64, 1e4, 0, 1., 1., 32., 1., None, ctypes.addressof(m)) == INVALID


def test_marshalling_module_refuses_what_it_cannot_read(lib):
    m = binding._load_marshal()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(TypeError, match="arguments"):
        m.page_plan(1, 2)
    with pytest.raises(TypeError, match="cached_lens must be a torch.Tensor"):
        kda.kda_page_plan([1, 2], i32(3), i32(2, 4), i32(5), 16, 0)
    with pytest.raises(TypeError, match="num_tokens must be an integer"):
        kda.kda_page_plan(i32(2), i32(3), i32(2, 4), i32(5), 16, 1.5)
    x = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="q must have shape"):
        kda.kda_qk_norm_rope(x[0], x, i32(3), None)
    with pytest.raises(ValueError, match="k must have shape"):
        kda.kda_qk_norm_rope(x, x[0], i32(3), None)
    with pytest.raises(KeyError):
        m.bind({})
    binding._fast = None                       # bound again by the next call
    assert binding._load_marshal() is m


@pytest.mark.parametrize("original_len", [4096, 65536, 131072, 1 << 22])
def test_rope_inv_freq_yarn_ramp_written_out(original_len):
    """Every channel of the ramp, also where its slow end lies past the last pair: a pair that
    still turns more than beta_slow times is never interpolated whole."""
    pairs, theta, factor, fast, slow = 64, 1e4, 4.0, 32.0, 1.0
    # the (fractional) index of the pair that turns b times in original_len tokens
    index = lambda b: pairs * math.log(original_len / (2 * math.pi * b)) / math.log(theta)
    lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), 2 * pairs - 1)
    want = []
    for i in range(pairs):
        f = theta ** (-i / pairs)
        share = min(max((i - lo) / (hi - lo), 0.0), 1.0) if hi > lo else float(i > lo)
        want.append(f * (1 - share) + f / factor * share)
    a, _ = kda.rope_inv_freq(2 * pairs, theta, "yarn", factor, original_len, fast, slow)
    assert near(a, want)
    turns = original_len * theta ** (-np.arange(pairs) / pairs) / (2 * math.pi)
    kept = a.double().numpy() > theta ** (-np.arange(pairs) / pairs) / factor * (1 + 1e-6)
    assert kept[turns > slow * 1.0001].all() and not kept[turns < slow / 1.2].any()


@pytest.mark.parametrize("original_len", [0.5, 4.0, 6.0])
def test_rope_inv_freq_yarn_shorter_than_a_turn(original_len):
    """No pair turns once in the trained length: all take f / factor."""
    f = 1e4 ** (-np.arange(32) / 32)
    assert near(kda.rope_inv_freq(64, 1e4, "yarn", 4.0, original_len)[0], f / 4)


@pytest.mark.parametrize("what", ["torch", "interpreter"])
def test_marshalling_module_of_another_version_is_not_loaded(lib, monkeypatch, what):
    """It uses interfaces that change between versions: one that was compiled for others does
    not count as built, nor is it imported."""
    binding._load_marshal()
    assert os.path.exists(_build.marshal_path()) and _build.up_to_date()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    else:
        monkeypatch.setattr(_build.sys.implementation, "cache_tag", "cpython-000")
    assert not _build.up_to_date()
    monkeypatch.setattr(binding, "_fast", None)
    with pytest.raises(RuntimeError, match="build it with"):
        kda.kda_page_plan(*[torch.zeros(1)] * 4, 16, 0)


# ---------------------------------------------------------------- kernels, by their source
def test_decode_allocates_tensor_memory_after_its_wait():
    """A CTA that may start while the kernel before it runs holds no tensor memory while it
    waits: that kernel may signal first and allocate its own afterwards."""
    src = open(os.path.join(_build.CSRC, "kda_paged_decode_tc.cu")).read()
    body = src[src.index("paged_decode_tc_kernel(DecodeArgs"):]
    assert 0 < body.index("wait_for_previous();") < body.index("tmem_alloc(") < body.index("__syncthreads();")
