"""Refusals of attention for several tokens at the ends of the arguments' types (no GPU, no
kernel launched)."""
import ctypes

import pytest

from kimi_delta_attention_10_gb300 import binding

from test_attention_host import BWD, FWD, PROMPT, UNSUPPORTED, call, lib  # noqa: F401

LONGEST = (1 << 63) - 1


@pytest.mark.parametrize("T", [LONGEST, LONGEST - 1, 1 << 62, 1 << 32, (1 << 32) + 10, 1 << 31])
@pytest.mark.parametrize("N", [1, 2, 1 << 16])
def test_tokens_beyond_the_indices(lib, T, N):  # noqa: F811
    """T + N must not wrap, nor T be cut to 32 bits."""
    n = ctypes.c_int64(-1)
    for name in ("kda_attention", "kda_attention_bwd", "kda_paged_prompt"):
        assert getattr(lib, name + "_workspace_size")(N, T, 1, 1, 64, ctypes.byref(n)) == UNSUPPORTED
    assert n.value == -1
    for fn, args in ((lib.kda_attention_fwd, FWD), (lib.kda_attention_bwd, BWD), (lib.kda_paged_prompt, PROMPT)):
        # a workspace of no bytes: what passed the sizes is refused before any launch
        assert call(fn, args, N=N, T=T, ws_bytes=-1) == UNSUPPORTED


def test_hooks_of_lost_arrivals(lib):  # noqa: F811
    """The kernels that the test hook can name, and no other number."""
    known = {getattr(binding, x) for x in dir(binding) if x.startswith("KDA_TEST_FAULT_")}
    try:
        for where in range(-2, 40):
            assert lib.kda_test_set_fault(where) == (binding.KDA_OK if where in known else binding.KDA_ERR_INVALID_ARG)
    finally:
        assert lib.kda_test_set_fault(binding.KDA_TEST_FAULT_NONE) == binding.KDA_OK
