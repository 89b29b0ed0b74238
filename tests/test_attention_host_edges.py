"""Refusals of attention for several tokens at the ends of the arguments' types (no GPU, no
kernel launched)."""
import ctypes

import pytest

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
