"""Attention for several tokens at the edges of its documentation: offsets of any 32-bit
value, rows of padded batches, gradients through rows without weight, long sequences.
Tolerances and helpers are those of test_gpu_attention."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_10_gb300 as kda
from kimi_delta_attention_10_gb300.binding import KDA_ERR_DEVICE_ARG

from test_gpu_attention import BF16, F32, ints, paged_case, projected, randn, status_word

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
