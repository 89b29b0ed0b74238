"""Bounded waits of attention's tensor-core kernels that run out, on purpose, through the
test hook: CTA 0 of one kernel never gives a place of its copies back, the copy that would take
it is waited for about a second, and the kernel reports KDA_ERR_TIMEOUT, lets its copies and products in
flight finish and returns without a CUDA error.  The next call gives exactly the bits of a call
before.  Nothing here traps or faults the GPU: the lost arrival is a flag that nothing sets, and
every wait on it is bounded."""
import pytest
import torch

import kimi_delta_attention_10_gb300 as kda
from kimi_delta_attention_10_gb300 import binding

from test_gpu_attention import BF16, ints, offsets, projected, randn, status_word

pytestmark = pytest.mark.gpu


# the first CTA has thirty tiles of keys or rows, so that it needs the lost place again; a
# second sequence gives other CTAs work
@pytest.mark.parametrize("lens,Hq,Hk,D", [([4000, 40], 8, 4, 64), ([4000, 40], 16, 8, 128)])
@pytest.mark.parametrize("where", [binding.KDA_TEST_FAULT_ATTENTION, binding.KDA_TEST_FAULT_ATTENTION_BWD_Q,
                                   binding.KDA_TEST_FAULT_ATTENTION_BWD_KV])
def test_lost_place_times_out_and_the_next_call_is_clean(where, lens, Hq, Hk, D):
    cu = ints(offsets(lens))
    T = sum(lens)
    q, k, v = projected(T, Hq, Hk, D, BF16, 3)
    dout = randn(T, Hq, D, seed=4, dtype=BF16)

    def step():
        st = status_word()
        out, lse = kda.kda_attention_fwd(q, k, v, cu, want_lse=True, status=st)
        grads = kda.kda_attention_bwd(q, k, v, out, lse, dout, cu, status=st)
        torch.cuda.synchronize()                 # raises if a kernel faulted
        return [out, lse, *grads], int(st[0])

    clean, st = step()
    assert st == 0
    binding.set_test_fault(where)
    try:
        _, st = step()
    finally:
        binding.set_test_fault(binding.KDA_TEST_FAULT_NONE)
    assert st == binding.KDA_ERR_TIMEOUT
    again, st = step()
    assert st == 0 and all(torch.equal(a, b) for a, b in zip(clean, again))
