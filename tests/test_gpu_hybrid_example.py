"""The hybrid serving example: a KDA layer and a paged attention layer, prompts then a
captured step, against the same tokens as one prompt."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(__file__), "..", "examples", "hybrid_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_decode", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_token_by_token_equals_one_prompt(example):
    # FP32 throughout: two layers of products over at most 512 terms, each mode of the KDA
    # layer within 1e-5 of the recurrence
    assert example.main(["--requests", "5", "--steps", "20"]) < 1e-4


def test_bf16_steps_without_a_graph(example):
    model = example.Hybrid(torch.bfloat16, seed=1)
    lengths, steps = [40, 1, 17], 18
    gen = torch.Generator().manual_seed(2)
    x = [torch.randn(n + steps, example.WIDTH, generator=gen).to("cuda", torch.bfloat16)
         for n in lengths]
    a = example.Server(model, 3, 64)
    a.prompt(torch.cat([r[:n] for r, n in zip(x, lengths)]), lengths)
    for i in range(steps):
        y = a.step(torch.stack([r[n + i] for r, n in zip(x, lengths)]))
    b = example.Server(model, 3, 64)
    ref = b.prompt(torch.cat(x), [n + steps for n in lengths])
    assert int(a.status[0]) == 0 and int(b.status[0]) == 0
    assert a.lens.tolist() == [n + steps for n in lengths] == b.lens.tolist()
    # roundings to BF16 along the way: a handful of 2^-8 each, on sums of unit size
    assert (y.float() - ref.float()).norm() / ref.float().norm() < 8 * 2.0 ** -8


def test_running_out_of_pages_is_reported(example):
    model = example.Hybrid(torch.bfloat16)
    s = example.Server(model, 2, 32)
    s.free = s.free[:3]                            # two pages for request 0, one for request 1
    s.prompt(torch.randn(40, example.WIDTH, device="cuda").bfloat16(), [20, 20])
    assert int(s.status[0]) == example.kda.binding.KDA_ERR_NO_PAGES
    assert s.lens.tolist() == [20, 0]
