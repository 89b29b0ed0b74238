"""Serving a small hybrid stack: a KDA layer and a full-attention layer.

Prompts of different lengths are taken in one packed call each layer, then every
request gets one token a step.  The KDA layer carries a state of fixed size
(kda_chunk_fwd_gated, then kda_gate and kda_recurrent_step); the attention layer keeps
keys and values in pages: kda_page_plan finds their places from the lengths on the
device, kda_qk_norm_rope_append norms, rotates and writes them, kda_paged_decode attends.
Nothing of a step comes back to the host, so the step is one CUDA graph.

    python examples/hybrid_decode.py [--requests 8] [--steps 32]

The attention layer is the last one here: of a prompt it attends for the last token only,
which is what kda_paged_decode does.  A layer above it would need all of them, which
kda_paged_prompt gives.

Weights and inputs are random: the program shows the calls, and checks that going token
by token gives what one long prompt gives.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import kimi_delta_attention_10_gb300 as kda  # noqa: E402

H, K = 4, 128                  # KDA heads and channels
HQ, HK, D = 8, 2, 64           # attention: query heads, key-value heads, channels
WIDTH = H * K
PAGE = 16


class Hybrid:
    """The two layers' weights."""

    def __init__(self, dtype=torch.float32, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        mat = lambda i, o: (torch.randn(i, o, generator=gen) * i ** -0.5).to(device, dtype)
        self.kda_in, self.kda_f, self.kda_b = mat(WIDTH, 3 * H * K), mat(WIDTH, H * K), mat(WIDTH, H)
        self.kda_out = mat(H * K, WIDTH)
        self.A_log = (torch.rand(H, generator=gen) * 1.4).to(device)
        self.dt_bias = (torch.randn(H, K, generator=gen) * 0.5).to(device)
        self.attn_in, self.attn_out = mat(WIDTH, (HQ + 2 * HK) * D), mat(HQ * D, WIDTH)
        self.q_weight = (torch.rand(D, generator=gen) + 0.5).to(device)
        self.k_weight = (torch.rand(D, generator=gen) + 0.5).to(device)
        self.inv_freq, self.rope_scale = kda.rope_inv_freq(D, device=device)
        self.dtype, self.device = dtype, device


class Server:
    """N requests: their KDA states, their pages, and the lengths, all on the device."""

    def __init__(self, model: Hybrid, requests: int, max_len: int):
        self.m, self.N = model, requests
        i32 = dict(dtype=torch.int32, device=model.device)
        rows = -(-max_len // PAGE)
        self.state = torch.zeros(requests, H, K, K, dtype=torch.float32, device=model.device)
        self.k_cache, self.v_cache = torch.zeros(2, requests * rows, HK, PAGE, D, dtype=model.dtype,
                                                 device=model.device).unbind(0)
        self.table = torch.full((requests, rows), -1, **i32)
        self.free = torch.randperm(requests * rows).to(**i32)
        self.taken = torch.zeros(1, **i32)
        self.lens = torch.zeros(requests, **i32)
        self.status = torch.zeros(4, **i32)
        self.one_each = torch.arange(requests + 1, **i32)

    def attend(self, x, cu):
        """The attention layer on packed new tokens x [T, WIDTH]; the last token's output."""
        m = self.m
        lens, positions, slots, taken = kda.kda_page_plan(
            self.lens, cu, self.table, self.free, PAGE, x.shape[0], free_start=self.taken,
            status=self.status)
        self.lens.copy_(lens)
        self.taken.copy_(taken)
        qkv = (x @ m.attn_in).view(x.shape[0], HQ + 2 * HK, D)
        q = kda.kda_qk_norm_rope_append(
            qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], positions, slots, self.k_cache,
            self.v_cache, m.inv_freq, m.q_weight, m.k_weight, rope_scale=m.rope_scale,
            status=self.status)
        last = cu[1:].long() - 1
        o, _ = kda.kda_paged_decode(q[last], self.k_cache, self.v_cache, self.table, lens,
                                    status=self.status)
        return x[last] + o.view(self.N, HQ * D) @ m.attn_out

    def prompt(self, x, lengths):
        """Packed prompts x [sum(lengths), WIDTH]; each request's last output [N, WIDTH]."""
        m, T = self.m, x.shape[0]
        host = [0]
        for n in lengths:
            host.append(host[-1] + n)
        cu = torch.tensor(host, dtype=torch.int32, device=m.device)
        q, k, v = ((x @ m.kda_in).view(T, 3, H, K)[:, i].contiguous() for i in range(3))
        o, self.state = kda.kda_chunk_fwd_gated(
            q, k, v, (x @ m.kda_f).view(T, H, K), m.A_log, m.dt_bias, x @ m.kda_b, cu,
            mode="fp32_exact" if m.dtype == torch.float32 else "bf16_tc", initial_state=self.state,
            cu_seqlens_host=host)
        return self.attend(x + o.view(T, H * K) @ m.kda_out, cu)

    def step(self, x):
        """One token of each request, x [N, WIDTH]."""
        m, N = self.m, self.N
        q, k, v = ((x @ m.kda_in).view(N, 3, H, K)[:, i].contiguous() for i in range(3))
        g, beta = kda.kda_gate((x @ m.kda_f).view(N, H, K), m.A_log, m.dt_bias, x @ m.kda_b)
        o = kda.kda_recurrent_step(q, k, v, g, beta, self.state)
        return self.attend(x + o.view(N, H * K) @ m.kda_out, self.one_each)


def step_graph(server: Server):
    """(input buffer, output buffer, graph) of a step; the server is left as it was."""
    x = torch.zeros(server.N, WIDTH, dtype=server.m.dtype, device=server.m.device)
    kept = [t.clone() for t in (server.state, server.table, server.taken, server.lens)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        server.step(x)                       # set-up that a capture must not meet
    torch.cuda.current_stream().wait_stream(side)
    for t, old in zip((server.state, server.table, server.taken, server.lens), kept):
        t.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = server.step(x)
    return x, y, graph


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    model = Hybrid()
    lengths = [1 + 37 * n % 300 for n in range(a.requests)]
    x = [torch.randn(n + a.steps, WIDTH, device="cuda") for n in lengths]

    server = Server(model, a.requests, max(lengths) + a.steps)
    server.prompt(torch.cat([r[:n] for r, n in zip(x, lengths)]), lengths)
    buf, y, graph = step_graph(server)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(a.steps):
        buf.copy_(torch.stack([r[n + i] for r, n in zip(x, lengths)]))
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps

    whole = Server(model, a.requests, max(lengths) + a.steps)
    ref = whole.prompt(torch.cat(x), [n + a.steps for n in lengths])
    off = ((y - ref).norm() / ref.norm()).item()
    assert int(server.status[0]) == 0 and int(whole.status[0]) == 0
    print(f"{a.requests} requests, prompts of {min(lengths)} to {max(lengths)} tokens, {a.steps} steps: "
          f"{t * 1e6:.0f} us a step; last outputs token by token against one prompt: {off:.1e}")
    return off


if __name__ == "__main__":
    main()
