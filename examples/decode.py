"""Serving with the 4-bit step: prompts through a PLE layer and an attention
block, then single tokens, the step captured once in a CUDA graph.

    python examples/decode.py [--requests 64] [--prompt 500] [--steps 100]

Weights and tokens are random; hidden size and hash constants are those of the
tiny workload. Prints the time of the prompts, of a step, and what the cache
takes next to one in bf16.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from hashed_gram_embedding_gb300 import PLEAttention, PLELayer, pack_w4  # noqa: E402
from hashed_gram_embedding_gb300 import workloads as wl  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE, GROUP = 16, 4, 128, 16, 128


def rotation(positions, dim):
    angle = torch.arange(positions)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2) / dim)
    return torch.cat((angle.cos(), angle.sin()), 1).float().cuda()


def random_w4(rows, columns):
    return pack_w4(torch.randn(rows, columns, device="cuda") * columns ** -0.5, GROUP)


def main():
    args = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    args.add_argument("--requests", type=int, default=64)
    args.add_argument("--prompt", type=int, default=500)
    args.add_argument("--steps", type=int, default=100)
    args = args.parse_args()
    R, P, total = args.requests, args.prompt, args.prompt + args.steps + 4
    torch.manual_seed(0)

    w = wl.WORKLOADS["tiny"]
    host = wl.host_inputs(w)
    dense = wl.dense_inputs(torch, w, "cuda")
    layer = PLELayer(*wl.make_table(torch, w, "cuda"), host["multipliers"][0], host["V"], host["O"],
                     w.eos_token_id, w.heads_per_ngram, dense["w_kv"], dense["gamma_h"], dense["gamma_k"],
                     dense["conv_w"], w.dilation)
    pages = -(-total // PAGE)
    block = PLEAttention(random_w4((HEADS + 2 * KV_HEADS) * DIM, w.hidden), random_w4(w.hidden, HEADS * DIM),
                         HEADS, KV_HEADS, DIM, R * pages, PAGE, R * P, cos_sin=rotation(total, DIM))
    block_table = torch.randperm(R * pages, device="cuda").to(torch.int32).view(R, pages)
    kv_lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    dev_err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # what the layer carries from step to step, in two buffers in turn
    reach = (w.conv_k - 1) * w.dilation
    context = [torch.full((R, w.ctx_len), w.eos_token_id, dtype=torch.int32, device="cuda") for _ in range(2)]
    state = [torch.zeros((R, reach, w.hidden), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step(ids, qsl, hidden, longest, turn):
        """hidden -> hidden, both parts added to it, in place."""
        hidden.add_(layer.forward(ids, qsl, hidden, ngram_context=context[turn], ngram_context_out=context[1 - turn],
                                  conv_state=state[turn], conv_state_out=state[1 - turn], dev_err=dev_err))
        hidden.add_(block.forward(hidden, block_table, qsl, kv_lens, max_query_len=longest, dev_err=dev_err))

    def tokens(n):
        return torch.randint(3, w.token_vocab, (n,), device="cuda", dtype=torch.int32)

    def timed(run):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        run()
        end.record()
        end.synchronize()
        return begin.elapsed_time(end)

    kv_lens.fill_(P)
    hidden = torch.randn(R * P, w.hidden, device="cuda").to(torch.bfloat16)
    qsl = torch.arange(0, R * P + 1, P, dtype=torch.int32, device="cuda")
    prompt_ms = timed(lambda: step(tokens(R * P), qsl, hidden, P, 0))
    hidden = hidden[P - 1::P].contiguous()

    ids, qsl = tokens(R), torch.arange(R + 1, dtype=torch.int32, device="cuda")

    def two_steps():
        for turn in (1, 0):
            kv_lens.add_(1)
            step(ids, qsl, hidden, 1, turn)

    two_steps()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        two_steps()
    torch.cuda.synchronize()
    pairs = (args.steps + 1) // 2
    step_ms = timed(lambda: [graph.replay() for _ in range(pairs)]) / pairs / 2

    if int(dev_err.item()) != 0 or not torch.isfinite(hidden).all():
        sys.exit(f"decode: device error word {int(dev_err.item())}, or a result that is not finite")
    cache = block.cache.numel() / 2 ** 20
    plain = R * pages * PAGE * KV_HEADS * DIM * 4 / 2 ** 20
    print(f"{R} prompts of {P} tokens: {prompt_ms:.2f} ms (first calls); a step of {R} tokens: {step_ms * 1e3:.1f} us; "
          f"cache {cache:.1f} MiB (bf16: {plain:.1f} MiB)")


if __name__ == "__main__":
    main()
