"""PLEAttention on the GPU: prompts and single tokens through its four calls,
against the float64 oracle of the same chain.

Bound: the projections' outputs agree with the oracle's to a rounding of 2^-8;
where that rounding falls the other way, a 4-bit code may move by one step of
its row's range / 15 (0.4 of the values' deviation), which one of the H D >= 256
columns of the output projection carries on: 0.4 / sqrt(256) of rms(y) for a row
that sees a single position, less for others. With the roundings of the
attention and of the result that stays below CHAIN_ATOL_FRAC = 3e-2 of rms(y)
plus 3e-2 of the element."""

import numpy as np
import pytest
import torch

from hashed_gram_embedding_gb300 import PLEAttention, PLELayer, PleError, pack_w4
from hashed_gram_embedding_gb300 import _lib

from _four_bit import oracle, rotation_table
from _helpers import CHAIN_ATOL_FRAC, assert_close, bits, dev_err_word, tiny_case

pytestmark = pytest.mark.gpu


def weights(N, E, group, seed, std):
    w = torch.randn(N, E, generator=torch.Generator().manual_seed(seed)) * std
    return pack_w4(w, group)


def block_case(C, H, Hk, D, page, group=32, positions=256, max_tokens=256, pages=64, seed=0, **more):
    w_qkv = weights((H + 2 * Hk) * D, C, group, seed, C ** -0.5)
    w_out = weights(C, H * D, group, seed + 1, (H * D) ** -0.5)
    table = torch.from_numpy(rotation_table(positions, D))
    block = PLEAttention([t.cuda() for t in w_qkv], [t.cuda() for t in w_out], H, Hk, D, pages, page,
                         max_tokens, cos_sin=table.cuda(), **more)
    return block, w_qkv, w_out, table.numpy()


def oracle_block(hidden, w_qkv, w_out, table, cache, block_table, qsl, lens, H, Hk, D, group, window=0):
    """The same chain in the oracle; ``cache`` is updated."""
    bf16 = oracle.f64_to_bf16
    qkv, _ = oracle.proj_w4(hidden, w_qkv[0].numpy(), bits(w_qkv[1]), w_qkv[2].numpy(), group)
    rows = bf16(qkv).reshape(-1, H + 2 * Hk, D)
    q = oracle.append(rows[:, :H], rows[:, H:H + Hk], rows[:, H + Hk:], table, cache, block_table, qsl, lens)
    mixed, _, _ = oracle.attention(q, cache, block_table, qsl, lens, D ** -0.5, window=window)
    y, _ = oracle.proj_w4(bf16(mixed).reshape(-1, H * D), w_out[0].numpy(), bits(w_out[1]), w_out[2].numpy(), group)
    return bf16(y)


@pytest.mark.parametrize("C,H,Hk,D,page,window", [(256, 4, 1, 64, 16, 0), (512, 4, 4, 128, 48, 20), (320, 2, 1, 256, 32, 0)])
def test_prompts_then_single_tokens(C, H, Hk, D, page, window):
    group = 32 if C == 320 else 64
    block, w_qkv, w_out, table = block_case(C, H, Hk, D, page, group, window=window)
    cache = block.cache.cpu().numpy().copy()
    rng = np.random.default_rng(1)
    block_table = rng.permutation(64)[:3 * 12].reshape(3, 12).astype(np.int32)
    lens = np.zeros(3, np.int32)
    err = dev_err_word()
    for step, queries in enumerate([(37, 1, 90), (1, 1, 1), (1, 4, 1), (1, 1, 1)]):
        qsl = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
        lens = lens + np.array(queries, np.int32)
        hidden = torch.randn(int(qsl[-1]), C, generator=torch.Generator().manual_seed(step)).to(torch.bfloat16)
        y = block.forward(hidden.cuda(), *(torch.from_numpy(a).cuda() for a in (block_table, qsl, lens)),
                          max_query_len=max(queries), dev_err=err)
        torch.cuda.synchronize()
        want = oracle_block(bits(hidden), w_qkv, w_out, table, cache, block_table, qsl, lens, H, Hk, D, group, window)
        assert_close(bits(y), want, rtol=3e-2, atol_frac=CHAIN_ATOL_FRAC, atol=1.0, what=f"step {step}")
    assert int(err.item()) == 0


def test_behind_a_layer_in_a_graph():
    """A PLE layer's output through the block, the step captured once and
    replayed with the lengths counted up on the device, gives the bits of the
    calls made one by one."""
    w, host, dense, table, _ = tiny_case()
    d = {k: v.cuda() for k, v in dense.items()}
    layer = PLELayer(table.cuda(), None, host["multipliers"][0], host["V"], host["O"], w.eos_token_id,
                     w.heads_per_ngram, d["w_kv"], d["gamma_h"], d["gamma_k"], d["conv_w"], w.dilation)
    block, _, _, _ = block_case(w.hidden, 8, 2, 64, 16, 128, max_tokens=w.num_tokens)
    R = 4
    ids = torch.from_numpy(host["input_ids"][:R]).cuda()
    qsl = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    block_table = torch.arange(R * 4, dtype=torch.int32, device="cuda").view(R, 4)
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    x = d["hidden"][:R].clone()
    y = torch.empty_like(x)

    def step():
        lens.add_(1)
        block.forward(layer.forward(ids, qsl, x), block_table, qsl, lens, max_query_len=1, out=y)
        x.add_(y)

    start = x.clone()
    want = []
    for _ in range(20):
        step()
        want.append(x.clone())
    lens.zero_()
    x.copy_(start)
    block.cache.zero_()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(20):
        graph.replay()
        assert torch.equal(x, want[i]), i


def test_no_tokens():
    block, _, _, _ = block_case(256, 4, 1, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    y = block.forward(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 1, **i32),
                      torch.zeros(2, **i32), torch.zeros(1, **i32))
    assert y.shape == (0, 256)


def test_refusals():
    block, _, _, _ = block_case(256, 4, 1, 64, 16, max_tokens=8)
    i32 = dict(dtype=torch.int32, device="cuda")
    one, table = torch.ones(1, **i32), torch.zeros(1, 4, **i32)
    qsl = torch.tensor([0, 1], **i32)
    x = torch.zeros(1, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        block.forward(torch.zeros(9, 256, dtype=torch.bfloat16, device="cuda"), table, qsl, one)  # past max_tokens
    with pytest.raises(ValueError):
        block.forward(x.float(), table, qsl, one)
    with pytest.raises(ValueError):
        block.forward(x, table.long(), qsl, one)
    with pytest.raises(ValueError):
        block.forward(x, table, qsl, torch.ones(2, **i32))
    for heads, kv, dim, page in ((4, 1, 96, 16), (4, 3, 64, 16), (4, 1, 64, 24), (4, 1, 64, 0)):
        rows = torch.zeros((heads + 2 * kv) * dim, 128, dtype=torch.uint8, device="cuda")
        out = torch.zeros(256, heads * dim // 2, dtype=torch.uint8, device="cuda")
        with pytest.raises(ValueError):
            PLEAttention((rows, None, None), (out, None, None), heads, kv, dim, 4, page, 8)
    with pytest.raises(ValueError):
        pack_w4(torch.zeros(4, 100), 32)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(PleError):  # too small a workspace
        _lib.ple_kv_attention(torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda"), block.cache, table, qsl, one,
                              torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda"), ws)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_packed_weights(group):
    """A weight's distance to its 4-bit form: half a step, and where the zero
    point's own rounding shifts an end of the range, half a step more; a step
    of 2^-8 relative is lost to the scale's rounding over 15 steps."""
    w = torch.randn(64, 256, generator=torch.Generator().manual_seed(3))
    codes, scales, zeros = pack_w4(w, group)
    got = torch.stack((codes & 15, codes >> 4), 2).view(64, 256 // group, group).float()
    got = (got - zeros[..., None]) * scales.float()[..., None]
    far = (got.view(64, 256) - w).abs().view(64, -1, group)
    assert (far <= scales.float()[..., None] * (1.0 + 15 * 2.0 ** -8)).all()
