"""PLEFeedForward on the GPU: the 8-bit step's calls in a run, as they are used."""

import numpy as np
import pytest
import torch

import hashed_gram_embedding_gb300 as ple
from hashed_gram_embedding_gb300 import PLEFeedForward, pack_mx8
from oracle import eight_bit as oracle

from _helpers import bits, bf16_values, dev_err_word

pytestmark = pytest.mark.gpu

C, I = 512, 896


def f64(t):
    return bf16_values(bits(t)).reshape(t.shape)


def weights(seed=0):
    rng = np.random.default_rng(seed)
    w1 = torch.from_numpy((rng.normal(0, C ** -0.5, (2 * I, C))).astype(np.float32))
    w2 = torch.from_numpy((rng.normal(0, I ** -0.5, (C, I))).astype(np.float32))
    g = torch.from_numpy(rng.normal(1, 0.1, C).astype(np.float32)).to(torch.bfloat16)
    return w1, w2, g


def values(weight):
    codes, scales = pack_mx8(weight)
    return oracle.values(codes.numpy(), oracle.pick(scales.numpy(), *weight.shape))


def block(max_tokens, activation="silu", seed=0):
    w1, w2, g = weights(seed)
    pack = lambda w: tuple(a.cuda() for a in pack_mx8(w))  # noqa: E731
    return PLEFeedForward(pack(w1), pack(w2), g.cuda(), max_tokens, activation=activation)


def hidden(t, seed=1):
    return torch.from_numpy(np.random.default_rng(seed).normal(0, 1, (t, C)).astype(np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("t", [1, 20, 130, 700])
@pytest.mark.parametrize("activation,delta", [("silu", True), ("gelu", False)])
def test_block(t, activation, delta):
    """The whole block against float64 with the format's own roundings. Where
    a float32 value falls on the other side of a code's border than the
    float64 one does (a share of about 2^-18 * 2^5 of the codes, each by 2^-3
    of itself at most), the result moves with it: by the 2-norm that is
    sqrt(2^-13) * 2^-3 < 0.002 of the product for each of the two
    quantisations, beside bf16's 0.0017."""
    w1, w2, g = weights()
    ff = block(t + 3, activation)
    h, d = hidden(t), hidden(t, 2) if delta else None
    err = dev_err_word()
    y = ff.forward(h, d, dev_err=err)
    assert int(err.item()) == 0
    s, n = oracle.norm(f64(h), None if d is None else f64(d), f64(g), 1e-6)
    q = oracle.values(*oracle.quantise(n))
    m = oracle.values(*oracle.quantise(oracle.gated(q, values(w1), activation)))
    want = m @ values(w2).T
    stream = bf16_values(bits(torch.from_numpy(s).to(torch.float32).to(torch.bfloat16))).reshape(s.shape)
    got = f64(y) - stream
    # y is rounded to bf16 with the stream in it
    off = 2.0 ** -8 * np.linalg.norm(want + stream) + 0.004 * np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= off
    assert y.dtype is torch.bfloat16 and y.shape == (t, C)


def test_fused_calls_are_the_calls():
    t = 50
    ff = block(64)
    h, d = hidden(t), hidden(t, 2)
    y = ff.forward(h, d)
    codes = torch.empty((t, C), dtype=torch.uint8, device="cuda")
    scales = torch.empty(ple.ple_mx8_scale_bytes(t, C), dtype=torch.uint8, device="cuda")
    total = torch.empty_like(h)
    ple.ple_norm_mx8(h, ff.gamma, codes, scales, residual=d, sum_out=total)
    hc = torch.empty((t, I), dtype=torch.uint8, device="cuda")
    hs = torch.empty(ple.ple_mx8_scale_bytes(t, I), dtype=torch.uint8, device="cuda")
    ple.ple_gated_mx8(codes, scales, *ff.w_gate_up, hc, hs)
    out = torch.empty_like(h)
    ple.ple_proj_mx8(hc, hs, *ff.w_down, out, residual=total)
    assert torch.equal(out, y)
    # in place
    same = h.clone()
    assert torch.equal(ff.forward(same, d, out=same), y)
    same = h.clone()
    alone = ff.forward(h)
    assert torch.equal(ff.forward(same, out=same), alone)


@pytest.mark.parametrize("t", [1, 100, 400])
def test_captured(t):
    ff = block(t)
    h, d, out = hidden(t), hidden(t, 2), torch.empty((t, C), dtype=torch.bfloat16, device="cuda")
    want = ff.forward(h, d).clone()
    ff.forward(h, d, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ff.forward(h, d, out=out)
    other = hidden(t, 9)
    want2 = ff.forward(other, d).clone()
    out.zero_()
    graph.replay()
    assert torch.equal(out, want)
    h.copy_(other)
    graph.replay()
    assert torch.equal(out, want2)


def test_streams():
    ff = block(200)
    h, d = hidden(200), hidden(200, 2)
    want = ff.forward(h, d).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = ff.forward(h, d, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    # two blocks at once
    other = block(200, seed=5)
    want2 = other.forward(h, d).clone()
    torch.cuda.synchronize()
    for _ in range(10):
        a, b = ff.forward(h, d, stream=side), other.forward(h, d)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want2)


def test_with_an_attention_block():
    """Between an attention block and the next layer: forward(hidden, delta)."""
    heads, kv, dim, t = 4, 2, 128, 70
    g = torch.Generator().manual_seed(3)
    w4 = lambda n, e: tuple(a.cuda() for a in ple.pack_w4(torch.randn(n, e, generator=g) * e ** -0.5))  # noqa: E731
    attention = ple.PLEAttention(w4((heads + 2 * kv) * dim, C), w4(C, heads * dim), heads, kv, dim, 8, 16, t)
    ff = block(t)
    h = hidden(t)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    qsl = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    lens = torch.tensor([t], dtype=torch.int32, device="cuda")
    delta = attention.forward(h, table, qsl, lens, max_query_len=t)
    y = ff.forward(h, delta)
    assert torch.isfinite(y.float()).all()
    # nothing added by the block leaves the stream: with w_down = 0 the result is h + delta
    ff.w_down = (torch.zeros_like(ff.w_down[0]), ff.w_down[1])
    assert torch.equal(ff.forward(h, delta), (h.float() + delta.float()).to(torch.bfloat16))


def test_refusals():
    w1, w2, g = weights()
    pack = lambda w: tuple(a.cuda() for a in pack_mx8(w))  # noqa: E731
    with pytest.raises(ValueError):
        PLEFeedForward(pack(w1[:I]), pack(w2), g.cuda(), 4)
    with pytest.raises(ValueError):
        PLEFeedForward(pack(w1), pack(w2), g.cuda(), 4, activation="relu")
    ff = block(4)
    with pytest.raises(ValueError):
        ff.forward(hidden(5))
    with pytest.raises(ValueError):
        ff.forward(hidden(3), hidden(2))
    ff.activation = "relu"
    with pytest.raises(ValueError):
        ff.forward(hidden(3))


def test_no_tokens():
    assert block(4).forward(hidden(0)).shape == (0, C)


def test_the_serving_example_runs():
    import os
    import subprocess
    import sys
    root = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")
    run = subprocess.run([sys.executable, os.path.join(root, "examples", "decode.py"), "--requests", "3", "--prompt", "21",
                          "--steps", "4"], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    assert "a step of 3 tokens" in run.stdout
