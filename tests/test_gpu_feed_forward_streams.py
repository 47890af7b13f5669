"""PLEFeedForward: a first step on another stream than the one it was built on."""

import numpy as np
import pytest
import torch

from hashed_gram_embedding_gb300 import PLEFeedForward, pack_mx8

pytestmark = pytest.mark.gpu

T, C, I = 2000, 1024, 2048


def test_first_step_on_another_stream():
    """The block's buffers may be memory that its own stream's earlier work
    still writes: that work has to be over before any stream takes a step."""
    rng = np.random.default_rng(0)
    pack = lambda n, e: tuple(a.cuda() for a in pack_mx8(  # noqa: E731
        torch.from_numpy(rng.normal(0, e ** -0.5, (n, e)).astype(np.float32))))
    w1, w2 = pack(2 * I, C), pack(C, I)
    h = torch.from_numpy(rng.normal(0, 1, (T, C)).astype(np.float32)).to(torch.bfloat16).cuda()
    first = PLEFeedForward(w1, w2, None, T)
    want = first.forward(h, h).clone()
    side, out = torch.cuda.Stream(), torch.empty_like(h)
    names = lambda ff: [*ff.normed, *ff.gated, ff.sum]  # noqa: E731
    old = names(first)
    places = {t.data_ptr() for t in old}
    fills = torch.cuda.CUDAGraph()
    with torch.cuda.graph(fills):
        for _ in range(100):
            for t in old:
                t.fill_(0x7F)
    torch.cuda.synchronize()
    for _ in range(30):  # some milliseconds
        fills.replay()
    del first, old, t
    ff = PLEFeedForward(w1, w2, None, T)
    assert places & {t.data_ptr() for t in names(ff)}  # as torch hands out what it got back
    ff.forward(h, h, stream=side, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
