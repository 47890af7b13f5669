"""PLEAttention on streams other than the current one: its result's memory and its first step."""

import torch
import pytest

from _four_bit import bits
from test_gpu_attention_layer import block_case

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000  # some 50 ms


def inputs(T, C):
    i32 = dict(dtype=torch.int32, device="cuda")
    hidden = torch.randn(T, C, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    return (hidden, torch.arange(16, **i32).view(1, 16), torch.tensor([0, T], **i32), torch.tensor([T], **i32))


def test_a_result_on_another_stream_takes_no_memory_that_the_current_one_still_reads():
    block, _, _, _ = block_case(256, 4, 1, 64, 16)
    args = inputs(48, 256)
    want = block.forward(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    held = torch.full((48, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    copy = torch.empty_like(held)
    torch.cuda._sleep(CYCLES)
    copy.copy_(held)
    del held  # the current stream's allocator may hand its memory out again
    y = block.forward(*args, stream=side)
    side.synchronize()
    got = bits(y)
    torch.cuda.synchronize()
    assert (copy == 3.0).all()
    assert (got == bits(want)).all() and (bits(y) == got).all()


def test_the_first_step_on_another_stream_finds_the_workspace_filled():
    args = inputs(48, 256)
    reference, _, _, _ = block_case(256, 4, 1, 64, 16)
    want = reference.forward(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    junk = torch.full((reference.workspace.numel(),), 255, dtype=torch.uint8, device="cuda")
    del junk  # its memory is likely to become the workspace
    torch.cuda._sleep(CYCLES)
    block, _, _, _ = block_case(256, 4, 1, 64, 16)
    y = block.forward(*args, stream=side)
    side.synchronize()
    assert (bits(y) == bits(want)).all()
    assert (block.workspace[:256] == 0).all()


def test_a_result_on_the_current_stream_and_one_given():
    block, _, _, _ = block_case(256, 4, 1, 64, 16)
    args = inputs(48, 256)
    want = bits(block.forward(*args))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty(48, 256, dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    assert block.forward(*args, stream=side, out=out) is out
    side.synchronize()
    assert (bits(out) == want).all()
