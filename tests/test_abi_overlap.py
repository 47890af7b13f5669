"""Refusals of outputs that share bytes with inputs (no GPU: nothing is enqueued, no pointer is followed)."""

import random

import pytest

from test_abi_four_bit import INVALID, append, attention, lib, proj  # noqa: F401


BASE = 1 << 20


def rows(at, stride, count, width):
    return {at + i * stride + x for i in range(count) for x in range(0, width, 16)}


def q_out_refused(lib, T, q, qs, qo, qos, k, ks, v, vs):
    """Of ple_kv_append with 1 head of q, k and v of 64 elements; strides in bytes. A negative num_positions ends
    the call behind the check."""
    status = append(lib, T=T, H=1, Hk=1, D=64, rot=64, npos=-1, q=q, qs=qs // 2, qo=qo, qos=qos // 2, k=k, ks=ks // 2,
                    v=v, vs=vs // 2)
    text = lib.ple_last_error()
    assert status == INVALID and (b"overlaps" in text or b"num_positions" in text), (status, text)
    return b"overlaps" in text


def test_columns_of_one_tensor_are_no_overlap(lib):
    for T in (1, 2, 1000):
        # q, k, v side by side, q_out in place, or behind them
        assert not q_out_refused(lib, T, BASE, 512, BASE, 512, BASE + 128, 512, BASE + 256, 512)
        assert not q_out_refused(lib, T, BASE, 512, BASE + 384, 512, BASE + 128, 512, BASE + 256, 512)
        # on k, on v, half on q
        assert q_out_refused(lib, T, BASE, 512, BASE + 128, 512, BASE + 128, 512, BASE + 256, 512)
        assert q_out_refused(lib, T, BASE, 512, BASE + 144, 512, BASE + 384, 512, BASE + 256, 512)
        assert q_out_refused(lib, T, BASE, 512, BASE + 16, 512, BASE + 384, 512, BASE + 256, 512)
    # a row further on: only where there is one
    far = 1 << 30
    assert q_out_refused(lib, 2, BASE, 512, BASE + 512, 512, far, 512, far, 512)
    assert not q_out_refused(lib, 1, BASE, 512, BASE + 512, 512, far, 512, far, 512)
    # the same pointer at another stride is not the same tensor
    assert q_out_refused(lib, 2, BASE, 512, BASE, 1024, far, 512, far, 512)


def test_against_the_bytes_themselves(lib):
    rng = random.Random(1)
    for _ in range(4000):
        T, stride = rng.randint(1, 5), 16 * rng.randint(0, 24)
        qo = BASE + 16 * rng.randint(0, 80)
        k, v = (BASE + 16 * rng.randint(0, 80) for _ in range(2))
        far = 1 << 30
        want = any(rows(qo, stride, T, 128) & rows(x, stride, T, 128) for x in (k, v))
        assert q_out_refused(lib, T, far, 512, qo, stride, k, stride, v, stride) == want, (T, stride, qo, k, v)
        negative = any(rows(qo, -stride, T, 128) & rows(x, -stride, T, 128) for x in (k, v))
        assert q_out_refused(lib, T, far, 512, qo, -stride, k, -stride, v, -stride) == negative


def test_one_piece_against_rows(lib):
    """ple_proj_w4's out is one piece: between two rows of x it overlaps neither."""
    def refused(out, T=2, N=64):
        status = proj(lib, x=BASE, xs=4096, T=T, E=256, group=64, N=N, out=out, codes=BASE + (1 << 25) + 8)
        return status == INVALID and b"overlaps" in lib.ple_last_error()

    # 512 bytes of x at BASE and at BASE + 8192; T * N * 2 = 256 bytes of out
    for out, want in ((BASE - 256, False), (BASE - 240, True), (BASE + 496, True), (BASE + 512, False),
                      (BASE + 7936, False), (BASE + 7952, True), (BASE + 8703, True), (BASE + 8704, False)):
        assert refused(out) == want, out - BASE
    assert refused(BASE + 512, N=2000)


def test_attention_in_place_or_apart(lib):
    def refused(out, out_stride=512, T=2):
        status = attention(lib, T=T, q=BASE, qs=512, out=out, os=out_stride, ws=None)
        assert status == INVALID
        return b"overlaps" in lib.ple_last_error()

    # rows of 4 heads of 128: 1024 bytes, 1024 apart
    assert not refused(BASE) and not refused(BASE + 2048) and not refused(BASE - 2048)
    assert refused(BASE + 16) and refused(BASE + 1024) and refused(BASE, 1024) and refused(BASE - 1024)
    assert not refused(BASE + 1024, T=1) and refused(BASE + 1008, T=1)


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("stride", [0, 2 ** 60, -(2 ** 60)])
def test_strides_of_any_size(lib, T, stride):
    assert not q_out_refused(lib, T, BASE, stride, BASE, stride, BASE + 4096, stride, BASE + 8192, stride)
    assert q_out_refused(lib, T, BASE, stride, BASE, stride, BASE + 16, stride, BASE + 8192, stride)
