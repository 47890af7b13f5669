"""ple_kv_append and ple_kv_read on the GPU. The cache's bytes follow from
float32 operations rounded one by one, so they equal the oracle's exactly, as
do the rotated queries and the values read back (one bf16 rounding)."""

import numpy as np
import pytest
import torch

from hashed_gram_embedding_gb300 import _lib

from _four_bit import Batch, bits, oracle, rotation_table
from _helpers import dev_err_word

pytestmark = pytest.mark.gpu


def _append(b, q, k, v, cs, interleaved=False, positions=None, err=None, in_place=False):
    cache, table, qsl, lens = b.device()
    dq = None if q is None else q.cuda()
    out = None if q is None else dq if in_place else torch.full_like(dq, 7.0)
    _lib.ple_kv_append(dq, k.cuda(), v.cuda(), None if cs is None else torch.from_numpy(cs).cuda(),
                       cache, table, qsl, lens, out, interleaved=interleaved,
                       positions=None if positions is None else torch.from_numpy(positions).cuda(),
                       dev_err=err)
    torch.cuda.synchronize()
    return out, cache


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 4), (128, 10, 5), (128, 8, 1), (256, 6, 2)])
@pytest.mark.parametrize("page", [16, 48])
@pytest.mark.parametrize("rot,interleaved", [("all", False), ("all", True), (32, False), (16, True), (None, False)])
def test_append_matches_the_oracle_byte_for_byte(dim, heads, kv_heads, page, rot, interleaved):
    b = Batch([1, 0, 5, 33, 2], [17, 9, 5, 40, 96], heads, kv_heads, dim, page, seed=dim + page, pad=2)
    q, k, v = b.rows(heads), b.rows(kv_heads), b.rows(kv_heads)
    cs = None if rot is None else rotation_table(100, dim if rot == "all" else rot)
    want_cache = b.cache.copy()
    want_q = oracle.append(bits(q), bits(k), bits(v), cs, want_cache, b.table, b.qsl, b.lens,
                           interleaved=interleaved)
    err = dev_err_word()
    out, cache = _append(b, q, k, v, cs, interleaved, err=err)
    assert int(err.item()) == 0
    assert np.array_equal(bits(out), want_q)
    assert np.array_equal(cache.cpu().numpy(), want_cache)
    out, cache = _append(b, q, k, v, cs, interleaved, in_place=True)
    assert np.array_equal(bits(out), want_q)
    out, cache = _append(b, None, k, v, cs, interleaved)
    assert np.array_equal(cache.cpu().numpy(), want_cache)


def test_append_takes_columns_of_a_fused_projection_and_given_positions():
    b = Batch([3, 4], [3, 50], 6, 2, 128, 16, seed=5)
    qkv = torch.randn(b.T, 10 * 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, 128)) for x in qkv.split([768, 256, 256], 1))
    cs = rotation_table(200, 128)
    positions = np.array([199, 0, 7, 7, 100, 3, 50], np.int32)
    want_cache = b.cache.copy()
    want_q = oracle.append(*(bits(x) for x in (q, k, v)), cs, want_cache, b.table, b.qsl, b.lens, positions)
    dev = qkv.cuda()
    dq, dk, dv = (x.unflatten(1, (-1, 128)) for x in dev.split([768, 256, 256], 1))
    cache, table, qsl, lens = b.device()
    side = torch.cuda.Stream()  # not the tensors' own stream
    side.wait_stream(torch.cuda.current_stream())
    _lib.ple_kv_append(dq, dk, dv, torch.from_numpy(cs).cuda(), cache, table, qsl, lens, dq,
                       positions=torch.from_numpy(positions).cuda(), stream=side)
    side.synchronize()
    assert np.array_equal(bits(dq), want_q)
    assert np.array_equal(cache.cpu().numpy(), want_cache)


def test_append_flags_places_outside_the_cache_and_writes_nothing_there():
    b = Batch([2, 3, 2, 1], [1, 3, 20, 5], 2, 2, 64, 16, seed=3)
    b.table[2, 1] = b.pages      # request 2's second page is outside the cache
    b.table[3, 0] = -1
    q, k, v = b.rows(2), b.rows(2), b.rows(2)
    cs = rotation_table(19, 64)  # request 2's last position, 19, is past the table
    want_cache = b.cache.copy()
    want_q = oracle.append(bits(q), bits(k), bits(v), cs, want_cache, b.table, b.qsl, b.lens)
    err = dev_err_word()
    out, cache = _append(b, q, k, v, cs, err=err)
    assert int(err.item()) == _lib.PLE_DEVERR_BOUNDS
    assert np.array_equal(cache.cpu().numpy(), want_cache)
    got, live = bits(out), np.ones(b.T, bool)
    live[[0, 6]] = False  # position -1 (not in the table either) and position 19: zero rows
    assert np.array_equal(got[live], want_q[live]) and not got[~live].any()


def test_constant_extreme_and_non_finite_rows():
    b = Batch([6], [6], 1, 1, 64, 16, seed=4)
    k, v = b.rows(1), b.rows(1)
    k[0] = 3.25                    # constant: scale 0, read back exactly
    k[1, 0, 5] = float("inf")
    k[2, 0, 9] = float("nan")
    k[3] = 0.0
    k[4, 0, 0], k[4, 0, 1] = 1e30, -1e30
    k[5] = 1e-38 * torch.arange(64)  # scale near the subnormals
    out, cache = _append(b, None, k, v, None)
    _, table, qsl, lens = b.device()
    ko, vo = (torch.empty(6, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _lib.ple_kv_read(cache, table, qsl, lens, ko, vo)
    ko, vo = ko.cpu().float(), vo.cpu().float()
    assert torch.equal(ko[0], torch.full((1, 64), 3.25)) and torch.equal(ko[3], torch.zeros(1, 64))
    assert ko[1].isnan().all() and ko[2].isnan().all() and torch.isfinite(vo).all()
    # half a step, the offset's rounding, the scale's rounding over 15 codes, the output's
    for row in (4, 5):
        x = k[row].float()
        step = float(x.max() - x.min()) / 15
        bound = step / 2 + 2 ** -9 * (abs(float(x.min())) + 15 * step) + 2 ** -8 * x.abs()
        assert ((ko[row] - x).abs() <= bound + 1e-40).all()


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_read_gives_the_stored_values(dim, page):
    b = Batch([7, 0, 40], [7, 11, 70], 4, 3, dim, page, seed=dim, pad=3)
    b.table[2, 2 * 32 // page] = b.pages + 5  # position 64 on (page 32 or 64)
    cache, table, qsl, lens = b.device()
    ko, vo = (torch.full((b.T, 3, dim), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = dev_err_word()
    _lib.ple_kv_read(cache, table, qsl, lens, ko, vo, dev_err=err)
    want = np.zeros((2, b.T, 3, dim))
    bad = False
    for t, r, p in oracle.tokens(b.qsl, b.lens, b.T):
        x = oracle.read(b.cache, b.table, r, p, dim)
        bad |= x is None
        if x is not None:
            want[:, t] = x
    assert bool(int(err.item()) & _lib.PLE_DEVERR_BOUNDS) == bad
    want = torch.from_numpy(want).to(torch.bfloat16)  # of the exact value: one rounding
    assert torch.equal(ko.cpu(), want[0]) and torch.equal(vo.cpu(), want[1])
    only = torch.empty_like(ko)
    _lib.ple_kv_read(cache, table, qsl, lens, None, only)
    assert torch.equal(only.cpu(), want[1])


def test_malformed_query_start_loc_is_flagged():
    b = Batch([2, 2], [2, 2], 1, 1, 64, 16)
    cache, table, _, lens = b.device()
    k = b.rows(1).cuda()
    for qsl in ([0, 3, 2], [1, 2, 4], [0, 2, 9]):
        err = dev_err_word()
        _lib.ple_kv_append(None, k, k, None, cache, table, torch.tensor(qsl, dtype=torch.int32, device="cuda"),
                           lens, None, dev_err=err)
        assert int(err.item()) & _lib.PLE_DEVERR_QSL


def test_append_past_32_bit_offsets():
    """A cache of 4.4 GB: the last page's blocks start past 2^32 bytes."""
    pages, hk, dim = 2_000_000, 1, 128
    cache = torch.zeros((pages, hk, 1, 16 * (dim + 8)), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    qsl = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 20, hk, dim, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    k, v = x.cuda()
    _lib.ple_kv_append(None, k, v, None, cache, table, qsl, lens, None)
    small = np.zeros((2, hk, 1, 16 * (dim + 8)), np.uint8)
    oracle.append(np.zeros((20, 1, dim), np.uint16), bits(x[0]), bits(x[1]), None, small,
                  np.array([[1, 0]]), np.array([0, 20]), np.array([20]))
    assert np.array_equal(cache[-2:].cpu().numpy(), small)
    assert not cache[:-2].any()
