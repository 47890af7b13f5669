"""ple_kv_attention on the GPU against the float64 oracle on the same cache.

Bound of an element, with u = 2^-8 (bf16 has 8 significant bits):
  * the result's rounding: u |o|;
  * the weights' rounding for the second product: u sum_p w_p |v_p| <= u max|V|;
  * the values' rounding, where a kernel rounds them: another u max|V|;
  * the keys' rounding, where a kernel rounds them: a score moves by at most
    d = u scale max_p sum_d |q_d K_pd|, a weight by a factor within e^(2d), so
    the result by (e^(2d) - 1) 2 max|V| at the very most;
  * float32 arithmetic: 2^-14 of max|V|, far above its accumulated roundings.
Over a whole output these are independent and average: each of the four is at
most u / sqrt(3) relative to rms(V) and rms(o) > rms(V) / sqrt(positions); with
few positions in a row the 2-norm of the error is within 4 * 2^-9 of the
result's."""

import math

import numpy as np
import pytest
import torch

from hashed_gram_embedding_gb300 import _lib

from _four_bit import Batch, bits, oracle
from _helpers import bf16_values, dev_err_word

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def attend(b, q, causal=True, window=0, hint=0, scale=None, err=None, ws=None, stream=None, strided=False):
    cache, table, qsl, lens = b.device()
    dq = q.cuda()
    if strided:  # rows of a wider tensor
        wide = torch.full((b.T, b.heads + 3, b.dim), 5.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:1 + b.heads] = dq
        dq = wide[:, 1:1 + b.heads]
    out = torch.full((b.T, b.heads, b.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = torch.zeros(_lib.ple_kv_attention_workspace(b.heads, b.kv_heads, b.dim), dtype=torch.uint8,
                         device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    _lib.ple_kv_attention(dq, cache, table, qsl, lens, out, ws, causal=causal, window=window, scale=scale,
                          max_query_len=hint, dev_err=err, stream=stream)
    torch.cuda.synchronize()
    return out


def check(out, want, kmax, vmax):
    got = bf16_values(bits(out))
    assert np.isfinite(got).all()
    d = U * kmax
    bound = U * np.abs(want) + (2 * U + 2.0 ** -14 + 2 * np.expm1(2 * d))[..., None] * vmax[..., None]
    assert (np.abs(got - want) <= bound).all(), np.abs(got - want).max()
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= 2 * U * norm


def run(b, causal=True, window=0, scale=None, q_scale=1.0, **kw):
    q = b.rows(b.heads, q_scale)
    err = dev_err_word()
    out = attend(b, q, causal, window, scale=scale, err=err, **kw)
    assert int(err.item()) == 0
    want, kmax, vmax = oracle.attention(bits(q), b.cache, b.table, b.qsl, b.lens,
                                        b.dim ** -0.5 if scale is None else scale, causal, window)
    check(out, want, kmax, vmax)
    return q, out


LAYOUTS = [(4, 4, 64), (8, 1, 64), (8, 2, 128), (10, 5, 128), (12, 1, 128), (33, 3, 128), (6, 2, 256), (5, 1, 256)]


@pytest.mark.parametrize("heads,kv_heads,dim", LAYOUTS)
@pytest.mark.parametrize("page", [16, 48, 128])
def test_single_tokens(heads, kv_heads, dim, page):
    """Decode: one token a request, lengths around the blocks' and tiles' edges, none among them."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 129, 200]
    run(Batch([1] * len(lens), lens, heads, kv_heads, dim, page, seed=dim + heads), hint=1)


@pytest.mark.parametrize("heads,kv_heads,dim", LAYOUTS)
@pytest.mark.parametrize("hint", [0, 9])
def test_few_tokens_ragged(heads, kv_heads, dim, hint):
    """Speculative decode: 0 to 9 tokens a request, padding tokens after the last."""
    run(Batch([4, 1, 0, 9, 2, 3], [70, 1, 5, 9, 133, 40], heads, kv_heads, dim, 16, seed=7, pad=3), hint=hint)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 2, 128), (5, 1, 128), (33, 3, 128), (2, 1, 256)])
@pytest.mark.parametrize("page", [16, 64, 80])
def test_prefill_chunks(heads, kv_heads, dim, page):
    """Chunks of many tokens, with and without cached positions before them, beside single tokens."""
    run(Batch([97, 1, 130, 3, 64], [97, 30, 300, 3, 191], heads, kv_heads, dim, page, seed=page), hint=130)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_long_request_is_split(dim):
    """One token over a long cache of odd length: the splits' partial results are joined."""
    b = Batch([1], [2777], 4, 2, dim, 16, seed=11)
    run(b, hint=1)


@pytest.mark.parametrize("queries,lens", [([1, 1, 4, 40], [50, 300, 100, 140]), ([150], [260])])
@pytest.mark.parametrize("window", [1, 7, 33, 100, 1000])
def test_window(queries, lens, window):
    run(Batch(queries, lens, 8, 2, 128, 16, seed=13), window=window)


@pytest.mark.parametrize("queries,lens", [([1, 4, 40], [50, 100, 60]), ([150, 30], [260, 31])])
def test_without_the_causal_mask(queries, lens):
    run(Batch(queries, lens, 8, 2, 128, 32, seed=17), causal=False)


def test_rows_that_see_nothing_are_zero():
    """Fewer cached positions than tokens: the first tokens stand before position 0."""
    b = Batch([5, 3, 90, 1], [2, 0, 70, 0], 8, 2, 128, 16, seed=19)
    _, out = run(b)
    got = bits(out)
    for rows in (slice(0, 3), slice(5, 8), slice(8, 28), slice(98, 99)):
        assert not got[rows].any()


def test_pages_outside_the_cache_are_not_seen():
    for queries, lens in (([1, 2], [100, 60]), ([120, 2], [200, 60])):
        b = Batch(queries, lens, 8, 2, 128, 16, seed=23)
        b.table[0, 2], b.table[0, 5], b.table[1, 0] = b.pages, -7, 1 << 30
        q = b.rows(8)
        err = dev_err_word()
        out = attend(b, q, err=err)
        assert int(err.item()) == _lib.PLE_DEVERR_BOUNDS
        check(out, *oracle.attention(bits(q), b.cache, b.table, b.qsl, b.lens, 128 ** -0.5))


@pytest.mark.parametrize("tokens", [1, 3, 100])
def test_pages_behind_the_window_may_be_gone(tokens):
    """What lies wholly behind every token's window is not looked up."""
    b = Batch([tokens], [300], 8, 2, 128, 16, seed=27)
    b.table[0, :(300 - tokens - 20 + 1) // 16] = -1
    run(b, window=20)


def test_lengths_past_the_block_table_are_flagged():
    b = Batch([1], [40], 4, 2, 128, 16, seed=29)
    b.lens[0] = 16 * b.table.shape[1] + 500
    q = b.rows(4)
    err = dev_err_word()
    out = attend(b, q, err=err)
    assert int(err.item()) == _lib.PLE_DEVERR_BOUNDS
    assert out.shape == (1, 4, 128)


@pytest.mark.parametrize("queries,lens", [([1, 3], [90, 40]), ([100], [150])])
def test_large_scores_and_offsets(queries, lens):
    """Scores of hundreds (one position takes all the weight) and keys far from zero."""
    run(Batch(queries, lens, 8, 2, 128, 16, seed=31, k_mean=0.1), scale=3.0, q_scale=4.0)
    b = Batch(queries, lens, 8, 2, 128, 16, seed=37, k_mean=30.0)
    run(b, scale=0.02)


def test_nan_in_a_seen_position_reaches_only_rows_that_see_it():
    for queries, lens in (([4, 1], [40, 30]), ([100, 1], [130, 30])):
        b = Batch(queries, lens, 4, 2, 64, 16, seed=41)
        page, sub, slot = oracle.place(b.cache, b.table, 0, lens[0] - 2)
        oracle.block_parts(b.cache[page, 1, sub], 64)[3][slot] = 0x7FC0  # V of head 1
        q = b.rows(4)
        out = attend(b, q).cpu().float()
        n = queries[0]
        assert out[n - 2:n, 2:].isnan().all()
        out[n - 2:n, 2:] = 0
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("queries,lens", [([1] * 5, [700, 3, 90, 1500, 1]), ([200, 1], [300, 60])])
def test_same_bits_again_strided_on_another_stream_and_replayed(queries, lens):
    b = Batch(queries, lens, 8, 2, 128, 16, seed=43)
    q = b.rows(8)
    ws = torch.zeros(_lib.ple_kv_attention_workspace(8, 2, 128), dtype=torch.uint8, device="cuda")
    first = attend(b, q, ws=ws)
    for kw in (dict(), dict(strided=True), dict(stream=torch.cuda.Stream())):
        assert torch.equal(bits_t(attend(b, q, ws=ws, **kw)), bits_t(first))
    # captured into a graph and replayed
    cache, table, qsl, lens_d = b.device()
    dq, out = q.cuda(), torch.zeros((b.T, 8, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _lib.ple_kv_attention(dq, cache, table, qsl, lens_d, out, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits_t(out), bits_t(first))


def bits_t(t):
    return t.cpu().view(torch.int16)


def test_one_workspace_for_many_shapes():
    """The workspace's counters are zero again after each call, whatever ran before."""
    ws = torch.zeros(max(_lib.ple_kv_attention_workspace(h, k, d) for h, k, d in LAYOUTS), dtype=torch.uint8,
                     device="cuda")
    for i, (h, k, d) in enumerate(LAYOUTS):
        b = Batch([1, 2, 50][: 1 + i % 3], [900, 40, 120][: 1 + i % 3], h, k, d, 16, seed=i)
        run(b, ws=ws)


def test_more_requests_than_threads():
    """Several hundred requests, most of one or two positions."""
    rng = np.random.default_rng(47)
    lens = rng.integers(0, 4, 700)
    lens[[3, 500]] = 90, 150
    run(Batch([1] * 700, lens, 2, 1, 64, 16, seed=47), hint=1)


@pytest.mark.parametrize("tokens", [1, 128])
def test_cache_past_32_bit_offsets(tokens):
    """Pages of a 4.4 GB cache, some of them past 2^32 bytes."""
    small = Batch([tokens], [200], 4, 1, 128, 16, seed=53)
    big = 2_000_000
    cache = torch.zeros((big, 1, 1, 16 * 136), dtype=torch.uint8, device="cuda")
    where = np.linspace(0, big - 1, small.pages).astype(np.int64)
    cache[torch.from_numpy(where).cuda()] = torch.from_numpy(small.cache).cuda()
    q = small.rows(4)
    ws = torch.zeros(_lib.ple_kv_attention_workspace(4, 1, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty((tokens, 4, 128), dtype=torch.bfloat16, device="cuda")
    _, _, qsl, lens = small.device()
    _lib.ple_kv_attention(q.cuda(), cache, torch.from_numpy(where[small.table].astype(np.int32)).cuda(), qsl, lens,
                          out, ws)
    check(out, *oracle.attention(bits(q), small.cache, small.table, small.qsl, small.lens, 128 ** -0.5))
    assert math.isclose(where[-1], big - 1)


@pytest.mark.parametrize("factor", [1e-20, 1e4, 3e6, 1e12])
def test_values_of_any_size(factor):
    """Values far below and above one; a scale above 2^18 takes a path of its own."""
    for queries, lens in (([1, 3], [150, 40]), ([100], [150])):
        b = Batch(queries, lens, 8, 2, 128, 16, seed=61)
        for r, n in enumerate(lens):
            for p in range(0, n, 2):  # every other position, so that both kinds meet in a step
                b.put(r, p, b.rng.normal(0, 1, (2, 128)), b.rng.normal(0, factor, (2, 128)))
        run(b)


@pytest.mark.parametrize("queries,lens,H,Hk,D,page,causal,window", [
    ([30], [5000], 4, 1, 128, 64, True, 0),
    ([100, 2, 40, 300], [2500, 900, 4100, 300], 4, 1, 64, 16, True, 0),
    ([70, 33], [3001, 2049], 8, 2, 128, 112, False, 0),
    ([300], [2800], 2, 2, 64, 32, True, 1100),
    ([128, 64], [0, 1700], 6, 2, 128, 16, True, 0),
    ([512], [4096], 3, 1, 128, 128, True, 1),
])
def test_few_rows_on_long_contexts(queries, lens, H, Hk, D, page, causal, window):
    """The positions of the same rows are shared out between CTAs and the results joined."""
    b = Batch(queries, lens, H, Hk, D, page, seed=sum(queries), pad=3)
    run(b, causal=causal, window=window)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_hint_too_small_loses_no_rows(dim):
    run(Batch([1, 60, 5], [90, 100, 5], 4, 2, dim, 16, seed=73), hint=1)


def test_shared_positions_then_single_tokens_in_one_workspace():
    """Calls of every kind after one another leave each other nothing."""
    ws = torch.zeros(_lib.ple_kv_attention_workspace(8, 2, 128), dtype=torch.uint8, device="cuda")
    for queries, lens in (([40], [2600]), ([1] * 5, [700, 3, 40, 1500, 90]), ([40, 1, 3], [1500, 2000, 77]), ([1], [2500])):
        b = Batch(queries, lens, 8, 2, 128, 32, seed=len(lens))
        q = b.rows(8)
        check(attend(b, q, ws=ws), *oracle.attention(bits(q), b.cache, b.table, b.qsl, b.lens, 128 ** -0.5))


@pytest.mark.parametrize("even,odd", [(1e-25, 1e-25), (1e30, 1e30), (1e30, 1e-12), (1e-3, 600.0)])
def test_values_all_beyond_one(even, odd):
    """No value of ordinary size among them; a long request, so that tiles of both kinds follow one another."""
    for queries, lens in (([2, 100], [40, 150]), ([150], [700])):
        b = Batch(queries, lens, 8, 2, 64, 32, seed=71)
        for r, n in enumerate(lens):
            for p in range(n):
                b.put(r, p, b.rng.normal(0, 1, (2, 64)), b.rng.normal(0, odd if p % 2 or p > 300 else even, (2, 64)))
        run(b)


@pytest.mark.parametrize("factor,q_scale", [(1e-4, 1e3), (1e3, 1e-2), (1e12, 1e-12), (1e-20, 1e18)])
def test_keys_of_any_size(factor, q_scale):
    """Keys far below and above one, among ordinary ones, and queries to match."""
    for queries, lens in (([1, 3], [150, 40]), ([100], [150])):
        b = Batch(queries, lens, 8, 2, 128, 16, seed=67, k_mean=0.0)
        for r, n in enumerate(lens):
            for p in range(n):
                if p % 2 == 0 or q_scale < 1:  # ordinary keys meet small queries as nothing, large ones not at all
                    b.put(r, p, b.rng.normal(0, factor, (2, 128)), b.rng.normal(0, 1, (2, 128)))
                else:
                    b.put(r, p, np.zeros((2, 128)), b.rng.normal(0, 1, (2, 128)))
        run(b, q_scale=q_scale)


@pytest.mark.parametrize("at", [0, 20, 40, 70, 100, 127, 130, 200, 255])
def test_scores_that_leap(at):
    """One key far above all others, met in each part of a tile, after rows of ordinary scores."""
    b = Batch([120], [256], 4, 2, 128, 16, seed=at, k_mean=0.0)
    q = b.rows(4)
    q[:] = q.abs() + 0.5
    b.put(0, at, np.full((2, 128), 20.0) + b.rng.normal(0, 1, (2, 128)), b.rng.normal(0, 1, (2, 128)))
    out = attend(b, q, scale=1.0)
    check(out, *oracle.attention(bits(q), b.cache, b.table, b.qsl, b.lens, 1.0))
