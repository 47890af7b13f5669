"""The 4-bit serving operators: cases, inputs, plain forms and exact values.

An attention block's step over a paged key/value cache that is held in 4 bits, next to a
per-layer embedding layer:

  append     rotate q and k by position, quantise k and v to 4 bits into the paged cache
             (ple_kv_append), and read the appended tokens back as values (ple_kv_read)
  attention  grouped-query attention of ragged requests over the 4-bit cache
             (ple_kv_attention), from one query token a request to long prefill chunks
  proj       y = x W^T with a weight of 4-bit codes, a scale and (optionally) a zero point
             for each group of columns (ple_proj_w4), for steps of few tokens

`run` computes an operator in elementary torch operations in 32 bits where `own` is false, and
through the library's entry points where it is true. `exact` computes it in 64 bits.

The cache is a uint8 tensor [pages, kv_heads, page_size / 16, 16 * (D + 8)]: a block holds 16
tokens of one head, as K codes [16][D/2], V codes [16][D/2], K (scale, offset) [16][2] and
V (scale, offset) [16][2] in bf16. Element d of a row is the low (even d) or high (odd d) half
of byte d/2, and stands for code * scale + offset with scale = bf16((max - min) / 15) and
offset = bf16(min) of its row.
"""

import math
import random

import torch

own = False

# Head layouts (query heads, kv heads, head dim): 32 x 128 makes up the 4096-wide hidden state of
# the serving workloads, the others are its smaller and wider relatives.
LAYOUTS = ((32, 8, 128), (32, 4, 128), (8, 8, 64), (24, 3, 64), (16, 2, 256), (10, 5, 128), (12, 1, 128))
PAGES = (16, 32, 64, 128)
MAX_BYTES = 1.2e9      # of cache in a drawn attention case
MAX_SCORES = 2.0e9     # padded (row, position) pairs in a drawn attention case
MAX_FLOPS = 5.0e11
WORKSPACE = 64 << 20   # bytes a serving program sets aside for the attention's partial results


def listed():
    h = dict(heads=32, kv_heads=8, dim=128)
    return [
        # One user, one token: the latency of a single decode step.
        dict(name="append_1", op="append", requests=1, query=1, context=700, ragged=False, lengths=1, page=16, rotary=128, interleaved=False, **h),
        # Speculative decode, 256 requests with 4 tokens each.
        dict(name="append_256x4", op="append", requests=256, query=4, context=4096, ragged=True, lengths=2, page=16, rotary=128, interleaved=False, **h),
        # A ragged prefill of about 8192 tokens over 16 requests.
        dict(name="append_prefill", op="append", requests=16, query=1024, context=0, ragged=True, lengths=3, page=64, rotary=128, interleaved=False, **h),
        # One user's decode step over a short conversation: latency alone.
        dict(name="attention_1x700", op="attention", requests=1, query=1, context=699, ragged=False, lengths=4, page=16, window=0, **h),
        # One user's decode step over a long document of odd length: the cache split over the whole card.
        dict(name="attention_1x131071", op="attention", requests=1, query=1, context=131070, ragged=False, lengths=5, page=64, window=0, **h),
        # Batched decode, 256 ragged requests.
        dict(name="attention_256x1", op="attention", requests=256, query=1, context=8192, ragged=True, lengths=6, page=16, window=0, **h),
        # Speculative decode, 256 requests with 4 tokens each.
        dict(name="attention_256x4", op="attention", requests=256, query=4, context=4096, ragged=True, lengths=7, page=16, window=0, **h),
        # A ragged prefill of about 8192 tokens over 16 requests, each behind a cached prefix.
        dict(name="attention_prefill", op="attention", requests=16, query=1024, context=2000, ragged=True, lengths=8, page=64, window=0, **h),
        # A chunk of a long document's prefill.
        dict(name="attention_2048x16k", op="attention", requests=1, query=2048, context=14336, ragged=False, lengths=9, page=128, window=0, **h),
        # The merged key/value projection of one decode token, 2048 -> 2 x 4096.
        dict(name="proj_1", op="proj", tokens=1, columns=2048, rows=8192, group=128, zeros=False),
        # A batch of odd size through a square projection of the hidden state, with zero points.
        dict(name="proj_13", op="proj", tokens=13, columns=4096, rows=4096, group=64, zeros=True),
        # The widest batch of a decode step through a wide projection.
        dict(name="proj_64", op="proj", tokens=64, columns=4096, rows=16384, group=128, zeros=True),
    ]


def _log(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1.0))))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "attention", "proj"))
    if op == "proj":
        group = rng.choice((32, 64, 128))
        columns = group * _log(rng, 512 // group, 8192 // group)
        return dict(op=op, tokens=_log(rng, 1, 64), columns=columns - group if columns == 3072 else columns,
                    rows=8 * _log(rng, 32, 1024) + rng.randint(1, 7), group=group, zeros=rng.random() < 0.5)
    heads, kv_heads, dim = rng.choice(LAYOUTS)
    case = dict(op=op, requests=_log(rng, 1, 256), query=1, context=0, ragged=rng.random() < 0.8, lengths=rng.randrange(1 << 20),
                page=rng.choice(PAGES), heads=heads, kv_heads=kv_heads, dim=dim)
    if op == "append":
        case["query"] = _log(rng, 1, max(1, 8192 // case["requests"]))
        case["context"] = _log(rng, 1, 4096)
        case["rotary"] = rng.choice((dim, dim, dim // 2))
        case["interleaved"] = rng.random() < 0.3
        return case
    case["window"] = rng.choice((0, 0, 0, _log(rng, 16, 4096)))
    case["query"] = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 9, 1024)))
    case["context"] = _log(rng, 1, 131072)
    while True:  # shorter until it costs no more than the largest listed case
        n, c, r = case["query"], case["context"], case["requests"]
        scores = r * heads * n * (n + c)
        if r * (n + c) * kv_heads * (dim + 8) <= MAX_BYTES and scores <= MAX_SCORES and 4.0 * scores * dim <= MAX_FLOPS:
            return case
        if c > n:
            case["context"] = c * 3 // 4
        elif r > 1:
            case["requests"] = r * 3 // 4
        else:
            case["query"] = n * 3 // 4


def _lengths(case):
    """Query tokens and cache length (these tokens included) of each request."""
    rng = random.Random(case["lengths"])
    queries, lens = [], []
    for _ in range(case["requests"]):
        n, c = case["query"], case["context"]
        if case["ragged"]:
            n = n if n <= 8 else rng.randint(1, n)
            c = rng.randint(c // 8, c)
        queries.append(n)
        lens.append(n + c)
    return queries, lens


def _quantise(x):
    """4-bit codes, scale and offset of rows of float32 values."""
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale, offset = ((high - low) / 15).bfloat16(), low.bfloat16()
    s = scale.float()
    code = torch.where(s > 0, (x - offset.float()) / s, torch.zeros_like(x)).round().clamp(0, 15)
    return code.to(torch.uint8), torch.cat([scale, offset], -1)


def _blocks(k, v):
    """Cache blocks of keys and values [..., 16, D]: uint8 [..., 16 * (D + 8)]."""
    parts = []
    for x in (k, v):
        code, pair = _quantise(x)
        parts.append(((code[..., 0::2] | (code[..., 1::2] << 4)).flatten(-2), pair.view(torch.uint8).flatten(-2)))
    return torch.cat([parts[0][0], parts[1][0], parts[0][1], parts[1][1]], -1)


def _values(blocks, dim):
    """Keys and values [..., 16, D] in float32 of cache blocks."""
    n = 8 * dim
    pairs = blocks[..., 2 * n:].contiguous().view(torch.bfloat16).float().unflatten(-1, (2, 16, 2))
    out = []
    for i in range(2):
        b = blocks[..., i * n:(i + 1) * n].unflatten(-1, (16, dim // 2))
        code = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
        out.append(code * pairs[..., i, :, :1] + pairs[..., i, :, 1:])
    return out


def _filled(pages, case, g, dev):
    """A cache whose pages hold keys with channel offsets, as rotated keys have, and centred values."""
    hk, d, sub = case["kv_heads"], case["dim"], case["page"] // 16
    cache = torch.empty((pages, hk, sub, 16 * (d + 8)), dtype=torch.uint8, device=dev)
    means = torch.randn((hk, 1, 1, d), generator=g, device=dev)
    step = max(1, (1 << 27) // (hk * sub * 16 * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn((2, n, hk, sub, 16, d), generator=g, device=dev)
        cache[i:i + n] = _blocks(x[0] + means, x[1])
    return cache


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    if case["op"] == "proj":
        t, e, n, group = case["tokens"], case["columns"], case["rows"], case["group"]
        s = dict(op="proj", group=group)
        s["x"] = torch.randn((t, e), generator=g, device=dev).bfloat16()
        s["codes"] = torch.randint(0, 256, (n, e // 2), generator=g, device=dev, dtype=torch.uint8)
        s["scales"] = (0.004 * (0.5 + torch.rand((n, e // group), generator=g, device=dev))).bfloat16()
        s["zeros"] = torch.randint(5, 11, (n, e // group), generator=g, device=dev, dtype=torch.uint8) if case["zeros"] else None
        s["out"] = torch.empty((t, n), dtype=torch.bfloat16, device=dev)
        return s
    queries, lens = _lengths(case)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    t, most = sum(queries), max(-(-n // page) for n in lens)
    pages = sum(-(-n // page) for n in lens)
    order = torch.randperm(pages, generator=g, device=dev).int()
    used = torch.tensor([-(-n // page) for n in lens], device=dev)
    first = used.cumsum(0) - used
    at = torch.arange(most, device=dev)
    table = torch.where(at < used[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], 0).int()
    s = dict(op=case["op"], dim=d, heads=hq, kv_heads=hk, page=page, queries=max(queries), longest=max(lens), block_table=table.contiguous())
    s["query_start_loc"] = torch.tensor([0] + queries, device=dev).cumsum(0).int()
    s["kv_lens"] = torch.tensor(lens, device=dev).int()
    if case["op"] == "append":
        s["cache"] = torch.zeros((pages, hk, page // 16, 16 * (d + 8)), dtype=torch.uint8, device=dev)
        # q, k and v are columns of one fused projection
        s["qkv"] = torch.randn((t, (hq + 2 * hk) * d), generator=g, device=dev).bfloat16()
        rot = case["rotary"]
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        angle = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
        s["interleaved"] = case["interleaved"]
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.empty((t, hk, d), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty((t, hk, d), dtype=torch.bfloat16, device=dev)
        return s
    s["cache"] = _filled(pages, case, g, dev)
    s["q"] = torch.randn((t, hq, d), generator=g, device=dev).bfloat16()
    s["out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
    s["window"] = case["window"]
    s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=dev)
    return s


def _split(s):
    """q, k and v of the fused projection, as heads."""
    hq, hk, d = s["heads"], s["kv_heads"], s["dim"]
    q, k, v = s["qkv"].split([hq * d, hk * d, hk * d], 1)
    return q.unflatten(1, (hq, d)), k.unflatten(1, (hk, d)), v.unflatten(1, (hk, d))


def _places(s, t):
    """Request and position of every token."""
    start = s["query_start_loc"].long()
    at = torch.arange(t, device=start.device)
    r = torch.searchsorted(start, at, right=True) - 1
    return r, at - start[r + 1] + s["kv_lens"].long()[r]


def _rotated(x, cos, sin, rot, interleaved):
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = [a * cos - b * sin, b * cos + a * sin]
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    q, k, v = (x.float() for x in _split(s))
    d, page, rot = s["dim"], s["page"], s["cos_sin"].shape[1]
    r, pos = _places(s, q.shape[0])
    cos, sin = s["cos_sin"][pos].unsqueeze(1).split(rot // 2, -1)
    q, k = (_rotated(x, cos, sin, rot, s["interleaved"]) for x in (q, k))
    block, slot = s["block_table"][r, pos // page].long(), pos % page
    cells, n = s["cache"], 8 * d
    where = (block[:, None], torch.arange(k.shape[1], device=k.device), slot[:, None] // 16)
    for i, x in enumerate((k, v)):
        code, pair = _quantise(x)
        row = cells[..., i * n:(i + 1) * n].unflatten(-1, (16, d // 2))
        row[where + (slot[:, None] % 16,)] = code[..., 0::2] | (code[..., 1::2] << 4)
        row = cells[..., 2 * n + 64 * i:2 * n + 64 * (i + 1)].unflatten(-1, (16, 4))
        row[where + (slot[:, None] % 16,)] = pair.view(torch.uint8)
    tokens = torch.arange(k.shape[0], device=k.device)[:, None]
    heads = torch.arange(k.shape[1], device=k.device)
    back = [x[tokens, heads, slot[:, None] % 16] for x in _values(cells[where], d)]
    return dict(q=q.bfloat16(), k=back[0].bfloat16(), v=back[1].bfloat16())


def _plain_attention(s):
    hq, hk, d, page = s["heads"], s["kv_heads"], s["dim"], s["page"]
    start, lens = s["query_start_loc"].long(), s["kv_lens"].long()
    n, used = start[1:] - start[:-1], -(-s["longest"] // page)
    i = torch.arange(s["queries"], device=n.device)
    live = i < n[:, None]
    q = s["q"][(start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.unflatten(2, (hk, hq // hk)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    blocks = s["cache"][s["block_table"][:, :used].long()].transpose(1, 2)
    k, v = (x.flatten(2, 4) for x in _values(blocks, d))
    score = torch.matmul(q * d ** -0.5, k.transpose(2, 3))
    del k
    last = lens[:, None] - n[:, None] + i
    p = torch.arange(score.shape[-1], device=n.device)
    seen = p <= last[..., None]
    if s["window"]:
        seen = seen & (p > last[..., None] - s["window"])
    seen = seen[:, None, :, None, :].expand(-1, hk, -1, hq // hk, -1).flatten(2, 3)
    score = score.masked_fill_(~seen, float("-inf"))
    score = score.sub_(score.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, v) / torch.where(total > 0, total, 1.0)
    out = out.unflatten(2, (-1, hq // hk)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return out[live].bfloat16()


def _plain_proj(s):
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(1).unflatten(1, (-1, s["group"])).float()
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w = ((code - zero) * s["scales"].float()[..., None]).flatten(1)
    return torch.matmul(s["x"].float(), w.T).bfloat16()


def run(s):
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "proj": _plain_proj}[s["op"]](s)
    import hashed_gram_embedding_gb300 as ple
    if s["op"] == "append":
        q, k, v = _split(s)
        ple.ple_kv_append(q, k, v, s["cos_sin"], s["cache"], s["block_table"], s["query_start_loc"], s["kv_lens"], s["q_out"],
                          interleaved=s["interleaved"])
        ple.ple_kv_read(s["cache"], s["block_table"], s["query_start_loc"], s["kv_lens"], s["k_out"], s["v_out"])
        return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
    if s["op"] == "attention":
        ple.ple_kv_attention(s["q"], s["cache"], s["block_table"], s["query_start_loc"], s["kv_lens"], s["out"], s["workspace"],
                             window=s["window"], max_query_len=s["queries"])
        return s["out"]
    ple.ple_proj_w4(s["x"], s["codes"], s["scales"], s["out"], zeros=s["zeros"])
    return s["out"]


def work(case):
    if case["op"] == "proj":
        t, e, n, groups = case["tokens"], case["columns"], case["rows"], case["columns"] // case["group"]
        return {"bytes": n * e // 2 + n * groups * (3 if case["zeros"] else 2) + 2 * t * (e + n), "flops": 2.0 * t * e * n}
    queries, lens = _lengths(case)
    t, hq, hk, d = sum(queries), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        # q, k, v and the rotations in; q and the cache rows out; the values read back from them
        return {"bytes": t * (2 * hq * d * 2 + 2 * hk * d * 2 + 4 * case["rotary"] + hk * (d + 8) + 2 * hk * d * 2),
                "flops": t * (3.0 * (hq + hk) * case["rotary"] + 8.0 * hk * d)}
    window = case["window"] or 1 << 40
    read = sum(min(n, window + q - 1) for q, n in zip(queries, lens))
    pairs = sum(min(n - q + i + 1, window) for q, n in zip(queries, lens) for i in range(q))
    return {"bytes": 4 * t * hq * d + read * hk * (d + 8), "flops": 4.0 * pairs * hq * d}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "proj":
        e, group, c = case["columns"], case["group"], s["codes"].to(torch.int32)
        w = torch.empty((case["rows"], e), dtype=f64, device=c.device)
        w[:, 0::2], w[:, 1::2] = c % 16, c // 16
        column = torch.arange(e, device=c.device) // group
        w -= 8 if s["zeros"] is None else s["zeros"].to(f64)[:, column]
        w *= s["scales"].to(f64)[:, column]
        return s["x"].to(f64) @ w.T
    queries, lens = _lengths(case)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(n - q, n) for q, n in zip(queries, lens)])
        rot = case["rotary"]
        turn = torch.complex(*s["cos_sin"].cpu()[pos].to(f64).split(rot // 2, 1))
        out = {}
        for name, x in zip("qkv", _split(s)):
            x = x.cpu().to(f64).clone()
            if name != "v":
                pairs = [x[..., i:rot:2] for i in (0, 1)] if case["interleaved"] else [x[..., :rot // 2], x[..., rot // 2:rot]]
                z = torch.complex(*(p.clone() for p in pairs)) * turn[:, None]
                pairs[0].copy_(z.real)
                pairs[1].copy_(z.imag)
            if name != "q":
                scale = ((x.amax(-1) - x.amin(-1)) / 15).bfloat16().to(f64)[..., None]
                offset = x.amin(-1).bfloat16().to(f64)[..., None]
                x = ((x - offset) / scale).round().clamp(0, 15) * scale + offset
            out[name] = x
        return out
    out, t0 = [], 0
    for r, (n, length) in enumerate(zip(queries, lens)):
        pages = s["block_table"][r, :-(-length // page)].long()
        raw = s["cache"][pages].permute(1, 0, 2, 3).reshape(hk, -1, 16 * (d + 8))
        pair = raw[..., 16 * d:].reshape(-1).contiguous().view(torch.bfloat16).to(f64).view(hk, -1, 2, 16, 2)
        kv = []
        for i in (0, 1):
            byte = raw[..., i * 8 * d:(i + 1) * 8 * d].reshape(hk, -1, 16, d // 2, 1).to(torch.int32)
            code = torch.cat([byte % 16, byte // 16], -1).reshape(hk, -1, 16, d).to(f64)
            kv.append((code * pair[:, :, i, :, 0:1] + pair[:, :, i, :, 1:2]).reshape(hk, -1, d)[:, :length])
        qs = s["q"][t0:t0 + n].to(f64)
        t0 += n
        last = torch.arange(length - n, length, device=qs.device)[:, None]
        p = torch.arange(length, device=qs.device)
        hidden = (p > last) | (p <= last - (case["window"] or length + 1))
        each = []
        for h in range(hq):
            a = (qs[:, h] @ kv[0][h // (hq // hk)].T) / math.sqrt(d)
            each.append(torch.softmax(a.masked_fill(hidden, -math.inf), -1) @ kv[1][h // (hq // hk)])
        out.append(torch.stack(each, 1))
    return torch.cat(out)
