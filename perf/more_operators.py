"""The 8-bit feed-forward step: cases, inputs, plain forms and exact values.

What stands around the attention block of a served layer, weights and activations in 8 bits:

  norm   the residual's addition and the root-mean-square norm, its result in 8 bits
         (ple_norm_mx8), read back as values (ple_mx8_read)
  gated  h = act(x Wg^T) * (x Wu^T), both products, the activation and the result's
         quantisation in one call (ple_gated_mx8), read back as values (ple_mx8_read)
  proj   y = residual + x W^T (ple_proj_mx8), from one token to a prefill's thousands

`run` computes an operator in elementary torch operations in 32 bits where `own` is false, and
through the library's entry points where it is true. `exact` computes it in 64 bits.

8-bit tensors are e4m3 codes, uint8 [rows, columns], with a power of two for each 32 columns of a
row: a byte b stands for 2^(b - 127), 255 for NaN. The largest value of a block decides: the least
power with which it stays within e4m3's 448. The bytes lie as
[rows / 128, rounded up][columns / 128][row % 32][row % 128 / 32][block % 4].
"""

import math
import random

import torch

own = False

MAX_FLOPS = 2.2e12     # of a drawn product: the largest listed one's
MAX_NORM = 8192 * 4096  # elements of a drawn norm
EPS = 1e-6


def listed():
    return [
        # One user, one token, a hidden state of the serving workloads' width: latency alone.
        dict(name="norm_1", op="norm", tokens=1, hidden=4096, residual=True),
        # Speculative decode, 256 requests with 4 tokens each.
        dict(name="norm_256x4", op="norm", tokens=1024, hidden=4096, residual=True),
        # The first norm of a ragged batch, of odd length and width, nothing to add yet.
        dict(name="norm_odd", op="norm", tokens=3001, hidden=2176, residual=False),
        # A prefill step.
        dict(name="norm_prefill", op="norm", tokens=8192, hidden=4096, residual=True),
        # One user's decode step: 138 MB of weights for one token.
        dict(name="gated_1", op="gated", tokens=1, hidden=4096, inner=16384, act="silu"),
        # A batched decode step.
        dict(name="gated_64", op="gated", tokens=64, hidden=4096, inner=16384, act="silu"),
        # A chunk of odd length through a smaller block, tanh-form gelu.
        dict(name="gated_odd", op="gated", tokens=777, hidden=2176, inner=5504, act="gelu"),
        # A prefill step.
        dict(name="gated_prefill", op="gated", tokens=8192, hidden=4096, inner=16384, act="silu"),
        # The second product of one user's decode step: few rows, many columns.
        dict(name="proj_1", op="proj", tokens=1, columns=16384, rows=4096, residual=True),
        # The second product of a batched decode step of odd size.
        dict(name="proj_203", op="proj", tokens=203, columns=16384, rows=4096, residual=True),
        # A chunk of odd length through a projection with an odd number of rows, nothing added.
        dict(name="proj_odd", op="proj", tokens=1023, columns=2048, rows=8195, residual=False),
        # The second product of a prefill step.
        dict(name="proj_prefill", op="proj", tokens=8192, columns=16384, rows=4096, residual=True),
    ]


def _log(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1.0))))))


def draw(rng):
    op = rng.choice(("norm", "gated", "gated", "proj", "proj"))
    if op == "norm":
        hidden = 128 * _log(rng, 4, 64)
        return dict(op=op, tokens=_log(rng, 1, MAX_NORM // hidden), hidden=hidden, residual=rng.random() < 0.7)
    case = dict(op=op, tokens=_log(rng, 1, 8192))
    if op == "gated":
        case.update(hidden=128 * _log(rng, 4, 64), inner=128 * _log(rng, 4, 128), act=rng.choice(("silu", "silu", "gelu")))
        flops = 4.0 * case["hidden"] * case["inner"]
    else:
        case.update(columns=128 * _log(rng, 4, 128), rows=_log(rng, 256, 8192), residual=rng.random() < 0.6)
        flops = 2.0 * case["columns"] * case["rows"]
    case["tokens"] = max(1, min(case["tokens"], int(MAX_FLOPS / flops)))
    return case


def _power(byte):
    """2^(byte - 127) of scale bytes, in float32."""
    bits = byte.to(torch.int32) << 23
    bits = torch.where(byte == 0, 1 << 22, bits)
    return torch.where(byte == 255, 0x7FC00000, bits).view(torch.float32)


def _quantise(x):
    """e4m3 codes [R, C] and scale bytes [R, C / 32] of float32 rows."""
    x = x.unflatten(1, (-1, 32))
    top = x.abs().amax(-1)
    part, power = torch.frexp(top)  # part in [0.5, 1): 448 is 0.875 * 2^9
    byte = (power - 9 + (part > 0.875) + 127).clamp(0, 254)
    byte = torch.where(top > 0, byte, 0)
    code = (x * _power(254 - byte)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    byte = torch.where(torch.isfinite(top), byte, 255)
    return code.flatten(1), byte.to(torch.uint8)


def _laid_out(byte):
    """Scale bytes [R, C / 32] as the products read them."""
    rows, blocks = byte.shape
    whole = torch.zeros((-(-rows // 128) * 128, blocks), dtype=torch.uint8, device=byte.device)
    whole[:rows] = byte
    return whole.view(-1, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4).contiguous().flatten()


def _values(codes, scales):
    """float32 values of codes and laid-out scales."""
    rows, columns = codes.shape
    byte = scales.view(-1, columns // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, columns // 32)[:rows]
    return (codes.view(torch.float8_e4m3fn).float().unflatten(1, (-1, 32)) * _power(byte)[..., None]).flatten(1)


def _packed(x):
    codes, byte = _quantise(x)
    return codes, _laid_out(byte)


def _random_weight(rows, columns, g, dev):
    codes = torch.empty((rows, columns), dtype=torch.uint8, device=dev)
    byte = torch.empty((rows, columns // 32), dtype=torch.uint8, device=dev)
    step = 4096
    for i in range(0, rows, step):
        n = min(step, rows - i)
        codes[i:i + n], byte[i:i + n] = _quantise(torch.randn((n, columns), generator=g, device=dev) * columns ** -0.5)
    return codes, _laid_out(byte)


def _room(rows, columns, dev):
    """Codes and scales of a result."""
    return (torch.empty((rows, columns), dtype=torch.uint8, device=dev),
            torch.empty(-(-rows // 128) * (columns // 128) * 512, dtype=torch.uint8, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = case["tokens"]
    s = dict(op=case["op"])
    if case["op"] == "norm":
        c = case["hidden"]
        # a few channels of a hidden state are far larger than the others
        size = 1.0 + 20.0 * (torch.rand(c, generator=g, device=dev) < 0.005)
        s["x"] = (torch.randn((t, c), generator=g, device=dev) * size).bfloat16()
        s["residual"] = (2.0 * torch.randn((t, c), generator=g, device=dev) * size).bfloat16() if case["residual"] else None
        s["sum"] = torch.empty((t, c), dtype=torch.bfloat16, device=dev) if case["residual"] else None
        s["gamma"] = (1.0 + 0.1 * torch.randn(c, generator=g, device=dev)).bfloat16()
        s["codes"], s["scales"] = _room(t, c, dev)
        s["out"] = torch.empty((t, c), dtype=torch.bfloat16, device=dev)
        return s
    columns = case["hidden"] if case["op"] == "gated" else case["columns"]
    x = torch.randn((t, columns), generator=g, device=dev)
    if case["op"] == "gated":
        s["act"], i = case["act"], case["inner"]
        s["w"], s["w_scales"] = _random_weight(2 * i, columns, g, dev)
        s["codes"], s["scales"] = _room(t, i, dev)
        s["out"] = torch.empty((t, i), dtype=torch.bfloat16, device=dev)
    else:
        x = torch.sigmoid(x) * x * torch.randn((t, columns), generator=g, device=dev)  # as a gated block gives them
        n = case["rows"]
        s["w"], s["w_scales"] = _random_weight(n, columns, g, dev)
        s["residual"] = torch.randn((t, n), generator=g, device=dev).bfloat16() if case["residual"] else None
        s["out"] = torch.empty((t, n), dtype=torch.bfloat16, device=dev)
    s["x"], s["x_scales"] = _packed(x)
    return s


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    out = _values(*_packed(n)).bfloat16()
    return dict(out=out) if s["residual"] is None else dict(out=out, sum=x.bfloat16())


def _plain_gated(s):
    gate, up = torch.matmul(_values(s["x"], s["x_scales"]), _values(s["w"], s["w_scales"]).T).chunk(2, 1)
    turn = gate if s["act"] == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate * gate * gate)
    return _values(*_packed(gate / (1.0 + torch.exp(-turn)) * up)).bfloat16()


def _plain_proj(s):
    y = torch.matmul(_values(s["x"], s["x_scales"]), _values(s["w"], s["w_scales"]).T)
    return (y if s["residual"] is None else y + s["residual"].float()).bfloat16()


def run(s):
    if not own:
        return {"norm": _plain_norm, "gated": _plain_gated, "proj": _plain_proj}[s["op"]](s)
    import hashed_gram_embedding_gb300 as ple
    if s["op"] == "norm":
        ple.ple_norm_mx8(s["x"], s["gamma"], s["codes"], s["scales"], residual=s["residual"], sum_out=s["sum"], eps=EPS)
        ple.ple_mx8_read(s["codes"], s["scales"], s["out"])
        return dict(out=s["out"]) if s["residual"] is None else dict(out=s["out"], sum=s["sum"])
    if s["op"] == "gated":
        ple.ple_gated_mx8(s["x"], s["x_scales"], s["w"], s["w_scales"], s["codes"], s["scales"], activation=s["act"])
        ple.ple_mx8_read(s["codes"], s["scales"], s["out"])
        return s["out"]
    ple.ple_proj_mx8(s["x"], s["x_scales"], s["w"], s["w_scales"], s["out"], residual=s["residual"])
    return s["out"]


def work(case):
    t = case["tokens"]
    eight = 33.0 / 32.0  # bytes of a code and its share of a scale
    if case["op"] == "norm":
        # x (and the residual) in, the sum, the codes and the values read from them out
        c = case["hidden"]
        return {"bytes": t * c * (2 + (4 if case["residual"] else 0) + eight + 2) + 2 * c, "flops": 10.0 * t * c}
    if case["op"] == "gated":
        c, i = case["hidden"], case["inner"]
        return {"bytes": eight * (2 * i * c + t * c + t * i) + 2 * t * i, "flops": 4.0 * t * c * i}
    e, n = case["columns"], case["rows"]
    return {"bytes": eight * (n * e + t * e) + t * n * (4 if case["residual"] else 2), "flops": 2.0 * t * e * n}


def _decoded(codes, scales):
    """float64 values, element by element from the definition."""
    r, c = codes.shape
    row = torch.arange(r, device=codes.device)[:, None]
    block = torch.arange(c // 32, device=codes.device)
    at = (row // 128 * (c // 128) + block // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + block % 4
    power = torch.exp2(scales[at].double() - 127)
    code = torch.arange(256, device=codes.device)
    field, part = code // 8 % 16, (code % 8).double()
    value = torch.where(field > 0, (1 + part / 8) * torch.exp2(field.double() - 7), part / 8 * 2.0 ** -6)
    value = torch.where(code % 128 == 127, math.nan, torch.where(code < 128, value, -value))
    return value[codes.int()] * power.repeat_interleave(32, 1)


def _rounded(x):
    """The values that float64 rows have in 8 bits."""
    x = x.view(x.shape[0], -1, 32)
    top = x.abs().max(2, keepdim=True).values
    low = torch.floor(torch.log2(top / 448)).nan_to_num(neginf=-127)  # one less where the logarithm is a whole number
    for _ in range(2):
        low = torch.where(top > 448 * torch.exp2(low), low + 1, low)
    power = torch.exp2(low.clamp(min=-127))
    y = x / power
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step * power).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        if s["residual"] is not None:
            x += s["residual"].double()
        norm = x / torch.sqrt((x * x).sum(1, keepdim=True) / case["hidden"] + EPS)
        out = _rounded(norm * s["gamma"].double())
        return dict(out=out) if s["residual"] is None else dict(out=out, sum=x)
    y = _decoded(s["x"], s["x_scales"]) @ _decoded(s["w"], s["w_scales"]).T
    if case["op"] == "proj":
        return y if s["residual"] is None else y + s["residual"].double()
    gate, up = y[:, :case["inner"]], y[:, case["inner"]:]
    if case["act"] == "silu":
        return _rounded(torch.sigmoid(gate) * gate * up)
    return _rounded(0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))) * up)
