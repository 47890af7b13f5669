"""PLEFeedForward: the gated feed-forward block that stands behind an
attention block, its weights and what passes between its products in 8 bits.

Three libple calls on one stream: the residual's addition and the norm
(ple_norm_mx8), both projections with the activation and their product
(ple_gated_mx8), and the projection back with the residual added
(ple_proj_mx8). Device memory comes from PyTorch, once, at construction; a
step allocates nothing unless its result has no place given, so it can be
captured in a CUDA graph.
"""

import torch

from . import _lib


def pack_mx8(weight):
    """(codes, scales) of a weight [N, E] as the 8-bit products read it: e4m3
    codes uint8 [N, E] and the powers of two of each 32 columns, laid out as
    include/ple.h says. Preparation in PyTorch, on the weight's device."""
    N, E = weight.shape
    if E % 128 != 0:
        raise ValueError(f"{E} columns are not a multiple of 128")
    w = weight.to(torch.float32).contiguous().view(N, E // 32, 32)  # codes lie as w does
    top = w.abs().amax(2)
    part, power = torch.frexp(top)  # top = part * 2^power, part in [0.5, 1); 448 = 0.875 * 2^9
    byte = torch.where(top > 0, (power + (part > 0.875) + 118).clamp(min=0), 0)
    # 2^(127 - b), written as its bits: b is 247 at most for a finite block
    inverse = ((254 - byte.clamp(max=253)).to(torch.int32) << 23).view(torch.float32)
    codes = (w * inverse[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(N, E)
    byte = torch.where(torch.isfinite(top), byte, 255).to(torch.uint8)
    rows = -(-N // 128) * 128
    scales = torch.zeros((rows, E // 32), dtype=torch.uint8, device=weight.device)
    scales[:N] = byte
    return codes, scales.view(-1, 4, 32, E // 128, 4).permute(0, 3, 2, 1, 4).reshape(-1)


class PLEFeedForward:
    """Weights and buffers of one feed-forward block.

    Args:
      w_gate_up: (codes, scales) of the merged weight [2 I, C], the gate's rows
        before the other half's (see pack_mx8).
      w_down: the same of the weight [C, I].
      gamma: bf16 [C] of the norm, or None for 1.
      max_tokens: the most tokens of a step.
      activation: "silu" or "gelu" (its tanh form).
      eps: of the norm.

    Building one waits for the current stream's work, and so is no part of a
    graph's capture.
    """

    def __init__(self, w_gate_up, w_down, gamma, max_tokens, activation="silu", eps=1e-6):
        self.w_gate_up, self.w_down, self.gamma = w_gate_up, w_down, gamma
        self.activation, self.eps = activation, float(eps)
        self.max_tokens = int(max_tokens)
        (rows, self.hidden), (out, self.inner) = _lib._mx8("w_gate_up", *w_gate_up), _lib._mx8("w_down", *w_down)
        if rows != 2 * self.inner or out != self.hidden:
            raise ValueError(f"w_gate_up {tuple(w_gate_up[0].shape)} and w_down {tuple(w_down[0].shape)} "
                             "are not [2 I, C] and [C, I]")
        if activation not in _lib._ACTIVATIONS:
            raise ValueError(f"activation {activation!r}: one of {', '.join(_lib._ACTIVATIONS)} is needed")
        device = w_gate_up[0].device

        def room(columns):
            scales = _lib.ple_mx8_scale_bytes(self.max_tokens, columns)
            return (torch.empty((self.max_tokens, columns), dtype=torch.uint8, device=device),
                    torch.empty((scales,), dtype=torch.uint8, device=device))

        self.normed, self.gated = room(self.hidden), room(self.inner)
        self.sum = torch.empty((self.max_tokens, self.hidden), dtype=torch.bfloat16, device=device)
        # torch may give memory that this stream's earlier work still uses, and
        # a first step may be on any stream
        torch.cuda.current_stream(device).synchronize()

    def forward(self, hidden, delta=None, dev_err=None, stream=None, out=None):
        """hidden [T, C] bf16, delta [T, C] bf16 or None (the attention block's
        result, not yet added) -> s + FFN(norm(s)), s = hidden + delta, as
        [T, C] bf16. out may be hidden. The steps of one block run one after
        another (they share its buffers): a step on another stream than the
        last one's has to wait for it. A result that has no place given is a
        tensor of the stream that the step runs on."""
        T = hidden.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens, and buffers for {self.max_tokens}")
        if out is None:
            with torch.cuda.stream(stream):  # where its memory may be written at once (None: the current one)
                out = torch.empty((T, self.hidden), dtype=torch.bfloat16, device=hidden.device)
        (codes, scales), (h_codes, h_scales) = self.normed, self.gated
        codes, h_codes, total = codes[:T], h_codes[:T], hidden
        if delta is not None:
            total = self.sum[:T]
        _lib.ple_norm_mx8(hidden, self.gamma, codes, scales, residual=delta,
                          sum_out=None if delta is None else total, eps=self.eps, stream=stream)
        _lib.ple_gated_mx8(codes, scales, *self.w_gate_up, h_codes, h_scales, activation=self.activation,
                           dev_err=dev_err, stream=stream)
        _lib.ple_proj_mx8(h_codes, h_scales, *self.w_down, out, residual=total, dev_err=dev_err, stream=stream)
        return out
