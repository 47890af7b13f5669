"""PLEAttention: the attention block that stands between two PLE layers, with
everything that grows or is read whole each step in 4 bits.

Four libple calls on one stream: the fused q, k, v projection (ple_proj_w4),
rotation and the store into the paged cache (ple_kv_append), attention over the
cache (ple_kv_attention) and the output projection (ple_proj_w4). Device memory
comes from PyTorch, once, at construction; a step allocates nothing unless its
result has no place given, so it can be captured in a CUDA graph.
"""

import torch

from . import _lib


def pack_w4(weight, group=128):
    """(codes, scales, zeros) of a weight [N, E] as ple_proj_w4 reads them: the
    range of each group of columns, widened to hold 0, in 15 steps. Preparation
    in PyTorch, on the weight's device."""
    N, E = weight.shape
    if E % group != 0:
        raise ValueError(f"{E} columns are not a multiple of the group {group}")
    w = weight.to(torch.float32).view(N, E // group, group)
    low, high = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
    scales = ((high - low) / 15).clamp(min=2.0 ** -126).to(torch.bfloat16)  # as the kernel will use them
    step = scales.to(torch.float32)
    zeros = (-low / step).round().clamp(0, 15)
    codes = ((w / step[..., None]).round() + zeros[..., None]).clamp(0, 15).to(torch.uint8).view(N, E)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales, zeros.to(torch.uint8)


class PLEAttention:
    """Weights, paged cache and buffers of one attention block.

    Args:
      w_qkv: (codes, scales, zeros) of the merged weight [(H + 2 Hk) D, C], rows
        in the order q, k, v (see pack_w4; zeros None: 8 everywhere).
      w_out: the same of the output weight [C, H D].
      num_heads, num_kv_heads, head_dim: H, Hk (a divisor of H), D (64, 128, 256).
      num_pages, page_size: of the cache; page_size a multiple of 16.
      max_tokens: the most tokens of a step.
      cos_sin: float32 [positions, rotary_dim], cos then sin, or None.
      interleaved: rotate neighbouring elements instead of the halves.
      window: positions that a token sees, itself among them; 0: all before it.
      scale: of the scores; 1 / sqrt(D) by default.
      cache: a cache to use, uint8 [num_pages, Hk, page_size / 16, 16 (D + 8)],
        or None for one of its own.
    """

    def __init__(self, w_qkv, w_out, num_heads, num_kv_heads, head_dim, num_pages, page_size,
                 max_tokens, cos_sin=None, interleaved=False, window=0, scale=None, cache=None):
        self.w_qkv, self.w_out = w_qkv, w_out
        self.num_heads, self.num_kv_heads, self.head_dim = int(num_heads), int(num_kv_heads), int(head_dim)
        self.cos_sin, self.interleaved = cos_sin, bool(interleaved)
        self.window, self.scale = int(window), scale
        self.max_tokens = int(max_tokens)
        device = w_qkv[0].device
        rows = (self.num_heads + 2 * self.num_kv_heads) * self.head_dim
        if w_qkv[0].shape[0] != rows or w_out[0].shape[1] * 2 != self.num_heads * self.head_dim:
            raise ValueError(f"w_qkv has {w_qkv[0].shape[0]} rows and w_out {w_out[0].shape[1] * 2} columns, "
                             f"not {rows} and {self.num_heads * self.head_dim}")
        self.hidden = w_out[0].shape[0]
        block = _lib.ple_kv_block_bytes(self.head_dim)
        room = _lib.ple_kv_attention_workspace(self.num_heads, self.num_kv_heads, self.head_dim)
        if block == 0 or room == 0 or page_size < 16 or page_size % 16 != 0:
            raise ValueError(f"{num_heads} heads, {num_kv_heads} kv heads of {head_dim} in pages of "
                             f"{page_size} are not supported")
        shape = (int(num_pages), self.num_kv_heads, page_size // 16, block)
        self.cache = torch.zeros(shape, dtype=torch.uint8, device=device) if cache is None else cache
        if tuple(self.cache.shape) != shape:
            raise ValueError(f"cache has the shape {tuple(self.cache.shape)}, not {shape}")
        # zero-filled once: each completed call leaves it ready for the next
        self.workspace = torch.zeros((room,), dtype=torch.uint8, device=device)
        self.qkv = torch.empty((self.max_tokens, rows), dtype=torch.bfloat16, device=device)
        self.mixed = torch.empty((self.max_tokens, self.num_heads, self.head_dim), dtype=torch.bfloat16,
                                 device=device)
        # the fills above are on this stream, and a first step may be on any
        torch.cuda.current_stream(device).synchronize()

    def forward(self, hidden, block_table, query_start_loc, kv_lens, positions=None, max_query_len=0,
                dev_err=None, stream=None, out=None):
        """hidden [T, C] bf16 -> [T, C] bf16 (no residual added): prompts, single
        tokens and both in one batch. block_table int32 [R, max_pages],
        query_start_loc int32 [R + 1], kv_lens int32 [R] (this step's tokens
        included); positions int32 [T] or None for the places in the cache;
        max_query_len: the most tokens of a request, if known (0 costs steps of
        single tokens several times the attention's time). The steps of one
        block run one after another (they share its buffers): a step on another
        stream than the last one's has to wait for it. A result that has no
        place given is a tensor of the stream that the step runs on."""
        T = hidden.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens, and buffers for {self.max_tokens}")
        H, Hk, D = self.num_heads, self.num_kv_heads, self.head_dim
        qkv, mixed = self.qkv[:T], self.mixed[:T]
        if out is None:
            with torch.cuda.stream(stream):  # where its memory may be written at once (None: the current one)
                out = torch.empty((T, self.hidden), dtype=torch.bfloat16, device=hidden.device)
        codes, scales, zeros = self.w_qkv
        _lib.ple_proj_w4(hidden, codes, scales, qkv, zeros=zeros, dev_err=dev_err, stream=stream)
        q, k, v = qkv.view(T, H + 2 * Hk, D).split((H, Hk, Hk), dim=1)
        _lib.ple_kv_append(q, k, v, self.cos_sin, self.cache, block_table, query_start_loc, kv_lens, q,
                           positions=positions, interleaved=self.interleaved, dev_err=dev_err,
                           stream=stream)
        _lib.ple_kv_attention(q, self.cache, block_table, query_start_loc, kv_lens, mixed, self.workspace,
                              scale=self.scale, window=self.window, max_query_len=max_query_len,
                              dev_err=dev_err, stream=stream)
        codes, scales, zeros = self.w_out
        _lib.ple_proj_w4(mixed.view(T, H * D), codes, scales, out, zeros=zeros, dev_err=dev_err,
                         stream=stream)
        return out
