"""A decoder layer with int4 weights, served from a paged cache: prefill of prompts that
share a system prompt, then decoding, all between the norms in this library.

    python examples/quantized_decoder_layer.py [--tokens 4]

One layer of 7B size (32 query and 8 key / value heads of 128, feed-forward 11008) with
random weights: query / key / value projection -> rotary append -> attention -> output
projection -> gated feed-forward -> down projection.  The system prompt is computed once
and its pages are shared by every sequence.  Ends with one step of adapter training
through the frozen feed-forward (its input's gradient).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_quantized_mixed_amd.device import PagedKV, QGated, QGemm  # noqa: E402

HIDDEN, INNER, Q_HEADS, KV_HEADS, HEAD_DIM, GROUP, PAGE = 4096, 11008, 32, 8, 128, 128, 16


def int4(n, k, gen):
    """Random canonical int4 words [n, k / 8] and fp16 scales [n, k / GROUP]."""
    words = torch.randint(-2**31, 2**31, (n, k // 8), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    scales = (torch.rand((n, k // GROUP), generator=gen, device="cuda") * 0.5 + 0.75) / (4.6 * k**0.5)
    return words, scales.half()


def rms_norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5)).half()


class Layer:
    """The layer's plans, packed weights and cache for up to max_rows tokens a call."""

    def __init__(self, max_rows, n_pages, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.widths = [Q_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM]
        shapes = {"qkv": (sum(self.widths), HIDDEN), "out": (HIDDEN, Q_HEADS * HEAD_DIM), "down": (HIDDEN, INNER)}
        self.plans = {name: QGemm(max_rows, n, k, "i4", GROUP) for name, (n, k) in shapes.items()}
        self.packed = {name: self.plans[name].pack(*int4(n, k, gen)) for name, (n, k) in shapes.items()}
        self.ffn = QGated(max_rows, INNER, HIDDEN, "i4", GROUP, act="silu")
        (wg, sg), (wu, su) = int4(INNER, HIDDEN, gen), int4(INNER, HIDDEN, gen)
        self.ffn_packed = self.ffn.pack(wg, wu, sg, su)
        self.cache = PagedKV(n_pages, PAGE, KV_HEADS, HEAD_DIM)
        angles = torch.arange(8192, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, HEAD_DIM, 2, device="cuda") / HEAD_DIM)
        self.cos, self.sin = angles.cos().float().contiguous(), angles.sin().float().contiguous()

    def product(self, name, x):
        return self.plans[name].run(x, self.packed[name], M=x.shape[0])

    def __call__(self, x, positions, slots, starts, lens, tables, max_q, max_len, prefix_table=None, prefix_len=0):
        rows = x.shape[0]
        q, k, v = self.product("qkv", rms_norm(x)).split(self.widths, dim=1)
        q = self.cache.append(q, k, v, self.cos, self.sin, positions, slots)
        y = self.cache.attend(q, starts, lens, tables, max_q, max_len, prefix_table, prefix_len)
        x = x + self.product("out", y.view(rows, -1))
        return x + self.product("down", self.ffn.run(rms_norm(x), self.ffn_packed, M=rows))


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def slots_of(table, tokens):
    """Cache slots of tokens (numbers within a sequence) from its page table."""
    return table.long()[tokens // PAGE] * PAGE + tokens % PAGE


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4, help="tokens to decode for each sequence")
    args = ap.parse_args()
    prefix, prompts = 1000, [37, 120, 5, 64]
    room = max(prompts) + args.tokens
    width = -(-room // PAGE)
    n_prefix = -(-prefix // PAGE)
    layer = Layer(1024, n_prefix + len(prompts) * width)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def hidden(n):
        return torch.randn((n, HIDDEN), generator=gen, device="cuda").half()

    # the system prompt, once
    pages = torch.arange(n_prefix, dtype=torch.int32, device="cuda")
    t = torch.arange(prefix, device="cuda")
    layer(hidden(prefix), t.int(), slots_of(pages, t), int32([0, prefix]), int32([prefix]), pages[None], prefix, prefix)

    # the prompts behind it, together
    tables = (n_prefix + torch.arange(len(prompts) * width, dtype=torch.int32, device="cuda")).view(len(prompts), width)
    own = [torch.arange(n, device="cuda") for n in prompts]
    starts = [0]
    for n in prompts:
        starts.append(starts[-1] + n)
    y = layer(hidden(starts[-1]), (prefix + torch.cat(own)).int(), torch.cat([slots_of(tb, o) for tb, o in zip(tables, own)]),
              int32(starts), int32(prompts), tables, max(prompts), room, pages, prefix)
    x = y[int32(starts[1:]).long() - 1]
    print("prefill:", tuple(y.shape), "finite:", bool(torch.isfinite(y).all()))

    # one token for each sequence at a time
    lens = int32(prompts)
    for _ in range(args.tokens):
        slots = torch.stack([slots_of(tb, n) for tb, n in zip(tables, lens.long())])
        positions = prefix + lens
        lens = lens + 1
        x = layer(rms_norm(x), positions, slots, int32(list(range(len(prompts) + 1))), lens, tables, 1, room, pages, prefix)
    print("decoded:", args.tokens, "tokens of", len(prompts), "sequences, finite:", bool(torch.isfinite(x).all()))

    # adapter training: the gradient of the frozen feed-forward's input
    h, preact = rms_norm(y), layer.ffn.new_preact(y.shape[0])
    out = layer.ffn.run(h, layer.ffn_packed, preact=preact, M=y.shape[0])
    dA = layer.ffn.backward(h, layer.ffn_packed, preact, torch.ones_like(out), M=y.shape[0])["dA"]
    print("input gradient:", tuple(dA.shape), "finite:", bool(torch.isfinite(dA).all()))


if __name__ == "__main__":
    main()
