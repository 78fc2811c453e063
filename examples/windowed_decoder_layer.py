"""The decoder layer with normed heads and a sliding window, its pages managed on the device.

    python examples/windowed_decoder_layer.py [--steps 12]

The int4 layer of quantized_decoder_layer.py, whose queries and keys are normed for each head and
whose queries see their last WINDOW tokens and the first SINKS.  A step takes new tokens of
several sequences, prompts and single tokens together: a pool gives their slots, positions and
block tables from the counts alone, and takes back the pages of ended sequences and of tokens
that fell out of the window, so that sequences may grow far past what the pool holds.  Decoding
is captured in a graph once and replayed.  Ends with the gradients of the norms, as training needs them.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_decoder_layer import HEAD_DIM, HIDDEN, PAGE, Layer, int32, rms_norm  # noqa: E402
from weight_quantized_mixed_amd.device import PagePool, norm_rotate, norm_rotate_backward  # noqa: E402

WINDOW, SINKS, EPS = 96, 4, 1e-6


class WindowedLayer(Layer):
    """The layer for up to max_rows tokens a step of `sequences` sequences, from n_pages pages."""

    def __init__(self, max_rows, n_pages, sequences, longest, seed=0):
        super().__init__(max_rows, n_pages, seed)
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.q_weight, self.k_weight = ((1 + 0.1 * torch.randn(HEAD_DIM, generator=gen, device="cuda")).half() for _ in range(2))
        self.pool = PagePool(n_pages, PAGE, sequences, -(-longest // PAGE), window=WINDOW, sinks=SINKS)

    def step(self, x, new_tokens, max_q):
        """The layer's output for the rows of x: new_tokens [sequences] of each sequence (-1: it ends), and what the pool said."""
        rows, n = x.shape[0], self.pool
        r = n.extend(new_tokens, rows)
        q, k, v = self.product("qkv", rms_norm(x)).split(self.widths, dim=1)
        q = self.cache.append(q, k, v, self.cos, self.sin, r["positions"], r["slots"], norm_eps=EPS, q_weight=self.q_weight,
                              k_weight=self.k_weight)
        y = torch.zeros_like(q)  # (rows behind the last token are of no sequence)
        self.cache.attend(q, r["q_starts"], r["kv_lens"], n.tables, max_q, n.table_width * PAGE, out=y, window=WINDOW, sinks=SINKS)
        x = x + self.product("out", y.view(rows, -1))
        return x + self.product("down", self.ffn.run(rms_norm(x), self.ffn_packed, M=rows)), r


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=12, help="steps of prompts and single tokens, and of decoding")
    args = ap.parse_args()
    B, rows = 4, 192
    # pages for the windows and the first tokens, and for a step's new tokens three times over: a step's tokens leave the window
    # at the next step, and the pages that this gives back serve the one after it
    layer = WindowedLayer(rows, B * (WINDOW // PAGE + 3) + 3 * rows // PAGE, B, 4096)
    gen = torch.Generator(device="cuda").manual_seed(2)

    def hidden(n):
        return torch.randn((n, HIDDEN), generator=gen, device="cuda").half()

    refused = 0
    for i in range(args.steps):  # a chunk of one sequence's prompt beside single tokens of the others; now and then one ends
        new = [1] * B
        new[i % B] = 150
        if i % 5 == 4:
            new[(i + 1) % B] = -1
        y, r = layer.step(hidden(rows), int32(new), 150)
        refused += int(r["refused"].sum())
    held = layer.pool.n_pages - int(layer.pool.state[-1])
    print("steps:", args.steps, "tokens in the cache's sequences:", layer.pool.lens.tolist(), "pages held:", held, "refused:", refused,
          "finite:", bool(torch.isfinite(y).all()))

    # decoding: one token of each sequence, captured once; each replay extends the sequences by one
    x, ones = hidden(B), int32([1] * B)
    layer.step(x, ones, 1)  # (workspaces are made before the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = layer.step(x, ones, 1)
    for _ in range(args.steps):
        graph.replay()
        x.copy_(rms_norm(out))
    print("decoded:", args.steps, "tokens from a graph, lengths:", layer.pool.lens.tolist(), "finite:", bool(torch.isfinite(out).all()))

    # training: the gradients of the normed and rotated heads, into the gradient of their projection's output
    T = 64
    qkv, at = layer.product("qkv", rms_norm(hidden(T))), torch.arange(T, device="cuda", dtype=torch.int32)
    q, k, _ = qkv.split(layer.widths, dim=1)
    same = {"q_weight": layer.q_weight, "k_weight": layer.k_weight, "eps": EPS}
    qo, ko = norm_rotate(q, k, HEAD_DIM, layer.cos, layer.sin, at, **same)
    d_qkv = torch.zeros_like(qkv)
    dq, dk, _ = d_qkv.split(layer.widths, dim=1)
    g = norm_rotate_backward(q, k, torch.ones_like(qo), torch.ones_like(ko), layer.cos, layer.sin, at, dq=dq, dk=dk, **same)
    print("gradients:", tuple(d_qkv.shape), tuple(g["dq_weight"].shape), "finite:",
          bool(torch.isfinite(d_qkv).all() & torch.isfinite(g["dq_weight"]).all() & torch.isfinite(g["dk_weight"]).all()))


if __name__ == "__main__":
    main()
