"""The example's decoder layer: decoding token by token from the cache gives what one call
over all tokens gives, and a shared prefix gives what private copies of it give."""
import os
import sys

import pytest
import torch

from gpu_helpers import say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import quantized_decoder_layer as ex  # noqa: E402


def test_decoding_agrees_with_prefill_and_with_private_prefixes():
    say("case decoder layer")
    prefix, n, B = 70, 40, 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    P = torch.randn((prefix, ex.HIDDEN), generator=gen, device="cuda").half()
    X = torch.randn((B, n, ex.HIDDEN), generator=gen, device="cuda").half()
    pages = lambda a, k: torch.arange(a, a + k, dtype=torch.int32, device="cuda")  # noqa: E731
    npre, width = 5, 8
    layer = ex.Layer(512, npre + B * width)
    t = torch.arange(prefix, device="cuda")

    # private: prefix and tokens of each sequence in one call
    tables = pages(npre, B * width).view(B, width)
    both = torch.arange(prefix + n, device="cuda")
    x = torch.cat([torch.cat([P, X[b]]) for b in range(B)])
    private = layer(x, both.int().repeat(B), torch.cat([ex.slots_of(tb, both) for tb in tables]),
                    ex.int32([b * (prefix + n) for b in range(B + 1)]), ex.int32([prefix + n] * B), tables, prefix + n, prefix + n)
    want = private.view(B, prefix + n, -1)[:, prefix:].float()

    # shared: the prefix once, then the tokens one by one
    shared = pages(0, npre)
    layer(P, t.int(), ex.slots_of(shared, t), ex.int32([0, prefix]), ex.int32([prefix]), shared[None], prefix, prefix)
    got = []
    for i in range(n):
        slots = torch.stack([ex.slots_of(tb, torch.tensor(i, device="cuda")) for tb in tables])
        got.append(layer(X[:, i].contiguous(), ex.int32([prefix + i] * B), slots, ex.int32(list(range(B + 1))), ex.int32([i + 1] * B),
                         tables, 1, n, shared, prefix))
    got = torch.stack(got, 1).float()
    # both are fp16 results of the same sums in other orders and parts: every kernel on the
    # way rounds its outputs to 2^-11, five of them one after the other
    err = (got - want).norm() / want.norm()
    assert err < 5 * 2.0**-11, float(err)


def test_example_runs(capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["quantized_decoder_layer.py", "--tokens", "2"])
    ex.main()
    out = capsys.readouterr().out
    assert out.count("finite: True") == 3
