"""Calls given a stream of their own: what they allocate belongs to that stream's memory, so
that no block still in use on the current stream is written, and results are the same."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import Case, say
from weight_quantized_mixed_amd.device import PagedKV, QGated, QGemm, host_to_device, quantize_rows

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)


def owner(t):
    """The stream whose memory holds a tensor."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


def agree(call, *scratch):
    """call(stream) on a side stream: its tensors, and the workspaces after it, are of that stream and
    the values those of the current one; scratch: the objects' workspaces, not used before."""
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side)
    side.synchronize()
    for t in got:
        assert owner(t) == side.cuda_stream
    for w in scratch:
        assert w.buffers and owner(w.buffers[-1]) == side.cuda_stream
    want = call(None)
    for a, b in zip(got, want):
        assert owner(b) == torch.cuda.current_stream().cuda_stream and torch.equal(a, b)
    torch.cuda.synchronize()


def half(rng, *shape):
    return host_to_device(rng.standard_normal(shape).astype(np.float16))


def test_products():
    say("case streams products")
    c = Case(40, 300, 1000, "i4", 0, k_parts=2, deterministic=True, seed=3)
    agree(lambda s: [c.q.pack(c.w, c.s, c.z, stream=s)])
    agree(lambda s: [c.q.run(c.A, c.packed, stream=s)], c.q._ws)
    A = half(np.random.default_rng(1), 40, 256)
    agree(lambda s: quantize_rows(A, stream=s))
    codes, rows = quantize_rows(A)
    p = synth.make_problem(40, 72, 256, "i8", seed=4)
    plan = QGemm(40, 72, 256, "i8", dequant_output=True)
    packed, cols = plan.pack(host_to_device(p.w)), host_to_device(synth.draw_col_scales(72, 5))
    agree(lambda s: [plan.run_scaled(codes, packed, rows, cols, stream=s)])


def test_gated():
    say("case streams gated")
    rng = np.random.default_rng(2)
    M, N, K = 70, 72, 100  # K off the granule: padded activations in the workspace
    plan = QGated(M, N, K, "f16")
    A, wg, wu, dC = half(rng, M, K), half(rng, N, K), half(rng, N, K), half(rng, M, N)
    agree(lambda s: [plan.pack(wg, wu, stream=s)])
    packed, preact = plan.pack(wg, wu), plan.new_preact()
    agree(lambda s: [plan.run(A, packed, preact=preact, stream=s)], plan._ws)
    agree(lambda s: [*plan.backward(A, packed, preact, dC, bias_grads=True, stream=s).values()], plan._backward_ws)
    agree(lambda s: [plan.new_output(stream=s).zero_(), plan.new_preact(stream=s).zero_()])


def test_paged_cache():
    say("case streams cache")
    rng = np.random.default_rng(6)
    T, hq, hkv, D, page = 1, 4, 2, 64, 16
    cache = PagedKV(64, page, hkv, D)
    cache.k.copy_(half(rng, *cache.k.shape))
    cache.v.copy_(half(rng, *cache.v.shape))
    row, table = half(rng, T, (hq + 2 * hkv) * D), torch.ones((8, 32), device="cuda")
    q, k, v = row.split([hq * D, hkv * D, hkv * D], dim=1)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    agree(lambda s: [cache.append(q, k, v, table, table, i32(3), torch.tensor([900], device="cuda"), stream=s)])
    pages, starts, lens, x = i32(*range(60))[None], i32(0, 1), i32(901), q.view(T, hq, D)
    agree(lambda s: [cache.attend(x, starts, lens, pages, 1, 901, stream=s)], cache._workspace)


def test_a_workspace_waits_for_every_stream_that_used_it():
    """A plan dropped while another stream still runs it: its workspace is not handed out before that stream is done."""
    plan = QGated(70, 72, 100, "f16")
    A = torch.zeros((70, 100), dtype=torch.float16, device="cuda")
    w = torch.zeros((72, 100), dtype=torch.float16, device="cuda")
    packed = plan.pack(w, w)
    C = plan.run(A, packed)  # the workspace is the current stream's
    torch.cuda.synchronize()
    at, size = plan._ws.buffers[-1].data_ptr(), plan._ws.buffers[-1].numel()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        plan.run(A, packed, C=C)
    done = side.record_event()
    del plan
    again = torch.empty(size, dtype=torch.uint8, device="cuda")
    busy = not done.query()
    side.synchronize()
    assert busy and again.data_ptr() != at
