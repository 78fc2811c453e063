"""Normed heads, block tables and windowed attention at sizes and over memory that their other GPU tests leave out: sums over
millions of heads, many pages that come back at once, tiles of wide heads, workspaces that begin as junk."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import say
from test_paged_kv_gpu import assert_near, dev, halves
from test_windowed_layer_gpu import PoolCase, WindowCase
from weight_quantized_mixed_amd import qgemm as q
from weight_quantized_mixed_amd.device import norm_rotate_backward

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)


def f64(t):
    return t.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T,hq,hkv,D,kinds,one_sign", [(2**21, 32, 1, 8, 1, True), (40001, 32, 3, 128, 97, False), (70001, 3, 16, 200, 89, False)])
def test_weight_gradients_over_millions_of_heads(T, hq, hkv, D, kinds, one_sign):
    """Token t is that of t mod kinds, so the sums are known; terms of one sign lose most where a sum in fp32 is long."""
    say(f"case weight gradients T={T} hq={hq} hkv={hkv} D={D}")
    rng = np.random.default_rng(D)
    draw = (lambda *s: rng.uniform(0.5, 2, s).astype(np.float16)) if one_sign else (lambda *s: halves(rng, *s))
    xq, xk, dyq, dyk = draw(kinds, hq, D), draw(kinds, hkv, D), draw(kinds, hq, D), draw(kinds, hkv, D)
    if one_sign:  # one head for all, so that every sum has one term over and over
        xq, dyq = np.repeat(xq[:, :1], hq, 1), np.repeat(dyq[:, :1], hq, 1)
    qw, kw = draw(D), draw(D)
    times = np.bincount(np.arange(T) % kinds, minlength=kinds)[:, None, None]
    at = torch.arange(T, device="cuda") % kinds
    spread = lambda x: dev(x)[at]  # noqa: E731
    none, pos = torch.zeros((1, 0), device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    args = (spread(xq).view(T, -1), spread(xk).view(T, -1), spread(dyq), spread(dyk), none, none, pos)
    r = norm_rotate_backward(*args, q_weight=dev(qw), k_weight=dev(kw), eps=1e-5)
    t = np.zeros((kinds, 0))
    for name, x, w, dy in (("q", xq, qw, dyq), ("k", xk, kw, dyk)):
        dx, _, ex, _ = oracle.norm_rotate_grads_ref(x, w, 1e-5, t, t, False, dy)
        unit = x / np.sqrt((x.astype(np.float64) ** 2).mean(-1, keepdims=True) + 1e-5)
        terms = times * unit * dy
        # the reference's bound: 2**-17 of the sum of magnitudes
        assert_near(f64(r[f"d{name}_weight"]), terms.sum((0, 1)), 2.0**-17 * np.abs(terms).sum((0, 1)), f"d{name}_weight")
        assert_near(f64(r[f"d{name}"][:kinds]).reshape(dx.shape), dx, ex, f"d{name}")
        assert torch.equal(r[f"d{name}"], r[f"d{name}"][at])
    again = norm_rotate_backward(*args, q_weight=dev(qw), k_weight=dev(kw), eps=1e-5)
    assert all(torch.equal(r[n], again[n]) for n in r)
    need = q.qgemm_norm_rotate_backward_workspace(T, hq, hkv, D, True)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    again = norm_rotate_backward(*args, q_weight=dev(qw), k_weight=dev(kw), eps=1e-5, ws=ws)
    assert all(torch.equal(r[n], again[n]) for n in r)


def kernels_of(call):
    """Names of the kernels that a call runs."""
    call()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [e.name for e in p.events()]


def assert_tiles(c, D, parts):
    """The tiles of 128 rows for heads past 128, and the keys in so many parts: where a rule of the split moves a case away from
    them, the case has to move too."""
    names = kernels_of(c.run)
    want = f"window_rows_kernel<256, {'true' if D == 256 else 'false'}>"
    assert any(want in n for n in names), names
    assert any("attend_join_kernel" in n for n in names) == (parts > 1), names
    T = sum(c.qs)
    need = q.qgemm_attention_window_workspace(c.cache.desc, T, c.hq, len(c.qs), max(c.qs), max(c.lens), c.prefix, c.window, c.sinks)
    assert need == (parts * T * c.hq * (D + 2) * 4 if parts > 1 else 0)


WIDE = [  # q_heads, kv_heads, D, page, queries, own tokens, prefix, window, sinks, parts
    (6, 2, 136, 16, [500, 499, 480, 500, 470, 500], [500, 499, 700, 510, 470, 500], 5, 64, 9, 1),
    (8, 2, 256, 64, [500, 499, 480, 500, 470, 500], [500, 499, 700, 510, 470, 500], 5, 64, 9, 1),
    (10, 2, 192, 16, [700, 650, 700], [900, 650, 701], 30, 300, 40, 1), (14, 2, 256, 1, [400, 390, 400, 399], [800, 390, 400, 700], 0, 100, 0, 1),
    (16, 4, 256, 16, [300, 301, 299, 250], [300, 500, 290, 600], 20, 100, 30, 1), (4, 2, 256, 16, [520], [9000], 0, 8000, 100, 13),
    (4, 2, 136, 32, [1000], [4000], 0, 3000, 50, 7), (6, 2, 256, 16, [520], [6000], 100, 5000, 100, 9),
    (6, 2, 248, 64, [1, 520], [30, 6000], 100, 5000, 100, 9), (8, 2, 256, 128, [1000], [4000], 0, 3000, 50, 4),
    (3, 1, 256, 16, [1000, 900], [2000, 3000], 0, 2000, 50, 5),
]


@pytest.mark.parametrize("hq,hkv,D,page,qs,lens,prefix,window,sinks,parts", WIDE)
def test_wide_heads_that_share_keys(hq, hkv, D, page, qs, lens, prefix, window, sinks, parts):
    """Several query heads of a key head, two to seven, in tiles that begin between a token's heads; keys whole and in parts."""
    say(f"case wide heads hq={hq} hkv={hkv} D={D} page={page} q={qs} lens={lens} prefix={prefix} window={window} sinks={sinks}")
    c = WindowCase(hq, hkv, D, page, qs, lens, prefix, window, sinks, seed=D + hq).upload()
    assert_tiles(c, D, parts)
    c.check()


# ---- infinite values

@pytest.mark.parametrize("hq,hkv,D,qs,lens,prefix,window,sinks", [
    (4, 2, 128, [200], [700], 0, 64, 300), (4, 2, 64, [150], [600], 70, 40, 257), (8, 2, 256, [500, 499, 480, 500, 470, 500], [900, 499, 700, 510, 470, 500], 5, 64, 209),
    (8, 1, 128, [90], [2000], 0, 900, 1000), (8, 2, 128, [5], [400], 0, 90, 200)])
def test_infinite_values_behind_vanishing_probabilities(hq, hkv, D, qs, lens, prefix, window, sinks):
    """One key that every row scores far below the others, among first keys that whole tiles see, at the window's edge, and both: its
    infinite value reaches no other place and no row that does not see it."""
    say(f"case vanishing hq={hq} hkv={hkv} D={D} q={qs} window={window} sinks={sinks}")
    c = WindowCase(hq, hkv, D, 16, qs, lens, prefix, window, sinks, seed=D)
    c.q[:] = 1  # (scores of about 1, and of -30 sqrt(D) for keys of -30: e^-240 and less, which is 0 in fp32)
    seen = c.visible(0)
    partly = np.flatnonzero(seen.any(0) & ~seen.all(0))
    partly = partly[partly >= prefix]
    first, edge = prefix + 10, partly[len(partly) // 2]
    assert seen[:, first].all()
    for at in ([first], [edge], [first, edge]):
        k, v = c.k.copy(), c.v.copy()
        for t in at:
            page, i = c.tables[0, (t - prefix) // 16], (t - prefix) % 16
            c.k[page, :, i] = -30
        plain, _ = c.upload().run()
        for t in at:
            c.v[c.tables[0, (t - prefix) // 16], :, (t - prefix) % 16, 7] = np.inf
        got, _ = c.upload().run()
        hit = np.zeros(plain.shape, bool)
        hit[:qs[0], :, 7] = seen[:, at].any(1)[:, None]
        assert np.array_equal(got[~hit], plain[~hit])
        assert (np.isposinf(got[hit]) | np.isnan(got[hit]) | (got[hit] == plain[hit])).all()
        c.k, c.v = k, v


@pytest.mark.parametrize("hq,hkv,D,qs,lens,prefix,window,sinks", [
    (8, 2, 256, [500, 499, 480, 500, 470, 500], [900, 499, 700, 510, 470, 500], 5, 64, 209), (6, 2, 136, [1000], [4000], 0, 3000, 500),
    (4, 2, 128, [200], [700], 0, 64, 300), (8, 1, 128, [90], [2000], 0, 900, 1000)])
def test_infinities_among_first_keys_and_at_the_edges(hq, hkv, D, qs, lens, prefix, window, sinks):
    """Infinities in blocks of first keys that whole tiles see, beside ones that some rows do not; keys whole and in parts."""
    c = WindowCase(hq, hkv, D, 16, qs, lens, prefix, window, sinks, seed=D + 1)
    rng = np.random.default_rng(D)
    say(f"case infinities {hq}/{hkv} heads of {D}")
    plain, _ = c.upload().run()
    want = plain.copy()
    for b, n in enumerate(lens):
        seen = c.visible(b)
        edge = [t for t in np.flatnonzero(seen.any(0) & ~seen.all(0)) if t >= prefix]
        tokens = {prefix + int(t) for t in rng.integers(0, min(sinks, n), 3)} | {int(t) for t in rng.choice(edge, 5, replace=False)}
        for t in sorted(tokens):
            h, e, value = int(rng.integers(hkv)), int(rng.integers(D)), float(rng.choice([np.inf, -np.inf, np.nan]))
            c.v[c.tables[b, (t - prefix) // 16], h, (t - prefix) % 16, e] = value
            rows, heads = np.flatnonzero(seen[:, t]) + c.starts[b], range(h * (hq // hkv), (h + 1) * (hq // hkv))
            with np.errstate(invalid="ignore"):
                want[np.ix_(rows, heads, [e])] += np.asarray(value, want.dtype)
    got, _ = c.upload().run()
    finite = np.isfinite(want)
    assert not finite.all() and np.array_equal(got[finite], plain[finite]) and np.array_equal(got[~finite], want[~finite], equal_nan=True)


# ---- many pages given back

@pytest.mark.parametrize("B,page,most,prefix,window,sinks,ends", [
    (1, 1, 30000, 0, 0, 0, 1.0), (1, 1, 8193, 0, 0, 0, 1.0), (1, 1, 8192, 0, 0, 0, 1.0), (3, 1, 30000, 5, 40, 90, 0.4), (48, 1, 2500, 0, 0, 0, 0.5), (300, 4, 900, 10, 64, 30, 0.3),
    (1500, 1, 200, 0, 20, 7, 0.1), (2048, 1, 60, 0, 0, 0, 0.6), (2048, 1, 9, 0, 0, 0, 1.0), (40, 1, 5000, 0, 4000, 600, 0.5)])
def test_many_pages_come_back(B, page, most, prefix, window, sinks, ends):
    """Steps of few tokens in which long sequences end or their windows first move on: thousands of pages, of sequences of mixed
    lengths, some of which hold none."""
    say(f"case pages back B={B} page={page} lens={most} window={window} sinks={sinks}")
    rng = np.random.default_rng(B + most)
    lens = rng.integers(0, most + 1, B)
    lens[rng.random(B) < 0.2] = 0
    lens[0] = most
    new = np.where(rng.random(B) < ends, -1, rng.integers(0, 2, B))
    c = PoolCase(B, page, -(-(most + 1) // page), int((-(-lens // page)).sum()) + 40, lens, prefix, window, sinks, seed=B, gone=False)
    got, want, pool = c.check(new, int(np.maximum(new, 0).sum()) + 3)
    assert want["free"] - c.free > 5000 and q.qgemm_kv_extend_workspace(B, int(np.maximum(new, 0).sum()) + 3) == 0
    c.check(new, int(np.maximum(new, 0).sum()), None, torch.full_like(pool.state, -5))


# ---- memory

@pytest.mark.parametrize("T", [700, 7000])
def test_results_and_workspaces_may_begin_as_anything(T):
    """Every array that the calls write, their workspaces among them, begins as NaN, zeros or junk; one launch and two."""
    rng = np.random.default_rng(T)
    rows, hq, hkv, D, rot = 300, 8, 2, 96, 64
    x, dyq, dyk = dev(halves(rng, rows, (hq + hkv) * D)), dev(halves(rng, rows, hq, D)), dev(halves(rng, rows, hkv, D))
    qw, kw, cos, sin = dev(halves(rng, D)), dev(halves(rng, D)), *(dev(rng.standard_normal((9, rot // 2)).astype(np.float32)) for _ in range(2))
    pos = dev(rng.integers(-1, 9, rows).astype(np.int32))
    B, page, width = 50, 16, 40
    c = PoolCase(B, page, width, 900, np.arange(B) * 7, window=64, sinks=4)
    new = dev(np.where(np.arange(B) % 7 == 6, -1, T // 60).astype(np.int32))
    norm_ws, extend_ws = q.qgemm_norm_rotate_backward_workspace(rows, hq, hkv, D, True), q.qgemm_kv_extend_workspace(B, T)
    assert norm_ws > 0 and (extend_ws > 0) == (T == 7000)
    results = []
    for fill in (0xFF, 0x00, 0x7B):
        def junk(*shape, dtype=torch.float16):
            return torch.full((int(np.prod(shape)) * dtype.itemsize,), fill, dtype=torch.uint8, device="cuda").view(dtype).view(shape)

        turn = (qw.data_ptr(), kw.data_ptr(), 1e-5, cos.data_ptr(), sin.data_ptr(), 9, rot, 1, pos.data_ptr())
        src = (x.data_ptr(), (hq + hkv) * D, x.data_ptr() + 2 * hq * D, (hq + hkv) * D)
        qo, ko, dq, dk = junk(rows, hq, D), junk(rows, hkv, D), junk(rows, hq * D), junk(rows, hkv * D)
        dw, ws = junk(2, D, dtype=torch.float32), junk(norm_ws, dtype=torch.uint8)
        q.qgemm_norm_rotate(rows, hq, hkv, D, *src, *turn, qo.data_ptr(), ko.data_ptr())
        q.qgemm_norm_rotate_backward(rows, hq, hkv, D, *src, *turn, dyq.data_ptr(), dyk.data_ptr(), dq.data_ptr(), hq * D, dk.data_ptr(), hkv * D,
                                     dw.data_ptr(), dw.data_ptr() + 4 * D, ws.data_ptr(), norm_ws)
        pool, i32 = c.pool(), torch.int32
        starts, after, where, slots, refused = junk(B + 1, dtype=i32), junk(2 * B + 2, dtype=i32), junk(T, dtype=i32), junk(T, dtype=torch.int64), junk(B, dtype=i32)
        ws = junk(max(extend_ws, 16), dtype=torch.uint8)
        at, to = pool.state.data_ptr(), after.data_ptr()
        q.qgemm_kv_extend(B, T, page, new.data_ptr(), at, at + 4 * B, at + 8 * B, pool.ring.data_ptr(), len(c.ring), pool.tables.data_ptr(), width, 0, 64, 4,
                          starts.data_ptr(), to, to + 4 * B, to + 8 * B, where.data_ptr(), slots.data_ptr(), refused.data_ptr(), ws.data_ptr(), extend_ws)
        results.append([t.view(torch.uint8) for t in (qo, ko, dq, dk, dw, starts, after, where, slots, refused, pool.ring, pool.tables)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for other in results[1:] for a, b in zip(results[0], other))
    want = oracle.extend_ref(new.cpu().numpy(), c.lens, c.gone, c.head, c.free, c.ring, c.tables, page, T, 0, 64, 4)
    assert np.array_equal(slots.cpu().numpy(), want["slots"]) and np.array_equal(refused.cpu().numpy(), want["refused"])
