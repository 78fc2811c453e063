"""GPU parity of the rotary append and of attention over the paged cache with the float64
references: head layouts, page sizes, ragged and empty sequences, shared prefixes, values
that must not matter."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import say
from weight_quantized_mixed_amd import qgemm as q
from weight_quantized_mixed_amd.device import PagedKV

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)


def halves(rng, *shape):
    return rng.standard_normal(shape, dtype=np.float32).astype(np.float16)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def assert_near(got, ref, bound, what):
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) > bound
    if over.any():
        at = np.argwhere(over)[:4]
        raise AssertionError(f"{what}: {int(over.sum())} outside the bound, first "
                             f"{[(tuple(i), float(got[tuple(i)]), float(ref[tuple(i)]), float(bound[tuple(i)])) for i in at]}")


# ---- append

APPEND = [  # T, q_heads, kv_heads, D, rot, page, interleaved
    (1, 4, 4, 128, 128, 16, False), (3, 8, 2, 64, 64, 1, True), (48, 32, 8, 128, 128, 16, False),
    (17, 6, 2, 80, 80, 32, False), (17, 6, 2, 80, 40, 32, True), (9, 3, 1, 8, 8, 2, False), (9, 3, 1, 8, 2, 2, True),
    (33, 4, 4, 96, 20, 64, False), (300, 8, 8, 256, 128, 256, False), (5, 2, 1, 40, 0, 4, False), (7, 2, 2, 24, 12, 8, True),
    (7, 2, 2, 24, 6, 8, False),
]


@pytest.mark.parametrize("T,hq,hkv,D,rot,page,il", APPEND)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_append(T, hq, hkv, D, rot, page, il, pad):
    """pad: values between the rows of the projection's output (3: rows not 16-byte aligned)."""
    say(f"case append T={T} hq={hq} hkv={hkv} D={D} rot={rot} page={page} il={il} pad={pad}")
    rng = np.random.default_rng(T + D + pad)
    width = (hq + 2 * hkv) * D
    wide = halves(rng, T, width + pad)
    n_pos = 50
    ang = rng.uniform(-np.pi, np.pi, (n_pos, rot // 2)).astype(np.float32)
    cos, sin = np.cos(ang), np.sin(ang)
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    n_pages = T // page + 3
    slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
    k0, v0 = halves(rng, n_pages, hkv, page, D), halves(rng, n_pages, hkv, page, D)
    cache = PagedKV(n_pages, page, hkv, D, k=dev(k0), v=dev(v0))
    x = dev(wide)[:, :width]
    qt, kt, vt = x.split([hq * D, hkv * D, hkv * D], dim=1)
    out = cache.append(qt, kt, vt, dev(cos), dev(sin), dev(pos), dev(slots), interleaved=il)
    torch.cuda.synchronize()
    heads = wide[:, :width].reshape(T, hq + 2 * hkv, D)
    ref, err = oracle.rotate_ref(heads[:, :hq + hkv], cos[pos], sin[pos], il)
    assert_near(out.cpu().numpy().astype(np.float64), ref[:, :hq], err[:, :hq], "q")
    want_v = v0.copy()
    want_v[slots // page, :, slots % page] = heads[:, hq + hkv:]
    assert np.array_equal(cache.v.cpu().numpy(), want_v)
    want_k, err_k = k0.astype(np.float64), np.zeros(k0.shape)
    want_k[slots // page, :, slots % page] = ref[:, hq:]
    err_k[slots // page, :, slots % page] = err[:, hq:]
    assert_near(cache.k.cpu().numpy().astype(np.float64), want_k, err_k, "k")


def test_append_leaves_out_what_is_outside():
    """Slots outside the cache are not stored; a position outside the table gives NaN queries and no key."""
    rng = np.random.default_rng(5)
    T, hq, hkv, D, page, n_pages = 8, 4, 2, 64, 4, 5
    x = dev(halves(rng, T, (hq + 2 * hkv) * D))
    qt, kt, vt = x.split([hq * D, hkv * D, hkv * D], dim=1)
    pos = np.array([0, 1, 2, 3, 10, -1, 4, 2**31 - 1], np.int32)
    slots = np.array([3, -1, 20, 7, 8, 9, 2**40, 10], np.int64)
    cache = PagedKV(n_pages, page, hkv, D)
    table = dev(np.ones((10, 32), np.float32))
    out = cache.append(qt, kt, vt, table, table, dev(pos), dev(slots)).cpu().numpy()
    bad = np.array([4, 5, 7])
    assert np.isnan(out[bad]).all() and np.isfinite(np.delete(out, bad, 0)).all()
    stored = np.zeros(n_pages * page, bool)
    stored[[3, 7]] = True
    for c in (cache.k, cache.v):
        flat = c.cpu().numpy().transpose(0, 2, 1, 3).reshape(n_pages * page, -1)
        assert np.array_equal((flat != 0).any(1), stored)


def test_append_in_place_and_empty():
    rng = np.random.default_rng(6)
    x = dev(halves(rng, 12, 4 * 64))
    kv = dev(halves(rng, 12, 64))
    t = dev(np.cos(rng.uniform(-3, 3, (9, 16))).astype(np.float32))
    pos, slots = dev(rng.integers(0, 9, 12).astype(np.int32)), torch.arange(12, device="cuda")
    cache = PagedKV(2, 8, 1, 64)
    ref = cache.append(x, kv, kv, t, t, pos, slots)
    got = cache.append(x, kv, kv, t, t, pos, slots, q_out=x.view(12, 4, 64))
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, ref)
    assert cache.append(x[:0], kv[:0], kv[:0], t, t, pos[:0], slots[:0]).shape == (0, 4, 64)


# ---- attention

class AttnCase:
    def __init__(self, hq, hkv, D, page, qs, lens, prefix=0, seed=0, extra_pages=3, spread=1.0):
        rng = self.rng = np.random.default_rng(seed + D + page)
        self.hq, self.hkv, self.D, self.page, self.qs, self.lens, self.prefix = hq, hkv, D, page, list(qs), list(lens), prefix
        B = len(qs)
        self.width = max(1, -(-max(lens) // page))
        n_prefix = -(-prefix // page)
        self.n_pages = B * self.width + n_prefix + extra_pages
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.prefix_table, self.tables = order[:n_prefix], order[n_prefix:n_prefix + B * self.width].reshape(B, self.width).copy()
        # every slot that holds no token is NaN: nothing may read it into a result
        self.k = np.full((self.n_pages, hkv, page, D), np.nan, np.float16)
        self.v = self.k.copy()
        self.tokens = []
        for table, n in [(self.prefix_table, prefix)] + list(zip(self.tables, lens)):
            kt, vt = halves(rng, n, hkv, D), halves(rng, n, hkv, D)
            t = np.arange(n)
            self.k[table[t // page], :, t % page], self.v[table[t // page], :, t % page] = kt, vt
            self.tokens.append((kt, vt))
        for b, n in enumerate(lens):  # entries past the last page point nowhere
            self.tables[b, -(-n // page):] = -1
        self.q = (halves(rng, sum(qs), hq, D).astype(np.float32) * spread).astype(np.float16)
        self.starts = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)

    def upload(self):
        self.cache = PagedKV(self.n_pages, self.page, self.hkv, self.D, k=dev(self.k), v=dev(self.v))
        self.dq, self.dstarts = dev(self.q), dev(self.starts)
        self.dlens, self.dtables = dev(np.array(self.lens, np.int32)), dev(self.tables)
        self.dprefix = dev(self.prefix_table) if self.prefix else None
        return self

    def run(self, scale=None, max_q=None, max_len=None, q=None, **kw):
        lse = torch.full((self.q.shape[0], self.hq), 7.0, device="cuda")
        out = self.cache.attend(self.dq if q is None else q, self.dstarts, self.dlens, self.dtables,
                                max_q=max(self.qs) if max_q is None else max_q,
                                max_len=max(self.lens) if max_len is None else max_len,
                                prefix_table=self.dprefix, prefix_len=self.prefix, scale=scale, lse=lse, **kw)
        torch.cuda.synchronize()
        return out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)

    def reference(self, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        G = self.hq // self.hkv
        out, lse, bound = (np.zeros((self.q.shape[0], self.hq) + s) for s in ((self.D,), (), (self.D,)))
        for b, (n, L) in enumerate(zip(self.qs, self.lens)):
            r = slice(self.starts[b], self.starts[b + 1])
            visible = np.concatenate([np.ones((n, self.prefix), bool),
                                      np.arange(L)[None] <= (L - n + np.arange(n))[:, None]], axis=1)
            for h in range(self.hq):
                kt, vt = (np.concatenate([self.tokens[0][i][:, h // G], self.tokens[b + 1][i][:, h // G]]) for i in (0, 1))
                out[r, h], lse[r, h], bound[r, h] = oracle.attention_ref(self.q[r, h], kt, vt, visible, scale)
        return out, lse, bound

    def check(self, scale=None, **kw):
        (got, lse), (ref, ref_lse, bound) = self.run(scale, **kw), self.reference(scale)
        assert_near(got, ref, bound, "out")
        empty = ~np.isfinite(ref_lse)
        assert np.array_equal(empty, np.isneginf(lse))
        assert (np.abs(lse[~empty] - ref_lse[~empty]) <= 1e-4 + 1e-5 * np.abs(ref_lse[~empty])).all()


ATTN = [  # q_heads, kv_heads, D, page, queries, own tokens, prefix
    (4, 4, 128, 16, [1], [1], 0), (4, 4, 128, 16, [1], [777], 0), (8, 2, 64, 16, [1, 1, 1], [5, 0, 130], 0),
    (8, 1, 128, 1, [1, 1], [33, 64], 0), (6, 2, 80, 32, [1] * 5, [1, 31, 32, 33, 100], 40),
    (32, 8, 128, 16, [1] * 9, [0, 1, 2, 63, 64, 65, 200, 17, 500], 1000), (4, 2, 256, 16, [1, 1], [70, 3], 130),
    (4, 2, 256, 64, [40, 90], [40, 300], 0), (2, 1, 256, 16, [200], [260], 33), (3, 1, 8, 2, [2, 5], [9, 5], 3),
    (16, 2, 128, 16, [3, 1, 0, 2], [40, 1, 20, 2], 70), (8, 8, 64, 16, [20, 1, 17], [25, 90, 17], 0),
    (8, 8, 96, 16, [20, 1, 17], [25, 90, 17], 65), (4, 4, 128, 64, [150, 64, 65], [150, 64, 400], 0),
    (8, 2, 128, 16, [100, 33], [130, 33], 200), (16, 2, 40, 256, [50], [700], 0), (64, 8, 128, 16, [1] * 3, [300, 40, 0], 0),
    (24, 8, 192, 32, [7, 9], [100, 9], 500), (12, 4, 64, 1, [5] * 4, [5, 40, 6, 77], 129), (4, 1, 128, 16, [1], [0], 0),
    (4, 1, 128, 16, [3], [0], 0), (8, 2, 64, 16, [300], [300], 0), (40, 40, 128, 16, [1] * 2, [3000, 10], 2500),
]


@pytest.mark.parametrize("hq,hkv,D,page,qs,lens,prefix", ATTN)
def test_attention(hq, hkv, D, page, qs, lens, prefix):
    say(f"case attention hq={hq} hkv={hkv} D={D} page={page} q={qs} lens={lens} prefix={prefix}")
    AttnCase(hq, hkv, D, page, qs, lens, prefix, seed=len(qs)).upload().check()


def test_attention_with_loose_bounds_and_other_scales():
    """Host bounds above the true sizes (other splits), sharp and flat softmaxes."""
    c = AttnCase(8, 2, 128, 16, [1, 2, 1], [100, 37, 8], 50, seed=4, spread=4.0).upload()
    c.check()
    c.check(max_q=90, max_len=5000)
    c.check(max_q=17, max_len=130)
    c.check(scale=1e-6)
    c.check(scale=1.0)


@pytest.mark.parametrize("qs,lens,prefix", [([40], [40], 0), ([3], [40], 0), ([1, 150], [20, 150], 90)])
def test_future_values_never_matter(qs, lens, prefix):
    """NaN and infinities in the last own tokens reach only the queries that see those tokens."""
    for what in (np.nan, np.inf, -np.inf):
        c = AttnCase(4, 2, 128, 16, qs, lens, prefix, seed=11).upload()
        clean, _ = c.run()
        b, n, L = len(qs) - 1, qs[-1], lens[-1]
        page, at = c.tables[b, (L - 1) // 16], (L - 1) % 16
        c.k[page, :, at, 5] = c.v[page, :, at, 7] = what
        c.k[page, :, at, 6] = np.nan
        c.upload()
        got, _ = c.run()
        assert np.array_equal(got[:-1], clean[:-1]) and not np.isfinite(got[-1]).any(), what
        # infinities of one sign in V alone come out as they are
        c.k[page, :, at, 5] = c.k[page, :, at, 6] = 0
        c.upload()
        got, _ = c.run()
        assert np.array_equal(got[:-1], clean[:-1])
        assert np.array_equal(got[-1][:, 7], np.full(4, what), equal_nan=True) and np.isfinite(np.delete(got[-1], 7, 1)).all()


def test_attention_results_do_not_depend_on_the_call_before():
    c = AttnCase(32, 8, 128, 16, [1] * 6, [0, 900, 30, 64, 5, 1], 3000, seed=2).upload()
    first = c.run()
    c.cache._workspace.buffers[-1].fill_(0xFF)  # NaN in every partial result
    again = c.run()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_attention_rows_of_no_sequence_are_left_alone():
    c = AttnCase(4, 2, 64, 16, [1, 2], [40, 50], 100, seed=8)
    c.q = np.concatenate([c.q, np.full((3, 4, 64), np.nan, np.float16)])
    c.upload()
    out = torch.full((6, 4, 64), 3.0, dtype=torch.float16, device="cuda")
    got, _ = c.run(out=out)
    ref, _, bound = c.reference()
    assert_near(got[:3], ref[:3], bound[:3], "out")
    assert (got[3:] == 3.0).all()


def test_strided_queries_other_stream_and_graph():
    c = AttnCase(8, 2, 128, 16, [1, 1, 1, 1], [90, 17, 0, 300], 200, seed=9).upload()
    base, _ = c.run()
    wide = torch.zeros((4, 8 * 128 + 24), dtype=torch.float16, device="cuda")
    wide[:, 8:8 + 1024] = c.dq.flatten(1)
    view = wide[:, 8:8 + 1024].view(4, 8, 128)
    assert np.array_equal(c.run(q=view)[0], base)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = c.cache.attend(c.dq, c.dstarts, c.dlens, c.dtables, 1, 300, c.dprefix, 200)
    side.synchronize()
    assert np.array_equal(out.cpu().numpy().astype(np.float64), base)
    # captured once, replayed with other lengths
    lens, out = c.dlens.clone(), torch.empty_like(c.dq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.cache.attend(c.dq, c.dstarts, lens, c.dtables, 1, 300, c.dprefix, 200, out=out)
    full = list(c.lens)
    for cut in (0, 16, 5):
        c.lens = [max(0, n - cut) for n in full]
        lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        saved = c.tokens
        c.tokens = [saved[0]] + [(k[:n], v[:n]) for (k, v), n in zip(saved[1:], c.lens)]
        ref, _, bound = c.reference()
        c.tokens = saved
        assert_near(out.cpu().numpy().astype(np.float64), ref, bound, f"replay {cut}")


def test_cache_offsets_past_32_bits():
    """Pages whose byte and value offsets pass 2**32 (9 GB of keys, as many of values)."""
    hkv, D, page = 8, 128, 256
    n_pages = (2**32 + 2**27) // (hkv * D * page)
    shape = (n_pages, hkv, page, D)
    k, v = (torch.empty(shape, dtype=torch.float16, device="cuda") for _ in range(2))
    cache = PagedKV(n_pages, page, hkv, D, k=k, v=v)
    rng = np.random.default_rng(1)
    T = 300
    rows = dev(halves(rng, T, 3 * hkv * D))
    qt, kt, vt = rows.split([hkv * D] * 3, dim=1)
    pages = np.array([n_pages - 1, n_pages - 3], np.int32)
    t = np.arange(T)
    slots = pages[t // page].astype(np.int64) * page + t % page
    none = torch.empty((1, 0), device="cuda")
    qo = cache.append(qt, kt, vt, none, none, torch.zeros(T, dtype=torch.int32, device="cuda"), dev(slots))
    assert torch.equal(k[n_pages - 3, :, : T - page].transpose(0, 1), kt[page:].view(-1, hkv, D))
    out = cache.attend(qo[-1:], dev(np.array([0, 1], np.int32)), dev(np.array([T], np.int32)), dev(pages[None]), 1, T)
    got = out.cpu().numpy().astype(np.float64)
    kh, vh, qh = (x.reshape(T, hkv, D).cpu().numpy() for x in (kt, vt, qt))
    for h in range(hkv):
        ref, _, bound = oracle.attention_ref(qh[-1:, h], kh[:, h], vh[:, h], np.ones((1, T), bool), D ** -0.5)
        assert_near(got[:, h], ref, bound, f"head {h}")


def test_pages_outside_the_cache_read_page_zero():
    c = AttnCase(4, 2, 64, 16, [1], [40], seed=3)
    c.tables[0, 1] = 10**6
    c.k[0] = c.v[0] = 0
    c.upload()
    got, _ = c.run()
    assert np.isfinite(got).all()


def test_paged_kv_rejects_wrong_tensors():
    c = AttnCase(4, 2, 64, 16, [1], [40], seed=3).upload()
    with pytest.raises(ValueError):
        c.run(q=c.dq.float())
    with pytest.raises(ValueError):
        c.run(q=c.dq[:, :, :32])
    with pytest.raises(q.QGemmError):
        c.run(scale=0.0)
    with pytest.raises(ValueError):
        PagedKV(4, 16, 2, 64, k=torch.zeros((4, 16, 2, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        c.cache.append(c.dq.flatten(1), c.dq.flatten(1), c.dq.flatten(1), *[torch.ones((4, 32), device="cuda")] * 2,
                       torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"))


def test_an_outgrown_workspace_stays_with_its_graph():
    """A graph replays a call whose workspace a later, larger call has outgrown."""
    c = AttnCase(8, 2, 128, 16, [1, 1], [400, 300], 600, seed=12).upload()
    base, _ = c.run()
    out = torch.empty_like(c.dq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.cache.attend(c.dq, c.dstarts, c.dlens, c.dtables, 1, 400, c.dprefix, 600, out=out)
    n = len(c.cache._workspace.buffers)
    c.run(max_q=60, max_len=20000)
    assert len(c.cache._workspace.buffers) > n
    junk = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy().astype(np.float64), base)
    assert all((j == 0xFF).all() for j in junk)


@pytest.mark.parametrize("hq,hkv,D,qs,lens,prefix,max_q,max_len,width", [
    (8, 2, 128, [5, 2], [40, 30], 0, 3, 40, 9), (8, 2, 128, [5, 2], [140, 100], 70, 5, 77, 9), (4, 1, 64, [1, 1], [140, 100], 70, 1, 140, 5),
    (4, 2, 128, [100, 150], [130, 190], 0, 70, 190, 12), (4, 2, 128, [100, 150], [130, 190], 33, 150, 100, 12),
    (2, 2, 256, [90], [400], 0, 60, 300, 15), (8, 1, 128, [6], [6], 0, 2, 6, 1)])
def test_rows_and_tokens_past_the_bounds_are_left_out(hq, hkv, D, qs, lens, prefix, max_q, max_len, width):
    """More queries, tokens or pages than max_q, max_len and the table's width: the rows within
    max_q see the tokens that they would see, as far as those are read; other rows stay as they were."""
    say(f"case bounds q={qs} lens={lens} max_q={max_q} max_len={max_len} width={width}")
    c = AttnCase(hq, hkv, D, 16, qs, lens, prefix, seed=13).upload()
    c.dtables = dev(c.tables[:, :width])
    out = torch.full((sum(qs), hq, D), 3.0, dtype=torch.float16, device="cuda")
    got, lse = c.run(max_q=max_q, max_len=max_len, out=out)
    for b, (n, L) in enumerate(zip(qs, lens)):
        m, held, r0 = min(n, max_q), min(L, max_len, width * 16), c.starts[b]
        seen = np.concatenate([np.ones((m, prefix), bool), np.arange(held)[None] <= (L - n + np.arange(m))[:, None]], axis=1)
        for h in range(hq):
            kt, vt = (np.concatenate([c.tokens[0][i][:, h // (hq // hkv)], c.tokens[b + 1][i][:held, h // (hq // hkv)]]) for i in (0, 1))
            ref, ref_lse, bound = oracle.attention_ref(c.q[r0:r0 + m, h], kt, vt, seen, D ** -0.5)
            assert_near(got[r0:r0 + m, h], ref, bound, f"sequence {b} head {h}")
            assert (np.abs(lse[r0:r0 + m, h] - ref_lse) <= 1e-4 + 1e-5 * np.abs(ref_lse)).all()
        assert (got[r0 + m:c.starts[b + 1]] == 3.0).all()


def test_a_single_token_cut_from_any_array():
    """One row of a wider array whose row length is odd: its step to a next row does not exist."""
    rng = np.random.default_rng(15)
    hq, hkv, D, page = 4, 2, 64, 16
    wide = dev(halves(rng, 5, (hq + 2 * hkv) * D + 3))
    row = wide[:1, :(hq + 2 * hkv) * D]
    table = dev(np.cos(rng.uniform(-3, 3, (9, 32))).astype(np.float32))
    pos, slot = dev(np.array([4], np.int32)), torch.tensor([20], device="cuda")
    got, want = PagedKV(4, page, hkv, D), PagedKV(4, page, hkv, D)
    results = []
    for cache, x in ((got, row), (want, row.clone(memory_format=torch.contiguous_format))):
        q0, k, v = x.split([hq * D, hkv * D, hkv * D], dim=1)
        cache.append(q0, k, v, table, table, pos, slot)
        pages = [dev(np.array(a, np.int32)) for a in ([0, 1], [21], [[0, 1]])]
        results.append(cache.attend(q0.view(1, hq, D), *pages, 1, 21))
    assert torch.equal(*results) and torch.equal(got.k, want.k) and torch.equal(got.v, want.v)


@pytest.mark.parametrize("B", [0, 3])
def test_attention_of_an_empty_batch(B):
    c = AttnCase(4, 2, 64, 16, [1], [40], seed=3).upload()
    starts, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B + 1, B))
    assert c.cache.attend(c.dq[:0], starts, lens, torch.zeros((B, 2), dtype=torch.int32, device="cuda"), 0, 0).shape == (0, 4, 64)


def test_append_of_more_tokens_than_one_launch_holds():
    """2^24 + 5 rows (a launch ends below 2^32 threads of 256 a token): the last ones are turned and stored too."""
    T, D = 2**24 + 5, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-2000, 2000, (T, 3 * D), generator=gen, device="cuda", dtype=torch.int16).half()
    qt, kt, vt = x.split([D] * 3, dim=1)
    cos, sin = torch.tensor([[0.0], [1.0]], device="cuda"), torch.tensor([[1.0], [0.0]], device="cuda")
    pos = (torch.arange(T, device="cuda", dtype=torch.int32) & 1) ^ 1  # every other token: a quarter turn of pair (0, 1)
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    kept = torch.tensor([0, 2**23 - 1, 2**23, 2**24 - 1, 2**24, T - 1], device="cuda")
    slots[kept] = torch.arange(6, device="cuda")
    cache = PagedKV(1, 8, 1, D)
    out = cache.append(qt, kt, vt, cos, sin, pos, slots, interleaved=True)[:, 0]
    turned = qt.clone()
    turned[1::2, 0], turned[1::2, 1] = -qt[1::2, 1], qt[1::2, 0]
    assert torch.equal(out, turned)
    k = kt[kept].clone()
    odd = (kept & 1).bool()
    k[odd, 0], k[odd, 1] = -kt[kept][odd, 1], kt[kept][odd, 0]
    assert torch.equal(cache.k[0, 0, :6], k) and torch.equal(cache.v[0, 0, :6], vt[kept])


def test_attention_at_the_largest_scale():
    """Scores of 0 stay 0 at the largest scale that is taken: the mean of the values."""
    c = AttnCase(4, 2, 64, 16, [1, 3], [40, 7], 20, seed=16)
    c.q[:] = 0
    c.upload().check(scale=2.3e38)


@pytest.mark.parametrize("D", [40, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("qs,lens,prefix", [([1, 1], [90, 40], 70), ([30], [150], 0)])
def test_infinite_keys_have_their_weight(D, qs, lens, prefix):
    """A key that a query sees with a score of minus infinity weighs nothing, in every head dimension."""
    c = AttnCase(4, 2, D, 16, qs, lens, prefix, seed=17)
    c.q[..., 3] = np.abs(c.q[..., 3]) + np.float16(0.125)
    c.upload()
    at = [(c.tables[0, 1], 5, 21)] + ([(c.prefix_table[2], 1, 33)] if prefix else [])
    for page, place, _ in at:
        c.k[page, :, place, 3] = -np.inf
    c.upload()
    got, lse = c.run()
    for b, (n, L) in enumerate(zip(qs, lens)):
        seen = np.concatenate([np.ones((n, prefix), bool), np.arange(L)[None] <= (L - n + np.arange(n))[:, None]], axis=1)
        seen[:, prefix + 21] &= b != 0
        if prefix:
            seen[:, 33] = False
        r = slice(c.starts[b], c.starts[b + 1])
        for h in range(4):
            kt, vt = (np.concatenate([c.tokens[0][i][:, h // 2], c.tokens[b + 1][i][:, h // 2]]) for i in (0, 1))
            ref, ref_lse, bound = oracle.attention_ref(c.q[r, h], kt, vt, seen, D ** -0.5)
            assert_near(got[r, h], ref, bound, f"sequence {b} head {h}")
            assert (np.abs(lse[r, h] - ref_lse) <= 1e-4 + 1e-5 * np.abs(ref_lse)).all()


@pytest.mark.parametrize("hq,hkv,D,qs,lens,prefix", [
    (2, 1, 64, [1, 1], [1, 2398], 0), (1, 1, 8, [1], [700], 0), (2, 1, 40, [1], [1500], 0), (4, 1, 64, [2, 1], [3000, 2500], 4000),
    (2, 1, 128, [1, 1], [4100, 3000], 4500), (2, 2, 80, [1, 2], [4100, 100], 4500), (1, 1, 256, [1, 1], [4100, 300], 4500),
    (2, 1, 96, [1], [9000], 0), (8, 1, 64, [9, 9], [2000, 1500], 3000)])
def test_many_parts_of_the_keys(hq, hkv, D, qs, lens, prefix):
    """More parts than a row has 16-byte pieces of fp32, up to 32 of the prefix and 32 of the own tokens: all of them count."""
    say(f"case parts hq={hq} hkv={hkv} D={D} q={qs} lens={lens} prefix={prefix}")
    c = AttnCase(hq, hkv, D, 64, qs, lens, prefix, seed=19).upload()
    c.check()
    need = q.qgemm_attention_workspace(c.cache.desc, sum(qs), hq, len(qs), max(qs), max(lens), prefix)
    assert need // (sum(qs) * hq * (D * 4 + 8)) > 5
