"""GPU parity of normed appends, norms with their gradients, block tables and windowed attention
with the float64 references, and a run of them together."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import say
from test_paged_kv_gpu import AttnCase, assert_near, dev, halves
from weight_quantized_mixed_amd import qgemm as q
from weight_quantized_mixed_amd.device import PagedKV, PagePool, norm_rotate, norm_rotate_backward

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

I32 = torch.int32


def f64(t):
    return t.cpu().numpy().astype(np.float64)


def ints(a):
    return dev(np.asarray(a, np.int32))


# ---- norms and rotation

NORM = [  # T, q_heads, kv_heads, D, rot, page, interleaved, weights
    (1, 4, 4, 128, 128, 16, False, True), (3, 8, 2, 64, 64, 1, True, True), (48, 32, 8, 128, 128, 16, False, True),
    (17, 6, 2, 80, 80, 32, False, False), (17, 6, 2, 80, 40, 32, True, True), (9, 3, 1, 8, 8, 2, False, True), (9, 3, 1, 8, 2, 2, True, False),
    (33, 4, 4, 96, 20, 64, False, True), (300, 8, 8, 256, 128, 256, False, True), (5, 2, 1, 40, 0, 4, False, True),
    (7, 2, 2, 24, 12, 8, True, True), (7, 2, 2, 24, 6, 8, False, True), (19, 1, 1, 192, 192, 16, True, True), (70, 64, 1, 64, 32, 16, False, True),
    (2, 70, 70, 16, 16, 8, False, False),
]


class NormCase:
    def __init__(self, T, hq, hkv, D, rot, il, weights, pad=0, eps=1e-5, seed=0, wscale=1.0):
        rng = self.rng = np.random.default_rng(T + D + pad + seed)
        self.T, self.hq, self.hkv, self.D, self.il, self.eps = T, hq, hkv, D, il, eps
        self.width = (hq + 2 * hkv) * D
        # heads of sizes from 1/16 to 16, so that the norm and the mean of its gradient matter
        size = 2.0 ** rng.integers(-4, 5, (T, hq + 2 * hkv, 1))
        self.wide = np.zeros((T, self.width + pad), np.float16)
        self.wide[:, :self.width] = (rng.standard_normal((T, hq + 2 * hkv, D)) * size).reshape(T, -1)
        self.wide[:, self.width:] = np.nan
        self.n_pos = 50
        ang = rng.uniform(-np.pi, np.pi, (self.n_pos, rot // 2)).astype(np.float32)
        self.cos, self.sin = np.cos(ang), np.sin(ang)
        self.pos = rng.integers(0, self.n_pos, T).astype(np.int32)
        self.qw, self.kw = ((rng.standard_normal(D) * wscale).astype(np.float16) if weights else None for _ in range(2))
        self.heads = self.wide[:, :self.width].reshape(T, hq + 2 * hkv, D)

    def split(self):
        hq, hkv, D = self.hq, self.hkv, self.D
        return dev(self.wide)[:, :self.width].split([hq * D, hkv * D, hkv * D], dim=1)

    def tables(self):
        return dev(self.cos), dev(self.sin), dev(self.pos)

    def weights(self):
        return {"q_weight": None if self.qw is None else dev(self.qw), "k_weight": None if self.kw is None else dev(self.kw)}

    def ref(self):
        """(queries, their bound, keys, their bound)."""
        c, s = self.cos[self.pos], self.sin[self.pos]
        return (*oracle.norm_rotate_ref(self.heads[:, :self.hq], self.qw, self.eps, c, s, self.il),
                *oracle.norm_rotate_ref(self.heads[:, self.hq:self.hq + self.hkv], self.kw, self.eps, c, s, self.il))


@pytest.mark.parametrize("T,hq,hkv,D,rot,page,il,weights", NORM)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_append_norm(T, hq, hkv, D, rot, page, il, weights, pad):
    say(f"case append_norm T={T} hq={hq} hkv={hkv} D={D} rot={rot} page={page} il={il} weights={weights} pad={pad}")
    c = NormCase(T, hq, hkv, D, rot, il, weights, pad)
    n_pages = T // page + 3
    slots = c.rng.permutation(n_pages * page)[:T].astype(np.int64)
    k0, v0 = halves(c.rng, n_pages, hkv, page, D), halves(c.rng, n_pages, hkv, page, D)
    cache = PagedKV(n_pages, page, hkv, D, k=dev(k0), v=dev(v0))
    out = cache.append(*c.split(), *c.tables(), dev(slots), interleaved=il, norm_eps=c.eps, **c.weights())
    rq, eq, rk, ek = c.ref()
    assert_near(f64(out), rq, eq, "q")
    want_v = v0.copy()
    want_v[slots // page, :, slots % page] = c.heads[:, hq + hkv:]
    assert np.array_equal(cache.v.cpu().numpy(), want_v)
    want_k, err_k = k0.astype(np.float64), np.zeros(k0.shape)
    want_k[slots // page, :, slots % page], err_k[slots // page, :, slots % page] = rk, ek
    assert_near(f64(cache.k), want_k, err_k, "k")


@pytest.mark.parametrize("T,hq,hkv,D,rot,page,il,weights", NORM)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_norm_rotate_and_gradients(T, hq, hkv, D, rot, page, il, weights, pad):
    say(f"case norm_rotate T={T} hq={hq} hkv={hkv} D={D} rot={rot} il={il} weights={weights} pad={pad}")
    c = NormCase(T, hq, hkv, D, rot, il, weights, pad)
    qt, kt, _ = c.split()
    args = {**c.weights(), "eps": c.eps, "interleaved": il}
    qo, ko = norm_rotate(qt, kt, D, *c.tables(), **args)
    rq, eq, rk, ek = c.ref()
    assert_near(f64(qo), rq, eq, "q")
    assert_near(f64(ko), rk, ek, "k")
    dq, dk = halves(c.rng, T, hq, D), halves(c.rng, T, hkv, D)
    # gradients into slices of one array, whose other places stay
    grad = torch.full((T, c.width + pad), 3.0, dtype=torch.float16, device="cuda")
    gq, gk, gv = grad[:, :c.width].split([hq * D, hkv * D, hkv * D], dim=1)
    r = norm_rotate_backward(qt, kt, dev(dq), dev(dk), *c.tables(), dq=gq, dk=gk, **args)
    turn = (c.cos[c.pos], c.sin[c.pos], il)
    for name, x, w, dy in (("q", c.heads[:, :hq], c.qw, dq), ("k", c.heads[:, hq:hq + hkv], c.kw, dk)):
        dx, dw, ex, ew = oracle.norm_rotate_grads_ref(x, w, c.eps, *turn, dy)
        assert_near(f64(r[f"d{name}"]).reshape(dx.shape), dx, ex, f"d{name}")
        if w is None:
            assert r[f"d{name}_weight"] is None
        else:
            assert_near(f64(r[f"d{name}_weight"]), dw, ew, f"d{name}_weight")
    assert (gv == 3.0).all() and (grad[:, c.width:] == 3.0).all()
    again = norm_rotate_backward(qt, kt, dev(dq), dev(dk), *c.tables(), **args)
    assert all(torch.equal(r[n], again[n]) for n in r if r[n] is not None)


def test_weight_gradients_over_many_rows():
    """More rows than the workgroups take in one pass, as training has them; and only one weight's gradient asked for."""
    c = NormCase(3000, 16, 2, 128, 128, False, True, seed=3)
    qt, kt, _ = c.split()
    dq, dk = halves(c.rng, c.T, 16, 128), halves(c.rng, c.T, 2, 128)
    args = (dev(dq), dev(dk), *c.tables())
    r = norm_rotate_backward(qt, kt, *args, eps=c.eps, **c.weights())
    turn = (c.cos[c.pos], c.sin[c.pos], False)
    for name, x, w, dy in (("q", c.heads[:, :16], c.qw, dq), ("k", c.heads[:, 16:18], c.kw, dk)):
        dx, dw, ex, ew = oracle.norm_rotate_grads_ref(x, w, c.eps, *turn, dy)
        assert_near(f64(r[f"d{name}"]).reshape(dx.shape), dx, ex, f"d{name}")
        assert_near(f64(r[f"d{name}_weight"]), dw, ew, f"d{name}_weight")
    one = norm_rotate_backward(qt, kt, *args, eps=c.eps, k_weight=dev(c.kw))
    assert one["dq_weight"] is None and torch.equal(one["dk_weight"], r["dk_weight"])
    none = norm_rotate_backward(qt, kt, *args, eps=c.eps, weight_grads=False, **c.weights())
    assert none["dk_weight"] is None and torch.equal(none["dq"], r["dq"]) and torch.equal(none["dk"], r["dk"])


def test_norm_of_zeros_and_of_the_largest_values():
    """A head of zeros stays zeros (its gradient is w dy / sqrt(eps)); squares past fp16 do not overflow; a tiny eps is taken."""
    T, H, D, eps = 4, 1, 64, 2.0**-12
    x = np.zeros((T, H, D), np.float16)
    x[1], x[2], x[3, 0, 5] = 65504, -65504, 2.0**-24
    pos, t = np.zeros(T, np.int32), np.zeros((1, 0), np.float32)
    flat = dev(x.reshape(T, D))
    none = torch.zeros((1, 0), device="cuda")
    qo, ko = norm_rotate(flat, flat, D, none, none, dev(pos), eps=eps)
    y, e = oracle.norm_rotate_ref(x, None, eps, t[pos], t[pos], False)
    assert_near(f64(qo), y, e, "q")
    assert torch.equal(qo, ko) and not qo[0].any()
    dy = halves(np.random.default_rng(0), T, H, D)
    r = norm_rotate_backward(flat, flat, dev(dy), dev(dy), none, none, dev(pos), eps=eps)
    dx, _, ex, _ = oracle.norm_rotate_grads_ref(x, None, eps, t[pos], t[pos], False, dy)
    assert_near(f64(r["dq"]).reshape(dx.shape), dx, ex, "dq")
    qo, _ = norm_rotate(flat, flat, D, none, none, dev(pos), eps=1e-38)
    assert not qo[0].any() and torch.isfinite(qo).all()


def test_positions_outside_the_table():
    """NaN results for such tokens, nothing stored, zero gradients, and nothing in the weights' gradients."""
    c = NormCase(8, 4, 2, 64, 64, False, True, seed=5)
    bad = np.array([1, 4, 7])
    c.pos[bad] = [50, -1, 2**31 - 1]
    qt, kt, vt = c.split()
    args = {"eps": c.eps, **c.weights()}
    qo, ko = norm_rotate(qt, kt, 64, *c.tables(), **args)
    nan = torch.isnan(qo).all((1, 2)).cpu().numpy()
    assert np.flatnonzero(nan).tolist() == bad.tolist() and torch.isnan(ko[bad]).all()
    good = np.delete(np.arange(8), bad)
    assert torch.isfinite(qo[good]).all() and torch.isfinite(ko[good]).all()
    dq, dk = halves(c.rng, 8, 4, 64), halves(c.rng, 8, 2, 64)
    dq[bad] = np.nan
    r = norm_rotate_backward(qt, kt, dev(dq), dev(dk), *c.tables(), **args)
    assert not r["dq"][bad].any() and not r["dk"][bad].any()
    turn = (c.cos[c.pos[good]], c.sin[c.pos[good]], False)
    _, dw, _, ew = oracle.norm_rotate_grads_ref(c.heads[good, :4], c.qw, c.eps, *turn, dq[good])
    assert_near(f64(r["dq_weight"]), dw, ew, "dq_weight")
    cache = PagedKV(2, 8, 2, 64)
    slots = torch.arange(8, device="cuda")
    slots[good[0]] = -1
    slots[good[1]] = 16
    out = cache.append(qt, kt, vt, *c.tables(), slots, norm_eps=c.eps, **c.weights())
    assert torch.equal(torch.isnan(out).all((1, 2)).cpu(), torch.from_numpy(nan))
    stored = (cache.k != 0).any(3).any(1).flatten().cpu().numpy()
    assert np.flatnonzero(stored).tolist() == good[2:].tolist()
    assert torch.equal(cache.k[0].transpose(0, 1)[good[2:]], ko[good[2:]])


def test_norms_in_place_and_empty():
    c = NormCase(12, 4, 1, 64, 32, True, True, seed=6)
    qt, kt, vt = (x.contiguous() for x in c.split())
    t, args = c.tables(), {"eps": c.eps, "interleaved": True, **c.weights()}
    qo, ko = norm_rotate(qt, kt, 64, *t, **args)
    dq, dk = dev(halves(c.rng, 12, 4, 64)), dev(halves(c.rng, 12, 1, 64))
    r = norm_rotate_backward(qt, kt, dq, dk, *t, **args)
    same = norm_rotate_backward(qt, kt, dq, dk, *t, dq=dq.view(12, 256), dk=dk.view(12, 64), **args)
    assert same["dq"].data_ptr() == dq.data_ptr() and all(torch.equal(r[n], same[n]) for n in r)
    slots = torch.arange(12, device="cuda")
    cache = PagedKV(2, 8, 1, 64)
    first = cache.append(qt, kt, vt, *t, slots, interleaved=True, norm_eps=c.eps, **c.weights())
    assert torch.equal(first, qo)
    kept = qt.clone()
    got = cache.append(qt, kt, vt, *t, slots, interleaved=True, norm_eps=c.eps, q_out=qt.view(12, 4, 64), **c.weights())
    assert got.data_ptr() == qt.data_ptr() and torch.equal(got, qo)
    got = norm_rotate(kept, kt, 64, *t, q_out=kept.view(12, 4, 64), k_out=kt.view(12, 1, 64), **args)
    assert torch.equal(got[0], qo) and torch.equal(got[1], ko)
    e = [x[:0] for x in (qt, kt, vt)]
    assert cache.append(*e, t[0], t[1], t[2][:0], slots[:0], norm_eps=1e-6).shape == (0, 4, 64)
    assert norm_rotate(e[0], e[1], 64, t[0], t[1], t[2][:0])[1].shape == (0, 1, 64)
    r = norm_rotate_backward(e[0], e[1], dq[:0], dk[:0], t[0], t[1], t[2][:0], **args)
    assert r["dq"].shape == (0, 256) and not r["dq_weight"].any() and not r["dk_weight"].any()
    with pytest.raises(ValueError):
        cache.append(qt, kt, vt, *t, slots, q_weight=dev(c.qw))


def test_norms_of_more_tokens_than_one_launch_holds():
    """2^24 + 5 rows of 33 heads of 4 lanes (a launch takes 2^31 lanes): those of the second launch are normed too, and row
    offsets pass 2^32 values."""
    T, hq, D = 2**24 + 5, 32, 8
    most = 2**31 // (33 * 4)
    assert most < T
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-500, 500, (T, hq * D), generator=gen, device="cuda", dtype=torch.int16).half()
    cos, sin = torch.tensor([[1.0], [0.0]], device="cuda"), torch.tensor([[0.0], [1.0]], device="cuda")
    pos = torch.arange(T, device="cuda", dtype=I32) & 1
    qo, ko = norm_rotate(x, x[:, :D], D, cos, sin, pos, eps=1e-5, interleaved=True)
    at = torch.tensor([0, 1, most - 1, most, most + 1, T - 1], device="cuda")
    heads = x[at].view(-1, hq, D).cpu().numpy()
    c, s = cos.cpu().numpy()[pos[at].cpu()], sin.cpu().numpy()[pos[at].cpu()]
    y, e = oracle.norm_rotate_ref(heads, None, 1e-5, c, s, True)
    assert_near(f64(qo[at]), y, e, "q")
    assert torch.equal(ko[at][:, 0], qo[at][:, 0])
    r = norm_rotate_backward(x, x[:, :D], qo, ko, cos, sin, pos, eps=1e-5, interleaved=True)
    dx, _, ex, _ = oracle.norm_rotate_grads_ref(heads, None, 1e-5, c, s, True, qo[at].cpu().numpy())
    assert_near(f64(r["dq"][at]).reshape(dx.shape), dx, ex, "dq")


def test_norms_on_other_streams_and_in_graphs():
    c = NormCase(40, 8, 2, 128, 128, False, True, seed=8)
    qt, kt, vt = c.split()
    t, args = c.tables(), {"eps": c.eps, **c.weights()}
    dq, dk = dev(halves(c.rng, 40, 8, 128)), dev(halves(c.rng, 40, 2, 128))
    base = norm_rotate(qt, kt, 128, *t, **args), norm_rotate_backward(qt, kt, dq, dk, *t, **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = norm_rotate(qt, kt, 128, *t, stream=side, **args), norm_rotate_backward(qt, kt, dq, dk, *t, stream=side, **args)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[0], base[0])) and all(torch.equal(got[1][n], base[1][n]) for n in base[1])
    x = qt.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = norm_rotate(x, kt, 128, *t, **args)
        grads = norm_rotate_backward(x, kt, dq, dk, *t, **args)
    for f in (1.0, -0.5, 3.0):
        x.copy_(qt * f)
        graph.replay()
        want = norm_rotate(x, kt, 128, *t, **args), norm_rotate_backward(x, kt, dq, dk, *t, **args)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[0])) and all(torch.equal(grads[n], want[1][n]) for n in grads), f


# ---- block tables

class PoolCase:
    def __init__(self, B, page, width, R, lens, prefix=0, window=0, sinks=0, seed=0, gone=True):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.page, self.width, self.prefix, self.window, self.sinks = B, page, width, prefix, window, sinks
        self.lens = np.asarray(lens, np.int64)
        first = -(-max(0, sinks - prefix) // page)
        self.gone = np.zeros(B, np.int64)
        if window and gone:
            self.gone = np.maximum(0, self.lens - rng.integers(1, 20, B) - window + 1) // page
            self.gone[self.gone <= first] = 0
        pages = -(-self.lens // page)
        held = (np.arange(width) < pages[:, None]) & ~((np.arange(width) >= first) & (np.arange(width) < self.gone[:, None]))
        order = rng.permutation(R)
        self.tables = np.full((B, width), -1)
        self.free = R - int(held.sum())
        assert self.free >= 0
        self.tables[held] = order[self.free:]
        self.head = int(rng.integers(0, R))
        self.ring = np.full(R, -1)
        self.ring[(self.head + np.arange(self.free)) % R] = order[:self.free]

    def pool(self):
        p = PagePool(len(self.ring), self.page, self.B, self.width, self.prefix, self.window or None, self.sinks, ring=ints(self.ring),
                     tables=ints(self.tables))
        p.state.copy_(ints(np.concatenate([self.lens, self.gone, [self.head, self.free]])))
        return p

    def check(self, new, T, pool=None, state_out=None):
        pool = pool or self.pool()
        want = oracle.extend_ref(new, self.lens, self.gone, self.head, self.free, self.ring, self.tables, self.page, T, self.prefix,
                                 self.window, self.sinks)
        got = pool.extend(ints(new), T, state_out=state_out)
        state = pool.state if state_out is None else state_out
        for name in ("q_starts", "kv_lens", "positions", "slots", "refused"):
            assert np.array_equal(got[name].cpu().numpy(), want[name]), name
        assert np.array_equal(state.cpu().numpy(), np.concatenate([want["kv_lens"], want["gone"], [want["head"], want["free"]]]))
        assert np.array_equal(pool.tables.cpu().numpy(), want["tables"]) and np.array_equal(pool.ring.cpu().numpy(), want["ring"])
        return got, want, pool


EXTEND = [  # B, page, lens up to, new up to, prefix, window, sinks, ends, spare pages, rows behind the last
    (1, 16, 777, 1, 0, 0, 0, 0.0, 5, 0), (1, 1, 5, 9, 0, 0, 0, 0.0, 20, 3), (7, 16, 100, 40, 33, 0, 0, 0.3, 60, 5),
    (64, 16, 900, 1, 100, 256, 4, 0.1, 64, 0), (64, 16, 900, 1, 0, 256, 40, 0.1, 10, 9), (65, 4, 300, 30, 0, 50, 0, 0.1, 100, 1),
    (130, 64, 2000, 90, 17, 500, 100, 0.05, 40, 700), (1024, 16, 60, 3, 0, 20, 2, 0.2, 300, 0), (1025, 1, 20, 3, 0, 4, 1, 0.2, 2000, 0),
    (2048, 16, 60, 2, 0, 0, 0, 0.2, 3000, 2), (2049, 2, 60, 1, 5, 16, 9, 0.2, 3000, 2), (5000, 16, 300, 2, 0, 64, 0, 0.1, 1000, 100),
    (3, 65536, 200000, 9000, 1, 70000, 3, 0.0, 3, 0), (3, 16, 5000, 9000, 0, 700, 20, 0.0, 2000, 0), (20, 256, 9000, 1, 0, 1, 0, 0.5, 9, 44),
    (8, 16, 3000, 1500, 0, 500, 4, 0.1, 1500, 60), (8, 1, 300, 2500, 0, 0, 0, 0.0, 1000, 3),
]


@pytest.mark.parametrize("B,page,most,new_most,prefix,window,sinks,ends,spare,pad", EXTEND)
def test_extend(B, page, most, new_most, prefix, window, sinks, ends, spare, pad):
    say(f"case extend B={B} page={page} lens={most} new={new_most} prefix={prefix} window={window} sinks={sinks}")
    rng = np.random.default_rng(B + page)
    lens = rng.integers(0, most + 1, B)
    lens[rng.random(B) < 0.2] = 0
    new = np.where(rng.random(B) < ends, -1, rng.integers(0, new_most + 1, B))
    width = int(-(-(most + new_most) // page))
    held = int((-(-lens // page)).sum())
    c = PoolCase(B, page, width, held + spare, lens, prefix, window, sinks, seed=B)
    T = int(np.maximum(new, 0).sum()) + pad
    got, want, pool = c.check(new, T)
    # the same step from the same state into another place, and what it wrote before changes nothing
    again = c.pool()
    other = torch.full_like(again.state, -5)
    c.check(new, T, again, other)
    c.check(new, T, c.pool(), other)
    assert np.array_equal(again.state.cpu().numpy(), np.concatenate([c.lens, c.gone, [c.head, c.free]]))
    # one row fewer than the tokens
    if T > pad:
        c.check(new, T - pad - 1)


def test_extend_refuses_what_finds_no_room():
    """For want of pages (and who comes after whom), past the table's width, past T, past the last position."""
    c = PoolCase(6, 16, 4, 14, [10, 20, 0, 60, 30, 16], prefix=5)
    assert c.free == 14 - 10
    for new, T, refused in (([1, 1, 1, 1, 1, 1], 6, [0] * 6), ([7, 13, 16, 2, 0, 1], 60, [0, 0, 0, 0, 0, 0]),
                            ([23, 13, 33, 2, 0, 1], 99, [0, 0, 1, 0, 0, 1]), ([7, 13, 65, 5, 35, 1], 200, [0, 0, 1, 1, 1, 0]),
                            ([1, 1, 1, 1, 1, 1], 4, [0, 0, 0, 0, 1, 1]), ([2**31 - 1] * 6, 4, [1] * 6), ([1, -1, 2**31 - 1, -1, -1, 16], 17, None)):
        got, want, _ = c.check(new, T)
        assert refused is None or got["refused"].tolist() == refused, new
    c.prefix = 2**31 - 1 - 40  # the fourth passes the last position; the first three take all four free pages
    got, _, _ = c.check([20, 20, 20, 1, 9, 20], 200)
    assert got["refused"].tolist() == [0, 0, 0, 1, 1, 1] and got["positions"].max() == 2**31 - 2


def test_extend_of_nothing():
    c = PoolCase(3, 16, 4, 20, [10, 20, 0])
    c.check([0, 0, 0], 0)
    c.check([-1, -1, -1], 0)
    c.check([0, -1, 0], 5)
    none = PoolCase(0, 16, 4, 20, [])
    none.check([], 0)
    none.check([], 7)
    none.check([], 5000)
    none.check([], 20000)


def test_extend_with_states_that_no_call_left():
    """Lengths, places and counts out of range touch nothing outside the arrays."""
    for lens, gone, head, free in (([2**31 - 1, 500, -7], [0, 3, -4], 0, 5), ([5, 70, 9], [2**31 - 1, 2, 1], 20, 21), ([5, 70, 9], [0, 0, 0], -3, -3),
                                   ([64, 64, 64], [0, 0, 0], 19, 20)):
        for new in ([1, 1, 1], [-1, -1, -1], [30, 0, 3]):
            c = PoolCase(3, 16, 4, 20, [10, 20, 0], window=8, sinks=3)
            c.lens, c.gone, c.head, c.free = np.array(lens), np.array(gone), head, free
            guard = torch.full((3, 200), 7, dtype=I32, device="cuda")
            pool = c.pool()
            ring, tables = guard[0, 50:70], guard[1, 50:62].view(3, 4)
            ring.copy_(pool.ring)
            tables.copy_(pool.tables)
            pool.ring, pool.tables = ring, tables
            c.check(new, 40, pool)
            outside = torch.cat([guard[0, :50], guard[0, 70:], guard[1, :50], guard[1, 62:], guard[2]])
            assert (outside == 7).all()


def test_extend_step_by_step_in_a_graph():
    """A captured step replayed as a server runs it: the pool's own state advances, other counts each time; the same on
    another stream."""
    rng = np.random.default_rng(3)
    B, T, page = 9, 40, 4
    c = PoolCase(B, page, 30, 150, np.zeros(B, int), prefix=7, window=21, sinks=10)
    pool, new = c.pool(), torch.zeros(B, dtype=I32, device="cuda")
    big = c.pool()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pool.extend(new, T)
        wide = big.extend(new, 20000)  # the form of two launches
    side = torch.cuda.Stream()
    for step in range(25):
        n = np.where(rng.random(B) < 0.1, -1, rng.integers(0, 8, B))
        want = oracle.extend_ref(n, c.lens, c.gone, c.head, c.free, c.ring, c.tables, page, T, 7, 21, 10)
        new.copy_(ints(n))
        if step % 5 == 4:  # an eager one between the replays
            side.wait_stream(torch.cuda.current_stream())
            eager = pool.extend(new, T, stream=side)
            big.extend(new, 20000, stream=side)
            torch.cuda.current_stream().wait_stream(side)
            outs = eager
        else:
            graph.replay()
            outs = got
            assert np.array_equal(wide["slots"].cpu().numpy()[:T], want["slots"]) and (wide["slots"][T:] == -1).all()
        torch.cuda.synchronize()
        for name in ("q_starts", "kv_lens", "positions", "slots", "refused"):
            assert np.array_equal(outs[name].cpu().numpy(), want[name]), (step, name)
        assert torch.equal(pool.state, big.state) and torch.equal(pool.ring, big.ring) and torch.equal(pool.tables, big.tables)
        c.lens, c.gone, c.head, c.free, c.ring, c.tables = (want[k] for k in ("kv_lens", "gone", "head", "free", "ring", "tables"))
        assert np.array_equal(pool.state.cpu().numpy(), np.concatenate([c.lens, c.gone, [c.head, c.free]])), step


# ---- windowed attention

class WindowCase(AttnCase):
    """Keys and values that no query sees are NaN, and their pages' entries point nowhere."""

    def __init__(self, hq, hkv, D, page, qs, lens, prefix, window, sinks, **kw):
        super().__init__(hq, hkv, D, page, qs, lens, prefix, **kw)
        self.window, self.sinks = window, sinks
        used = np.zeros(prefix, bool)
        for b, (n, L) in enumerate(zip(qs, lens)):
            seen = self.visible(b).any(0)
            used |= seen[:prefix]
            own = seen[prefix:]
            for t in np.flatnonzero(~own):
                page_, at = self.tables[b, t // page], t % page
                self.k[page_, :, at] = self.v[page_, :, at] = np.nan
            for p in range(-(-L // page)):
                if not own[p * page:(p + 1) * page].any():
                    self.tables[b, p] = (-1, 10**6)[p % 2]
        for t in np.flatnonzero(~used):
            page_, at = self.prefix_table[t // page], t % page
            self.k[page_, :, at] = self.v[page_, :, at] = np.nan

    def visible(self, b, held=None):
        L = self.lens[b]
        return oracle.window_visible(self.qs[b], L if held is None else held, L, self.prefix, self.window, self.sinks)

    def run(self, scale=None, **kw):
        return super().run(scale, window=self.window, sinks=self.sinks, **kw)

    def reference(self, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        G = self.hq // self.hkv
        out, lse, bound = (np.zeros((self.q.shape[0], self.hq) + s) for s in ((self.D,), (), (self.D,)))
        for b in range(len(self.qs)):
            r = slice(self.starts[b], self.starts[b + 1])
            seen = self.visible(b)
            used = seen.any(0)
            for h in range(self.hq):
                kt, vt = (np.concatenate([self.tokens[0][i][:, h // G], self.tokens[b + 1][i][:, h // G]]) for i in (0, 1))
                out[r, h], lse[r, h], bound[r, h] = oracle.attention_ref(self.q[r, h], kt[used], vt[used], seen[:, used], scale)
        return out, lse, bound


WINDOW = [  # q_heads, kv_heads, D, page, queries, own tokens, prefix, window, sinks
    (4, 4, 128, 16, [1], [1], 0, 1, 0), (4, 4, 128, 16, [1], [777], 0, 100, 4), (4, 4, 128, 16, [1], [777], 0, 1, 0),
    (8, 2, 64, 16, [1, 1, 1], [5, 0, 130], 0, 64, 1), (8, 1, 128, 1, [1, 1], [33, 64], 0, 32, 32), (6, 2, 80, 32, [1] * 5, [1, 31, 32, 33, 100], 40, 33, 3),
    (32, 8, 128, 16, [1] * 9, [0, 1, 2, 63, 64, 65, 200, 17, 500], 1000, 300, 20), (32, 8, 128, 16, [1] * 4, [0, 3000, 1, 900], 70, 2000, 90),
    (4, 2, 256, 16, [1, 1], [70, 3], 130, 60, 150), (4, 2, 256, 64, [40, 90], [40, 300], 0, 50, 2), (2, 1, 256, 16, [200], [260], 33, 20, 40),
    (3, 1, 8, 2, [2, 5], [9, 5], 3, 2, 1), (16, 2, 128, 16, [3, 1, 0, 2], [40, 1, 20, 2], 70, 7, 0), (8, 8, 64, 16, [20, 1, 17], [25, 90, 17], 0, 5, 5),
    (8, 8, 96, 16, [20, 1, 17], [25, 90, 17], 65, 100, 10), (4, 4, 128, 64, [150, 64, 65], [150, 64, 400], 0, 64, 0),
    (4, 4, 128, 64, [150, 64, 65], [150, 64, 400], 0, 129, 65), (8, 2, 128, 16, [100, 33], [130, 33], 200, 150, 190), (8, 2, 128, 16, [300], [700], 0, 256, 4),
    (8, 2, 128, 16, [300], [300], 0, 1, 0), (8, 2, 128, 16, [300], [300], 0, 1, 100), (8, 2, 128, 16, [300], [300], 0, 3, 1000), (2, 2, 64, 16, [700], [900], 50, 333, 17),
    (8, 2, 64, 16, [300], [300], 0, 5000, 4), (16, 2, 40, 256, [50], [700], 0, 90, 64), (64, 8, 128, 16, [1] * 3, [300, 40, 0], 0, 30, 0),
    (24, 8, 192, 32, [7, 9], [100, 9], 500, 505, 1), (12, 4, 64, 1, [5] * 4, [5, 40, 6, 77], 129, 40, 33), (4, 1, 128, 16, [1], [0], 0, 9, 9),
    (4, 1, 128, 16, [3], [0], 0, 9, 9), (4, 1, 128, 16, [3], [1], 20, 9, 2), (1, 1, 64, 16, [400], [400], 0, 2**31 - 1, 2**31 - 1),
    (2, 1, 128, 16, [260], [2000], 0, 1100, 70), (1, 1, 128, 16, [513], [513], 128, 128, 128),
]


@pytest.mark.parametrize("hq,hkv,D,page,qs,lens,prefix,window,sinks", WINDOW)
def test_windowed_attention(hq, hkv, D, page, qs, lens, prefix, window, sinks):
    say(f"case window hq={hq} hkv={hkv} D={D} page={page} q={qs} lens={lens} prefix={prefix} window={window} sinks={sinks}")
    WindowCase(hq, hkv, D, page, qs, lens, prefix, window, sinks, seed=len(qs)).upload().check()


def test_windowed_attention_with_loose_bounds_and_other_scales():
    c = WindowCase(8, 2, 128, 16, [1, 2, 1], [100, 37, 300], 50, 60, 5, seed=4, spread=4.0).upload()
    c.check()
    c.check(max_q=90, max_len=5000)
    c.check(max_q=17, max_len=330)
    c.check(scale=1e-6)
    c.check(scale=1.0)


@pytest.mark.parametrize("hq,hkv,D,qs,lens,prefix,window,sinks", [
    (2, 1, 64, [1, 1], [1, 5398], 0, 5000, 100), (1, 1, 8, [1], [9000], 0, 8000, 0), (4, 1, 64, [2, 1], [3000, 2500], 4000, 6000, 300),
    (2, 2, 256, [1], [6000], 4500, 9999, 9), (8, 1, 64, [9, 9], [2000, 1500], 3000, 4000, 2), (2, 1, 128, [30], [6000], 0, 5000, 1000)])
def test_many_parts_of_a_window(hq, hkv, D, qs, lens, prefix, window, sinks):
    say(f"case window parts hq={hq} hkv={hkv} D={D} q={qs} lens={lens} prefix={prefix} window={window} sinks={sinks}")
    c = WindowCase(hq, hkv, D, 64, qs, lens, prefix, window, sinks, seed=19).upload()
    c.check()
    need = q.qgemm_attention_window_workspace(c.cache.desc, sum(qs), hq, len(qs), max(qs), max(lens), prefix, window, sinks)
    assert need // (sum(qs) * hq * (D * 4 + 8)) > 3


@pytest.mark.parametrize("qs,lens,prefix,window,sinks", [([40], [40], 0, 10, 2), ([3], [40], 0, 10, 0), ([1, 150], [20, 150], 90, 60, 3),
                                                         ([200], [300], 0, 128, 5)])
def test_values_outside_a_window_never_matter(qs, lens, prefix, window, sinks):
    """NaN and infinities of one token reach only the queries that see it, at either edge of the window and among the sinks."""
    c = WindowCase(4, 2, 128, 16, qs, lens, prefix, window, sinks, seed=11).upload()
    clean, _ = c.run()
    b = len(qs) - 1
    seen = c.visible(b)
    some = [t for t in range(prefix, seen.shape[1]) if 0 < seen[:, t].sum()]
    for t in sorted({some[0], some[len(some) // 2], some[-1], prefix + lens[-1] - qs[-1]}):
        own = t - prefix
        page, at = c.tables[b, own // 16], own % 16
        for what in (np.nan, np.inf, -np.inf):
            k, v = c.k[page, :, at].copy(), c.v[page, :, at].copy()
            c.v[page, :, at, 7] = what
            got, _ = c.upload().run()
            hit = np.zeros(len(got), bool)
            hit[c.starts[b]:] = seen[:, t]
            assert np.array_equal(got[~hit], clean[~hit]), (t, what)
            assert np.array_equal(got[hit][..., 7], np.full((hit.sum(), 4), what), equal_nan=True), (t, what)
            c.k[page, :, at, 5] = what
            c.k[page, :, at, 6] = np.nan
            got, _ = c.upload().run()
            assert np.array_equal(got[~hit], clean[~hit]) and not np.isfinite(got[hit]).any(), (t, what)
            c.k[page, :, at], c.v[page, :, at] = k, v


@pytest.mark.parametrize("hq,hkv,D,qs,lens,prefix,window,sinks,max_q,max_len,width", [
    (8, 2, 128, [5, 2], [40, 30], 0, 12, 3, 3, 40, 9), (8, 2, 128, [5, 2], [140, 100], 70, 60, 9, 5, 77, 9), (4, 1, 64, [1, 1], [140, 100], 70, 90, 3, 1, 140, 5),
    (4, 2, 128, [100, 150], [130, 190], 0, 64, 1, 70, 190, 12), (4, 2, 128, [100, 150], [130, 190], 33, 100, 0, 150, 100, 12),
    (8, 1, 128, [6], [6], 0, 2, 1, 2, 6, 1), (2, 2, 256, [90], [400], 0, 70, 150, 60, 300, 15)])
def test_rows_and_tokens_past_the_bounds_are_left_out_of_windows(hq, hkv, D, qs, lens, prefix, window, sinks, max_q, max_len, width):
    say(f"case window bounds q={qs} lens={lens} window={window} max_q={max_q} max_len={max_len} width={width}")
    c = WindowCase(hq, hkv, D, 16, qs, lens, prefix, window, sinks, seed=13).upload()
    c.dtables = dev(c.tables[:, :width])
    out = torch.full((sum(qs), hq, D), 3.0, dtype=torch.float16, device="cuda")
    got, lse = c.run(max_q=max_q, max_len=max_len, out=out)
    for b, (n, L) in enumerate(zip(qs, lens)):
        m, held, r0 = min(n, max_q), min(L, max_len, width * 16), c.starts[b]
        seen = c.visible(b, held)[:m]
        used = seen.any(0)
        for h in range(hq):
            kt, vt = (np.concatenate([c.tokens[0][i][:, h // (hq // hkv)], c.tokens[b + 1][i][:held, h // (hq // hkv)]]) for i in (0, 1))
            ref, ref_lse, bound = oracle.attention_ref(c.q[r0:r0 + m, h], kt[used], vt[used], seen[:, used], D ** -0.5)
            assert_near(got[r0:r0 + m, h], ref, bound, f"sequence {b} head {h}")
            live = np.isfinite(ref_lse)
            assert np.array_equal(np.isneginf(lse[r0:r0 + m, h]), ~live)
            assert (np.abs(lse[r0:r0 + m, h] - ref_lse)[live] <= 1e-4 + 1e-5 * np.abs(ref_lse[live])).all()
        assert (got[r0 + m:c.starts[b + 1]] == 3.0).all()


def test_windowed_attention_on_another_stream_and_in_a_graph():
    c = WindowCase(8, 2, 128, 16, [1, 1, 1, 1], [90, 17, 0, 300], 200, 150, 6, seed=9).upload()
    base, _ = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = c.cache.attend(c.dq, c.dstarts, c.dlens, c.dtables, 1, 300, c.dprefix, 200, stream=side, window=150, sinks=6)
    side.synchronize()
    assert np.array_equal(f64(out), base)
    again, _ = c.run()
    assert np.array_equal(again, base)
    # captured once, replayed with other lengths (whose windows see tokens that are NaN here, so these get values first)
    for arr in (c.k, c.v):
        arr[np.isnan(arr)] = 0.5
    for b, L in enumerate(c.lens):
        c.tables[b, :-(-L // 16)] = np.arange(-(-L // 16)) + 40 * b
    c.upload()
    lens, out = c.dlens.clone(), torch.empty_like(c.dq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.cache.attend(c.dq, c.dstarts, lens, c.dtables, 1, 300, c.dprefix, 200, out=out, window=150, sinks=6)
    for cut in (0, 16, 5):
        lens.copy_(torch.tensor([max(0, n - cut) for n in c.lens], dtype=I32))
        graph.replay()
        want = c.cache.attend(c.dq, c.dstarts, lens, c.dtables, 1, 300, c.dprefix, 200, window=150, sinks=6)
        torch.cuda.synchronize()
        assert torch.equal(out, want), cut
    with pytest.raises(ValueError):
        c.cache.attend(c.dq, c.dstarts, lens, c.dtables, 1, 300, sinks=6)


def test_a_wide_window_sees_what_no_window_sees():
    c = WindowCase(8, 2, 128, 16, [1, 40, 1], [90, 170, 0], 200, 10**6, 0, seed=21).upload()
    c.check()
    plain, _ = AttnCase.run(c)
    got, _ = c.run()
    _, _, bound = c.reference()
    assert_near(got, plain, 2 * bound, "out")


# ---- a run of them together

@pytest.mark.parametrize("hq,hkv,D,rot,window,sinks,prefix", [(8, 2, 64, 64, 37, 5, 21), (4, 4, 80, 40, 16, 0, 0), (8, 1, 128, 128, 50, 40, 9)])
def test_serving_with_a_window(hq, hkv, D, rot, window, sinks, prefix):
    """Prompts and single tokens of sequences that come and go, through extend, append and attend, from a pool that only lasts
    because windows give pages back; checked against attention over each sequence's own rounded keys and values."""
    say(f"case serving hq={hq} hkv={hkv} D={D} window={window} sinks={sinks} prefix={prefix}")
    rng = np.random.default_rng(D)
    B, page, T, eps, n_prefix = 4, 8, 96, 1e-5, -(-prefix // 8)
    held = (sinks + window) // page + 4                      # pages that a sequence needs beside those of a step's new tokens
    R = B * held + T // page
    cache = PagedKV(n_prefix + R, page, hkv, D)
    pool = PagePool(R, page, B, 60, prefix, window, sinks, ring=torch.arange(n_prefix, n_prefix + R, dtype=I32, device="cuda"))
    ang = rng.uniform(-np.pi, np.pi, (2000, rot // 2)).astype(np.float32)
    cos, sin, qw, kw = np.cos(ang), np.sin(ang), (1 + 0.2 * rng.standard_normal(D)).astype(np.float16), halves(rng, D)
    tabs = dev(cos), dev(sin)
    prefix_table = torch.arange(n_prefix, dtype=I32, device="cuda") if prefix else None

    def project(n):
        x = halves(rng, n, (hq + 2 * hkv) * D)
        return x, dev(x).split([hq * D, hkv * D, hkv * D], dim=1)

    def stored(slots):
        flat = lambda c: c.transpose(1, 2).reshape(-1, hkv, D)[slots].cpu().numpy()  # noqa: E731
        return flat(cache.k), flat(cache.v)

    if prefix:
        _, parts = project(prefix)
        at = torch.arange(prefix, device="cuda")
        cache.append(*parts, *tabs, at.int(), at, norm_eps=eps, q_weight=dev(qw), k_weight=dev(kw))
        first = stored(at)
    else:
        first = (np.zeros((0, hkv, D), np.float16),) * 2
    past = [first] * B
    for step in range(30):
        new = rng.integers(0, 2, B)
        new[rng.integers(0, B)] = rng.integers(1, 25)
        if step % 4 == 3:
            new[rng.integers(0, B)] = -1
        for b in range(B):  # a sequence ends before its table does
            if len(past[b][0]) + new[b] > 300:
                new[b] = -1
        x, parts = project(T)
        r = pool.extend(ints(new), T)
        assert not r["refused"].any(), step
        qo = cache.append(*parts, *tabs, r["positions"], r["slots"], norm_eps=eps, q_weight=dev(qw), k_weight=dev(kw))
        out = f64(cache.attend(qo, r["q_starts"], r["kv_lens"], pool.tables, T, 400, prefix_table, prefix, window=window, sinks=sinks))
        starts, qh = r["q_starts"].cpu().numpy(), qo.cpu().numpy()
        for b in range(B):
            n, r0 = max(int(new[b]), 0), starts[b]
            if new[b] < 0:
                past[b] = first
            if n == 0:
                continue
            before = len(past[b][0])
            pos = np.arange(before, before + n)
            heads = x[r0:r0 + n].reshape(n, hq + 2 * hkv, D)
            want_q, eq = oracle.norm_rotate_ref(heads[:, :hq], qw, eps, cos[pos], sin[pos], False)
            want_k, ek = oracle.norm_rotate_ref(heads[:, hq:hq + hkv], kw, eps, cos[pos], sin[pos], False)
            kt, vt = stored(r["slots"][r0:r0 + n])
            assert_near(qh[r0:r0 + n].astype(np.float64), want_q, eq, f"step {step} queries")
            assert_near(kt.astype(np.float64), want_k, ek, f"step {step} keys")
            assert np.array_equal(vt, heads[:, hq + hkv:])
            past[b] = tuple(np.concatenate([p, y]) for p, y in zip(past[b], (kt, vt)))
            seen = oracle.window_visible(n, before + n - prefix, before + n - prefix, prefix, window, sinks)
            for h in range(hq):
                ks, vs = (p[:, h // (hq // hkv)] for p in past[b])
                ref, _, bound = oracle.attention_ref(qh[r0:r0 + n, h], ks, vs, seen, D ** -0.5)
                assert_near(out[r0:r0 + n, h], ref, bound, f"step {step} sequence {b} head {h}")


def test_windowed_example_runs(capsys, monkeypatch):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import windowed_decoder_layer as ex
    monkeypatch.setattr(sys, "argv", ["windowed_decoder_layer.py", "--steps", "11"])
    ex.main()
    out = capsys.readouterr().out
    assert out.count("finite: True") == 3 and "refused: 0" in out


# ---- other calls that the documentation allows

def test_windowed_cache_offsets_past_32_bits():
    """Pages whose byte and value offsets pass 2**32, for single tokens and for tiles of 128 rows."""
    hkv, D, page = 8, 128, 256
    n_pages = (2**32 + 2**27) // (hkv * D * page)
    k, v = (torch.empty((n_pages, hkv, page, D), dtype=torch.float16, device="cuda") for _ in range(2))
    cache = PagedKV(n_pages, page, hkv, D, k=k, v=v)
    rng = np.random.default_rng(2)
    T, window, sinks = 300, 100, 7
    rows = dev(halves(rng, T, 3 * hkv * D))
    qt, kt, vt = rows.split([hkv * D] * 3, dim=1)
    pages = np.array([n_pages - 1, n_pages - 3], np.int32)
    t = np.arange(T)
    slots = pages[t // page].astype(np.int64) * page + t % page
    none = torch.empty((1, 0), device="cuda")
    qo = cache.append(qt, kt, vt, none, none, torch.zeros(T, dtype=I32, device="cuda"), dev(slots), norm_eps=1e-5)
    assert torch.equal(v[n_pages - 3, :, : T - page].transpose(0, 1), vt[page:].view(-1, hkv, D))
    kn = k[n_pages - 1].transpose(0, 1), k[n_pages - 3, :, : T - page].transpose(0, 1)
    kh, vh, qh = torch.cat(kn).cpu().numpy(), vt.reshape(T, hkv, D).cpu().numpy(), qo.cpu().numpy()
    for n in (1, 200):
        got = f64(cache.attend(qo[T - n:], ints([0, n]), ints([T]), ints(pages[None]), n, T, window=window, sinks=sinks))
        seen = oracle.window_visible(n, T, T, 0, window, sinks)
        for h in range(hkv):
            ref, _, bound = oracle.attention_ref(qh[T - n:, h], kh[:, h], vh[:, h], seen, D ** -0.5)
            assert_near(got[:, h], ref, bound, f"{n} queries, head {h}")


def random_window_case(seed):
    rng = np.random.default_rng(1000 + seed)
    hkv = int(rng.choice([1, 2, 3]))
    G = int(rng.choice([1, 2, 5, 8]))
    B = int(rng.integers(1, 5))
    qs = [int(rng.choice([0, 1, 3, rng.integers(1, 200)])) for _ in range(B)]
    qs[0] = max(qs[0], 1)
    lens = [int(rng.integers(0, 400)) if rng.random() < 0.3 else n + int(rng.integers(0, 500)) for n in qs]
    return (hkv * G, hkv, int(rng.choice([8, 40, 64, 88, 128, 136])), int(rng.choice([1, 4, 16, 128])), qs, lens,
            int(rng.choice([0, rng.integers(1, 300)])), int(rng.choice([1, 2, 63, 64, 65, rng.integers(1, 600)])), int(rng.choice([0, 1, 64, rng.integers(0, 400)])))


@pytest.mark.parametrize("seed", range(40))
def test_windowed_attention_at_random(seed):
    """Mixed queries, lengths shorter than the queries among them, sinks past the windows, every page size."""
    a = random_window_case(seed)
    say("case window", a)
    WindowCase(*a, seed=seed).upload().check()


def test_calls_refuse_what_they_cannot_take():
    c = NormCase(6, 4, 2, 64, 64, False, True, seed=4)
    qt, kt, vt = c.split()
    cos, sin, pos = c.tables()
    slots = torch.arange(6, device="cuda")
    cache = PagedKV(2, 8, 2, 64)
    for eps in (0.0, -1.0, float("nan"), 1e-60):
        for f in (lambda: cache.append(qt, kt, vt, cos, sin, pos, slots, norm_eps=eps),
                  lambda: norm_rotate(qt, kt, 64, cos, sin, pos, eps=eps)):
            with pytest.raises(q.QGemmError) as e:
                f()
            assert e.value.status == q.QGEMM_ERR_INVALID_ARG
    d3 = torch.zeros((6, 4, 64), dtype=torch.float16, device="cuda")
    for what, f in (("positions:", lambda: norm_rotate(qt, kt, 64, cos, sin, pos.cpu())),
                    ("k:", lambda: cache.append(qt, kt.float(), vt, cos, sin, pos, slots, norm_eps=1e-5)),
                    ("v:", lambda: cache.append(qt, kt, vt[:, :64], cos, sin, pos, slots, norm_eps=1e-5)),
                    ("slots:", lambda: cache.append(qt, kt, vt, cos, sin, pos, slots.int(), norm_eps=1e-5)),
                    ("q_out:", lambda: cache.append(qt, kt, vt, cos, sin, pos, slots, norm_eps=1e-5, q_out=d3.transpose(0, 1))),
                    ("dk_out:", lambda: norm_rotate_backward(qt, kt, d3, d3[:, :2], cos, sin, pos)),
                    ("dq:", lambda: norm_rotate_backward(qt, kt, d3, d3[:, :2].contiguous(), cos, sin, pos, dq=d3[0])),
                    ("k:", lambda: norm_rotate(qt, kt[:5], 64, cos, sin, pos)), ("q:", lambda: norm_rotate(qt[0], kt, 64, cos, sin, pos))):
        with pytest.raises(ValueError, match=what):
            f()
    with pytest.raises(TypeError):
        q.binding().extend(0, 0)
    w = WindowCase(4, 2, 64, 16, [1], [40], 20, 30, 2, seed=3).upload()
    for kw, error in ((dict(window=0), q.QGemmError), (dict(window=-3), q.QGemmError), (dict(sinks=-1), q.QGemmError), (dict(prefix_table=None), ValueError),
                      (dict(tables=w.dtables.long()), ValueError), (dict(q_starts=w.dstarts[:1]), ValueError), (dict(q=w.dq.float()), ValueError),
                      (dict(q=w.dq[:, :, :32]), ValueError), (dict(lse=torch.zeros((1, 4), dtype=torch.float64, device="cuda")), ValueError)):
        args = dict(q=w.dq, q_starts=w.dstarts, kv_lens=w.dlens, tables=w.dtables, max_q=1, max_len=40, prefix_table=w.dprefix, prefix_len=20, window=30,
                    sinks=2)
        with pytest.raises(error):
            w.cache.attend(**{**args, **kw})
    pool = PagePool(6, 16, 3, 4)
    with pytest.raises(ValueError, match="new_tokens:"):
        pool.extend(torch.zeros(3, dtype=I32), 4)
    for page in (0, 24):
        with pytest.raises(q.QGemmError):
            PagePool(6, page, 3, 4).extend(torch.zeros(3, dtype=I32, device="cuda"), 4)
    with pytest.raises(ValueError):
        pool.extend(torch.zeros(3, dtype=I32, device="cuda"), -1)


def test_results_do_not_depend_on_what_memory_held():
    """Workspaces and results of every call begin as NaN or junk: the results are the same."""
    c = NormCase(700, 8, 2, 96, 64, True, True, seed=7)
    qt, kt, _ = c.split()
    dq, dk = dev(halves(c.rng, 700, 8, 96)), dev(halves(c.rng, 700, 2, 96))
    p = PoolCase(50, 16, 40, 900, np.arange(50) * 7, window=64, sinks=4)
    new = ints(np.where(np.arange(50) % 7 == 6, -1, 100))
    results = []
    for fill in (0xFF, 0x00, 0x7B):
        torch.cuda.empty_cache()
        junk = [torch.full((1 << 22,), fill, dtype=torch.uint8, device="cuda") for _ in range(24)]
        del junk
        r = norm_rotate_backward(qt, kt, dq, dk, *c.tables(), eps=c.eps, interleaved=True, **c.weights())
        pool = p.pool()
        e = pool.extend(new, 7000)
        results.append([*r.values(), *(t.clone() for t in e.values()), pool.tables.clone(), pool.ring.clone(), pool.state.clone()])
    assert all(torch.equal(a, b) for other in results[1:] for a, b in zip(results[0], other))


def test_workspaces_have_to_be_whole():
    """A workspace that is large by its shape alone is refused, and so is a small one."""
    byte = torch.zeros(1, dtype=torch.uint8, device="cuda")
    c = NormCase(6, 4, 2, 64, 64, False, True, seed=4)
    qt, kt, _ = c.split()
    d = [torch.zeros((6, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2)]
    w = WindowCase(4, 2, 64, 16, [1], [2000], 0, 1500, 2, seed=3).upload()
    pool = PagePool(6, 16, 3, 4)
    for ws, error in ((byte.expand(1 << 24), ValueError), (byte, q.QGemmError)):
        for f in (lambda: norm_rotate_backward(qt, kt, *d, *c.tables(), **c.weights(), ws=ws),
                  lambda: w.cache.attend(w.dq, w.dstarts, w.dlens, w.dtables, max_q=1, max_len=2000, window=1500, sinks=2, ws=ws),
                  lambda: pool.extend(torch.zeros(3, dtype=I32, device="cuda"), 50000, ws=ws)):
            with pytest.raises(error):
                f()


def test_windows_in_parts_do_not_depend_on_what_memory_held():
    w = WindowCase(8, 2, 128, 16, [1, 3, 40, 0], [3000, 5, 900, 60], 70, 1500, 40, seed=3).upload()
    need = q.qgemm_attention_window_workspace(w.cache.desc, 44, 8, 4, 40, 3000, 70, 1500, 40)
    assert need > 0
    results = []
    for fill in (0xFF, 0x00, 0x7B):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((44, 8, 128), float("nan"), dtype=torch.float16, device="cuda")
        lse = torch.full((44, 8), float("nan"), device="cuda")
        w.cache.attend(w.dq, w.dstarts, w.dlens, w.dtables, max_q=40, max_len=3000, prefix_table=w.dprefix, prefix_len=70, window=1500, sinks=40,
                       ws=ws, out=out, lse=lse)
        results.append((out, lse))
    assert not torch.isnan(results[0][0]).any()
    assert all(torch.equal(a, b) for other in results[1:] for a, b in zip(results[0], other))


@pytest.mark.parametrize("D", [136, 192, 256])
def test_windows_of_wide_heads_over_many_rows(D):
    """Enough tiles that those of 128 rows are taken for heads past 128 too (20 of 64 rows a sequence's heads, 256 CUs)."""
    say("case wide heads", D)
    WindowCase(16, 16, D, 16, [300, 301, 299, 250], [300, 500, 290, 600], 20, 100, 30, seed=D).upload().check()
    WindowCase(32, 16, D, 64, [150, 1, 170], [150, 900, 400], 0, 260, 0, seed=D + 1).upload().check()


@pytest.mark.parametrize("hq,hkv,D,qs,lens", [(4, 2, 64, [40, 150], [50, 150]), (4, 2, 128, [40, 150], [50, 150]), (16, 16, 256, [300, 301, 299, 250], [310, 500, 299, 600]),
                                              (16, 16, 136, [300, 301, 299, 250], [310, 500, 299, 600])])
def test_infinities_at_any_place_reach_the_rows_that_see_them(hq, hkv, D, qs, lens):
    c = WindowCase(hq, hkv, D, 16, qs, lens, 70, 90, 33, seed=D)
    rng = np.random.default_rng(D)
    bad = []  # (sequence, token, kv head, place, value)
    for b, n in enumerate(lens):
        for t in rng.choice(n, 12, replace=False):
            if c.visible(b)[:, 70 + t].any():
                bad.append((b, int(t), int(rng.integers(hkv)), int(rng.integers(D)), float(rng.choice([np.inf, -np.inf, np.nan]))))
    say(f"case infinities {hq}/{hkv} heads of {D}: {len(bad)}")
    plain, _ = c.upload().run()
    want = plain.copy()
    for b, t, h, e, value in bad:
        c.v[c.tables[b, t // 16], h, t % 16, e] = value
        rows = np.flatnonzero(c.visible(b)[:, 70 + t]) + c.starts[b]
        heads = range(h * (hq // hkv), (h + 1) * (hq // hkv))
        with np.errstate(invalid="ignore"):
            want[np.ix_(rows, heads, [e])] += np.asarray(value, want.dtype)
    got, _ = c.upload().run()
    finite = np.isfinite(want)
    assert not finite.all() and np.array_equal(got[finite], plain[finite]) and np.array_equal(got[~finite], want[~finite], equal_nan=True)


@pytest.mark.parametrize("hq,hkv,D,qs,lens,prefix,window,sinks", [
    (4, 2, 128, [200], [700], 0, 64, 300), (4, 2, 64, [200, 333], [250, 333], 150, 20, 257), (8, 1, 128, [90], [2000], 0, 900, 1000),
    (16, 16, 256, [300, 301, 299, 250], [310, 500, 299, 600], 20, 50, 250)])
def test_many_first_keys(hq, hkv, D, qs, lens, prefix, window, sinks):
    """Blocks of first keys that every row of a tile sees, behind ones of the window that some do not; keys split or not."""
    say(f"case first keys hq={hq} hkv={hkv} D={D} q={qs} lens={lens} prefix={prefix} window={window} sinks={sinks}")
    WindowCase(hq, hkv, D, 16, qs, lens, prefix, window, sinks, seed=sinks).upload().check()
