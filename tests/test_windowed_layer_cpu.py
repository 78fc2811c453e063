"""Host-side checks of normed appends, their gradients, block tables and windowed attention (no
device calls): the float64 references against brute force and differences, and every refusal
of the entry points."""
import numpy as np
import pytest

import oracle
from weight_quantized_mixed_amd import qgemm as q

P = 4096  # an aligned address that no refused call may touch
BAD, UNS = q.QGEMM_ERR_INVALID_ARG, q.QGEMM_ERR_UNSUPPORTED


def status(fn, *args):
    try:
        fn(*args)
    except q.QGemmError as e:
        return e.status
    return q.QGEMM_OK


def cache(**kw):
    a = dict(k=P, v=P, n_pages=10, page_size=16, kv_heads=2, head_dim=128)
    a.update(kw)
    return q.KVCacheDesc(*a.values())


# ---- the references

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_norm_gradients_against_differences(interleaved, weight):
    rng = np.random.default_rng(4)
    T, H, D, eps, h = 3, 2, 8, 1e-3, 1e-5
    x, dy, w = rng.standard_normal((T, H, D)), rng.standard_normal((T, H, D)), rng.standard_normal(D) if weight else None
    a = rng.uniform(-3, 3, (T, 3))
    turn = (np.cos(a), np.sin(a), interleaved)
    dx, dw, _, _ = oracle.norm_rotate_grads_ref(x, w, eps, *turn, dy)
    loss = lambda x, w: float((oracle.norm_rotate_ref(x, w, eps, *turn)[0] * dy).sum())  # noqa: E731
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        # central differences: h^2 / 6 of the third derivative (below 100 here), and rounding of the loss / h
        assert abs((loss(up, w) - loss(down, w)) / (2 * h) - dx[i]) < 1e-7, i
    for d in range(D if weight else 0):
        up, down = w.copy(), w.copy()
        up[d] += h
        down[d] -= h
        assert abs((loss(x, up) - loss(x, down)) / (2 * h) - dw[d]) < 1e-7, d


def test_norm_by_hand():
    x = np.array([[[3.0, 4.0, 0, 0, 0, 0, 0, 0]]])  # mean of squares 25 / 8
    y, _ = oracle.norm_rotate_ref(x, np.full(8, 2.0), 0.0, np.zeros((1, 1)), np.ones((1, 1)), True)
    assert np.allclose(y[0, 0, :2], np.array([-4.0, 3.0]) * 2 * np.sqrt(8) / 5) and not y[0, 0, 2:].any()


def test_windows_by_hand():
    see = lambda *a: ["".join("x" if v else "." for v in row) for row in oracle.window_visible(*a)]  # noqa: E731
    assert see(3, 4, 4, 2, 2, 1) == ["x.xx..", "x..xx.", "x...xx"]
    assert see(2, 5, 5, 0, 1, 0) == ["...x.", "....x"] and see(2, 5, 5, 0, 9, 0) == ["xxxx.", "xxxxx"]
    assert see(2, 1, 1, 2, 1, 0) == [".x.", "..x"]      # a query without own tokens sees the end of the prefix
    assert see(1, 3, 5, 0, 3, 1) == ["x.x"]             # of five tokens three are read


def test_extend_by_hand():
    # two sequences of 3 and 4 tokens on pages of 4, the first one grows over a page's end, the second ends
    r = oracle.extend_ref([3, -1], [3, 4], [0, 0], head=1, free=2, ring=[9, 7, 8, 5], tables=[[6, -1], [2, -1]], page=4, T=4, prefix=10)
    assert r["q_starts"].tolist() == [0, 3, 3] and r["kv_lens"].tolist() == [6, 0] and r["positions"].tolist() == [13, 14, 15, 0]
    assert r["slots"].tolist() == [27, 28, 29, -1] and r["tables"].tolist() == [[6, 7], [2, -1]]
    assert r["ring"].tolist() == [9, 7, 8, 2] and (r["head"], r["free"]) == (2, 2)


def test_extend_never_loses_a_page():
    """Over many steps of sequences that grow, end and begin: held and free pages are all pages, each once, and what a window
    sees is held."""
    rng = np.random.default_rng(7)
    B, width, page, R, window, sinks, prefix = 5, 12, 4, 40, 13, 6, 3
    tables, ring, lens, gone, head, free = np.full((B, width), -1), np.arange(R), np.zeros(B, int), np.zeros(B, int), 0, R
    first = -(-(sinks - prefix) // page)
    for step in range(300):
        new = np.where(rng.random(B) < 0.1, -1, rng.integers(0, 7, B))
        r = oracle.extend_ref(new, lens, gone, head, free, ring, tables, page, 40, prefix, window, sinks)
        before = lens
        tables, ring, lens, gone, head, free = (r[k] for k in ("tables", "ring", "kv_lens", "gone", "head", "free"))
        held = [tables[b, p] for b in range(B) for p in range(-(-lens[b] // page)) if not first <= p < gone[b]]
        assert sorted(held + [ring[(head + i) % R] for i in range(free)]) == list(range(R)), step
        for b in range(B):
            if new[b] > 0 and not r["refused"][b]:
                seen = oracle.window_visible(new[b], lens[b], lens[b], prefix, window, sinks).any(0)[prefix:]
                assert seen[before[b]:].all()
                assert not any(first <= t // page < gone[b] for t in np.flatnonzero(seen))


# ---- refusals

NORM = dict(qw=P, kw=P, eps=1e-6, cos=P, sin=P, n=9, rot=128, il=0)
BAD_NORM = (dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-50), dict(qw=P + 1), dict(kw=P + 1),
            dict(cos=0), dict(sin=0), dict(n=0), dict(rot=-2), dict(rot=7), dict(rot=130), dict(il=2), dict(cos=P + 2), dict(sin=P + 2))


def test_append_norm_refuses_bad_arguments():
    ok = dict(T=4, hq=8, q=P, qs=1024, k=P, ks=256, v=P, vs=256, **NORM, pos=P, slots=P, out=P)
    for kw in BAD_NORM + (dict(T=-1), dict(hq=0), dict(hq=5), dict(q=0), dict(k=0), dict(v=0), dict(qs=1023), dict(ks=255),
                          dict(vs=255), dict(pos=0), dict(slots=0), dict(out=0), dict(q=P + 1), dict(pos=P + 2), dict(slots=P + 4),
                          dict(out=P + 1)):
        assert status(q.qgemm_kv_append_norm, cache(), *{**ok, **kw}.values()) == BAD, kw
    assert status(q.qgemm_kv_append_norm, None, *ok.values()) == BAD
    for kw, want in ((dict(head_dim=100), UNS), (dict(page_size=24), UNS), (dict(kv_heads=3), BAD), (dict(k=0), BAD)):
        assert status(q.qgemm_kv_append_norm, cache(**kw), *ok.values()) == want, kw
    assert status(q.qgemm_kv_append_norm, cache(), *{**ok, "T": 0, "q": 0}.values()) == q.QGEMM_OK


def test_norm_rotate_refuses_bad_arguments():
    ok = dict(T=4, hq=8, hkv=2, D=128, q=P, qs=1024, k=P, ks=256, **NORM, pos=P, qo=P, ko=P)
    for kw in BAD_NORM + (dict(T=-1), dict(hq=0), dict(hkv=0), dict(D=0), dict(q=0), dict(k=0), dict(qs=1023), dict(ks=255),
                          dict(pos=0), dict(qo=0), dict(ko=0), dict(q=P + 1), dict(pos=P + 2), dict(ko=P + 1)):
        assert status(q.qgemm_norm_rotate, *{**ok, **kw}.values()) == BAD, kw
    for kw in (dict(D=100), dict(D=264, qs=3000, ks=3000), dict(T=2**31), dict(hq=65536, qs=2**30), dict(hkv=65536, ks=2**30)):
        assert status(q.qgemm_norm_rotate, *{**ok, **kw}.values()) == UNS, kw
    assert status(q.qgemm_norm_rotate, *{**ok, "T": 0, "q": 0}.values()) == q.QGEMM_OK


def test_norm_backward_refuses_bad_arguments():
    need = q.qgemm_norm_rotate_backward_workspace(4, 8, 2, 128, 1)
    assert need > 0 and q.qgemm_norm_rotate_backward_workspace(4, 8, 2, 128, 0) == 0
    ok = dict(T=4, hq=8, hkv=2, D=128, q=P, qs=1024, k=P, ks=256, **NORM, pos=P, dqo=P, dko=P, dq=P, dqs=1024, dk=P, dks=256, dqw=P, dkw=P,
              ws=P, wsb=need)
    for kw in BAD_NORM + (dict(T=-1), dict(hq=0), dict(hkv=0), dict(D=0), dict(q=0), dict(k=0), dict(qs=1023), dict(ks=255),
                          dict(dqs=1023), dict(dks=255), dict(pos=0), dict(dqo=0), dict(dko=0), dict(dq=0), dict(dk=0), dict(dqo=P + 1),
                          dict(dk=P + 1), dict(dqw=P + 2), dict(dkw=P + 2), dict(ws=0), dict(wsb=need - 1), dict(ws=P + 4), dict(pos=P + 2)):
        assert status(q.qgemm_norm_rotate_backward, *{**ok, **kw}.values()) == BAD, kw
    for kw in (dict(D=100), dict(T=2**28), dict(T=2**31)):
        assert status(q.qgemm_norm_rotate_backward, *{**ok, **kw}.values()) == UNS, kw
    assert status(q.qgemm_norm_rotate_backward_workspace, 2**28, 8, 2, 128, 1) == UNS
    assert status(q.qgemm_norm_rotate_backward_workspace, -1, 8, 2, 128, 1) == BAD
    # no tokens and no weights' gradients: nothing to do, nothing touched
    assert status(q.qgemm_norm_rotate_backward, *{**ok, "T": 0, "q": 0, "dqw": 0, "dkw": 0, "ws": 0}.values()) == q.QGEMM_OK


def test_extend_refuses_bad_arguments():
    ok = dict(B=4, T=9, page=16, new=P, lens=P, gone=P, st=P, ring=P, R=10, tables=P, width=3, prefix=0, window=0, sinks=0, starts=P, lo=P, go=P,
              so=P, pos=P, slots=P, ref=P, ws=0, wsb=0)
    for kw in (dict(B=-1), dict(T=-1), dict(page=0), dict(new=0), dict(lens=0), dict(gone=0), dict(st=0), dict(ring=0), dict(R=0),
               dict(tables=0), dict(width=-1), dict(prefix=-1), dict(window=-1), dict(sinks=-1), dict(starts=0), dict(lo=0), dict(go=0),
               dict(so=0), dict(pos=0), dict(slots=0), dict(ref=0), dict(new=P + 2), dict(slots=P + 4), dict(tables=P + 1),
               dict(T=100000), dict(T=100000, ws=P + 4, wsb=1 << 20), dict(T=100000, ws=P, wsb=16)):
        assert status(q.qgemm_kv_extend, *{**ok, **kw}.values()) == BAD, kw
    for kw in (dict(page=24), dict(page=1 << 17), dict(B=65536), dict(T=2**31), dict(R=2**31), dict(width=2**31), dict(prefix=2**31),
               dict(window=2**31), dict(sinks=2**31)):
        assert status(q.qgemm_kv_extend, *{**ok, **kw}.values()) == UNS, kw
    assert q.qgemm_kv_extend_workspace(64, 64) == 0 and q.qgemm_kv_extend_workspace(64, 100000) > 0
    assert status(q.qgemm_kv_extend_workspace, -1, 4) == BAD and status(q.qgemm_kv_extend_workspace, 4, 2**31) == UNS


def test_windowed_attention_refuses_bad_arguments():
    ok = dict(T=4, hq=8, q=P, qs=1024, B=2, starts=P, lens=P, tables=P, width=3, pt=P, pl=20, mq=2, ml=40, w=30, s=4, scale=0.1, out=P, lse=0,
              ws=P, wsb=1 << 40)
    for kw in (dict(w=0), dict(w=-1), dict(s=-1), dict(T=-1), dict(hq=7), dict(q=0), dict(qs=1016), dict(B=0), dict(starts=0), dict(lens=0),
               dict(tables=0), dict(pt=0), dict(mq=0), dict(scale=0.0), dict(scale=float("nan")), dict(out=0), dict(lse=P + 2),
               dict(ml=4000, w=5000, ws=0), dict(ml=4000, w=5000, wsb=16), dict(ml=4000, w=5000, ws=P + 4)):
        assert status(q.qgemm_attention_window, cache(), *{**ok, **kw}.values()) == BAD, kw
    for kw in (dict(w=2**31), dict(s=2**31), dict(B=70000), dict(pl=2**31 - 1)):
        assert status(q.qgemm_attention_window, cache(), *{**ok, **kw}.values()) == UNS, kw
    assert status(q.qgemm_attention_window, None, *ok.values()) == BAD
    assert status(q.qgemm_attention_window, cache(), *{**ok, "T": 0, "q": 0}.values()) == q.QGEMM_OK
    args = (4, 8, 2, 1, 100000, 0)
    assert status(q.qgemm_attention_window_workspace, cache(), *args, 0, 0) == BAD
    assert status(q.qgemm_attention_window_workspace, cache(), *args, 10, -1) == BAD
    # a window bounds the keys of a query, and with them the parts
    small, large = (q.qgemm_attention_window_workspace(cache(), *args, w, 4) for w in (100, 100000))
    assert small < large == q.qgemm_attention_workspace(cache(), *args)


def test_wrong_tensors_are_refused_before_any_address():
    torch = pytest.importorskip("torch")
    from weight_quantized_mixed_amd.device import PagePool, norm_rotate, norm_rotate_backward
    i32, half = torch.int32, torch.float16
    for kw in (dict(ring=torch.zeros(5, dtype=i32)), dict(ring=torch.zeros(6)), dict(tables=torch.zeros((2, 4), dtype=i32)),
               dict(tables=torch.zeros((3, 4))), dict(window=0)):
        with pytest.raises(ValueError, match=next(iter(kw)) + ":"):
            PagePool(6, 16, 3, 4, device="cpu", **kw)
    pool = PagePool(6, 16, 3, 4, device="cpu")
    assert pool.state.tolist() == [0] * 7 + [6] and pool.lens.shape == (3,)
    for kw in (dict(new_tokens=torch.zeros(2, dtype=i32)), dict(new_tokens=torch.zeros(3)), dict(state_out=torch.zeros(7, dtype=i32))):
        with pytest.raises(ValueError, match=next(iter(kw)) + ":"):
            pool.extend(**{"new_tokens": torch.zeros(3, dtype=i32), "T": 4, **kw})
    x, t, pos = torch.zeros((4, 64), dtype=half), torch.zeros((9, 16)), torch.zeros(4, dtype=i32)
    for kw in (dict(cos=t.double()), dict(sin=t[:8]), dict(positions=pos[:3]), dict(q_weight=torch.zeros(32)), dict(k_weight=torch.zeros(31, dtype=half))):
        with pytest.raises(ValueError, match=next(iter(kw)) + ":"):
            norm_rotate(x, x, 32, **{"cos": t, "sin": t, "positions": pos, **kw})
        with pytest.raises(ValueError, match=next(iter(kw)) + ":"):
            norm_rotate_backward(x, x, x.view(4, 2, 32), x.view(4, 2, 32), **{"cos": t, "sin": t, "positions": pos, **kw})
    with pytest.raises(ValueError, match="device tensors only"):
        norm_rotate(x, x, 32, t, t, pos)


def test_sizes_past_32_bits_are_refused_by_name():
    torch = pytest.importorskip("torch")
    from weight_quantized_mixed_amd.device import PagePool
    pool = PagePool(4, 2**32 + 16, 2, 4, device="cpu")
    with pytest.raises(ValueError, match="page_size"):
        pool.extend(torch.zeros(2, dtype=torch.int32), 0)
