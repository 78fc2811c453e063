"""Host-side checks of the decoder-layer operators (no device calls): the float64
references against brute force and differences, and every refusal of the entry points."""
import ctypes

import numpy as np
import pytest

import oracle
from weight_quantized_mixed_amd import qgemm as q

P = 4096  # an aligned address that no refused call may touch


# ---- the references

@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_against_differences(act):
    rng = np.random.default_rng(3)
    M, N, K, h = 3, 4, 5, 1e-5
    x = {"A": rng.standard_normal((M, K)), "Wg": rng.standard_normal((K, N)), "Wu": rng.standard_normal((K, N)),
         "bg": rng.standard_normal(N), "bu": rng.standard_normal(N)}
    dC = rng.standard_normal((M, N))

    def loss(y):
        return float((oracle.gated_ref(y["A"], y["Wg"], y["Wu"], act, y["bg"], y["bu"])[0] * dC).sum())

    _, g, u = oracle.gated_ref(x["A"], x["Wg"], x["Wu"], act, x["bg"], x["bu"])
    grads = oracle.gated_grads_ref(x["A"], x["Wg"], x["Wu"], g, u, dC, act)
    formula = {"A": grads["dA"], "Wg": grads["dw_gate"].T, "Wu": grads["dw_up"].T, "bg": grads["dbias_gate"], "bu": grads["dbias_up"]}
    for name, arr in x.items():
        for i in np.ndindex(arr.shape):
            up, down = ({**x, name: arr.copy()} for _ in range(2))
            up[name][i] += h
            down[name][i] -= h
            # central differences: h^2 / 6 of the third derivative, and rounding of the loss / h
            assert abs((loss(up) - loss(down)) / (2 * h) - formula[name][i]) < 1e-7, (name, i)


def test_activation_known_values():
    v, d = oracle.activation(np.array([0.0, 1.0, -1.0]), "silu")
    assert np.allclose(v, [0, 0.7310585786300049, -0.2689414213699951], atol=1e-15) and d[0] == 0.5
    v, d = oracle.activation(np.array([0.0, 1.0]), "gelu_tanh")
    assert np.allclose(v, [0, 0.8411919906082768], atol=1e-12) and d[0] == 0.5


def test_attention_reference_by_hand():
    q1, k, v = np.array([[1.0, 0.0]]), np.array([[0.0, 5.0], [np.log(3.0), 1.0], [9.0, 9.0]]), np.array([[1.0], [5.0], [np.pi]])
    out, lse, _ = oracle.attention_ref(q1, k, v, np.array([[True, True, False]]), 1.0)
    assert np.allclose(out, 0.25 * 1 + 0.75 * 5) and np.allclose(lse, np.log(4))
    out, lse, _ = oracle.attention_ref(q1, k, v, np.zeros((1, 3), bool), 1.0)
    assert out[0, 0] == 0 and np.isneginf(lse[0])


def test_rotation_reference_keeps_lengths():
    rng = np.random.default_rng(0)
    x, a = rng.standard_normal((4, 2, 12)), rng.uniform(-3, 3, (4, 4))
    for il in (False, True):
        y, _ = oracle.rotate_ref(x, np.cos(a), np.sin(a), il)
        assert np.allclose((y**2).sum(-1), (x**2).sum(-1)) and np.array_equal(y[..., 8:], x[..., 8:])
        back, _ = oracle.rotate_ref(y, np.cos(a), -np.sin(a), il)
        assert np.allclose(back, x)


# ---- refusals

def status(fn, *args):
    try:
        fn(*args)
    except q.QGemmError as e:
        return e.status
    return q.QGEMM_OK


def gated(**kw):
    a = dict(M=8, N=100, K=256, a="f16", w="i4", out="f16", acc="f32", g=128, z=0, act="silu")
    a.update(kw)
    return q.qgemm_create_gated(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(), q.QGEMM_OK), (dict(w="f16", g=0), q.QGEMM_OK), (dict(w="u4", z=1), q.QGEMM_OK),
    (dict(a="i8", w="i8", acc="i32", g=0), q.QGEMM_OK), (dict(a="i8", w="i2", acc="i32", g=0), q.QGEMM_OK),
    (dict(M=0), q.QGEMM_ERR_INVALID_ARG), (dict(N=0), q.QGEMM_ERR_INVALID_ARG), (dict(K=-1), q.QGEMM_ERR_INVALID_ARG),
    (dict(act=0), q.QGEMM_ERR_INVALID_ARG), (dict(act=3), q.QGEMM_ERR_INVALID_ARG),
    (dict(a="i8", w="i8", out="i32", acc="i32", g=0), q.QGEMM_ERR_UNSUPPORTED),
    (dict(N=2**31 - 1), q.QGEMM_ERR_UNSUPPORTED), (dict(N=2**30), q.QGEMM_ERR_UNSUPPORTED),
    (dict(K=200), q.QGEMM_ERR_UNSUPPORTED), (dict(z=1), q.QGEMM_ERR_UNSUPPORTED), (dict(g=48), q.QGEMM_ERR_UNSUPPORTED),
    (dict(w="i8", g=0), q.QGEMM_ERR_UNSUPPORTED), (dict(acc="f16"), q.QGEMM_ERR_UNSUPPORTED),
    (dict(M=2**24, K=256), q.QGEMM_ERR_UNSUPPORTED),
])
def test_create_gated(kw, want):
    try:
        plan, pb, _ = gated(**kw)
    except q.QGemmError as e:
        assert e.status == want
    else:
        assert want == q.QGEMM_OK and pb > 0
        q.qgemm_destroy(plan)


def test_gated_blob_holds_both_projections():
    plan, pb, wb = gated()
    inner = 256  # 2 * roundup(100, 16) = 224 columns, padded to 256
    assert pb == inner * 256 // 2 + inner * 2 * 2 and wb == 0
    q.qgemm_destroy(plan)


def test_gated_plans_and_plain_plans_do_not_mix():
    plan, pb, wb = gated()
    plain, _, _ = q.qgemm_create(8, 100, 256, "f16", "i4", "f16", "f32", 128)
    bad = q.QGEMM_ERR_INVALID_ARG
    assert status(q.qgemm_pack_weights, plan, P, P, 0, P) == bad
    assert status(q.qgemm_run, plan, P, P, P, 0, 0) == bad
    assert status(q.qgemm_run_ex, plan, 8, P, P, 0, P, 0, 0) == bad
    assert status(q.qgemm_run_noalloc, plan, 8, P, P, 0, P) == bad
    assert status(q.qgemm_run_scaled, plan, 8, P, P, P, P, 0, P, 0, 0) == bad
    assert status(q.qgemm_pack_gated, plain, P, P, 0, P, P, 0, P) == bad
    assert status(q.qgemm_run_gated, plain, 8, P, P, 0, 0, 0, 0, 0, 0, P, 0, 0) == bad
    assert status(q.qgemm_gated_backward, plain, 8, P, P, P, P, P, 0, 0, 0, 0, P, 1 << 40) == bad
    assert status(q.qgemm_gated_backward_workspace, plain, 8, 0) == bad
    q.qgemm_destroy(plan)
    q.qgemm_destroy(plain)


def test_gated_calls_refuse_bad_arguments():
    bad = q.QGEMM_ERR_INVALID_ARG
    plan, _, _ = gated(w="u4", z=1)
    for i in range(7):  # each array in turn missing
        args = [P] * 7
        args[i] = 0
        assert status(q.qgemm_pack_gated, plan, *args) == bad, i
    assert status(q.qgemm_pack_gated, plan, P + 2, P, P, P, P, P, P) == bad
    ok = dict(M=8, A=P, packed=P, rs=0, cg=0, cu=0, bg=0, bu=0, pre=0, C=P, ws=0, wsb=0)
    for kw in (dict(M=0), dict(M=9), dict(A=0), dict(packed=0), dict(C=0), dict(A=P + 2), dict(packed=P + 8), dict(rs=P),
               dict(cg=P), dict(cu=P), dict(bg=P + 1), dict(bu=P + 1), dict(pre=P + 1)):
        assert status(q.qgemm_run_gated, plan, *{**ok, **kw}.values()) == bad, kw
    assert status(q.qgemm_run_gated, None, *ok.values()) == bad
    q.qgemm_destroy(plan)
    plan, _, _ = gated(a="i8", w="i8", acc="i32", g=0)
    for kw in (dict(), dict(rs=P, cg=P), dict(rs=P, cu=P), dict(cg=P, cu=P), dict(rs=P + 2, cg=P, cu=P),
               dict(rs=P, cg=P, cu=P + 2)):
        assert status(q.qgemm_run_gated, plan, *{**ok, **kw}.values()) == bad, kw
    assert status(q.qgemm_gated_backward_workspace, plan, 8, 0) == q.QGEMM_ERR_UNSUPPORTED  # int8 activations
    q.qgemm_destroy(plan)


def test_backward_refuses_bad_arguments():
    bad = q.QGEMM_ERR_INVALID_ARG
    plan, _, _ = gated(w="f16", g=0)
    need = q.qgemm_gated_backward_workspace(plan, 8, 1)
    assert need > q.qgemm_gated_backward_workspace(plan, 8, 0) > 0
    ok = dict(M=8, A=P, packed=P, pre=P, dC=P, dA=P, dwg=P, dwu=P, dbg=P, dbu=P, ws=P, wsb=need)
    for kw in (dict(M=0), dict(M=9), dict(A=0), dict(packed=0), dict(pre=0), dict(dC=0), dict(dwg=0), dict(dwu=0), dict(ws=0),
               dict(wsb=need - 1), dict(A=P + 2), dict(packed=P + 2), dict(ws=P + 4), dict(pre=P + 1), dict(dA=P + 1),
               dict(dbu=P + 1), dict(dA=0, dwg=0, dwu=0, dbg=0, dbu=0)):
        assert status(q.qgemm_gated_backward, plan, *{**ok, **kw}.values()) == bad, kw
    assert status(q.qgemm_gated_backward_workspace, plan, 0, 0) == bad
    assert status(q.qgemm_gated_backward_workspace, plan, 9, 0) == bad
    q.qgemm_destroy(plan)
    plan, _, _ = gated()  # frozen int4 weights
    assert q.qgemm_gated_backward_workspace(plan, 8, 0) > 0
    assert status(q.qgemm_gated_backward_workspace, plan, 8, 1) == q.QGEMM_ERR_UNSUPPORTED
    assert status(q.qgemm_gated_backward, plan, *ok.values()) == q.QGEMM_ERR_UNSUPPORTED
    q.qgemm_destroy(plan)


def cache(**kw):
    a = dict(k=P, v=P, n_pages=10, page_size=16, kv_heads=2, head_dim=128)
    a.update(kw)
    return q.KVCacheDesc(*a.values())


BAD, UNS = q.QGEMM_ERR_INVALID_ARG, q.QGEMM_ERR_UNSUPPORTED
CACHES = [(dict(k=0), BAD), (dict(v=0), BAD), (dict(k=P + 8), BAD), (dict(n_pages=0), BAD), (dict(page_size=0), BAD),
          (dict(kv_heads=0), BAD), (dict(head_dim=0), BAD), (dict(kv_heads=3), BAD), (dict(page_size=24), UNS),
          (dict(page_size=1 << 17), UNS), (dict(head_dim=100), UNS), (dict(head_dim=264), UNS),
          (dict(n_pages=2**31), UNS), (dict(page_size=65536, kv_heads=1024, head_dim=256), BAD),
          (dict(page_size=65536, kv_heads=256, head_dim=256), BAD)]


@pytest.mark.parametrize("kw,want", CACHES)
def test_cache_descriptors(kw, want):
    args = [4, 8, P, 2000, P, 2000, P, 2000, P, P, 9, 8, 0, P, P, P]
    assert status(q.qgemm_kv_append, cache(**kw), *args) == want
    assert status(q.qgemm_attention_workspace, cache(**kw), 4, 8, 2, 1, 100, 0) == want
    assert status(q.qgemm_attention, cache(**kw), 4, 8, P, 2048, 2, P, P, P, 3, 0, 0, 1, 30, 1.0, P, 0, P, 1 << 40) == want


def test_a_page_is_below_four_gigabytes():
    c = cache(page_size=65536, kv_heads=128, head_dim=256)
    assert status(q.qgemm_attention_workspace, c, 4, 128, 2, 1, 100, 0) == UNS


def test_append_refuses_bad_arguments():
    ok = dict(T=4, hq=8, q=P, qs=1024, k=P, ks=256, v=P, vs=256, cos=P, sin=P, n=9, rot=128, il=0, pos=P, slots=P, out=P)
    for kw in (dict(T=-1), dict(hq=0), dict(hq=5), dict(q=0), dict(k=0), dict(v=0), dict(qs=1023), dict(ks=255), dict(vs=255),
               dict(cos=0), dict(sin=0), dict(n=0), dict(rot=-2), dict(rot=7), dict(rot=130), dict(il=2), dict(pos=0),
               dict(slots=0), dict(out=0), dict(q=P + 1), dict(cos=P + 2), dict(pos=P + 2), dict(slots=P + 4), dict(out=P + 1)):
        assert status(q.qgemm_kv_append, cache(), *{**ok, **kw}.values()) == BAD, kw
    assert status(q.qgemm_kv_append, None, *ok.values()) == BAD
    assert status(q.qgemm_kv_append, cache(), *{**ok, "T": 0, "q": 0}.values()) == q.QGEMM_OK  # nothing to do, nothing touched


def test_attention_refuses_bad_arguments():
    ok = dict(T=4, hq=8, q=P, qs=1024, B=2, starts=P, lens=P, tables=P, width=3, pt=P, pl=20, mq=2, ml=40, scale=0.1, out=P,
              lse=0, ws=P, wsb=1 << 40)
    for kw in (dict(T=-1), dict(hq=7), dict(q=0), dict(qs=1016), dict(qs=1028), dict(q=P + 8), dict(B=0), dict(starts=0),
               dict(lens=0), dict(tables=0), dict(width=-1), dict(pt=0), dict(pl=-1), dict(mq=0), dict(ml=-1),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=0),
               dict(out=P + 2), dict(lse=P + 2), dict(starts=P + 2), dict(ws=0), dict(wsb=16), dict(ws=P + 4)):
        assert status(q.qgemm_attention, cache(), *{**ok, **kw}.values()) == BAD, kw
    assert status(q.qgemm_attention, None, *ok.values()) == BAD
    assert status(q.qgemm_attention, cache(), *{**ok, "B": 70000}.values()) == UNS
    assert status(q.qgemm_attention, cache(), *{**ok, "pl": 2**31 - 1}.values()) == UNS
    assert status(q.qgemm_attention, cache(), *{**ok, "T": 0, "q": 0}.values()) == q.QGEMM_OK
    assert status(q.qgemm_attention_workspace, cache(), 4, 8, 0, 1, 1, 0) == BAD
    assert q.load().qgemm_attention_workspace(ctypes.byref(cache()), 4, 8, 2, 1, 10, 0, None) == BAD


def test_attention_of_an_empty_batch():
    ok = dict(T=0, hq=8, q=0, qs=1024, B=0, starts=0, lens=0, tables=0, width=0, pt=0, pl=0, mq=0, ml=0, scale=0.1, out=0,
              lse=0, ws=0, wsb=0)
    assert status(q.qgemm_attention, cache(), *ok.values()) == q.QGEMM_OK
    assert q.qgemm_attention_workspace(cache(), 0, 8, 0, 0, 0, 0) == 0
    for kw in (dict(B=-1), dict(mq=-1), dict(T=1), dict(T=1, B=1), dict(T=1, mq=1)):
        assert status(q.qgemm_attention, cache(), *{**ok, **kw}.values()) == BAD, kw


def test_attention_scale_stays_finite_in_powers_of_two():
    args = [4, 8, P, 1024, 2, P, P, P, 3, 0, 0, 1, 40]
    for scale in (2.4e38, 3e38, 3.4e38):
        assert status(q.qgemm_attention, cache(), *args, scale, P, 0, P, 1 << 40) == BAD, scale


def test_attention_items_fit_a_launch():
    """65535 sequences of one token and 300 heads are more workgroups of 256 than one launch holds (2^32 threads)."""
    wide = cache(kv_heads=300, head_dim=8)
    assert status(q.qgemm_attention_workspace, wide, 65535, 300, 65535, 1, 40, 0) == UNS
    assert status(q.qgemm_attention, wide, 65535, 300, P, 2400, 65535, P, P, P, 3, 0, 0, 1, 40, 1.0, P, 0, P, 1 << 40) == UNS
    assert status(q.qgemm_attention_workspace, wide, 50000, 300, 50000, 1, 40, 0) == q.QGEMM_OK


def test_workspace_holds_the_parts():
    assert q.qgemm_attention_workspace(cache(), 0, 8, 1, 1, 10, 0) == 0
    assert q.qgemm_attention_workspace(cache(), 1, 8, 1, 1, 60, 0) == 0          # one part: written directly
    n = q.qgemm_attention_workspace(cache(), 1, 8, 1, 1, 2000, 0)
    parts = n // (8 * 128 * 4 + 8 * 8)
    assert parts > 1 and n == parts * (8 * 128 * 4 + 8 * 8)                       # (o, m, l) of each


def test_gated_tensors_of_other_sizes_are_refused_before_any_address():
    """A blob of a smaller plan, or weights and tables of another shape, would be read past their end."""
    torch = pytest.importorskip("torch")
    from weight_quantized_mixed_amd.device import QGated
    plan = QGated(4, 32, 256, "u4", 64, True, device="cpu")
    w, t = torch.zeros((32, 32), dtype=torch.int32), torch.ones((32, 4), dtype=torch.float16)
    ok = dict(w_gate=w, w_up=w, s_gate=t, s_up=t, z_gate=t, z_up=t)
    for kw in (dict(w_gate=w[:31]), dict(w_up=w[:, :31]), dict(w_up=torch.zeros((33, 32), dtype=torch.int32)), dict(s_gate=t[:, :2]),
               dict(s_up=t.float()), dict(z_gate=t[:31]), dict(z_up=t.t())):
        with pytest.raises(ValueError, match=next(iter(kw)) + ":"):
            plan.pack(**{**ok, **kw})
    small = torch.zeros(plan.packed_bytes - 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="out: "):
        plan.pack(**ok, out=small)
    A, row = torch.zeros((4, 256), dtype=torch.float16), torch.zeros((4, 32), dtype=torch.float16)
    with pytest.raises(ValueError, match="packed: "):
        plan.run(A, small)
    with pytest.raises(ValueError, match="packed: "):
        plan.backward(A, small, torch.zeros((4, 64), dtype=torch.float16), row)
