"""What is measured of a quantised decoder layer's operators, beside the matrix product itself.

Three operators, in the order in which a layer runs them after its query / key / value projection:

* append: rotary positions on the queries and keys of new tokens, and their keys and values written into a paged cache;
* attend: attention of a ragged batch over that cache, where the batch may share a prefix whose keys and values exist once;
* gated: the gated feed-forward block act(A Wg + bg) * (A Wu + bu) with quantised or fp16 weights, and its gradients.

`run` takes the plain form (float32 torch operations, one rounding) where `own` is false and the library's kernels where it is true.
"""
import math

import torch

own = False

GELU_C = math.sqrt(2.0 / math.pi)
BITS = {"i4": 4, "u4": 4, "i2": 2, "i8": 8, "f16": 16}
INT8_A = ("i8", "i2")


# ---- cases ---------------------------------------------------------------------------------------------------------

def gated_case(name, M, N, K, w, g=0, zeros=False, act="silu", bias=False, train=False):
    c = {"op": "gated", "M": M, "N": N, "K": K, "w": w, "g": g, "zeros": zeros, "act": act, "bias": bias, "train": train}
    return c if name is None else {"name": name, **c}


def append_case(name, T, hq, hkv, D, rot, page, interleaved=False, padded=False):
    c = {"op": "append", "T": T, "hq": hq, "hkv": hkv, "D": D, "rot": rot, "page": page, "interleaved": interleaved, "padded": padded}
    return c if name is None else {"name": name, **c}


def attend_case(name, B, hq, hkv, D, page, q_min, q_max, own_min, own_max, prefix):
    c = {"op": "attend", "B": B, "hq": hq, "hkv": hkv, "D": D, "page": page, "q_min": q_min, "q_max": q_max,
         "own_min": own_min, "own_max": own_max, "prefix": prefix}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one token of a 7B layer's feed-forward, int4 weights with a scale per 128: the latency of decoding alone
        gated_case("gated_decode_i4", 1, 11008, 4096, "i4", 128),
        # a decode batch with zero points
        gated_case("gated_batch32_u4z", 32, 11008, 4096, "u4", 128, zeros=True),
        # int8 activations and weights (per-token and per-channel scales), a mid-sized batch
        gated_case("gated_batch128_i8", 128, 11008, 4096, "i8"),
        # prefill of one prompt
        gated_case("gated_prefill_i4", 2048, 11008, 4096, "i4", 128),
        # a small odd layer trained in fp16: rows, columns and depth off every tile, gelu, biases
        gated_case("gated_train_f16_odd", 333, 1250, 776, "f16", act="gelu_tanh", bias=True, train=True),
        # adapter training through frozen int4 weights: the input's gradient only
        gated_case("gated_train_i4", 1024, 11008, 4096, "i4", 128, train=True),
        # a full fp16 training step of the block: all gradients, weights laid out anew as they change each step
        gated_case("gated_train_f16", 2048, 11008, 4096, "f16", train=True),
        # one new token for each of 48 sequences, some slots of the batch unused
        append_case("append_decode", 48, 32, 8, 128, 128, 16, padded=True),
        # a prompt's tokens, all heads, partial rotation in the interleaved order
        append_case("append_prefill", 8190, 32, 32, 128, 64, 64, interleaved=True),
        # one sequence, one token, nothing shared: latency
        attend_case("attend_one", 1, 32, 32, 128, 16, 1, 1, 777, 777, 0),
        # a decode batch behind one long system prompt, short tails of their own (some slots unused)
        attend_case("attend_shared", 64, 32, 8, 128, 16, 1, 1, 0, 512, 8000),
        # prompts of mixed length, each beginning with the shared prefix, computed at once
        attend_case("attend_prefill", 4, 32, 8, 128, 64, 700, 1024, 700, 1500, 1000),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "append", "attend", "attend"])
    if op == "gated":
        w = rng.choice(["i4", "u4", "f16", "i8", "i2"])
        train = w in ("i4", "u4", "f16") and rng.random() < 0.4
        M = log_int(rng, 1, 2048)
        N = log_int(rng, 40, 11008)
        g = rng.choice([0, -1, 32, 64, 128]) if w in ("i4", "u4") else 0
        unit = g if g > 0 else {"i4": 8, "u4": 8, "i2": 16, "i8": 1, "f16": 1}[w]
        K = max(1, log_int(rng, 128, 4096) // unit) * unit
        return gated_case(None, M, N, K, w, g, zeros=w == "u4" and g != 0 and rng.random() < 0.6,
                          act=rng.choice(["silu", "gelu_tanh"]), bias=rng.random() < 0.4, train=train)
    D = rng.choice([64, 80, 96, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    hq, hkv = (hq, hkv) if hq <= 64 else (32, 8)
    page = rng.choice([1, 16, 16, 32, 64, 256])
    if op == "append":
        return append_case(None, log_int(rng, 1, 4096), hq, hkv, D, rng.choice([D, D, D // 2]), page,
                           interleaved=rng.random() < 0.5, padded=rng.random() < 0.5)
    while True:
        B = log_int(rng, 1, 64)
        q_max = rng.choice([1, 1, 1, log_int(rng, 2, 16), log_int(rng, 16, max(17, 2048 // B))])
        own_max = q_max + log_int(rng, 1, max(2, 16384 // B))
        c = attend_case(None, B, hq, hkv, D, page, rng.choice([1, q_max]), q_max, rng.choice([0, q_max, own_max]), own_max,
                        rng.choice([0, 0, log_int(rng, 1, 8192)]))
        if work(c)["flops"] <= 1e11:
            return c


# ---- inputs --------------------------------------------------------------------------------------------------------

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def spread(lo, hi, i, n):
    """The i-th of n sizes between lo and hi, in a fixed mixed order that begins with hi."""
    return hi - (hi - lo) * ((i * 37) % n) // max(1, n - 1) if n > 1 else hi


def lengths(c):
    """(queries, own tokens with the queries' among them, or none in an unused slot) of each sequence of an attend case."""
    qs = [spread(c["q_min"], c["q_max"], i, c["B"]) for i in range(c["B"])]
    own_tokens = [spread(c["own_min"], c["own_max"], i + 3, c["B"]) for i in range(c["B"])]
    return qs, [max(n, L) if L else 0 for n, L in zip(qs, own_tokens)]


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).half()


def uniform(gen, lo, hi, *shape):
    return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo


def weights(gen, c):
    """Canonical storage of one projection: words or values [N, K], scales and zero points [N, G]."""
    N, K, w, g = c["N"], c["K"], c["w"], c["g"]
    if w == "f16":
        return normal(gen, N, K, std=0.02), None, None
    if w == "i8":
        return torch.randint(-128, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8), None, None
    words = torch.randint(-2**31, 2**31, (N, K * BITS[w] // 32), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    G = 0 if g == 0 else 1 if g < 0 else K // g
    s = uniform(gen, 0.005, 0.02, N, G).half() if G else None
    z = uniform(gen, 6.0, 9.0, N, G).half() if c["zeros"] else None
    return words, s, z


def prepare(case, seed):
    return {"gated": prepare_gated, "append": prepare_append, "attend": prepare_attend}[case["op"]](case, generator(seed))


def prepare_gated(c, gen):
    M, N, K = c["M"], c["N"], c["K"]
    st = {"case": c}
    for p in ("gate", "up"):
        st["w_" + p], st["s_" + p], st["z_" + p] = weights(gen, c)
        st["b_" + p] = normal(gen, N, std=0.5) if c["bias"] else None
    if c["w"] in INT8_A:
        st["A"] = torch.randint(-128, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
        st["rs"] = uniform(gen, 0.001, 0.01, M)
        for p in ("gate", "up"):
            st["cs_" + p] = uniform(gen, 0.001, 0.01, N)
    else:
        # unscaled int4 sums are kept to the size of scaled ones by the activations
        st["A"] = normal(gen, M, K, std=0.0125 if c["w"] in ("i4", "u4") and c["g"] == 0 else 1.0)
    if c["train"]:
        st["dC"] = normal(gen, M, N, std=0.1)
    if own:  # the plan, and frozen weights in the library's layout
        from weight_quantized_mixed_amd.device import QGated
        st["plan"] = QGated(M, N, K, c["w"], c["g"], c["zeros"], act=c["act"])
        if not (c["train"] and c["w"] == "f16"):
            st["packed"] = st["plan"].pack(st["w_gate"], st["w_up"], st["s_gate"], st["s_up"], st["z_gate"], st["z_up"])
    return st


def prepare_append(c, gen):
    T, hq, hkv, D, rot, page = c["T"], c["hq"], c["hkv"], c["D"], c["rot"], c["page"]
    st = {"case": c, "qkv": normal(gen, T, (hq + 2 * hkv) * D)}
    n_pos = 4096 + T
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    ang = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * inv
    st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
    st["positions"] = torch.randint(0, n_pos, (T,), generator=gen, device="cuda", dtype=torch.int32)
    n_pages = -(-T * 5 // 4 // page) + 1
    slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:T]
    if c["padded"]:
        slots[5::11] = -1  # unused slots of the batch: rotated, not stored
    st["slots"] = slots
    st["k"], st["v"] = normal(gen, n_pages, hkv, page, D), normal(gen, n_pages, hkv, page, D)
    if own:
        from weight_quantized_mixed_amd.device import PagedKV
        st["cache"] = PagedKV(n_pages, page, hkv, D, k=st["k"], v=st["v"])
    return st


def prepare_attend(c, gen):
    B, hq, hkv, D, page, prefix = c["B"], c["hq"], c["hkv"], c["D"], c["page"], c["prefix"]
    qs, lens = lengths(c)
    width = max(1, -(-c["own_max"] // page))
    n_prefix = -(-prefix // page)
    n_pages = B * width + n_prefix
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    starts = [0]
    for n in qs:
        starts.append(starts[-1] + n)
    dev = {"device": "cuda", "dtype": torch.int32}
    st = {"case": c, "q": normal(gen, starts[-1], hq, D), "k": normal(gen, n_pages, hkv, page, D), "v": normal(gen, n_pages, hkv, page, D),
          "starts": torch.tensor(starts, **dev), "lens": torch.tensor(lens, **dev), "tables": order[n_prefix:].view(B, width).contiguous(),
          "prefix_table": order[:n_prefix].clone(), "scale": D ** -0.5}
    if own:
        from weight_quantized_mixed_amd.device import PagedKV
        st["cache"] = PagedKV(n_pages, page, hkv, D, k=st["k"], v=st["v"])
    return st


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    kind = c["op"] + ("_own" if own else "_plain")
    return {"gated_own": gated_own, "gated_plain": gated_plain, "append_own": append_own, "append_plain": append_plain,
            "attend_own": attend_own, "attend_plain": attend_plain}[kind](state, c)


def gated_own(st, c):
    q = st["plan"]
    if c["w"] in INT8_A:
        return q.run_scaled(st["A"], st["packed"], st["rs"], st["cs_gate"], st["cs_up"], bias_gate=st["b_gate"], bias_up=st["b_up"])
    if not c["train"]:
        return q.run(st["A"], st["packed"], bias_gate=st["b_gate"], bias_up=st["b_up"])
    learns = c["w"] == "f16"  # quantised weights are frozen
    packed = q.pack(st["w_gate"], st["w_up"]) if learns else st["packed"]
    preact = q.new_preact()
    C = q.run(st["A"], packed, bias_gate=st["b_gate"], bias_up=st["b_up"], preact=preact)
    grads = q.backward(st["A"], packed, preact, st["dC"], weight_grads=learns, bias_grads=learns and c["bias"])
    return {"C": C, **{k: v for k, v in grads.items() if v is not None}}


def append_own(st, c):
    hq, hkv, D = c["hq"], c["hkv"], c["D"]
    q, k, v = st["qkv"].split([hq * D, hkv * D, hkv * D], dim=1)
    out = st["cache"].append(q, k, v, st["cos"], st["sin"], st["positions"], st["slots"], interleaved=c["interleaved"])
    return {"q": out, "k": st["k"], "v": st["v"]}


def attend_own(st, c):
    return st["cache"].attend(st["q"], st["starts"], st["lens"], st["tables"], max_q=c["q_max"], max_len=c["own_max"],
                              prefix_table=st["prefix_table"] if c["prefix"] else None, prefix_len=c["prefix"], scale=st["scale"])


def dequantise(w, s, z, c, dtype):
    """[N, K] weight values of canonical storage."""
    kind, K = c["w"], c["K"]
    if kind in ("f16", "i8"):
        return w.to(dtype)
    bits = BITS[kind]
    q = (w[:, :, None] >> (bits * torch.arange(32 // bits, device=w.device, dtype=torch.int32))) & ((1 << bits) - 1)
    q = q.reshape(w.shape[0], K).to(dtype)
    if kind != "u4":  # two's complement
        q = torch.where(q >= 2 ** (bits - 1), q - 2**bits, q)
    if s is None:
        return q
    q = q.view(w.shape[0], s.shape[1], -1)
    if z is not None:
        q = q - z.to(dtype)[:, :, None]
    return (q * s.to(dtype)[:, :, None]).reshape(w.shape[0], K)


def activation(x, act):
    """act(x) and its derivative: both kinds are x sigmoid(t(x))."""
    if act == "silu":
        t, dt = x, 1.0
    else:  # 0.5 x (1 + tanh(c (x + 0.044715 x^3)))
        t, dt = 2 * GELU_C * (x + 0.044715 * x * x * x), 2 * GELU_C * (1 + 3 * 0.044715 * x * x)
    s = 1 / (1 + torch.exp(-t))
    return x * s, s + x * s * (1 - s) * dt


def gated_plain(st, c):
    Wg = dequantise(st["w_gate"], st["s_gate"], st["z_gate"], c, torch.float32)
    Wu = dequantise(st["w_up"], st["s_up"], st["z_up"], c, torch.float32)
    A = st["A"].float()
    G, U = A @ Wg.t(), A @ Wu.t()
    if c["w"] in INT8_A:
        G, U = G * st["rs"][:, None] * st["cs_gate"], U * st["rs"][:, None] * st["cs_up"]
    if c["bias"]:
        G, U = G + st["b_gate"].float(), U + st["b_up"].float()
    h, dh = activation(G, c["act"])
    C = (h * U).half()
    if not c["train"]:
        return C
    dC = st["dC"].float()
    dG, dU = dC * U * dh, dC * h
    out = {"C": C, "dA": (dG @ Wg + dU @ Wu).half()}
    if c["w"] == "f16":
        out["dw_gate"], out["dw_up"] = (dG.t() @ A).half(), (dU.t() @ A).half()
        if c["bias"]:
            out["dbias_gate"], out["dbias_up"] = dG.sum(0).half(), dU.sum(0).half()
    return out


def rotate(x, cos, sin, interleaved):
    """x [T, H, D] rotated in its first 2 * cos.shape[1] places by the angles of each token."""
    R = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * R:2], x[..., 1:2 * R:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R], x[..., R:2 * R]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., 2 * R:]], -1)


def append_plain(st, c):
    T, hq, hkv, D, page = c["T"], c["hq"], c["hkv"], c["D"], c["page"]
    q, k, v = st["qkv"].float().split([hq * D, hkv * D, hkv * D], dim=1)
    at = st["positions"].long()
    cos, sin = st["cos"][at], st["sin"][at]
    q = rotate(q.view(T, hq, D), cos, sin, c["interleaved"]).half()
    k = rotate(k.view(T, hkv, D), cos, sin, c["interleaved"]).half()
    v = v.view(T, hkv, D).half()
    if c["padded"]:
        keep = st["slots"] >= 0
        slots, k, v = st["slots"][keep], k[keep], v[keep]
    else:
        slots = st["slots"]
    st["k"][slots // page, :, slots % page] = k
    st["v"][slots // page, :, slots % page] = v
    return {"q": q, "k": st["k"], "v": st["v"]}


def gather(cache, table, n):
    """Tokens 0 .. n - 1 of a page table (or of each row of one), [..., n, heads, D] in float32."""
    page = cache.shape[2]
    t = torch.arange(n, device=cache.device)
    return cache[table.long()[..., t // page], :, t % page].float()


def attend_plain(st, c):
    B, hq, hkv, D, prefix, qm, om = c["B"], c["hq"], c["hkv"], c["D"], c["prefix"], c["q_max"], c["own_max"]
    G = hq // hkv
    starts, lens = st["starts"].long(), st["lens"].long()
    nq = starts[1:] - starts[:-1]
    i = torch.arange(qm, device="cuda")
    live = i < nq[:, None]                                                      # [B, qm]: rows of the padded batch that exist
    rows = (starts[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[rows] * st["scale"]                                    # [B, qm, hq, D]
    q = q.view(B, qm, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, qm * G, D)
    k, v = gather(st["k"], st["tables"], om), gather(st["v"], st["tables"], om)  # [B, om, hkv, D]
    s = q @ k.permute(0, 2, 3, 1).contiguous()                                 # [B, hkv, qm * G, om]
    last = lens[:, None] - nq[:, None] + i                                     # the last own token that each query sees
    seen = (torch.arange(om, device="cuda") <= last[..., None]) & live[..., None]
    seen = seen[:, None, :, None].expand(B, hkv, qm, G, om).reshape(B, hkv, qm * G, om)
    s = torch.where(seen, s, -torch.inf)
    if prefix:
        pk, pv = gather(st["k"], st["prefix_table"], prefix), gather(st["v"], st["prefix_table"], prefix)
        qp = q.permute(1, 0, 2, 3).reshape(hkv, B * qm * G, D)
        sp = (qp @ pk.permute(1, 2, 0).contiguous()).view(hkv, B, qm * G, prefix).permute(1, 0, 2, 3)
        m = torch.maximum(s.amax(-1), sp.amax(-1))
    else:
        m = s.amax(-1).clamp(min=-3e38)                                        # rows that see nothing
    p = torch.exp(s - m[..., None])
    total, o = p.sum(-1), p @ v.permute(0, 2, 1, 3).contiguous()
    if prefix:
        pp = torch.exp(sp - m[..., None])
        total = total + pp.sum(-1)
        o = o + (pp.permute(1, 0, 2, 3).reshape(hkv, -1, prefix) @ pv.permute(1, 0, 2).contiguous()).view(hkv, B, qm * G, D).permute(1, 0, 2, 3)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    o = o.view(B, hkv, qm, G, D).permute(0, 2, 1, 3, 4).reshape(B, qm, hq, D)
    return o[live].half()


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "append":
        T, width = c["T"], (c["hq"] + 2 * c["hkv"]) * c["D"]
        return {"bytes": 2 * T * width * 2 + T * (c["rot"] * 4 + 12), "flops": 3 * T * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "attend":
        qs, lens = lengths(c)
        keys = sum(n * c["prefix"] + sum(max(0, L - n + i + 1) for i in range(n)) for n, L in zip(qs, lens))
        held = 2 * 2 * c["hkv"] * c["D"] * (c["prefix"] + sum(lens))
        return {"bytes": held + 2 * 2 * sum(qs) * c["hq"] * c["D"], "flops": 4 * c["D"] * c["hq"] * keys}
    M, N, K = c["M"], c["N"], c["K"]
    G = 0 if c["g"] == 0 else 1 if c["g"] < 0 else K // c["g"]
    a = 1 if c["w"] in INT8_A else 2
    w = 2 * (N * K * BITS[c["w"]] // 8 + N * G * 2 * (2 if c["zeros"] else 1))
    extra = (4 * N if c["bias"] else 0) + (4 * (M + 2 * N) if a == 1 else 0)
    bytes_, flops = w + M * K * a + M * N * 2 + extra, 4 * M * N * K
    if c["train"]:
        bytes_, flops = bytes_ + M * N * 2 + M * K * 2, flops + 4 * M * N * K
        if c["w"] == "f16":
            bytes_, flops = bytes_ + w + (4 * N if c["bias"] else 0), flops + 4 * M * N * K
    return {"bytes": bytes_, "flops": flops}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"gated": gated_exact, "append": append_exact, "attend": attend_exact}[case["op"]](st, case)


def gated_exact(st, c):
    def weight(p):
        q, K = st["w_" + p], c["K"]
        if c["w"] in ("f16", "i8"):
            return q.double()
        bits = BITS[c["w"]]
        k = torch.arange(K, device="cuda")
        f = (q.long()[:, k * bits // 32] >> (k * bits % 32)) & (2**bits - 1)
        if c["w"] in ("i4", "i2"):
            f = (f + 2 ** (bits - 1)) % 2**bits - 2 ** (bits - 1)
        f = f.double()
        if c["g"]:
            grp = k // c["g"] if c["g"] > 0 else k * 0
            f = f - st["z_" + p].double()[:, grp] if c["zeros"] else f
            f = f * st["s_" + p].double()[:, grp]
        return f

    A, Wg, Wu = st["A"].double(), weight("gate"), weight("up")
    G, U = torch.mm(A, Wg.T.contiguous()), torch.mm(A, Wu.T.contiguous())
    if c["w"] in INT8_A:
        row = st["rs"].double().unsqueeze(1)
        G, U = G * (row * st["cs_gate"].double()), U * (row * st["cs_up"].double())
    if c["bias"]:
        G, U = G + st["b_gate"].double(), U + st["b_up"].double()
    if c["act"] == "silu":
        sg = torch.sigmoid(G)
        h, slope = G * sg, sg * (1 + G * (1 - sg))
    else:
        th = torch.tanh(GELU_C * (G + 0.044715 * G**3))
        h = 0.5 * G * (1 + th)
        slope = 0.5 * (1 + th) + 0.5 * G * (1 - th**2) * GELU_C * (1 + 0.134145 * G**2)
    if not c["train"]:
        return h * U
    dC = st["dC"].double()
    dU, dG = dC * h, dC * U * slope
    out = {"C": h * U, "dA": torch.mm(dG, Wg) + torch.mm(dU, Wu)}
    if c["w"] == "f16":
        out["dw_gate"], out["dw_up"] = torch.mm(dG.T.contiguous(), A), torch.mm(dU.T.contiguous(), A)
        if c["bias"]:
            out["dbias_gate"], out["dbias_up"] = dG.sum(0), dU.sum(0)
    return out


def append_exact(st, c):
    T, hq, hkv, D, page = c["T"], c["hq"], c["hkv"], c["D"], c["page"]
    x = st["qkv"].double().view(T, hq + 2 * hkv, D)
    half = c["rot"] // 2
    j = torch.arange(half, device="cuda")
    i0, i1 = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
    at = st["positions"].long()
    turn = torch.complex(st["cos"].double()[at], st["sin"].double()[at])[:, None]
    heads = x[:, :hq + hkv]
    turned = torch.complex(heads[..., i0], heads[..., i1]) * turn
    y = heads.clone()
    y[..., i0], y[..., i1] = turned.real, turned.imag
    flat_k = st["k"].double().transpose(1, 2).reshape(-1, hkv, D)
    flat_v = st["v"].double().transpose(1, 2).reshape(-1, hkv, D)
    kept = (st["slots"] >= 0).nonzero()[:, 0]
    flat_k[st["slots"][kept]] = y[kept, hq:]
    flat_v[st["slots"][kept]] = x[kept, hq + hkv:]
    back = lambda f: f.view(-1, page, hkv, D).transpose(1, 2).contiguous()  # noqa: E731
    return {"q": y[:, :hq].contiguous(), "k": back(flat_k), "v": back(flat_v)}


def attend_exact(st, c):
    hq, hkv, D, page = c["hq"], c["hkv"], c["D"], c["page"]
    if work(c)["flops"] > 4e12:
        return None
    qs, lens = lengths(c)
    out, row = [], 0

    def tokens(cache, table, n):
        return cache[table.long()].double().transpose(0, 1).reshape(hkv, -1, D)[:, :n]

    pk, pv = (tokens(st[x], st["prefix_table"], c["prefix"]) for x in ("k", "v"))
    for b, (n, L) in enumerate(zip(qs, lens)):
        k = torch.cat([pk, tokens(st["k"], st["tables"][b], L)], 1).repeat_interleave(hq // hkv, 0)
        v = torch.cat([pv, tokens(st["v"], st["tables"][b], L)], 1).repeat_interleave(hq // hkv, 0)
        q = st["q"][row:row + n].double().transpose(0, 1).contiguous()
        row += n
        s = torch.matmul(q, k.transpose(1, 2).contiguous()) * st["scale"]
        reach = c["prefix"] + (L - n + 1 + torch.arange(n, device="cuda")).clamp(min=0)  # keys that each query sees
        hidden = torch.arange(k.shape[1], device="cuda") >= reach[:, None]
        p = torch.softmax(s.masked_fill(hidden, -math.inf), -1).nan_to_num(0.0) if k.shape[1] else s
        out.append(torch.matmul(p, v).transpose(0, 1))
    return torch.cat(out)
