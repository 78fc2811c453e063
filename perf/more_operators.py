"""What is measured of serving with a windowed, normed decoder layer: the operators around its paged cache.

Three operators, in the order in which a step runs them:

* extend: block tables, slots, positions and lengths of a batch's new tokens from its request lengths, with pages taken from a
  pool and given back to it by ended sequences and by tokens that fell out of the window;
* norm: root-mean-square norms of queries and keys for each head with their rotation, in one pass: written into the paged
  cache ("append"), or as dense outputs with their gradients ("train");
* window: attention of a ragged batch over that cache where a query sees its last `window` tokens and the first `sinks` ones.

`run` takes the plain form (elementary torch operations in float32, one rounding) where `own` is false and the library's
kernels where it is true.
"""
import math

import torch

own = False
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------------------------------

def extend_case(name, B, len_min, len_max, new_min, new_max, page, prefix=0, window=0, sinks=0, ends=0, pad=0, short=False):
    """ends: every ends-th sequence ends (0: none); pad: unused rows behind the last token; short: a pool of too few pages."""
    c = {"op": "extend", "B": B, "len_min": len_min, "len_max": len_max, "new_min": new_min, "new_max": new_max, "page": page,
         "prefix": prefix, "window": window, "sinks": sinks, "ends": ends, "pad": pad, "short": short}
    return c if name is None else {"name": name, **c}


def norm_case(name, T, hq, hkv, D, rot, page=16, interleaved=False, padded=False, weight=True, train=False):
    c = {"op": "norm", "T": T, "hq": hq, "hkv": hkv, "D": D, "rot": rot, "page": page, "interleaved": interleaved,
         "padded": padded, "weight": weight, "train": train}
    return c if name is None else {"name": name, **c}


def window_case(name, B, hq, hkv, D, page, q_min, q_max, own_min, own_max, window, sinks, prefix=0):
    c = {"op": "window", "B": B, "hq": hq, "hkv": hkv, "D": D, "page": page, "q_min": q_min, "q_max": q_max,
         "own_min": own_min, "own_max": own_max, "window": window, "sinks": sinks, "prefix": prefix}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one sequence decoding alone: latency
        extend_case("extend_one", 1, 777, 777, 1, 1, 16),
        # a decode batch behind a system prompt, windowed; some sequences end, some rows of the batch are unused
        extend_case("extend_decode", 48, 0, 8000, 1, 1, 16, prefix=1000, window=1024, sinks=4, ends=9, pad=16),
        # chunks of prompts beside decoding sequences, from a pool that does not hold them all
        extend_case("extend_chunks", 24, 0, 6000, 1, 700, 16, window=2048, sinks=16, short=True),
        # a large server's step: many sequences, tens of thousands of new tokens
        extend_case("extend_many", 1500, 0, 8000, 0, 40, 32, window=4096, ends=50, pad=333),
        # one new token for each of 48 sequences, some slots of the batch unused
        norm_case("norm_decode", 48, 32, 8, 128, 128, padded=True),
        # a prompt's tokens, partial rotation in the interleaved order
        norm_case("norm_prefill", 8190, 32, 8, 128, 64, page=64, interleaved=True),
        # the same in training: dense outputs and all gradients
        norm_case("norm_train", 4096, 32, 8, 128, 128, train=True),
        # an odd small layer in training: a head of 80 of which half turns
        norm_case("norm_train_odd", 333, 6, 2, 80, 40, train=True),
        # one sequence, one token, far along: latency
        window_case("window_one", 1, 32, 8, 128, 16, 1, 1, 16000, 16000, 4096, 4),
        # a decode batch behind a system prompt whose beginning stays visible
        window_case("window_decode", 64, 32, 8, 128, 16, 1, 1, 0, 9000, 1024, 4, prefix=1000),
        # one long prompt at once
        window_case("window_prefill", 1, 32, 8, 128, 64, 8192, 8192, 8192, 8192, 1024, 16),
        # chunks of several prompts over what they hold already, heads of 64, sequences of mixed length
        window_case("window_chunks", 4, 32, 4, 64, 16, 700, 1024, 700, 6000, 2000, 130, prefix=300),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "norm", "norm", "window", "window"])
    page = rng.choice([1, 16, 16, 32, 64, 256])
    if op == "extend":
        B = log_int(rng, 1, 1500)
        page = max(page, 16)
        len_max = log_int(rng, 1, 8000)
        new_max = rng.choice([1, log_int(rng, 1, max(1, 30000 // B))])
        return extend_case(None, B, rng.choice([0, len_max]), len_max, rng.choice([0, new_max]), new_max, page,
                           prefix=rng.choice([0, log_int(rng, 1, 4000)]), window=rng.choice([0, log_int(rng, 16, 6000)]),
                           sinks=rng.choice([0, 4, log_int(rng, 1, 500)]), ends=rng.choice([0, rng.randint(2, 40)]),
                           pad=rng.choice([0, log_int(rng, 1, 500)]), short=rng.random() < 0.3)
    D = rng.choice([64, 80, 96, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    hq, hkv = (hq, hkv) if hq <= 64 else (32, 8)
    if op == "norm":
        return norm_case(None, log_int(rng, 1, 4096), hq, hkv, D, rng.choice([D, D, D // 2]), page, interleaved=rng.random() < 0.5,
                         padded=rng.random() < 0.5, weight=rng.random() < 0.8, train=rng.random() < 0.5)
    while True:
        B = log_int(rng, 1, 64)
        q_max = rng.choice([1, 1, 1, log_int(rng, 2, 16), log_int(rng, 16, max(17, 4096 // B))])
        own_max = q_max + log_int(rng, 1, max(2, 32768 // B))
        c = window_case(None, B, hq, hkv, D, page, rng.choice([1, q_max]), q_max, rng.choice([0, q_max, own_max]), own_max,
                        log_int(rng, 1, 4096), rng.choice([0, 4, log_int(rng, 1, 300)]), rng.choice([0, 0, log_int(rng, 1, 4096)]))
        # the plain form holds the scores of 256 queries of every sequence at once
        scores = B * hq * min(q_max, 256) * min(c["window"] + 256 + c["sinks"], own_max + c["prefix"])
        if work(c)["flops"] <= 1.2e11 and scores <= 1 << 28:
            return c


# ---- inputs --------------------------------------------------------------------------------------------------------

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def spread(lo, hi, i, n):
    """The i-th of n sizes between lo and hi, in a fixed mixed order that begins with hi."""
    return hi - (hi - lo) * ((i * 37) % n) // max(1, n - 1) if n > 1 else hi


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).half()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def up(x, y):
    return -(-x // y)


def requests(c):
    """(tokens in the cache, new tokens or -1 at its end, pages given back earlier) of each sequence of an extend case."""
    B, page = c["B"], c["page"]
    lens = [spread(c["len_min"], c["len_max"], i + 3, B) for i in range(B)]
    news = [-1 if c["ends"] and i % c["ends"] == c["ends"] - 1 else spread(c["new_min"], c["new_max"], i, B) for i in range(B)]
    s0 = up(max(0, c["sinks"] - c["prefix"]), page)
    gone = []
    for i, L in enumerate(lens):  # as the call before left them, which began some tokens earlier
        e = max(0, L - spread(1, max(1, min(L, 300)), i, B) - c["window"] + 1) // page if c["window"] else 0
        gone.append(e if e > s0 else 0)
    return lens, news, gone


def tables_of(c):
    """(table width, pages in the pool, free ones on entry) of an extend case."""
    lens, news, gone = requests(c)
    s0, page = up(max(0, c["sinks"] - c["prefix"]), c["page"]), c["page"]
    held = sum(up(L, page) - max(0, g - s0) for L, g in zip(lens, gone))
    need = sum(up(L + max(n, 0), page) - up(L, page) for L, n in zip(lens, news))
    free = need * 2 // 3 if c["short"] else need + 50
    return max(1, max(up(L + max(n, 0), page) for L, n in zip(lens, news))), max(1, held + free), free


def lengths(c):
    """(queries, own tokens with the queries' among them, or none in an unused slot) of each sequence of a window case."""
    qs = [spread(c["q_min"], c["q_max"], i, c["B"]) for i in range(c["B"])]
    own_tokens = [spread(c["own_min"], c["own_max"], i + 3, c["B"]) for i in range(c["B"])]
    return qs, [max(n, L) if L else 0 for n, L in zip(qs, own_tokens)]


def prepare(case, seed):
    return {"extend": prepare_extend, "norm": prepare_norm, "window": prepare_window}[case["op"]](case, generator(seed))


def prepare_extend(c, gen):
    B, page = c["B"], c["page"]
    lens, news, gone = requests(c)
    width, pool, free = tables_of(c)
    s0 = up(max(0, c["sinks"] - c["prefix"]), page)
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    st = {"case": c, "lens": ints(lens), "news": ints(news), "gone": ints(gone), "T": sum(max(n, 0) for n in news) + c["pad"]}
    col = torch.arange(width, device="cuda")
    held = (col < ((st["lens"] + page - 1) // page)[:, None]) & ~((col >= s0) & (col < st["gone"][:, None]))
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    tables[held] = order[free:]
    # the pool is a ring: the free pages begin anywhere in it
    head = int(torch.randint(0, pool, (1,), generator=gen, device="cuda"))
    ring = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(free, device="cuda")) % pool] = order[:free]
    st.update(tables=tables, ring=ring, head=ints([head]), free=ints([free]), page=page)
    if own:  # the pool that a server keeps, in this state
        from weight_quantized_mixed_amd.device import PagePool
        st["pool"] = PagePool(pool, page, B, width, prefix_len=c["prefix"], window=c["window"] or None, sinks=c["sinks"],
                              ring=ring, tables=tables)
        st["pool"].state.copy_(torch.cat([st["lens"], st["gone"], st["head"], st["free"]]))
        st["after"] = torch.empty_like(st["pool"].state)
    return st


def prepare_norm(c, gen):
    T, hq, hkv, D, rot, page = c["T"], c["hq"], c["hkv"], c["D"], c["rot"], c["page"]
    st = {"case": c, "qkv": normal(gen, T, (hq + 2 * hkv) * D)}
    for w in ("qw", "kw"):
        st[w] = (1 + 0.2 * torch.randn((D,), generator=gen, device="cuda")).half() if c["weight"] else None
    n_pos = 4096 + T
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    ang = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * inv
    st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
    st["positions"] = torch.randint(0, n_pos, (T,), generator=gen, device="cuda", dtype=torch.int32)
    if c["train"]:
        st["dq"], st["dk"] = normal(gen, T, hq, D, std=0.1), normal(gen, T, hkv, D, std=0.1)
        return st
    n_pages = up(T * 5, 4 * page) + 1
    slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:T]
    if c["padded"]:
        slots[5::11] = -1  # unused rows of the batch: normed and rotated, not stored
    st["slots"] = slots
    st["k"], st["v"] = normal(gen, n_pages, hkv, page, D), normal(gen, n_pages, hkv, page, D)
    if own:
        from weight_quantized_mixed_amd.device import PagedKV
        st["cache"] = PagedKV(n_pages, page, hkv, D, k=st["k"], v=st["v"])
    return st


def prepare_window(c, gen):
    B, hq, hkv, D, page, prefix = c["B"], c["hq"], c["hkv"], c["D"], c["page"], c["prefix"]
    qs, lens = lengths(c)
    width, n_prefix = max(1, up(c["own_max"], page)), up(prefix, page)
    n_pages = B * width + n_prefix
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    starts = [0]
    for n in qs:
        starts.append(starts[-1] + n)
    st = {"case": c, "q": normal(gen, starts[-1], hq, D), "k": normal(gen, n_pages, hkv, page, D), "v": normal(gen, n_pages, hkv, page, D),
          "starts": ints(starts), "lens": ints(lens), "tables": order[n_prefix:].view(B, width).contiguous(),
          "prefix_table": order[:n_prefix].clone(), "scale": D ** -0.5}
    if own:
        from weight_quantized_mixed_amd.device import PagedKV
        st["cache"] = PagedKV(n_pages, page, hkv, D, k=st["k"], v=st["v"])
    return st


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    kind = c["op"] + ("_train" if c.get("train") else "") + ("_own" if own else "_plain")
    return {"extend_own": extend_own, "extend_plain": extend_plain, "norm_own": norm_own, "norm_plain": norm_plain,
            "norm_train_own": norm_train_own, "norm_train_plain": norm_train_plain, "window_own": window_own,
            "window_plain": window_plain}[kind](state, c)


def extend_own(st, c):
    # the state after the step goes to a place of its own, so that a step can be tried again
    pool = st["pool"]
    r = pool.extend(st["news"], st["T"], state_out=st["after"])
    return {**r, "state": st["after"], "tables": pool.tables, "ring": pool.ring}


def norm_own(st, c):
    hq, hkv, D = c["hq"], c["hkv"], c["D"]
    q, k, v = st["qkv"].split([hq * D, hkv * D, hkv * D], dim=1)
    out = st["cache"].append(q, k, v, st["cos"], st["sin"], st["positions"], st["slots"], interleaved=c["interleaved"],
                             norm_eps=EPS, q_weight=st["qw"], k_weight=st["kw"])
    return {"q": out, "k": st["k"], "v": st["v"]}


def norm_train_own(st, c):
    from weight_quantized_mixed_amd.device import norm_rotate, norm_rotate_backward
    hq, hkv, D = c["hq"], c["hkv"], c["D"]
    q, k, _ = st["qkv"].split([hq * D, hkv * D, hkv * D], dim=1)
    args = {"q_weight": st["qw"], "k_weight": st["kw"], "eps": EPS, "interleaved": c["interleaved"]}
    qo, ko = norm_rotate(q, k, D, st["cos"], st["sin"], st["positions"], **args)
    grads = norm_rotate_backward(q, k, st["dq"], st["dk"], st["cos"], st["sin"], st["positions"], weight_grads=c["weight"], **args)
    return {"q": qo, "k": ko, **{name: g for name, g in grads.items() if g is not None}}


def window_own(st, c):
    return st["cache"].attend(st["q"], st["starts"], st["lens"], st["tables"], max_q=c["q_max"], max_len=c["own_max"],
                              prefix_table=st["prefix_table"] if c["prefix"] else None, prefix_len=c["prefix"], scale=st["scale"],
                              window=c["window"], sinks=c["sinks"])


def extend_plain(st, c):
    B, page, prefix, T = c["B"], c["page"], c["prefix"], st["T"]
    R, width = st["ring"].shape[0], st["tables"].shape[1]
    lens, news, gone = st["lens"].long(), st["news"].long(), st["gone"].long()
    head, free = st["head"].long(), st["free"].long()
    n = news.clamp(min=0)
    stop = n.cumsum(0)
    start = stop - n
    old, new = (lens + page - 1) // page, (lens + n + page - 1) // page
    alone = (new > width) | (prefix + lens + n > 2**31 - 1) | (stop > T)
    need = torch.where(alone, 0, new - old)
    taken = need.cumsum(0)
    refused = (n > 0) & (alone | ((need > 0) & (taken > free)))
    before = taken - need
    grow = torch.where(refused, 0, n)
    # tokens
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(stop, t, right=True)
    live, seq = seq < B, seq.clamp(max=B - 1)
    j = lens[seq] + t - start[seq]
    at = j // page
    fresh = at >= old[seq]
    pages = torch.where(fresh, st["ring"][(head + before[seq] + at - old[seq]) % R], st["tables"][seq, at.clamp(max=width - 1)])
    good = live & ~refused[seq]
    slots = torch.where(good, pages.long() * page + j % page, -1)
    positions = torch.where(good, prefix + j, torch.where(live, -1, 0)).int()
    # new pages into the tables, through one place more than they have for the tokens that bring none
    flat = torch.cat([st["tables"].reshape(-1), st["tables"].new_zeros(1)])
    flat[torch.where(good & fresh, seq * width + at, B * width)] = pages
    # pages that are given back, in the order of the sequences and of their pages
    col = torch.arange(width, device="cuda")
    s0 = up(max(0, c["sinks"] - prefix), page)
    held = (col < old[:, None]) & ~((col >= s0) & (col < gone[:, None]))
    past = (lens - c["window"] + 1).clamp(min=0) // page if c["window"] else gone * 0
    back = held & torch.where((news < 0)[:, None], True, (col >= s0) & (col < past[:, None]))
    rank = back.reshape(-1).cumsum(0)
    ring = torch.cat([st["ring"], st["ring"].new_zeros(1)])
    ring[torch.where(back.reshape(-1), (head + free + rank - 1) % R, R)] = st["tables"].reshape(-1)
    used = torch.where(refused, 0, need).sum().reshape(1)
    kv_lens = torch.where(news < 0, 0, lens + grow)
    gone = torch.where(news < 0, 0, torch.where(past > s0, torch.maximum(gone, past), gone))
    state = torch.cat([kv_lens, gone, (head + used) % R, free - used + rank[-1:]]).int()
    return {"q_starts": torch.cat([start.new_zeros(1), stop]).clamp(max=T).int(), "kv_lens": kv_lens.int(), "positions": positions,
            "slots": slots, "refused": refused.int(), "state": state, "tables": flat[:-1].view(B, width), "ring": ring[:-1]}


def turn(x, cos, sin, interleaved):
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


def norm_forward(st, c):
    """Normed and rotated queries and keys in float32, with the values."""
    T, hq, hkv, D = c["T"], c["hq"], c["hkv"], c["D"]
    q, k, v = st["qkv"].float().split([hq * D, hkv * D, hkv * D], dim=1)
    at = st["positions"].long()
    out = []
    for x, h, w in ((q, hq, st["qw"]), (k, hkv, st["kw"])):
        x = x.reshape(T, h, D)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if w is not None:
            x = x * w.float()
        out.append(turn(x, st["cos"][at], st["sin"][at], c["interleaved"]))
    return (*out, v.reshape(T, hkv, D))


def norm_plain(st, c):
    page = c["page"]
    q, k, v = norm_forward(st, c)
    slots, k, v = st["slots"], k.half(), v.half()
    if c["padded"]:
        keep = slots >= 0
        slots, k, v = slots[keep], k[keep], v[keep]
    st["k"][slots // page, :, slots % page] = k
    st["v"][slots // page, :, slots % page] = v
    return {"q": q.half(), "k": st["k"], "v": st["v"]}


def norm_train_plain(st, c):
    T, hq, hkv, D = c["T"], c["hq"], c["hkv"], c["D"]
    qo, ko, _ = norm_forward(st, c)
    out = {"q": qo.half(), "k": ko.half()}
    q, k, _ = st["qkv"].float().split([hq * D, hkv * D, hkv * D], dim=1)
    at = st["positions"].long()
    grads = {}
    for name, x, dy, h, w in (("q", q, st["dq"], hq, st["qw"]), ("k", k, st["dk"], hkv, st["kw"])):
        x = x.reshape(T, h, D)
        g = turn(dy.float(), st["cos"][at], -st["sin"][at], c["interleaved"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if w is not None:
            grads[f"d{name}_weight"] = (x * r * g).sum((0, 1), dtype=torch.float64).float()
            g = g * w.float()
        grads[f"d{name}"] = (r * g - x * r**3 * (x * g).mean(-1, keepdim=True)).half().view(T, h * D)
    return {**out, **grads}


def gather(cache, st, c, at):
    """Tokens at `at` [B, n], counted from the prefix's first one, as [B, n, heads, D] in float32."""
    page, prefix = c["page"], c["prefix"]
    mine = (at - prefix).clamp(min=0)
    pages = st["tables"].long().gather(1, (mine // page).clamp(max=st["tables"].shape[1] - 1))
    off = mine % page
    if prefix:
        first = at.clamp(max=prefix - 1)
        pages = torch.where(at < prefix, st["prefix_table"].long()[first // page], pages)
        off = torch.where(at < prefix, first % page, off)
    return cache[pages, :, off].float()


def window_plain(st, c):
    B, hq, hkv, D, prefix = c["B"], c["hq"], c["hkv"], c["D"], c["prefix"]
    W, S, G, step = c["window"], c["sinks"], hq // hkv, 256
    starts, lens = st["starts"].long(), st["lens"].long()
    nq = starts[1:] - starts[:-1]
    out = torch.empty_like(st["q"])
    for i0 in range(0, c["q_max"], step):  # queries of all sequences, some at a time, against the band that they see
        i = torch.arange(i0, min(i0 + step, c["q_max"]), device="cuda")
        m = i.shape[0]
        live = i < nq[:, None]
        rows = (starts[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
        q = (st["q"][rows].float() * st["scale"]).view(B, m, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, m * G, D)
        last = prefix + (lens[:, None] - nq[:, None] + i + 1).clamp(min=0)                   # keys up to each query [B, m]
        first = (last[:, :1] - W).clamp(min=S)                                               # where the band of all of them begins
        band = torch.arange(min(W + m, prefix + c["own_max"]), device="cuda")
        at = torch.cat([torch.arange(min(S, prefix + c["own_max"]), device="cuda").expand(B, -1), first + band], 1)   # [B, nk]
        k, v = gather(st["k"], st, c, at), gather(st["v"], st, c, at)
        s = q @ k.permute(0, 2, 3, 1).contiguous()
        at, end = at[:, None], last[..., None]
        seen = (at < end) & ((at >= end - W) | (at < S)) & live[..., None]                   # [B, m, nk]
        s = torch.where(seen[:, None, :, None].expand(B, hkv, m, G, -1).reshape(s.shape), s, -torch.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-3e38))
        total = p.sum(-1, keepdim=True)
        o = (p @ v.permute(0, 2, 1, 3).contiguous()) / total.clamp(min=1e-30)
        o = o.view(B, hkv, m, G, D).permute(0, 2, 1, 3, 4).reshape(B, m, hq, D)
        out[rows[live]] = o[live].half()
    return out


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def seen_keys(c):
    """(pairs of a query and a key that it sees, keys that any query of their sequence sees) of a window case."""
    pairs = keys = 0
    for n, L in zip(*lengths(c)):
        ends = [c["prefix"] + max(0, L - n + i + 1) for i in range(n)]
        pairs += sum(min(e, c["window"] + min(c["sinks"], max(0, e - c["window"]))) for e in ends)
        low = max(0, ends[0] - c["window"]) if n else 0
        keys += (ends[-1] - low + min(c["sinks"], low)) if n else 0
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "extend":
        lens, news, gone = requests(c)
        T = sum(max(n, 0) for n in news) + c["pad"]
        pages = sum(up(L + max(n, 0), c["page"]) - up(L, c["page"]) for L, n in zip(lens, news))
        back = sum(up(L, c["page"]) for L, n in zip(lens, news) if n < 0)
        return {"bytes": 28 * c["B"] + 12 * T + 8 * (pages + back) + 16, "flops": 10 * (c["B"] + T)}
    if c["op"] == "norm":
        T, rows, kv = c["T"], c["T"] * (c["hq"] + c["hkv"]), c["T"] * c["hkv"]
        angles = T * (c["rot"] * 4 + 4)
        if c["train"]:  # x and the outputs' gradients read, outputs and the inputs' gradients written
            return {"bytes": 8 * rows * c["D"] + angles + (12 * 2 * c["D"] if c["weight"] else 0), "flops": rows * (15 * c["D"] + 6 * c["rot"])}
        return {"bytes": 4 * (rows + kv) * c["D"] + angles + 8 * T, "flops": rows * (5 * c["D"] + 3 * c["rot"])}
    pairs, keys = seen_keys(c)
    return {"bytes": 4 * c["hkv"] * c["D"] * keys + 4 * sum(lengths(c)[0]) * c["hq"] * c["D"], "flops": 4 * c["D"] * c["hq"] * pairs}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "extend":
        return extend_exact(st, case)
    if case["op"] == "norm":
        return norm_exact(st, case)
    return window_exact(st, case)


def extend_exact(st, c):
    """One sequence and one page after the other, on the host."""
    page, prefix, T = c["page"], c["prefix"], st["T"]
    lens, news, gone = (st[x].tolist() for x in ("lens", "news", "gone"))
    tables, ring = st["tables"].cpu(), st["ring"].tolist()
    width, R, head, free = tables.shape[1], len(ring), int(st["head"]), int(st["free"])
    starts, positions, slots, refused, returned = [0], [0] * T, [-1] * T, [], []
    asked = used = row = 0
    keep = -(-max(0, c["sinks"] - prefix) // page)
    for b, (L, n) in enumerate(zip(lens, news)):
        have = -(-L // page)
        gap = range(keep, gone[b])
        if n < 0:
            returned += [int(tables[b, i]) for i in range(have) if i not in gap]
            lens[b] = gone[b] = 0
        elif c["window"]:
            to = max(0, L - c["window"] + 1) // page
            returned += [int(tables[b, i]) for i in range(keep, to) if i not in gap]
            gone[b] = max(gone[b], to) if to > keep else gone[b]
        n = max(n, 0)
        more = -(-(L + n) // page) - have
        fits = have + more <= width and prefix + L + n < 2**31 and row + n <= T
        asked += more if fits else 0
        no = n > 0 and (not fits or (more > 0 and asked > free))
        refused.append(int(no))
        if n and not no:
            for i in range(more):
                tables[b, have + i] = ring[(head + used) % R]
                used += 1
            lens[b] = L + n
        for i in range(min(n, T - row) if row < T else 0):
            positions[row + i] = -1 if no else prefix + L + i
            if not no:
                slots[row + i] = int(tables[b, (L + i) // page]) * page + (L + i) % page
        row += n
        starts.append(min(row, T))
    for i, p in enumerate(returned):
        ring[(head + free + i) % R] = p
    state = lens + gone + [(head + used) % R, free - used + len(returned)]
    return {"q_starts": ints(starts), "kv_lens": ints(lens), "positions": ints(positions),
            "slots": torch.tensor(slots, dtype=torch.int64, device="cuda"), "refused": ints(refused), "state": ints(state),
            "tables": tables.cuda(), "ring": ints(ring)}


def norm_exact(st, c):
    T, hq, hkv, D = c["T"], c["hq"], c["hkv"], c["D"]
    x = st["qkv"].double().view(T, hq + 2 * hkv, D)
    j = torch.arange(c["rot"] // 2, device="cuda")
    i0, i1 = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + c["rot"] // 2)
    at = st["positions"].long()
    angle = torch.complex(st["cos"].double()[at], st["sin"].double()[at])[:, None]

    def rotated(y, by):
        z = y.clone()
        t = torch.complex(y[..., i0], y[..., i1]) * by
        z[..., i0], z[..., i1] = t.real, t.imag
        return z

    ones = torch.ones(D, dtype=torch.float64, device="cuda")
    out = {}
    for name, heads, w, dy in (("q", x[:, :hq], st["qw"], st.get("dq")), ("k", x[:, hq:hq + hkv], st["kw"], st.get("dk"))):
        rms = (heads.square().sum(-1, keepdim=True) / D + EPS).sqrt()
        unit, w64 = heads / rms, ones if w is None else w.double()
        out[name] = rotated(unit * w64, angle)
        if c["train"]:
            g = rotated(dy.double(), angle.conj())
            if w is not None:
                out[f"d{name}_weight"] = (unit * g).sum((0, 1))
            g = g * w64
            out[f"d{name}"] = ((g - unit * (unit * g).sum(-1, keepdim=True) / D) / rms).reshape(T, -1)
    if c["train"]:
        return out
    page = c["page"]
    flat_k = st["k"].double().transpose(1, 2).reshape(-1, hkv, D)
    flat_v = st["v"].double().transpose(1, 2).reshape(-1, hkv, D)
    kept = (st["slots"] >= 0).nonzero()[:, 0]
    flat_k[st["slots"][kept]], flat_v[st["slots"][kept]] = out["k"][kept], x[kept, hq + hkv:]
    back = lambda f: f.view(-1, page, hkv, D).transpose(1, 2).contiguous()  # noqa: E731
    return {"q": out["q"].contiguous(), "k": back(flat_k), "v": back(flat_v)}


def window_exact(st, c):
    hq, hkv, D, W, S = c["hq"], c["hkv"], c["D"], c["window"], c["sinks"]
    qs, lens = lengths(c)
    if sum(hq * n * (L + c["prefix"]) for n, L in zip(qs, lens)) * D > 1e12:
        return None
    out, row = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), 0

    def tokens(cache, table, n):
        return cache[table.long()].double().transpose(0, 1).reshape(hkv, -1, D)[:, :n]

    pk, pv = (tokens(st[x], st["prefix_table"], c["prefix"]) for x in ("k", "v"))
    for b, (n, L) in enumerate(zip(qs, lens)):
        k = torch.cat([pk, tokens(st["k"], st["tables"][b], L)], 1)
        v = torch.cat([pv, tokens(st["v"], st["tables"][b], L)], 1)
        key = torch.arange(k.shape[1], device="cuda")
        for i0 in range(0, n, 1024) if k.shape[1] else ():
            i = torch.arange(i0, min(i0 + 1024, n), device="cuda")
            own_seen = (L - n + i + 1).clamp(min=0)
            dist = c["prefix"] + own_seen[:, None] - 1 - key  # of each key behind the query's own place
            hidden = (dist < 0) | ((dist >= W) & (key >= S))
            for h in range(hq):
                q = st["q"][row + i, h].double()
                s = torch.mm(q, k[h // (hq // hkv)].T.contiguous()) * st["scale"]
                p = torch.softmax(s.masked_fill(hidden, -math.inf), -1).nan_to_num(0.0)
                out[row + i, h] = torch.mm(p, v[h // (hq // hkv)])
        row += n
    return out
