"""Measured cases of the operators of a cached decode step: per-head norms of
queries and keys with the position rotation (forward and backward), the append
of keys and values to a paged cache, and attention for a tree of drafted
tokens over [memory ; cache ; tree].

With ``own`` false ``run`` computes each operator in elementary torch
operations in 32 bits (angles in 64), rounded once at the end; with ``own``
true it makes the calls a user makes of ``latent_memory_routing_b200.pipeline``.

Shared shapes: q [n_tok][Hq][D], k and v [n_tok][H][D] (tokens of all
sequences one after another, offsets [B+1]); cache pages [n_pages][H][page][D];
memory rows [B][m_cap][H][D].
"""

import math
import random

import torch

own = False

BASE = 10000.0
EPS = 1e-6
TOP_K = 16  # selected documents: a query's global positions start at this offset
DEV = "cuda"


def _dt(case):
    return torch.float32 if case["dt"] == "f32" else torch.bfloat16


def _es(case):
    return 4 if case["dt"] == "f32" else 2


# ---------------------------------------------------------------- the cases

def listed():
    model = {"Hq": 32, "H": 8, "D": 128, "dt": "bf16"}  # the heads of the bf16 banks
    tiny = {"Hq": 4, "H": 2, "D": 64, "dt": "f32"}      # the fp32 workload's heads
    return [
        # one decode step of 64 sequences: the launch decides
        dict(model, name="norm_decode_64", op="norm", n=64, fused=True),
        # a long prompt's queries and keys, slices of one projection's output
        dict(model, name="norm_prompt_32k", op="norm", n=32799, fused=True),
        # a training step's micro-batch, gradients in bf16
        dict(model, name="norm_back_16k", op="norm_back", n=16384, grad="bf16", fused=True),
        # the 16 x 180 tokens of the fp32 workload
        dict(tiny, name="norm_back_f32", op="norm_back", n=2880, grad="f32", fused=False),
        # one token for each of 64 sequences, the step's queries on the way
        dict(model, name="append_decode_64", op="append", B=64, n=1, L=2047, page=64,
             ragged=0, queries=True, norm=True),
        # the prompts of 16 sequences, of unlike lengths, into empty caches
        dict(model, name="append_prompts_16", op="append", B=16, n=2048, L=0, page=64,
             ragged=5, queries=False, norm=True),
        # a drafted tree a sequence, without norms, in fp32
        dict(tiny, name="append_tree_f32", op="append", B=3, n=13, L=117, page=16,
             ragged=7, queries=True, norm=False),
        # plain decode of 64 sequences over 2,048 local tokens and their memory rows
        dict(model, name="attend_decode_64", op="tree", B=64, n=1, L=2047, M=220, page=64,
             ragged=0),
        # one sequence, one token: latency
        dict(model, name="attend_decode_1", op="tree", B=1, n=1, L=4095, M=220, page=64,
             ragged=0),
        # trees of up to 48 drafted tokens over unlike caches
        dict(model, name="attend_trees_16", op="tree", B=16, n=48, L=8000, M=220, page=64,
             ragged=11),
        # full trees over long caches
        dict(model, name="attend_long_2", op="tree", B=2, n=64, L=150001, M=0, page=64,
             ragged=0),
        # the fp32 workload's heads
        dict(tiny, name="attend_tree_f32", op="tree", B=2, n=16, L=300, M=6, page=16,
             ragged=3),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "append", "tree", "tree"])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    H = rng.choice([1, 2, 4, 8])
    Hq = H * rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 128])
    case = {"op": op, "Hq": Hq, "H": H, "D": D, "dt": dt}
    if op in ("norm", "norm_back"):
        case.update(n=_logint(rng, 1, 32768), fused=rng.random() < 0.5)
        if op == "norm_back":
            case["grad"] = "f32" if dt == "f32" else rng.choice(["bf16", "f32"])
            case["n"] = _logint(rng, 1, 16384)
        # at most the bytes of the largest listed case
        while work(case)["bytes"] > 6.0e8:
            case["n"] = max(1, case["n"] // 2)
        return case
    case.update(B=_logint(rng, 1, 64), page=rng.choice([16, 32, 64, 128]),
                ragged=rng.choice([0, rng.randrange(1, 1 << 20)]))
    if op == "append":
        case.update(n=_logint(rng, 1, 4096), L=rng.choice([0, _logint(rng, 1, 4096)]),
                    queries=rng.random() < 0.5, norm=rng.random() < 0.7)
        while work(case)["bytes"] > 2.5e8 or case["B"] * (case["n"] + case["L"]) > 100000:
            case["B"] = max(1, case["B"] // 2)
            case["n"] = max(1, case["n"] * 2 // 3)
        return case
    case.update(n=_logint(rng, 1, 64), L=_logint(rng, 1, 150000),
                M=rng.choice([0, _logint(rng, 1, 700)]))
    top = 8e9 if dt == "f32" else 8e10
    while (work(case)["flops"] > top or work(case)["bytes"] > 6e8
           or case["B"] * case["L"] > 300000):
        if case["B"] > 1:
            case["B"] = max(1, case["B"] * 2 // 3)
        else:
            case["L"] = max(1, case["L"] * 2 // 3)
    return case


def _lens(case):
    """Tokens and cached tokens (and memory rows) of each sequence; unlike
    from sequence to sequence where the case is ragged."""
    B, n, L, M = case["B"], case["n"], case["L"], case.get("M", 0)
    if not case["ragged"]:
        return [n] * B, [L] * B, [M] * B
    r = random.Random(case["ragged"])
    ns = [n] + [r.randint(1 + n // 4, n) for _ in range(B - 1)]
    Ls = [L] + [r.randint(0, L) for _ in range(B - 1)]
    Ms = [M] + [r.randint(0, M) for _ in range(B - 1)]
    return ns, Ls, Ms


def work(case):
    es, Hq, H, D = _es(case), case["Hq"], case["H"], case["D"]
    if case["op"] == "norm":
        e = case["n"] * (Hq + H) * D
        return {"bytes": 2 * e * es + 4 * case["n"], "flops": 9 * e}
    if case["op"] == "norm_back":
        e = case["n"] * (Hq + H) * D
        gs = 4 if case["grad"] == "f32" else 2
        return {"bytes": e * (es + 2 * gs) + 4 * case["n"], "flops": 20 * e}
    ns, Ls, Ms = _lens(case)
    t = sum(ns)
    if case["op"] == "append":
        e = t * (2 * H + (Hq if case["queries"] else 0)) * D
        return {"bytes": 2 * e * es + 4 * t, "flops": 9 * e}
    keys = [n + L + M for n, L, M in zip(ns, Ls, Ms)]
    return {"bytes": 2 * sum(keys) * H * D * es + 2 * t * Hq * D * es,
            "flops": 4 * Hq * D * sum(n * k for n, k in zip(ns, keys))}


# --------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, dt, g):
    return torch.randn(shape, device=DEV, generator=g).to(dt)


def _qkv(case, n, g, need_v):
    """q, k (, v) of n tokens: slices of one projection's output where the
    case is fused, else tensors of their own."""
    Hq, H, D, dt = case["Hq"], case["H"], case["D"], _dt(case)
    if case.get("fused"):
        x = _randn((n, (Hq + 2 * H) * D), dt, g)
        q = x[:, :Hq * D].unflatten(1, (Hq, D))
        k = x[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        v = x[:, (Hq + H) * D:].unflatten(1, (H, D))
    else:
        q, k = _randn((n, Hq, D), dt, g), _randn((n, H, D), dt, g)
        v = _randn((n, H, D), dt, g) if need_v else None
    return q, k, v


def _weights(case, g):
    mk = lambda: (1.0 + 0.1 * torch.randn(case["D"], device=DEV, generator=g)).to(_dt(case))  # noqa: E731
    return mk(), mk()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tables(case, seed):
    """Offsets, cached lengths and a block table of shuffled pages, with the
    parents and depths of each sequence's drafted tokens."""
    r = random.Random(seed)
    ns, Ls, Ms = _lens(case)
    page = case["page"]
    need = [(n + L + page - 1) // page for n, L in zip(ns, Ls)]
    max_pages = max(need)
    n_pages = sum(need) + 3
    ids = list(range(n_pages))
    r.shuffle(ids)
    table, at = [], 0
    for c in need:
        table.append(ids[at:at + c] + [0] * (max_pages - c))
        at += c
    off = [0]
    for n in ns:
        off.append(off[-1] + n)
    parents, pos = [], []
    chain = case["n"] > 64 or case["n"] == 1
    for n, L in zip(ns, Ls):
        depth = []
        for i in range(n):
            p = i - 1 if chain else r.randrange(max(-1, i - 6), i)
            parents.append(p)
            depth.append(0 if p < 0 else depth[p] + 1)
            pos.append(TOP_K + L + depth[-1])
    return dict(off=torch.tensor(off, dtype=torch.int64, device=DEV), lens=_i32(Ls),
                mems=_i32(Ms), table=_i32(table), parents=_i32(parents), pos=_i32(pos),
                n_pages=n_pages, max_pages=max_pages, n_tok=off[-1])


def prepare(case, seed):
    g = _gen(seed)
    Hq, H, D, dt = case["Hq"], case["H"], case["D"], _dt(case)
    st = {"case": case}
    if case["op"] in ("norm", "norm_back"):
        n = case["n"]
        q, k, _ = _qkv(case, n, g, False)
        wq, wk = _weights(case, g)
        first = random.Random(seed).randrange(0, 1 << 16)
        pos = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
        st.update(q=q, k=k, wq=wq, wk=wk, pos=pos)
        if case["op"] == "norm_back":
            gd = torch.float32 if case["grad"] == "f32" else torch.bfloat16
            st.update(dq=_randn((n, Hq, D), gd, g), dk=_randn((n, H, D), gd, g))
        if own:
            from latent_memory_routing_b200 import pipeline
            st["call"] = pipeline.qk_norm_rope
            if case["op"] == "norm_back":
                st["call"] = pipeline.qk_norm_rope_backward
                st["ws"] = pipeline.qk_norm_rope_backward_workspace(q, k)
        return st
    t = _tables(case, seed)
    st.update(t)
    pages = (t["n_pages"], H, case["page"], D)
    kp, vp = _randn(pages, dt, g), _randn(pages, dt, g)
    if case["op"] == "append":
        q, k, v = _qkv(dict(case, fused=True), t["n_tok"], g, True)
        wq, wk = _weights(case, g) if case["norm"] else (None, None)
        st.update(q=q if case["queries"] else None, k=k, v=v, wq=wq, wk=wk)
    else:
        m_cap = case["M"]
        st["q"] = _randn((t["n_tok"], Hq, D), dt, g)
        st["km"] = _randn((case["B"], m_cap, H, D), dt, g) if m_cap else None
        st["vm"] = _randn((case["B"], m_cap, H, D), dt, g) if m_cap else None
    st.update(kp=kp, vp=vp)
    if own:
        from latent_memory_routing_b200 import pipeline
        c = pipeline.PagedCache(dt, t["n_pages"], case["page"], H, D, case["B"], t["max_pages"],
                                DEV)
        c.k_pages, c.v_pages = kp, vp
        c.block_table.copy_(t["table"])
        c.cache_len.copy_(t["lens"])
        st["cache"] = c
        if case["op"] == "tree":
            st["call"] = pipeline.TreeAttention(dt, case["B"], case["n"], Hq, H, D, case["M"],
                                                t["max_pages"], case["page"], DEV)
    return st


# ------------------------------------------------------------ the plain form

def _angles(pos, D):
    i = torch.arange(D // 2, device=DEV, dtype=torch.float64)
    th = pos.double()[:, None] * BASE ** (-2.0 * i / D)
    return th.cos().float()[:, None, :], th.sin().float()[:, None, :]


def _rotate(x, c, s):
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _norm_back(x, w, c, s, dy):
    x, w, dy = x.float(), w.float(), dy.float()
    dz = _rotate(dy, c, -s)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    g = dz * w
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (dz * xh).double().sum((0, 1)).float()


def _plain_append(st):
    c, s = _angles(st["pos"], st["case"]["D"])
    page = st["case"]["page"]
    t = torch.arange(st["n_tok"], device=DEV)
    seq = torch.searchsorted(st["off"][1:], t, right=True)
    slot = st["lens"].long()[seq] + t - st["off"][seq]
    pg = st["table"].long()[seq, slot // page]
    k = _rotate(_norm(st["k"], st["wk"]), c, s)
    st["kp"][pg, :, slot % page] = k.to(st["kp"].dtype)
    st["vp"][pg, :, slot % page] = st["v"]
    out = [st["kp"], st["vp"]]
    if st["q"] is not None:
        out.append(_rotate(_norm(st["q"], st["wq"]), c, s).to(st["q"].dtype))
    return out


def _plain_tree(st):
    """Padded to the longest sequence: scores over every key, a mask, one
    softmax, one product."""
    case = st["case"]
    B, n, H, D, page = case["B"], case["n"], case["H"], case["D"], case["page"]
    G, M = case["Hq"] // H, case["M"]
    off, lens, nt = st["off"], st["lens"].long(), st["n_tok"]
    cnt = off[1:] - off[:-1]
    i = torch.arange(n, device=DEV)
    live = i[None] < cnt[:, None]                                    # [B][n]
    tok = torch.clamp(off[:-1, None] + i, max=nt - 1)
    q = st["q"].float()[tok].view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    kc = st["kp"][st["table"].long()].permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    vc = st["vp"][st["table"].long()].permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    # ancestors: every token sees itself and what its parent sees
    par = torch.where(live, st["parents"].long()[tok], -1)
    anc = torch.eye(n, dtype=torch.bool, device=DEV).expand(B, n, n).clone()
    up = par
    hop = torch.zeros_like(anc)
    for _ in range(max(1, math.ceil(math.log2(max(n, 2))))):
        hop = torch.gather(anc, 1, up.clamp(min=0)[:, :, None].expand(B, n, n))
        anc = anc | (hop & (up >= 0)[:, :, None])
        up = torch.where(up >= 0, torch.gather(up, 1, up.clamp(min=0)), up)
    key = torch.arange(kc.shape[2], device=DEV)
    rel = key[None] - lens[:, None]                                  # [B][keys]
    see = torch.gather(anc, 2, rel.clamp(0, n - 1)[:, None].expand(B, n, -1))
    see = torch.where((rel < 0)[:, None], True, see & ((rel >= 0) & (rel < cnt[:, None]))[:, None])
    if M:
        kc = torch.cat((st["km"].permute(0, 2, 1, 3), kc), 2)
        vc = torch.cat((st["vm"].permute(0, 2, 1, 3), vc), 2)
        mem = torch.arange(M, device=DEV)[None] < st["mems"][:, None]
        see = torch.cat((mem[:, None].expand(B, n, M), see), 2)
    sc = torch.matmul(q, kc.float().transpose(-1, -2)) * (D ** -0.5)
    sc = sc.view(B, H, n, G, -1).masked_fill(~see[:, None, :, None], float("-inf"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, H, n * G, -1)
    o = torch.matmul(p, vc.float()).view(B, H, n, G, D).permute(0, 2, 1, 3, 4)
    return o.reshape(B, n, H * G, D)[live].to(st["q"].dtype)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        if op == "norm":
            return list(st["call"](st["q"], st["k"], st["pos"], st["wq"], st["wk"], eps=EPS,
                                   rope_base=BASE))
        if op == "norm_back":
            return list(st["call"](st["q"], st["k"], st["pos"], st["dq"], st["dk"], st["wq"],
                                   st["wk"], eps=EPS, rope_base=BASE, ws=st["ws"]))
        if op == "append":
            c = st["cache"]
            qo = c.append(st["k"], st["v"], st["off"], st["pos"], k_weight=st["wk"], q=st["q"],
                          q_weight=st["wq"], eps=EPS, rope_base=BASE)
            return [c.k_pages, c.v_pages] + ([] if qo is None else [qo])
        return st["call"](st["q"], st["off"], st["cache"], parents=st["parents"], k_mem=st["km"],
                          v_mem=st["vm"], mem_len=st["mems"])
    if op == "norm":
        c, s = _angles(st["pos"], case["D"])
        return [_rotate(_norm(st[x], st["w" + x]), c, s).to(st[x].dtype) for x in ("q", "k")]
    if op == "norm_back":
        c, s = _angles(st["pos"], case["D"])
        dq, dwq = _norm_back(st["q"], st["wq"], c, s, st["dq"])
        dk, dwk = _norm_back(st["k"], st["wk"], c, s, st["dk"])
        return [dq.to(st["dq"].dtype), dk.to(st["dk"].dtype), dwq, dwk]
    if op == "append":
        return _plain_append(st)
    return _plain_tree(st)


# ------------------------------------------------- the definition in 64 bits

def _turn(x, pos):
    """x [n][heads][D] turned by its positions: dims i and i + D/2 as one
    complex number times e^{i p base^(-2i/D)}."""
    D = x.shape[-1]
    f = torch.pow(torch.tensor(BASE, dtype=torch.float64, device=DEV),
                  -torch.arange(0, D, 2, dtype=torch.float64, device=DEV) / D)
    z = torch.complex(x[..., :D // 2], x[..., D // 2:])
    z = z * torch.polar(torch.ones_like(f), pos.double()[:, None] * f)[:, None]
    return torch.cat((z.real, z.imag), -1)


def _unit(x, w):
    if w is None:
        return x
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "norm":
        return [_turn(_unit(d(st[x]), d(st["w" + x])), st["pos"]) for x in ("q", "k")]
    if case["op"] == "norm_back":
        dxs, dws = [], []
        for x in ("q", "k"):
            xi = d(st[x]).requires_grad_(True)
            wi = d(st["w" + x]).requires_grad_(True)
            y = _turn(_unit(xi, wi), st["pos"])
            dx, dw = torch.autograd.grad(y, (xi, wi), d(st["d" + x]))
            dxs.append(dx)
            dws.append(dw)
        return dxs + dws
    off = st["off"].tolist()
    page, table, lens = case["page"], st["table"].tolist(), st["lens"].tolist()
    if case["op"] == "append":
        kp, vp = d(st["kp"]), d(st["vp"])
        k, v = _turn(_unit(d(st["k"]), d(st["wk"])), st["pos"]), d(st["v"])
        for b in range(case["B"]):
            t, slot = off[b], lens[b]
            while t < off[b + 1]:  # page by page
                row = slot % page
                m = min(page - row, off[b + 1] - t)
                pg = table[b][slot // page]
                kp[pg, :, row:row + m] = k[t:t + m].transpose(0, 1)
                vp[pg, :, row:row + m] = v[t:t + m].transpose(0, 1)
                t, slot = t + m, slot + m
        out = [kp, vp]
        if st["q"] is not None:
            out.append(_turn(_unit(d(st["q"]), d(st["wq"])), st["pos"]))
        return out
    H, D, G = case["H"], case["D"], case["Hq"] // case["H"]
    parents, mems = st["parents"].tolist(), st["mems"].tolist()
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        n, L, M = off[b + 1] - off[b], lens[b], mems[b]
        ids = torch.tensor(table[b][:(L + n + page - 1) // page], device=DEV)
        ks = st["kp"][ids].transpose(0, 1).reshape(H, -1, D)[:, :L + n]
        vs = st["vp"][ids].transpose(0, 1).reshape(H, -1, D)[:, :L + n]
        sees = [[False] * n for _ in range(n)]
        for i in range(n):
            a = i
            while a >= 0:
                sees[i][a] = True
                a = parents[off[b] + a]
        tree = torch.tensor(sees, device=DEV)
        for g in range(H):  # one KV head at a time
            kk, vv = ks[g].double(), vs[g].double()
            q = st["q"][off[b]:off[b + 1], g * G:(g + 1) * G].double()
            if M:
                kk = torch.cat((st["km"][b, :M, g].double(), kk))
                vv = torch.cat((st["vm"][b, :M, g].double(), vv))
            s = torch.einsum("tgd,jd->tgj", q, kk) / math.sqrt(D)
            s[:, :, M + L:] = torch.where(tree[:, None], s[:, :, M + L:],
                                          torch.full_like(s[:, :, M + L:], -math.inf))
            out[off[b]:off[b + 1], g * G:(g + 1) * G] = torch.einsum(
                "tgj,jd->tgd", torch.softmax(s, -1), vv)
    return out
