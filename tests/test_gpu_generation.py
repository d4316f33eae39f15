"""GPU parity of the generation operators (per-head norms with RoPE and their
gradient, the paged append, attention for drafted trees, and a run of them
together) against the float64 oracle.

Tolerances count roundings: U = 2^-24 is half a step of fp32, and a value
rounded to bf16 moves by at most 2^-8 of itself.

* Norms: the mean of D <= 128 squares by at most 16 chained additions and 5
  of a shuffle tree, halved by the root, rsqrt (2 steps), and three products:
  below 16 U of |z|.  The rotation mixes two components with (cos, sin) of an
  angle good to 1e-7 rad (2 U) and three roundings.  Together 24 U of
  |z_1| + |z_2|; far positions add the float64 oracle's own angle, p 2^-52.
* Gradients: the same per term; dx subtracts two such terms, so the bound is
  on the sum of their magnitudes.  A weight's gradient adds, in a lane, one
  product per head of each of its tokens (at most n / 1024 + 1 of them), then
  a few fixed trees.
* Attention, with A = sum_j p_j |v_j| and S = the largest scale sum |q k|: a
  score is off by (D + 4) U S, which moves a normalised weight by twice that;
  the sums over N keys by N U; bf16 weights move the output by 2^-8 A.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from latent_memory_routing_b200 import msa, pipeline

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from latent_memory_routing_b200 import build
    build.build()
    msa.lib()
    msa.msa_device_status(clear=True)
    yield
    torch.cuda.synchronize()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def status(want=0):
    torch.cuda.synchronize()
    assert msa.msa_device_status(clear=True) == want


def rnd(shape, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).to(dt)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def i64(x):
    return torch.tensor(x, dtype=torch.int64, device="cuda")


def step_of(dt):
    return BF if dt == BF16 else U


def close(got, want, tol):
    bad = np.abs(f64(got) - want) - tol
    assert not np.any(~(bad <= 0)), float(np.nanmax(bad))


def fused(n, Hq, H, D, dt, seed):
    """q, k, v as slices of one projection's output with a gap behind them."""
    x = rnd((n, (Hq + 2 * H) * D + 16), dt, seed)
    cut = [x[:, a * D:b * D].unflatten(1, (b - a, D)) if b > a else None
           for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H))]
    return x, cut


# ----------------------------------------------------------- norms and RoPE

NORMS = [  # dt, n, Hq, H, D, weights, positions
    (F32, 1, 4, 2, 64, "qk", "near"),
    (BF16, 1, 32, 8, 128, "qk", "near"),
    (F32, 37, 5, 1, 128, "qk", "far"),
    (BF16, 300, 3, 3, 64, "qk", "negative"),
    (BF16, 2000, 7, 2, 128, "q", "near"),
    (BF16, 5, 1, 0, 64, "qk", "far"),
    (F32, 5, 0, 3, 64, "k", "near"),
    (BF16, 130, 8, 2, 128, "qk", None),
    (F32, 33, 2, 1, 64, "", "near"),
    (BF16, 33, 64, 1, 64, "", "far"),
    (BF16, 5000, 4, 1, 128, "qk", "near"),
]


def norm_inputs(dt, n, Hq, H, D, weights, positions, seed):
    base, (q, k, _) = fused(n, Hq, H, D, dt, seed)
    w = rnd((2, D), dt, seed + 1) * 0.2 + 1
    wq, wk = (w[0] if "q" in weights else None), (w[1] if "k" in weights else None)
    pos = {None: None, "near": i32(np.arange(16, 16 + n)),
           "far": i32(2 ** 31 - 1 - 77777 * np.arange(n)),
           "negative": i32(-3 * np.arange(n) - 1)}[positions]
    return base, q, k, wq, wk, pos


def norm_tol(x, w, pos):
    """The bound of one forward output before its last rounding."""
    z = np.abs(oracle.head_norm(f64(x), f64(w), 1e-6))
    half = z.shape[-1] // 2
    z = np.concatenate([z[..., :half] + z[..., half:]] * 2, axis=-1)
    far = 0.0 if pos is None else float(np.abs(f64(pos)).max()) * 2.0 ** -52
    return z * (24 * U + far)


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_norm_rope(case):
    dt = case[0]
    _, q, k, wq, wk, pos = norm_inputs(*case, seed=3)
    got = pipeline.qk_norm_rope(q, k, pos, wq, wk)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        if x is None:
            assert y is None
            continue
        want = oracle.norm_rope(f64(x), f64(w), None if pos is None else pos.cpu().numpy())
        close(y, want, norm_tol(x, w, pos) * (1 + BF) + step_of(dt) * np.abs(want))
    status()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_an_infinite_element_stays_where_it_is_without_positions(dt, D):
    """r = 0 makes it NaN and the others 0; in a tensor that is neither normed
    nor rotated nothing changes."""
    q, k = rnd((7, 3, D), dt, 1), rnd((7, 2, D), dt, 2)
    at = [(0, 0, 0), (3, 2, D // 2), (6, 1, D - 1), (5, 0, 5)]
    for i, (t, h, d) in enumerate(at):
        q[t, h, d] = float("inf") * (-1) ** i
    k[4, 1, 9] = float("inf")
    w = rnd((D,), dt, 3) * 0.2 + 1
    yq, yk = pipeline.qk_norm_rope(q, k, None, w, None)
    assert torch.equal(yk, k)
    with np.errstate(invalid="ignore"):
        want = oracle.norm_rope(f64(q), f64(w), None)
    assert np.isnan(want).sum() == len(at)
    assert np.array_equal(np.isnan(f64(yq)), np.isnan(want))
    for t, h, _ in at:
        assert bool((yq[t, h] == 0).sum() == D - 1)
    # the gradient of such a row: as the formula's, element by element
    dy = rnd((7, 3, D), dt, 4)
    dq = pipeline.qk_norm_rope_backward(q, None, None, dy, None, w)[0]
    rows = torch.zeros((7, 3), dtype=torch.bool, device="cuda")
    for t, h, _ in at:
        rows[t, h] = True
    assert not bool(dq[~rows].isnan().any())
    status()


def test_norm_rope_in_place_is_the_same_bits():
    q, k = rnd((77, 6, 64), BF16, 1), rnd((77, 2, 64), BF16, 2)
    w, pos = rnd((64,), BF16, 3), i32(np.arange(77))
    want = pipeline.qk_norm_rope(q, k, pos, w, w)
    pipeline.qk_norm_rope(q, k, pos, w, w, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    status()


def test_norm_rope_of_nothing_writes_nothing():
    q = torch.empty((0, 4, 64), device="cuda")
    got = pipeline.qk_norm_rope(q, None, i32([]), rnd((64,), F32, 0))
    assert got[0].shape == (0, 4, 64) and got[1] is None
    w = torch.ones(64, device="cuda")
    _, _, dw, _ = pipeline.qk_norm_rope_backward(q, None, i32([]), q, None, w)
    assert torch.equal(dw, torch.zeros(64, device="cuda"))
    status()


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(x) for x in c[1:]))
@pytest.mark.parametrize("grad", [F32, BF16], ids=["f32", "bf16"])
def test_norm_rope_backward(case, grad):
    dt, n, Hq, H, D = case[:5]
    if dt == F32 and grad == BF16:
        pytest.skip("bf16 gradients need bf16 inputs")
    _, q, k, wq, wk, pos = norm_inputs(*case, seed=5)
    dq_out, dk_out = (rnd((n, h, D), grad, 7 + h) if h else None for h in (Hq, H))
    # dq and dk are slices of the projection's gradient; the gap stays
    base, (dq, dk, _) = fused(n, Hq, H, D, grad, 11)
    before = base.clone()
    dwq, dwk = (None if w is None or x is None else torch.full((D,), NAN, device="cuda")
                for x, w in ((q, wq), (k, wk)))
    pipeline.qk_norm_rope_backward(q, k, pos, dq_out, dk_out, wq, wk, out=(dq, dk, dwq, dwk))
    p = None if pos is None else pos.cpu().numpy()
    far = 0.0 if pos is None else float(np.abs(f64(pos)).max()) * 2.0 ** -52
    for x, w, dy, dx, dw in ((q, wq, dq_out, dq, dwq), (k, wk, dk_out, dk, dwk)):
        if x is None:
            continue
        want, wantw = oracle.norm_rope_backward(f64(x), f64(w), p, f64(dy))
        half = D // 2
        a = np.abs(f64(dy))
        a = np.concatenate([a[..., :half] + a[..., half:]] * 2, axis=-1)  # bounds |dz|
        rel = 40 * U + far
        if w is None:
            tol = a * rel
        else:
            xh = np.abs(oracle.head_norm(f64(x), np.ones(D), 1e-6))
            r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
            g = a * np.abs(f64(w))
            tol = r * (g + xh * (g * xh).mean(-1, keepdims=True)) * rel
            chain = x.shape[1] * (n // 1024 + 1) + 40
            close(dw, wantw, (a * xh).sum((0, 1)) * (rel + chain * U))
        close(dx, want, tol * (1 + BF) + step_of(grad) * np.abs(want))
    edge = (Hq + H) * D  # v's columns and the gap behind them
    assert torch.equal(base[:, edge:], before[:, edge:])
    status()


def test_norm_rope_backward_repeats_bit_for_bit():
    _, q, k, wq, wk, pos = norm_inputs(BF16, 3001, 8, 2, 128, "qk", "near", seed=1)
    dq, dk = rnd((3001, 8, 128), BF16, 2), rnd((3001, 2, 128), BF16, 3)
    a = pipeline.qk_norm_rope_backward(q, k, pos, dq, dk, wq, wk)
    for _ in range(10):
        b = pipeline.qk_norm_rope_backward(q, k, pos, dq, dk, wq, wk)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    status()


def test_a_training_steps_gradients_join_in_one_projection():
    """qk_norm_rope and its backward as an autograd step would chain them:
    the gradient of sum(y * c) against central differences of the operator's
    own float64 definition, through one projection's output."""
    n, Hq, H, D = 6, 4, 2, 64
    base, (q, k, _) = fused(n, Hq, H, D, F32, 21)
    w, pos = rnd((D,), F32, 22), i32(np.arange(9, 9 + n))
    cq, ck = rnd((n, Hq, D), F32, 23), rnd((n, H, D), F32, 24)
    yq, yk = pipeline.qk_norm_rope(q, k, pos, w, w)
    dq, dk, dwq, dwk = pipeline.qk_norm_rope_backward(q, k, pos, cq, ck, w, w)
    r = np.random.default_rng(0)
    eq, ek, ew = r.normal(size=(n, Hq, D)), r.normal(size=(n, H, D)), r.normal(size=D)
    h, p = 1e-5, pos.cpu().numpy()

    def loss(s):
        return sum(float((oracle.norm_rope(f64(x) + s * e, f64(w) + s * ew, p) * f64(c)).sum())
                   for x, e, c in ((q, eq, cq), (k, ek, ck)))

    want = (loss(h) - loss(-h)) / (2 * h)
    got = sum(float((f64(a) * b).sum()) for a, b in ((dq, eq), (dk, ek), (dwq, ew), (dwk, ew)))
    size = sum(float(np.abs(f64(a) * b).sum()) for a, b in ((dq, eq), (dk, ek), (dwq, ew),
                                                            (dwk, ew)))
    # fp32 gradients (100 U of each term) and the differences' h^2 term, whose
    # third derivative is of the size of the terms themselves
    assert abs(got - want) <= size * (100 * U + 100 * h * h)
    status()


# -------------------------------------------------------------- paged append

def paged(B, H, D, dt, page, need, seed, extra=3):
    """A cache whose sequences own shuffled pages for `need` rows each; every
    row holds NaN."""
    pages = [-(-n // page) for n in need]
    max_pages = max(1, max(pages))
    c = pipeline.PagedCache(dt, sum(pages) + extra, page, H, D, B, max_pages, "cuda")
    c.k_pages.fill_(NAN)
    c.v_pages.fill_(NAN)
    ids = np.random.default_rng(seed).permutation(c.n_pages)
    at = 0
    for b, n in enumerate(pages):
        if n:
            c.block_table[b, :n] = i32(ids[at:at + n])
        at += n
    return c


def rows_of(c, b, rows):
    at = oracle.paged_rows(b, rows, c.block_table.cpu().numpy(), c.page_size)
    return (torch.tensor([p for p, _ in at], dtype=torch.int64, device="cuda"),
            torch.tensor([r for _, r in at], dtype=torch.int64, device="cuda"))


APPENDS = [  # dt, page, Hq, H, D, lens, tokens, weights, lead
    (BF16, 64, 32, 8, 128, [0, 63, 64, 2047], [1, 1, 1, 1], "qk", 0),
    (F32, 16, 4, 2, 64, [0, 5, 117, 15], [13, 0, 33, 1], "qk", 0),
    (BF16, 16, 0, 1, 64, [31], [300], "k", 0),
    (BF16, 128, 5, 1, 128, [0, 127], [129, 257], "", 3),
    (F32, 32, 0, 3, 128, [7, 0, 0], [0, 0, 90], "", 2),
    (BF16, 32, 64, 2, 64, [0] * 40, [3] * 40, "qk", 1),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"{c[1]}-{c[2]}-{c[3]}-{c[4]}-{c[7]}")
def test_paged_append(case):
    dt, page, Hq, H, D, lens, toks, weights, lead = case
    B = len(lens)
    c = paged(B, H, D, dt, page, [a + b for a, b in zip(lens, toks)], 1)
    c.cache_len.copy_(i32(lens))
    off = lead + np.concatenate([[0], np.cumsum(toks)])
    n = int(off[-1]) + lead  # `lead` padding tokens on either side
    _, (q, k, v) = fused(n, Hq, H, D, dt, 2)
    w = rnd((2, D), dt, 3) * 0.2 + 1
    wq, wk = (w[0] if "q" in weights else None), (w[1] if "k" in weights else None)
    pos = i32(np.random.default_rng(4).integers(-5, 100000, n))
    q_out = None if q is None else torch.full((n, Hq, D), NAN, dtype=dt, device="cuda")
    got = c.append(k, v, i64(off), pos, wk, q, wq, q_out=q_out)
    p = pos.cpu().numpy()
    want = oracle.norm_rope(f64(k), f64(wk), p)
    tol = norm_tol(k, wk, pos) * (1 + BF) + step_of(dt) * np.abs(want)
    left = torch.ones(c.k_pages.shape[:3:2], dtype=torch.bool, device="cuda")
    for b in range(B):
        pg, row = rows_of(c, b, range(lens[b], lens[b] + toks[b]))
        t = slice(int(off[b]), int(off[b + 1]))
        close(c.k_pages[pg, :, row], want[t], tol[t])
        assert torch.equal(c.v_pages[pg, :, row], v[t])
        left[pg, row] = False
    left = left[:, None].expand(-1, H, -1)
    assert bool(c.k_pages[left].isnan().all()) and bool(c.v_pages[left].isnan().all())
    assert c.cache_len.tolist() == lens
    if q is not None:
        assert got is q_out
        wantq = oracle.norm_rope(f64(q), f64(wq), p)
        tolq = norm_tol(q, wq, pos) * (1 + BF) + step_of(dt) * np.abs(wantq)
        live = slice(int(off[0]), int(off[-1]))
        close(q_out[live], wantq[live], tolq[live])
        assert bool(q_out[:int(off[0])].isnan().all()) and bool(q_out[int(off[-1]):].isnan().all())
    status()


@pytest.mark.parametrize("what,code", [("page", -1), ("minus", -1), ("length", -1), ("full", -3)])
def test_append_skips_rows_it_cannot_place(what, code):
    c = paged(2, 2, 64, F32, 16, [32, 32], 5)
    if what == "page":
        c.block_table[1, 1] = c.n_pages
    if what == "minus":
        c.block_table[1, 1] = -1
    c.cache_len.copy_(i32([0, {"length": -2}.get(what, 31 if what == "full" else 15)]))
    k, v = rnd((6, 2, 64), F32, 6), rnd((6, 2, 64), F32, 7)
    # sequence 1 appends four rows, of which all, all, two or three have no place
    c.append(k, v, i64([0, 2, 6]), i32(np.arange(6)))
    status(code)
    pg, row = rows_of(c, 0, [0, 1])
    assert torch.equal(c.v_pages[pg, :, row], v[:2])
    written = int((~c.v_pages.isnan()).all(-1).all(1).sum())
    assert written == 2 + {"page": 1, "minus": 1, "length": 2, "full": 1}[what]


def test_a_negative_length_keeps_to_its_own_sequence():
    """Rows -2 and -1 have no place, rows 0 and 1 do, and the call reports it."""
    c = paged(3, 2, 64, F32, 16, [16, 16, 16], 5)
    c.cache_len.copy_(i32([3, -2, 0]))
    x = rnd((6, 2, 64), F32, 6)
    c.append(x, x, i64([0, 1, 5, 6]), i32(np.arange(6)))
    status(-1)
    want = torch.full_like(c.v_pages, NAN)
    for b, row, t in ((0, 3, 0), (1, 0, 3), (1, 1, 4), (2, 0, 5)):
        want[c.block_table[b, 0], :, row] = x[t]
    assert torch.equal(c.v_pages.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("case", ["past_the_reserved", "never_reserved", "released"])
def test_append_without_a_page_leaves_the_other_sequences_alone(case):
    """The rows of sequence 0, some of them on pages that sequence 1 had."""
    c = pipeline.PagedCache(F32, 6, 16, 2, 64, 2, 3, "cuda")
    c.k_pages.fill_(NAN)
    c.v_pages.fill_(NAN)
    if case == "released":
        c.reserve(1, 40)
        c.release(1)
    elif case == "past_the_reserved":
        c.reserve(1, 16)
    c.reserve(0, 48)
    k, v = rnd((48, 2, 64), F32, 1), rnd((48, 2, 64), F32, 2)
    c.append(k, v, i64([0, 48, 48]), i32(np.arange(48)))
    status()
    c.cache_len.copy_(i32([48, 15 if case == "past_the_reserved" else 0]))
    before = [p.clone() for p in (c.k_pages, c.v_pages)]
    new = rnd((3, 2, 64), F32, 3)
    c.append(new, new, i64([0, 0, 3]), i32(np.arange(3)))
    status(-1)
    if case == "past_the_reserved":       # its one row with a place
        pg = c.owned[1][0]
        assert torch.equal(c.v_pages[pg, :, 15], new[0])
        for p, b in zip((c.k_pages, c.v_pages), before):
            p[pg, :, 15] = b[pg, :, 15]
    assert all(torch.equal(p.view(torch.int32), b.view(torch.int32))
               for p, b in zip((c.k_pages, c.v_pages), before))


def test_two_tokens_of_a_sequence_cross_a_page():
    c = paged(1, 1, 64, BF16, 16, [48], 9)
    c.cache_len.fill_(15)
    k = rnd((2, 1, 64), BF16, 1)
    c.append(k, k, i64([0, 2]), i32([0, 0]))
    tab = c.block_table[0].tolist()
    assert torch.equal(c.v_pages[tab[0], 0, 15], k[0, 0])
    assert torch.equal(c.v_pages[tab[1], 0, 0], k[1, 0])
    status()


# ------------------------------------------------------------ tree attention

def tree_case(dt, page, Hq, H, D, lens, toks, mem, tree, seed=0, lead=0):
    """A filled cache, memory and queries; rows that no sequence owns, rows
    behind a sequence's last, and memory rows behind mem_len hold NaN."""
    B = len(lens)
    c = paged(B, H, D, dt, page, [a + b for a, b in zip(lens, toks)], seed)
    c.cache_len.copy_(i32(lens))
    for b in range(B):
        m = lens[b] + toks[b]
        pg, row = rows_of(c, b, range(m))
        c.k_pages[pg, :, row] = rnd((m, H, D), dt, seed + 10 * b + 1)
        c.v_pages[pg, :, row] = rnd((m, H, D), dt, seed + 10 * b + 2)
    off = lead + np.concatenate([[0], np.cumsum(toks)])
    n = int(off[-1]) + lead
    q = rnd((n, Hq, D), dt, seed + 3)
    m_cap = max(mem) if mem else 0
    km = vm = ml = None
    if mem:
        km, vm = rnd((B, m_cap, H, D), dt, seed + 4), rnd((B, m_cap, H, D), dt, seed + 5)
        for b, m in enumerate(mem):
            km[b, m:], vm[b, m:] = NAN, NAN
        ml = i32(mem)
    r = np.random.default_rng(seed + 6)
    parents = None
    if tree != "chain":
        parents = np.full(n, -1)
        for b in range(B):
            for i in range(toks[b]):
                p = int(r.integers(max(-1, i - 5), i)) if tree != "roots" else -1
                if tree == "pruned" and r.random() < 0.2:
                    p = -2
                parents[off[b] + i] = p
        parents = i32(parents)
    return c, q, i64(off), parents, km, vm, ml, m_cap


def run_tree(case, n_max, scale=0.0, **kw):
    c, q, off, parents, km, vm, ml, m_cap = case
    att = pipeline.TreeAttention(q.dtype, c.B, n_max, q.shape[1], c.H, c.D, m_cap, c.max_pages,
                                 c.page_size, "cuda")
    att.ws.view(torch.uint8).fill_(0xFF)
    out = torch.full_like(q, NAN)
    att(q, off, c, parents, km, vm, ml, scale, out, **kw)
    return out


def expected(case, scale=0.0):
    """The oracle's output and the bound on an output's distance from it."""
    c, q, off, parents, km, vm, ml, m_cap = case
    o = off.cpu().numpy()
    par = None if parents is None else parents.cpu().numpy()
    want, bound, top = oracle.tree_attn(
        f64(q), o, par, f64(km), f64(vm), None if ml is None else ml.cpu().numpy(),
        f64(c.k_pages), f64(c.v_pages), c.block_table.cpu().numpy(), c.cache_len.cpu().numpy(),
        scale)
    keys = m_cap + int((c.cache_len.long() + off[1:] - off[:-1]).max())
    D = q.shape[2]
    tol = bound * U * (2 * (D + 4) * top[..., None] + 2 * keys + 64)
    if q.dtype == BF16:
        tol = tol + BF * bound + BF * np.abs(want)
    return want, tol


def check_tree(case, out, scale=0.0):
    o = case[2].cpu().numpy()
    want, tol = expected(case, scale)
    live = slice(int(o[0]), int(o[-1]))
    close(out[live], want[live], tol[live])
    # rows of no sequence are left as they were
    assert bool(out[:int(o[0])].isnan().all()) and bool(out[int(o[-1]):].isnan().all())


TREES = [  # dt, page, Hq, H, D, lens, tokens, memory rows, tree, n_max
    (F32, 16, 4, 2, 64, [300, 0, 17], [16, 1, 5], [6, 0, 3], "tree", 16),
    (F32, 32, 3, 3, 128, [0, 31, 32], [1, 1, 1], [], "chain", 1),
    (F32, 128, 16, 1, 64, [1000], [128], [130], "pruned", 128),
    (F32, 64, 5, 1, 128, [0, 0], [7, 0], [], "roots", 9),
    (BF16, 64, 32, 8, 128, [2047, 1, 0, 63, 64, 128], [1] * 6, [220, 0, 1, 128, 129, 7],
     "chain", 1),
    (BF16, 64, 8, 2, 128, [517, 130], [48, 3], [220, 5], "tree", 48),
    (BF16, 16, 4, 4, 64, [100, 0, 16, 15], [17, 2, 16, 1], [], "tree", 17),
    (BF16, 16, 16, 1, 128, [255, 256, 257], [1, 1, 1], [], "chain", 1),
    (BF16, 32, 6, 2, 128, [1000, 40], [30, 43], [44, 0], "pruned", 64),
    (BF16, 128, 5, 1, 64, [390, 0], [64, 33], [], "roots", 64),
    (BF16, 64, 2, 1, 128, [3000], [128], [700], "tree", 128),
    (BF16, 128, 16, 1, 128, [700], [128], [128], "chain", 128),
    (BF16, 32, 13, 1, 64, [0, 0, 0], [1, 2, 128], [], "tree", 128),
    (BF16, 64, 15, 5, 64, [4095], [1], [1], "chain", 1),
    (BF16, 64, 40, 8, 64, [9, 1200], [2, 1], [0, 31], "chain", 4),
    (BF16, 16, 1, 1, 128, [20000], [1], [], "chain", 1),
    (BF16, 128, 3, 1, 128, [20000], [20], [64], "tree", 20),
    (BF16, 64, 4, 2, 128, [0, 200, 0], [0, 40, 0], [0, 0, 0], "chain", 40),
]


@pytest.mark.parametrize("case", TREES,
                         ids=lambda c: f"{'f32' if c[0] == F32 else 'bf16'}-{c[1]}-{c[2]}-{c[3]}-"
                         f"{c[4]}-{max(c[5])}-{max(c[6])}-{c[8]}")
def test_tree_attention(case):
    dt, page, Hq, H, D, lens, toks, mem, tree, n_max = case
    t = tree_case(dt, page, Hq, H, D, lens, toks, mem, tree, seed=len(lens) + n_max)
    check_tree(t, run_tree(t, n_max))
    status()


@pytest.mark.parametrize("dt,Hq,n", [(F32, 2, 2), (BF16, 2, 2), (BF16, 1, 18), (BF16, 8, 17)],
                         ids=["f32", "bf16", "bf16-18rows", "bf16-136rows"])
def test_many_short_sequences(dt, Hq, n):
    """More sequences than a CTA has threads, many of them without tokens."""
    B = 700
    r = np.random.default_rng(5)
    toks = [int(x) for x in r.integers(0, n + 1, B)]
    lens = [int(x) for x in r.integers(0, 40, B)]
    toks[17], lens[17] = n, 200
    t = tree_case(dt, 16, Hq, 1, 64, lens, toks, [], "chain", seed=1)
    check_tree(t, run_tree(t, n))
    status()


@pytest.mark.parametrize("lens,toks,H", [
    ([3] * 33, [6] * 33, 2), ([1, 0, 90, 7, 33, 5], [3] * 6, 4), ([130], [2], 1),
    ([2000], [1], 1), ([4100, 5], [1, 4], 2), ([20000], [1], 1)])
def test_few_rows_over_short_and_long_items(lens, toks, H):
    """Items kept whole, and cut into ranges of one slice and of more."""
    t = tree_case(BF16, 16, 2 * H, H, 64, lens, toks, [], "chain", seed=3)
    check_tree(t, run_tree(t, max(toks)))
    status()


@pytest.mark.parametrize("dt,Hq,H,D,lens,toks,mem,tree,n_max", [
    (F32, 16, 1, 64, [(i * 37) % 211 for i in range(300)], [i % 9 for i in range(300)], [], "tree",
     8),
    (F32, 16, 1, 64, [700, 0], [128, 77], [3, 0], "pruned", 128),
    (F32, 16, 4, 128, [0] * 8, [64] * 8, [], "chain", 64),
    (F32, 16, 8, 128, [3000] * 4, [0] * 4, [], "chain", 16),
    (F32, 4, 1, 64, [9000] + [1] * 60, [3] + [4] * 60, [0] * 60 + [50], "roots", 4),
    (BF16, 16, 4, 128, [9000] + [1] * 60, [3] + [4] * 60, [0] * 60 + [50], "roots", 4),
    (BF16, 16, 4, 128, [9000] + [1] * 60, [33] + [4] * 60, [0] * 60 + [50], "tree", 48),
    (BF16, 2, 1, 64, [4, 0], [0, 0], [], "chain", 1),
    (BF16, 1, 1, 64, [i % 3 for i in range(1000)], [i % 2 for i in range(1000)], [], "chain", 1)])
def test_unlike_and_empty_sequences(dt, Hq, H, D, lens, toks, mem, tree, n_max):
    t = tree_case(dt, 16, Hq, H, D, lens, toks, mem, tree, seed=1, lead=2)
    check_tree(t, run_tree(t, n_max))
    status()


@pytest.mark.parametrize("page,Hq,H,lens,toks,mem,tree,n_max", [
    (64, 8, 2, [18500] + [300, 0, 129] * 4, [64, 33, 1, 20] * 3 + [64], [], "tree", 64),
    (16, 14, 2, [9400, 12] * 10, [32, 31] * 10, [100, 0] * 10, "pruned", 32),
    (128, 16, 1, [70000, 0, 250, 2, 1], [128, 128, 17, 5, 0], [], "chain", 128)])
def test_two_query_tiles_share_a_pass(page, Hq, H, lens, toks, mem, tree, n_max):
    """More than 192 rows a KV head and room for more keys than the L2 keeps,
    most of it unused."""
    t = tree_case(BF16, page, Hq, H, 128, lens, toks, mem, tree, seed=19, lead=2)
    out = run_tree(t, n_max)
    check_tree(t, out)
    assert torch.equal(out.view(torch.int16), run_tree(t, n_max).view(torch.int16))
    status()


@pytest.mark.parametrize("page,Hq,H,D,lens,toks,mem,tree,n_max", [
    (16, 4, 2, 64, [6100, 0, 17], [16, 1, 5], [6, 0, 3], "tree", 16),
    (32, 3, 3, 128, [40000, 31], [1, 1], [], "chain", 1),
    (128, 5, 1, 64, [20000], [4], [130], "pruned", 5),
    (64, 2, 2, 128, [5000, 12], [9, 17], [], "roots", 17),
    (16, 16, 1, 128, [3000, 2999, 7, 0], [2, 1, 2, 0], [5, 0, 0, 9], "tree", 2),
    (64, 8, 4, 64, [4000] * 3, [1, 3, 0], [], "chain", 8)])
def test_long_fp32_items(page, Hq, H, D, lens, toks, mem, tree, n_max):
    """One and two row tiles of 16, with padding tokens before and behind."""
    t = tree_case(F32, page, Hq, H, D, lens, toks, mem, tree, seed=7, lead=3)
    out = run_tree(t, n_max)
    check_tree(t, out)
    assert torch.equal(out.view(torch.int32), run_tree(t, n_max).view(torch.int32))
    status()


@pytest.mark.parametrize("Hq,H,D,lens,toks,mem,tree", [
    (32, 8, 128, [2047, 5, 0, 640], [1] * 4, [220, 0, 1, 16], "chain"),
    (8, 2, 64, [4000, 9], [4, 3], [], "tree"),
    (16, 1, 128, [9000], [1], [33], "chain")])
def test_few_rows_in_bf16_round_once(Hq, H, D, lens, toks, mem, tree):
    """Up to 16 rows a KV head: an output is rounded to bf16 (BF of itself) and
    what is behind it is exact to the fp32 terms of `expected` and to the two
    bf16 terms of a weight (each leaves at most BF of what it is to hold)."""
    t = tree_case(BF16, 16, Hq, H, D, lens, toks, mem, tree, seed=12)
    out = run_tree(t, max(toks))
    want, tol = expected(t)
    c, q, off, parents, km, vm, ml, _ = t
    _, bound, _ = oracle.tree_attn(
        f64(q), off.cpu().numpy(), None if parents is None else parents.cpu().numpy(), f64(km),
        f64(vm), None if ml is None else ml.cpu().numpy(), f64(c.k_pages), f64(c.v_pages),
        c.block_table.cpu().numpy(), c.cache_len.cpu().numpy())
    behind = tol - BF * bound - BF * np.abs(want) + BF * BF * bound
    close(out, want, behind * (1 + BF) + BF * np.abs(want))
    status()


@pytest.mark.parametrize("n_max", [1, 4, 5, 8, 9, 32, 33, 100, 128])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_row_counts_around_the_kernels_tiles(dt, n_max):
    """Four heads a group: 4 to 512 rows, in full and in part."""
    t = tree_case(dt, 32, 4, 1, 128, [190, 7, 0], [n_max, 1, max(1, n_max // 2)], [33, 1, 0],
                  "tree", seed=n_max)
    check_tree(t, run_tree(t, n_max))
    status()


def test_few_tokens_where_many_were_allowed():
    """n_max bounds the work; the tokens may be fewer."""
    t = tree_case(BF16, 64, 8, 2, 128, [500, 70], [2, 1], [9, 0], "tree", seed=3)
    for n_max in (2, 20, 128):
        check_tree(t, run_tree(t, n_max))
    status()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_padding_tokens_are_left_alone_and_scale_is_used(dt):
    t = tree_case(dt, 32, 8, 4, 64, [40, 3], [5, 9], [10, 2], "tree", seed=2, lead=4)
    check_tree(t, run_tree(t, 9, scale=0.31), scale=0.31)
    status()


@pytest.mark.parametrize("dt,D,n,rows", [(F32, 64, 12, 45), (F32, 64, 20, 45), (F32, 64, 8, 12005),
                                         (F32, 64, 16, 7001), (BF16, 64, 8, 45),
                                         (BF16, 64, 20, 45), (BF16, 128, 100, 45),
                                         (BF16, 128, 100, 150001)])
def test_unseen_non_finite_values_do_not_reach_a_row(dt, D, n, rows):
    """A drafted token's NaN or infinite K and V reach the rows that see it
    and no others."""
    t = tree_case(dt, 16, 4, 2, D, [rows], [n], [], "tree", seed=31)
    c, q, off, parents, *_ = t
    clean = run_tree(t, n)
    see = oracle.ancestors(parents.cpu().numpy())
    j = next(j for j in range(2, n) if 1 < see[:, j].sum() < n // 2)
    pg, row = rows_of(c, 0, [rows + j])
    for poison_k, value in ((False, NAN), (False, float("inf")), (True, NAN)):
        keep = (c.k_pages if poison_k else c.v_pages)[pg, :, row].clone()
        (c.k_pages if poison_k else c.v_pages)[pg, :, row, :9] = value
        out = run_tree(t, n)
        blind = torch.from_numpy(~see[:, j]).cuda()
        assert torch.equal(out[blind], clean[blind])
        hit = out[~blind] if poison_k else out[~blind][..., :9]
        if value == value:
            assert bool((hit == value).all())
        else:
            assert bool(hit.isnan().all())
        if not poison_k:
            assert torch.equal(out[~blind][..., 9:], clean[~blind][..., 9:])
        (c.k_pages if poison_k else c.v_pages)[pg, :, row] = keep
    status()


SEEN_INF = {
    "simt-f32": (F32, 64, [90, 7], [3, 1]),
    "few-f32": (F32, 128, [6000, 7], [4, 1]),
    "few-f32-64": (F32, 64, [9000, 0], [20, 1]),
    "few-bf16": (BF16, 128, [3000, 7], [3, 1]),
    "few-bf16-64": (BF16, 64, [90, 0], [1, 1]),
    "tc": (BF16, 128, [900, 7], [30, 1]),
    "tc-64": (BF16, 64, [3000, 0], [30, 1]),
}


@pytest.mark.parametrize("name", SEEN_INF)
def test_an_infinite_value_that_is_seen(name):
    """In a memory row, a cached row and a sequence's only drafted token: the
    column becomes that infinity, NaN where two of unlike signs meet, and no
    other column changes."""
    dt, D, lens, toks = SEEN_INF[name]
    t = tree_case(dt, 16, 4, 2, D, lens, toks, [33, 5], "roots", seed=14)
    c, q, off, parents, km, vm, ml, m_cap = t
    clean = run_tree(t, max(toks))
    inf = float("inf")
    vm[0, 7, 0, 3], vm[1, 4, 1, D - 1] = inf, -inf
    for b, row, g, d, x in ((0, 11, 0, 40, -inf), (0, lens[0] - 1, 1, 5, inf),
                            (0, 20, 1, 5, -inf), (1, lens[1], 0, 2, inf),
                            (1, lens[1], 1, D - 2, -inf)):
        pg, r = rows_of(c, b, [row])
        c.v_pages[pg, g, r, d] = x
    want, n0 = clean.clone(), toks[0]
    want[:n0, :2, 3], want[:n0, :2, 40], want[:n0, 2:, 5] = inf, -inf, NAN
    want[n0:, 2:, D - 1], want[n0:, :2, 2], want[n0:, 2:, D - 2] = -inf, inf, -inf
    assert torch.equal(run_tree(t, max(toks)).nan_to_num(nan=1e9, posinf=2e9, neginf=3e9),
                       want.nan_to_num(nan=1e9, posinf=2e9, neginf=3e9))
    status()


@pytest.mark.parametrize("name", SEEN_INF)
def test_an_infinite_key_that_is_seen(name):
    """The rows whose score it makes infinite become NaN, those whose score it
    makes -inf come out as without it, and one without an element there (0 times
    infinity) is NaN too."""
    dt, D, lens, toks = SEEN_INF[name]
    t = tree_case(dt, 16, 4, 2, D, lens, toks, [33, 5], "roots", seed=15)
    c, q, off, parents, km, vm, ml, m_cap = t
    n, rows = toks[0], []
    q[0, 1, 6] = 0                                 # heads 0, 1 read KV head 0
    q[0, 0, 6], q[0, 2, 9], q[0, 3, 9] = 0.5, -1, -1.3   # few bits: a rest of 0
    pg, r = rows_of(c, 0, [lens[0] - 1])
    key = c.k_pages[pg, :, r].clone()
    c.k_pages[pg, 0, r, 6], c.k_pages[pg, 1, r, 9] = float("inf"), float("inf")
    out = run_tree(t, max(toks))
    nan = torch.stack([q[:n, :2, 6] >= 0, q[:n, 2:, 9] >= 0], 1).flatten(1)
    assert torch.equal(out[:n].isnan(), nan[..., None].expand_as(out[:n]))
    assert not bool(out[n:].isnan().any()) and bool(nan[0, 0]) and not bool(nan[0, 2])
    # without it: a key that is far from the query in the same way
    c.k_pages[pg, :, r] = key
    c.k_pages[pg, 0, r, 6], c.k_pages[pg, 1, r, 9] = 1e30, 1e30
    want = exact(t)[:n][~nan]
    got = out[:n][~nan].double()
    tol = 2.0 ** -6 if dt == BF16 else 2.0 ** -16
    assert bool(((got - want).abs() <= tol * want.abs().amax(-1, keepdim=True)).all())
    status()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_scores_of_thousands(dt):
    """Scores of +-thousands: one key takes all the weight, as in the formula."""
    t = tree_case(dt, 16, 2, 1, 64, [70], [3], [], "chain", seed=8)
    c, q, *_ = t
    q.mul_(64)
    c.k_pages.mul_(8)
    check_tree(t, run_tree(t, 3))
    status()


def test_a_nan_key_that_is_seen_makes_its_rows_nan():
    for dt in (F32, BF16):
        t = tree_case(dt, 16, 4, 2, 64, [33], [4], [], "chain", seed=9)
        c = t[0]
        pg, row = rows_of(c, 0, [5])
        c.k_pages[pg, 0, row] = NAN
        out = run_tree(t, 4)
        assert bool(out[:, :2].isnan().all()) and not bool(out[:, 2:].isnan().any())
    status()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_bad_arrays_are_recorded(dt):
    def fresh():
        return tree_case(dt, 16, 4, 2, 64, [30, 12], [4, 6], [3, 9], "tree", seed=4)

    t = fresh()
    want = run_tree(t, 6)
    t[3][2] = 2                                   # a token is its own parent: pruned
    out = run_tree(t, 6)
    status(-1)
    assert bool((out[2] == 0).all()) and torch.equal(out[4:], want[4:])
    t = fresh()
    t[6][1] = 10                                  # past m_cap: clamped
    out = run_tree(t, 6)
    status(-1)
    assert torch.equal(out, want)
    t = fresh()
    t[0].block_table[0, 0] = t[0].n_pages         # a page that is not there
    out = run_tree(t, 6)
    status(-1)
    assert torch.equal(out[4:], want[4:])
    t = fresh()
    t[2][2] = 9                                   # five tokens
    five = run_tree(t, 5)
    status()
    out = run_tree(fresh(), 5)                    # six, where five were promised
    status(-1)
    assert torch.equal(out[:9], five[:9]) and bool(out[9].isnan().all())
    t = fresh()
    t[0].cache_len[0] = 46                        # 46 + 4 rows, the table holds 48
    run_tree(t, 6)
    status(-3)
    t = fresh()
    exact, tol = expected(t)
    t[2][2] = 99                                  # offsets past the tokens: skipped
    out = run_tree(t, 6)
    status(-1)
    # the sequence that is left is cut into other parts, whose joining rounds
    # otherwise: each result keeps the formula's bound, not the other's bits
    close(out[:4], exact[:4], tol[:4])
    assert bool(out[4:].isnan().all())


@pytest.mark.parametrize("case", [TREES[0], TREES[5], TREES[4], TREES[11]],
                         ids=["f32", "tree", "decode", "chain"])
def test_tree_attention_repeats_bit_for_bit(case):
    dt, page, Hq, H, D, lens, toks, mem, tree, n_max = case
    t = tree_case(dt, page, Hq, H, D, lens, toks, mem, tree, seed=1)
    first = run_tree(t, n_max)
    for _ in range(20):
        assert torch.equal(run_tree(t, n_max), first)
    status()


def test_a_cache_past_32_bit_element_offsets():
    """Pages whose rows start past 2^32 elements of the pool."""
    H, D, page, L, n = 8, 128, 128, 300, 5
    n_pages = 2 ** 32 // (H * page * D) + 8
    c = pipeline.PagedCache(BF16, n_pages, page, H, D, 1, 3, "cuda")
    c.block_table.copy_(i32([[n_pages - 1, n_pages - 3, 7]]))
    k, v, q = (rnd((L + n, h, D), BF16, s) for h, s in ((H, 1), (H, 2), (16, 3)))
    pos = i32(np.arange(L + n))
    c.append(k, v, i64([0, L + n]), pos)
    c.cache_len.fill_(L)
    pg, row = rows_of(c, 0, range(L + n))
    assert torch.equal(c.v_pages[pg, :, row], v)
    small = pipeline.PagedCache(BF16, 3, page, H, D, 1, 3, "cuda")
    small.block_table.copy_(i32([[2, 0, 1]]))
    small.append(k, v, i64([0, L + n]), pos)
    small.cache_len.fill_(L)
    att = pipeline.TreeAttention(BF16, 1, n, 16, H, D, 0, 3, page, "cuda")
    a = att(q[:n].contiguous(), i64([0, n]), c)
    b = att(q[:n].contiguous(), i64([0, n]), small)
    assert torch.equal(a, b)
    status()


# ------------------------------------- long items, to their last slice
#
# The bounds of `expected` grow with the keys; these do not.

def exact(case):
    """The attention in float64 on the GPU, a sequence and KV head at a time."""
    c, q, off, parents, km, vm, ml, m_cap = case
    D, G = c.D, q.shape[1] // c.H
    o, lens = off.tolist(), c.cache_len.tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b in range(c.B):
        n, L, M = o[b + 1] - o[b], lens[b], ml[b].item() if m_cap else 0
        if n == 0:
            continue
        par = list(range(-1, n - 1)) if parents is None else parents[o[b]:o[b + 1]].tolist()
        tree = torch.from_numpy(oracle.ancestors(par)).cuda()
        ids = c.block_table[b, :-(-(L + n) // c.page_size)].long()
        for g in range(c.H):
            k, v = (p[ids, g].reshape(-1, D)[:L + n] for p in (c.k_pages, c.v_pages))
            if M:
                k, v = torch.cat((km[b, :M, g], k)), torch.cat((vm[b, :M, g], v))
            s = torch.einsum("tgd,jd->tgj", q[o[b]:o[b + 1], g * G:(g + 1) * G].double(),
                             k.double()) / D ** 0.5
            s[:, :, M + L:].masked_fill_(~tree[:, None], float("-inf"))
            live = tree.diagonal()
            out[o[b]:o[b + 1], g * G:(g + 1) * G][live] = torch.einsum(
                "tgj,jd->tgd", torch.softmax(s[live], -1), v.double())
    return out


# kernel: dt, page, Hq, H, D, lens, tokens, memory rows, tree, n_max
LONG = {
    "simt-f32": (F32, 16, 2, 1, 64, [1500, 3], [4, 2], [40, 0], "tree", 4),
    "few-f32": (F32, 64, 8, 4, 128, [32000, 31900, 32050, 7], [1] * 4, [100, 0, 64, 5], "chain",
                1),
    "few-f32-trees": (F32, 16, 8, 2, 64, [30011, 0, 8200], [17, 5, 33], [3, 0, 200], "tree", 33),
    "few-bf16": (BF16, 64, 8, 2, 128, [20000, 4097, 300], [3, 4, 1], [220, 0, 17], "chain", 4),
    "few-bf16-64": (BF16, 16, 5, 1, 64, [9000, 8999, 1, 0], [3, 1, 2, 3], [], "tree", 3),
    "tc": (BF16, 64, 8, 2, 128, [18500, 333, 0], [33, 20, 1], [700, 0, 129], "tree", 33),
    "tc-64": (BF16, 32, 16, 4, 64, [12000, 7000], [60, 33], [0, 31], "pruned", 64),
    "tc-rows": (BF16, 16, 6, 2, 128, [9001, 15], [64, 9], [], "chain", 64),
    "tc-two-tiles": (BF16, 128, 8, 2, 128, [80000, 79000, 5], [64, 50, 60], [130, 0, 1], "tree",
                     64),
}


def long_case(name, seed=5):
    dt, page, Hq, H, D, lens, toks, mem, tree, n_max = LONG[name]
    return tree_case(dt, page, Hq, H, D, lens, toks, mem, tree, seed=seed, lead=2), n_max


def test_the_float64_attention_is_the_oracles():
    t = tree_case(F32, 16, 4, 2, 64, [37, 0, 5], [6, 2, 0], [7, 0, 3], "pruned", seed=2, lead=1)
    want, _ = expected(t)
    assert np.abs(f64(exact(t)) - want).max() < 1e-13


@pytest.mark.parametrize("name", LONG)
def test_long_items_to_a_root_mean_square(name):
    """The error over a sequence's output against that output.  The errors of scores,
    weights and products are independent of the values they meet, so they add in
    squares, as the outputs do, and the bound does not grow with the keys; a
    slice that is lost or taken twice is (8 / keys)^(1/2) or more of an output,
    1.4% at 40,000.
    fp32: a score of size 1 by its split operands (2^-22 each) and its
    sum of 16 cut-off terms at most 2^-20 together, the weight's and the value's
    splits and a slice's cut-off sum again 2^-20, rounded sums and the joining
    2^-21: 2^-19 is twice the root of their squares; a split term that is lost
    is 2^-12.
    bf16: at most BF / 3^(1/2) of each value for the output's rounding (an even
    distribution), and in the tcgen05 kernel the same of each weight."""
    t, n_max = long_case(name)
    out = run_tree(t, n_max)
    if out.dtype == F32:
        bound = 2.0 ** -19
    else:
        bound = 1.02 * BF * (2 / 3 if name.startswith("tc") else 1 / 3) ** 0.5
    want, o = exact(t), t[2].tolist()
    for lo, hi in zip(o[:-1], o[1:]):
        err, size = (out[lo:hi].double() - want[lo:hi]).norm().item(), want[lo:hi].norm().item()
        assert err <= bound * size, (err / size, bound)
    status()


@pytest.mark.parametrize("name", LONG)
def test_every_slice_counts_once(name):
    """Scores of zero give every seen key the weight 1 / N; the values of each
    piece of keys are ones in one column (the next piece's in the next), so that
    N out counts the seen keys of the pieces of a column.  The counts are exact
    on the way; one rounding of 1 / N, one of the product, one of the output."""
    t, n_max = long_case(name)
    c, q, off, parents, km, vm, ml, m_cap = t
    D, H, G = c.D, c.H, q.shape[1] // c.H
    piece = 8 if q.dtype == F32 else 16
    q.zero_()
    o, lens = off.tolist(), c.cache_len.tolist()
    want = np.zeros(q.shape)
    for b in range(c.B):
        n, L, M = o[b + 1] - o[b], lens[b], ml[b].item() if m_cap else 0
        at = np.concatenate([np.arange(M) // piece, -(-M // piece) + np.arange(L + n) // piece])
        par = list(range(-1, n - 1)) if parents is None else parents[o[b]:o[b + 1]].tolist()
        tree = oracle.ancestors(par)
        pg, row = rows_of(c, b, range(L + n))
        for g in range(H):
            one = np.eye(D)[(at + 5 * g + 3 * b) % D]
            v = torch.from_numpy(one).cuda().to(q.dtype)
            c.v_pages[pg, g, row] = v[M:]
            if M:
                vm[b, :M, g] = v[:M]
            for i in range(n):
                if tree[i, i]:
                    seen = one[:M + L].sum(0) + one[M + L:][tree[i]].sum(0)
                    want[o[b] + i, g * G:(g + 1) * G] = seen / seen.sum()
    out = run_tree(t, n_max)
    live = slice(o[0], o[-1])
    close(out[live], want[live], want[live] * (step_of(q.dtype) + 4 * U))
    status()


@pytest.mark.parametrize("name", LONG)
def test_one_key_at_a_border_takes_all_the_weight(name):
    """Each row looks for a key of its own (a dim that no other key has), the
    first or last of a slice: the output is that key's value."""
    t, n_max = long_case(name)
    c, q, off, parents, km, vm, ml, m_cap = t
    D, H, G = c.D, c.H, q.shape[1] // c.H
    o, lens = off.tolist(), c.cache_len.tolist()
    dead = np.zeros(q.shape[0], dtype=bool)
    if parents is not None:
        for b in range(c.B):
            dead[o[b]:o[b + 1]] = ~oracle.ancestors(parents[o[b]:o[b + 1]].tolist()).diagonal()
    for turn in range(8):
        q.zero_()
        want = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        for b in range(c.B):
            n, L, M = o[b + 1] - o[b], lens[b], ml[b].item() if m_cap else 0
            ends = [j for j in range(M + L) if (j if j < M else j - M) % 8 in (0, 7)]
            if not ends or n == 0:
                dead[o[b]:o[b + 1]] = True
                continue
            pg, row = rows_of(c, b, range(L))
            for g in range(H):
                c.k_pages[pg, g, row] = 0
                if M:
                    km[b, :M, g] = 0
                for r in range(min(n * G, D)):
                    x = ((r * 8 + turn + g) * 0.6180339887498949) % 1.0
                    j = ends[int(x * len(ends))]
                    h = g * G + r % G
                    q[o[b] + r // G, h, r] = 64
                    if j < M:
                        km[b, j, g, r] = 64
                        want[o[b] + r // G, h] = vm[b, j, g].double()
                    else:
                        c.k_pages[pg[j - M], g, row[j - M], r] = 64
                        want[o[b] + r // G, h] = c.v_pages[pg[j - M], g, row[j - M]].double()
        # a score of 4096 / D^(1/2) above the others: their weights are 0.  (The
        # drafted keys keep their random values: 64 of one dim is at most 5 x 64
        # / D^(1/2), as far below.)
        out = run_tree(t, n_max).double()
        seek = (q != 0).any(-1) & torch.from_numpy(~dead).cuda()[:, None]
        assert int(seek.sum()) > 0
        diff = (out[seek] - want[seek]).abs()
        assert bool((diff <= want[seek].abs() * 2.0 ** -20).all()), diff.max()
    status()


# ------------------------------------------------------------- together

def bank(dt, H, D, seed):
    lengths = [180] * 6
    toff = np.concatenate([[0], np.cumsum(lengths)])
    coff = oracle.chunk_offsets_from_lengths(lengths)
    C = int(coff[-1])
    kr, kb, vb = (rnd((C, H, D), dt, seed + i) for i in range(3))
    return toff, coff, kr, kb, vb


@pytest.mark.parametrize("dt,Hq,H,D", [(F32, 4, 2, 64), (BF16, 8, 2, 128)])
def test_generation(dt, Hq, H, D):
    """Prompts, decode steps and a drafted tree whose accepted path is kept,
    against one oracle attention over everything a token may see."""
    B, T, k, page = 2, 9, 2, 16
    _, coff, kr, kb, vb = bank(dt, H, D, 40)
    m_cap = 6
    c = pipeline.PagedCache(dt, 20, page, H, D, B, 5, "cuda")
    c.k_pages.fill_(NAN)
    c.v_pages.fill_(NAN)
    n_max = 8
    g = pipeline.CachedPipeline(kr, kb, vb, i64(coff), c, T=T, n_max=n_max, Hq=Hq, k=k,
                                m_cap=m_cap)
    idx = g.select(rnd((B, T, H, D), dt, 50)).cpu().numpy()
    okm, ovm, oml = oracle.gather_kv(idx, coff, f64(kb), f64(vb))
    w = rnd((2, D), dt, 51) * 0.2 + 1
    kept = [[] for _ in range(B)]  # (k, v) rows each sequence has kept, unrotated

    def step(toks, parents, seed):
        off = np.concatenate([[0], np.cumsum(toks)])
        N = int(off[-1])
        q, kk, vv = (rnd((N, h, D), dt, seed + i) for i, h in enumerate((Hq, H, H)))
        par = parents or [i - 1 for n in toks for i in range(n)]
        depth, pos = [], []
        for b in range(B):
            for i in range(toks[b]):
                p = par[off[b] + i]
                depth.append(0 if p < 0 else depth[int(off[b]) + p] + 1)
                pos.append(k + len(kept[b]) + depth[-1])
            c.reserve(b, len(kept[b]) + toks[b])
        out = g.step(q, kk, vv, i64(off), i32(pos), None if parents is None else i32(parents),
                     w[0], w[1])
        # the oracle on the cache's own rows (append is checked above)
        want, bound, top = oracle.tree_attn(
            oracle_q(q, w[0], pos, dt), off, np.array(par), f64(g.k_mem), f64(g.v_mem), oml,
            f64(c.k_pages), f64(c.v_pages), c.block_table.cpu().numpy(),
            c.cache_len.cpu().numpy())
        tol = bound * U * (2 * (D + 4) * top[..., None] + 1000)
        if dt == BF16:
            tol = tol + BF * (bound + np.abs(want))
        else:
            # the queries' own rounding (24 U of them) in the scores
            tol = tol + bound * 2 * 24 * U * top[..., None]
        close(out, want, tol)
        return kk, vv, pos, off

    def oracle_q(q, wq, pos, dt):
        if dt == F32:
            return oracle.norm_rope(f64(q), f64(wq), pos)
        # bf16 queries are rounded by the operator: take its own
        return f64(pipeline.qk_norm_rope(q, None, i32(pos), wq)[0])

    def keep(kk, vv, tokens):
        for b, ts in enumerate(tokens):
            kept[b] += [(kk[t], vv[t]) for t in ts]
        c.cache_len.add_(i32([len(ts) for ts in tokens]))

    # prompts of unlike lengths, in pieces of n_max
    kk, vv, _, off = step([8, 5], None, 60)
    keep(kk, vv, [range(0, 8), range(8, 13)])
    kk, vv, _, off = step([8, 0], None, 70)
    keep(kk, vv, [range(0, 8), []])
    for s in range(3):  # decode
        kk, vv, _, off = step([1, 1], None, 80 + 3 * s)
        keep(kk, vv, [[0], [1]])
    # drafted trees; the path 0-2-3 of the first, 1 of the second is accepted
    kk, vv, pos, off = step([5, 3], [-1, 0, 0, 2, -1, -1, -1, 0], 100)
    path = [[0, 2, 3], [6]]
    ts = [t for p in path for t in p]
    c.append(kk[ts], vv[ts], i64([0, 3, 4]), i32([pos[t] for t in ts]), w[1])
    keep(kk, vv, path)
    kk, vv, _, off = step([1, 1], None, 110)
    keep(kk, vv, [[0], [1]])
    # the cache now holds every kept row, at consecutive positions
    for b in range(B):
        pg, row = rows_of(c, b, range(len(kept[b])))
        assert torch.equal(c.v_pages[pg, :, row], torch.stack([v for _, v in kept[b]]))
        ks = torch.stack([x for x, _ in kept[b]])
        want = pipeline.qk_norm_rope(None, ks, i32(k + np.arange(len(kept[b]))), None, w[1])[1]
        assert torch.equal(c.k_pages[pg, :, row], want)
    status()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_captured_steps_follow_the_caches_lengths(dt):
    """A decode step captured once and replayed as the cache grows gives the
    eager step's bits; a second captured step shares nothing with it."""
    Hq, H, D, B = 8, 2, 128, 3
    _, coff, kr, kb, vb = bank(dt, H, D, 3)

    def make():
        c = pipeline.PagedCache(dt, 30, 16, H, D, B, 6, "cuda")
        c.k_pages.fill_(NAN)
        c.v_pages.fill_(NAN)
        g = pipeline.CachedPipeline(kr, kb, vb, i64(coff), c, T=4, n_max=2, Hq=Hq, k=2, m_cap=6)
        for b in range(B):
            c.reserve(b, 60)
        g.select(rnd((B, 4, H, D), dt, 5))
        return c, g

    off = i64(np.arange(0, 2 * B + 1, 2))
    ins = [rnd((2 * B, h, D), dt, 9 + h) for h in (Hq, H)] + [rnd((2 * B, H, D), dt, 8)]
    pos = i32([0] * 2 * B)
    out = torch.empty((2 * B, Hq, D), dtype=dt, device="cuda")

    def fill(s):
        for i, x in enumerate(ins):
            x.copy_(rnd(x.shape, dt, 100 + 3 * s + i))
        pos.copy_(i32([2 + 2 * s, 3 + 2 * s] * B))

    caches = [make() for _ in range(3)]
    eager = []
    c, g = caches[0]
    for s in range(25):
        fill(s)
        eager.append(g.step(*ins, off, pos, out=out).clone())
        c.cache_len.add_(2)
    graphs = []
    for c, g in caches[1:]:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.step(*ins, off, pos, out=out)
        torch.cuda.current_stream().wait_stream(side)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            g.step(*ins, off, pos, out=out)
            c.cache_len.add_(2)
        graphs.append(gr)
    for s in range(25):
        fill(s)
        for gr in graphs:
            out.fill_(NAN)
            gr.replay()
            assert torch.equal(out, eager[s])
    status()


def test_calls_on_two_streams_at_once():
    dt, Hq, H, D = BF16, 8, 2, 128
    cases = [tree_case(dt, 64, Hq, H, D, [900 + 100 * i, 40], [3, 2], [20, 7], "tree", seed=i)
             for i in range(2)]
    want = [run_tree(t, 3) for t in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    atts = [pipeline.TreeAttention(dt, 2, 3, Hq, H, D, 20, t[0].max_pages, 64, "cuda")
            for t in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (t, s) in enumerate(zip(cases, streams)):
            c, q, off, parents, km, vm, ml, _ = t
            got[i].append(atts[i](q, off, c, parents, km, vm, ml, stream=s))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        assert all(torch.equal(w, x) for x in gs)
    status()


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_pages_are_handed_over_on_the_calls_stream(raw):
    """Reservations, appends and releases on a stream of their own, while the
    current stream is busy: the next append sees the pages of the last reserve."""
    s = torch.cuda.Stream()
    st = s.cuda_stream if raw else s
    c = pipeline.PagedCache(F32, 4, 16, 2, 64, 2, 2, "cuda")
    c.v_pages.fill_(NAN)
    k, off, pos = rnd((16, 2, 64), F32, 1), i64([0, 16, 16]), i32(np.arange(16))
    other = i64([0, 0, 16])
    busy = rnd((4096, 4096), F32, 2)
    torch.cuda.synchronize()
    for i in range(6):
        for _ in range(8):
            busy = busy @ busy * 1e-3
        b = i & 1
        c.reserve(b, 16, stream=st)
        c.append(k, k, other if b else off, pos, stream=st)
        if i < 5:
            c.release(b, stream=st)
    s.synchronize()
    assert torch.equal(c.v_pages[c.owned[1][0]].transpose(0, 1), k)
    torch.cuda.synchronize()
    assert c.block_table.tolist() == [[-1, -1], [c.owned[1][0], -1]]
    status()


def test_a_backward_call_on_another_stream():
    n, Hq, H, D = 4000, 8, 2, 128
    _, q, k, wq, wk, pos = norm_inputs(BF16, n, Hq, H, D, "qk", "near", seed=1)
    dq, dk = rnd((n, Hq, D), BF16, 2), rnd((n, H, D), BF16, 3)
    want = pipeline.qk_norm_rope_backward(q, k, pos, dq, dk, wq, wk)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [pipeline.qk_norm_rope_backward(q, k, pos, dq, dk, wq, wk, stream=s) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))
    status()


@pytest.fixture(params=["native", "python"])
def marshalling(request):
    """The calls' arguments checked by the native module, or in Python."""
    native = msa._native()
    assert native is not None
    if request.param == "python":
        msa._bound[1] = None
    yield request.param
    msa._bound[1] = native


def test_binding_takes_what_fits_and_refuses_the_rest(marshalling):
    dt, D = BF16, 64
    _, (q, k, v) = fused(6, 4, 2, D, dt, 1)
    w, pos, off = rnd((D,), dt, 2), i32(np.arange(6)), i64([0, 4, 6])
    c = pipeline.PagedCache(dt, 8, 16, 2, D, 2, 3, "cuda")
    for b in range(2):
        c.reserve(b, 40)
    qr = c.append(k, v, off, pos, w, q, w)
    att = pipeline.TreeAttention(dt, 2, 4, 4, 2, D, 0, 3, 16, "cuda")
    out = att(qr, off, c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = [att(qr, off, c, stream=side), att(qr, off, c, stream=side.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, out) for x in again)
    dq, dk = (x.float() for x in pipeline.qk_norm_rope(q, k, pos, w, w))
    pipeline.qk_norm_rope_backward(q, k, pos, dq, dk, w, w)
    torch.cuda.synchronize()

    def no(match, fn):
        with pytest.raises(ValueError, match=match):
            fn()

    no("v is torch.float32", lambda: c.append(k, v.float(), off, pos))
    no("tok_offsets is torch.int32", lambda: c.append(k, v, off.int(), pos))
    no("positions holds 5", lambda: c.append(k, v, off, pos[:5]))
    no("q must be contiguous", lambda: att(q, off, c))
    no("heads must be contiguous", lambda: c.append(k.transpose(0, 1).contiguous().transpose(0, 1),
                                                    v, off, pos))
    no("v has shape", lambda: c.append(k, v[:, :1], off, pos))
    no("parents is on cpu", lambda: att(qr, off, c, parents=torch.zeros(6, dtype=torch.int32)))
    no("q_weight is on cpu", lambda: pipeline.qk_norm_rope(q, k, pos, w.cpu()))
    no("dq_out is torch.float64", lambda: msa.msa_qk_norm_rope_backward(
        1, 0, 6, 4, 0, D, q, None, None, None, pos, 1e-6, 1e4, dq.double(), None, dq, None, None,
        None, None, 0))
    no("ws holds", lambda: msa.msa_tree_attn(
        1, 2, 6, 4, 4, 2, D, qr, off, None, None, None, None, 0, c.k_pages, c.v_pages, 8, 16,
        c.block_table, 3, c.cache_len, 0.0, out, att.ws, att.ws.numel() + 1))
    with pytest.raises(msa.MsaError) as e:
        msa.msa_tree_attn(1, 2, 6, 4, 4, 2, D, qr, off, None, None, None, None, 0, c.k_pages,
                          c.v_pages, 8, 16, c.block_table, 3, c.cache_len, 0.0, out, att.ws, 8)
    assert e.value.status == -6
    with pytest.raises(ctypes.ArgumentError):
        pipeline.qk_norm_rope(q, k, pos, w, w, eps="small")
    assert torch.equal(att(qr, off, c), out)
    status()


DEBUG_CHILD = r"""
import torch
from latent_memory_routing_b200 import msa, pipeline

assert msa.LIB_PATH.endswith("libmsa_debug.so"), msa.LIB_PATH
msa.lib()
msa.msa_device_status(clear=True)

def refused(fn, code):
    try:
        fn()
    except msa.MsaError as e:
        assert e.status == code, (e.status, code)
        msa.msa_device_status(clear=True)
        return
    raise AssertionError("the call was not refused")

def i32(x): return torch.tensor(x, dtype=torch.int32, device="cuda")
def i64(x): return torch.tensor(x, dtype=torch.int64, device="cuda")

for dt in (torch.float32, torch.bfloat16):
    c = pipeline.PagedCache(dt, 8, 16, 2, 64, 2, 3, "cuda")
    for b in range(2):
        c.reserve(b, 40)
    k, q = torch.randn(6, 2, 64, device="cuda").to(dt), torch.randn(6, 4, 64, device="cuda").to(dt)
    off, pos = i64([0, 4, 6]), i32([0, 1, 2, 3, 0, 1])
    att = pipeline.TreeAttention(dt, 2, 4, 4, 2, 64, 0, 3, 16, "cuda")
    c.append(k, k, off, pos)
    out = att(q, off, c)
    assert bool(torch.isfinite(out).all())
    refused(lambda: c.append(k, k, i64([0, 5, 4]), pos), -1)    # offsets that fall
    refused(lambda: att(q, i64([0, 5, 4]), c), -1)
    refused(lambda: att(q, off, c, parents=i32([0, 0, 0, 0, -1, 0])), -1)  # its own parent
    c.cache_len[1] = 49                                         # past the block table
    refused(lambda: c.append(k, k, off, pos), -1)
    refused(lambda: att(q, off, c), -1)
    c.cache_len[1] = 47                                         # its second row has no place
    refused(lambda: c.append(k, k, off, pos), -3)
    c.cache_len[1] = 0
    assert torch.equal(att(q, off, c), out)
    y = pipeline.qk_norm_rope(q, k, pos)
    dy = [x.float() for x in y]
    pipeline.qk_norm_rope_backward(q, k, pos, *dy)
    assert msa.msa_device_status(clear=True) == 0
print("debug build ok")
"""


def test_debug_library_refuses_bad_arrays(cuda_device):
    """The input-checking build returns what its calls find from the calls."""
    import os
    import subprocess
    import sys

    from latent_memory_routing_b200 import build
    build.build(debug=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", DEBUG_CHILD], cwd=root, capture_output=True,
                       text=True, env=dict(os.environ, MSA_DEBUG="1"), timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "debug build ok" in r.stdout
