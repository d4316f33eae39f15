"""CPU checks of the generation operators (per-head norms with RoPE, paged
append, tree attention): the oracle against differences and plainer
restatements, the host refusals of the library and of the binding, and the
page accounting of PagedCache."""

import os

import numpy as np
import pytest
import torch

import oracle
from latent_memory_routing_b200 import msa, pipeline

NULL = None
P = 256  # a 16-byte aligned address that no refused call reads


# ------------------------------------------------------------------- oracle

@pytest.mark.parametrize("rotated", [True, False])
def test_oracle_norm_gradient_matches_differences(rotated):
    r = np.random.default_rng(0)
    x, w, dy = r.normal(size=(3, 2, 8)), r.normal(size=8), r.normal(size=(3, 2, 8))
    pos = np.array([0, 5, -17]) if rotated else None
    dx, dw = oracle.norm_rope_backward(x, w, pos, dy, eps=1e-2)
    h = 1e-6

    def loss(x, w):
        return float((oracle.norm_rope(x, w, pos, eps=1e-2) * dy).sum())

    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(8):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[i]) < 1e-7


def test_oracle_rotation_only_is_orthogonal():
    r = np.random.default_rng(1)
    x, dy = r.normal(size=(4, 2, 8)), r.normal(size=(4, 2, 8))
    pos = np.array([3, 0, 9, 1000000])
    y = oracle.norm_rope(x, None, pos)
    dx, dw = oracle.norm_rope_backward(x, None, pos, dy)
    assert dw is None
    assert abs((y * dy).sum() - (x * dx).sum()) < 1e-12  # <R x, dy> = <x, R^T dy>


def test_oracle_ancestors():
    see = oracle.ancestors([-1, 0, 0, 1, -1, -2, 5, 3])
    want = {0: [0], 1: [0, 1], 2: [0, 2], 3: [0, 1, 3], 4: [4], 5: [], 6: [], 7: [0, 1, 3, 7]}
    for i, w in want.items():
        assert list(np.flatnonzero(see[i])) == w


def test_oracle_chain_is_the_causal_sparse_attention():
    """A chain over a paged cache, after the append's rotation, is the
    oracle's sparse attention over [memory ; local causal context]."""
    r = np.random.default_rng(2)
    Hq, H, D, page, L, n, M, k = 4, 2, 8, 4, 6, 3, 5, 2
    km, vm = r.normal(size=(1, M, H, D)), r.normal(size=(1, M, H, D))
    kl, vl = r.normal(size=(1, L + n, H, D)), r.normal(size=(1, L + n, H, D))
    q = r.normal(size=(1, n, Hq, D))
    want = oracle.sparse_attn(q, [km[0]], [vm[0]], kl, vl, k)
    pos = k + np.arange(L + n)
    table = np.array([[3, 0, 2]])
    kp, vp = r.normal(size=(5, H, page, D)), r.normal(size=(5, H, page, D))
    kr = oracle.norm_rope(kl[0], None, pos)
    kp = oracle.paged_append(kp, kr, [0, L + n], [0], table)
    vp = oracle.paged_append(vp, vl[0], [0, L + n], [0], table)
    got, _, _ = oracle.tree_attn(oracle.norm_rope(q[0], None, pos[L:]), [0, n], None, km, vm, [M],
                                 kp, vp, table, [L])
    assert np.max(np.abs(got - want[0])) < 1e-12


# ---------------------------------------------------------- host refusals

@pytest.fixture(scope="module")
def lib():
    return msa.lib()


def test_norm_refusals(lib):
    def f(dt=1, n=10, Hq=4, H=2, D=128, q=P, qs=512, k=P, ks=256, wq=P, wk=P, pos=P, eps=1e-6,
          base=1e4, qo=P, ko=P):
        return lib.msa_qk_norm_rope(dt, n, Hq, H, D, q, qs, k, ks, wq, wk, pos, eps, base, qo, ko,
                                    NULL)
    assert f(n=0) == 0                                     # nothing to do
    assert f(dt=7) == f(n=-1) == f(Hq=-1) == f(H=-1) == f(Hq=0, H=0) == -1
    assert f(D=96) == f(D=256) == f(n=2 ** 31) == f(Hq=1 << 20) == -2
    assert f(q=NULL) == f(k=NULL) == f(qo=NULL) == f(ko=NULL) == -1
    assert f(q=P + 8) == f(k=P + 2) == f(qo=P + 4) == f(ko=P + 8) == f(wq=P + 2) == -1
    assert f(qs=511) == f(qs=508) == f(ks=255) == f(ks=260) == -1  # short, or not 16-byte rows
    assert f(eps=-1.0) == f(eps=float("nan")) == f(base=0.0) == f(base=float("inf")) == -1


def test_norm_backward_refusals(lib):
    need = msa.msa_qk_norm_rope_backward_workspace_size(10, 128)
    assert need > 0
    assert msa.msa_qk_norm_rope_backward_workspace_size(0, 128) == 0

    def f(dt=1, gdt=0, n=10, Hq=4, H=2, D=128, q=P, qs=512, k=P, ks=256, wq=P, wk=P, pos=P,
          eps=1e-6, base=1e4, dqo=P, dko=P, dq=P, dqs=512, dk=P, dks=256, dwq=P, dwk=P, ws=P,
          nb=need):
        return lib.msa_qk_norm_rope_backward(dt, gdt, n, Hq, H, D, q, qs, k, ks, wq, wk, pos, eps,
                                             base, dqo, dko, dq, dqs, dk, dks, dwq, dwk, ws, nb,
                                             NULL)
    assert f(dt=0, gdt=1) == f(D=32) == -2
    assert f(gdt=5) == f(dqo=NULL) == f(dq=NULL) == f(dqs=300) == f(dks=258) == f(dko=P + 4) == -1
    assert f(dwq=NULL) == f(dwk=NULL) == -1                # a weight without its gradient
    assert f(wq=NULL) == f(wk=NULL) == -1                  # a gradient without its weight
    assert f(ws=NULL) == f(nb=need - 1) == f(ws=P + 8) == -6


def test_append_refusals(lib):
    def f(dt=1, B=2, n=5, Hq=4, H=2, D=128, q=P, qs=512, k=P, ks=256, v=P, vs=256, wq=P, wk=P,
          off=P, pos=P, eps=1e-6, base=1e4, tab=P, mp=4, cl=P, ps=64, npg=8, kp=P, vp=P, qo=P):
        return lib.msa_paged_append(dt, B, n, Hq, H, D, q, qs, k, ks, v, vs, wq, wk, off, pos, eps,
                                    base, tab, mp, cl, ps, npg, kp, vp, qo, NULL)
    assert f(n=0) == 0
    assert f(B=0) == f(H=0) == f(mp=0) == f(npg=0) == f(n=-1) == -1
    assert f(off=NULL) == f(tab=NULL) == f(cl=NULL) == f(pos=NULL) == -1
    assert f(k=NULL) == f(v=NULL) == f(kp=NULL) == f(vp=NULL) == f(q=NULL) == f(qo=NULL) == -1
    assert f(kp=P + 8) == f(vs=255) == f(v=P + 4) == -1
    assert f(ps=48) == f(ps=8) == f(ps=256) == f(D=80) == -2
    assert f(npg=1 << 24) == f(mp=1 << 26) == -2           # row numbers past 31 bits


def test_tree_refusals(lib):
    def f(dt=1, B=2, n=5, nm=3, Hq=4, H=2, D=128, q=P, off=P, par=P, km=P, vm=P, ml=P, mc=8, kp=P,
          vp=P, npg=8, ps=64, tab=P, mp=4, cl=P, sc=0.0, out=P, ws=P, nb=1 << 40):
        return lib.msa_tree_attn(dt, B, n, nm, Hq, H, D, q, off, par, km, vm, ml, mc, kp, vp, npg,
                                 ps, tab, mp, cl, sc, out, ws, nb, NULL)
    assert f(n=0) == 0
    assert f(dt=2) == f(B=0) == f(nm=0) == f(H=0) == f(mc=-1) == f(mp=0) == f(npg=0) == -1
    assert f(q=NULL) == f(off=NULL) == f(tab=NULL) == f(cl=NULL) == f(out=NULL) == -1
    assert f(km=NULL) == f(vm=NULL) == f(ml=NULL) == f(kp=NULL) == f(vp=NULL) == -1
    assert f(q=P + 8) == f(kp=P + 8) == f(km=P + 4) == f(out=P + 2) == f(sc=float("nan")) == -1
    assert f(nm=129) == f(Hq=5) == f(Hq=34) == f(D=96) == f(ps=24) == f(B=40000) == -2
    assert f(mp=1 << 26) == f(npg=1 << 24) == -2
    need = msa.msa_tree_attn_workspace_size(1, 2, 3, 4, 2, 128, 8, 4, 64)
    if need:
        assert f(ws=NULL) == f(nb=need - 1) == f(ws=P + 8) == -6
    assert msa.msa_tree_attn_workspace_size(1, 2, 129, 4, 2, 128, 8, 4, 64) == 0


# ------------------------------------------------------------------ binding

class _StubLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def stub(monkeypatch):
    s = _StubLib()
    monkeypatch.setattr(msa, "lib", lambda *a, **k: s)
    monkeypatch.setattr(msa, "_device_ok", lambda t, host_ok: True)
    monkeypatch.setattr(msa, "_stream", lambda s: 0)
    return s


def test_binding_takes_token_strides_of_a_fused_projection(stub):
    x = torch.zeros(5, 8 * 64)
    q, k = x[:, :256].unflatten(1, (4, 64)), x[:, 256:384].unflatten(1, (2, 64))
    pipeline.qk_norm_rope(q, k, torch.zeros(5, dtype=torch.int32))
    name, args = stub.calls[0]
    assert name == "msa_qk_norm_rope" and args[6] == 512 and args[8] == 512
    assert args[7] - args[5] == 256 * 4


def test_binding_refuses_other_layouts(stub):
    pos = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="q: a token's heads must be contiguous"):
        pipeline.qk_norm_rope(torch.zeros(4, 5, 64).transpose(0, 1), None, pos)
    with pytest.raises(ValueError, match="q: a token's heads must be contiguous"):
        pipeline.qk_norm_rope(torch.zeros(5, 4, 128)[:, :, ::2], None, pos)
    with pytest.raises(ValueError, match="16 bytes apart"):
        pipeline.qk_norm_rope(torch.zeros(5, 4 * 64 + 1)[:, :256].unflatten(1, (4, 64)), None, pos)
    with pytest.raises(ValueError, match="overlap"):
        pipeline.qk_norm_rope(torch.zeros(1, 4, 64).expand(5, 4, 64), None, pos)
    with pytest.raises(ValueError, match="positions is torch.int64"):
        pipeline.qk_norm_rope(torch.zeros(5, 4, 64), None, pos.long())
    with pytest.raises(ValueError, match="positions holds 4"):
        pipeline.qk_norm_rope(torch.zeros(5, 4, 64), None, pos[:4])
    with pytest.raises(ValueError, match="k is torch.bfloat16"):
        pipeline.qk_norm_rope(torch.zeros(5, 4, 64), torch.zeros(5, 2, 64).bfloat16(), pos)
    with pytest.raises(ValueError, match="q_weight"):
        pipeline.qk_norm_rope(torch.zeros(5, 4, 64), None, pos, torch.ones(32))
    assert stub.calls == []


def test_binding_refuses_operands_of_different_lengths(stub):
    """What a call left out would come back as uninitialised rows."""
    pos, off = torch.zeros(6, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    q, k, k6 = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64), torch.zeros(6, 2, 64)
    with pytest.raises(ValueError, match="both None"):
        pipeline.qk_norm_rope(None, None, pos)
    with pytest.raises(ValueError, match="both None"):
        pipeline.qk_norm_rope_backward(None, None, pos, None, None)
    with pytest.raises(ValueError, match="k has shape"):
        pipeline.qk_norm_rope(q, k6, pos)
    with pytest.raises(ValueError, match="k has shape"):
        pipeline.qk_norm_rope_backward(q, k6, pos, q, k6)
    with pytest.raises(ValueError, match="dk_out has the shape of k"):
        pipeline.qk_norm_rope_backward(q, k, pos, q, k6)
    with pytest.raises(ValueError, match="dk_out has the shape of k"):
        pipeline.qk_norm_rope_backward(q, k, pos, q, None)
    with pytest.raises(ValueError, match="dq_out has the shape of q"):
        pipeline.qk_norm_rope_backward(None, k, pos, q, k)
    c = pipeline.PagedCache(torch.float32, 4, 16, 2, 64, 2, 3, "cpu")
    with pytest.raises(ValueError, match="q has shape"):
        c.append(k, k, off, pos, q=torch.zeros(6, 4, 64))
    att = pipeline.TreeAttention(torch.float32, 2, 4, 4, 2, 64, 0, 3, 16, "cpu")
    with pytest.raises(ValueError, match="q has shape"):
        att(torch.zeros(5, 8, 64), off, c)
    assert [n for n, _ in stub.calls] == ["msa_tree_attn_workspace_size"]


def test_append_refuses_values_of_more_tokens_than_keys(stub):
    """Their rows would be written nowhere."""
    c = pipeline.PagedCache(torch.float32, 4, 16, 2, 64, 2, 3, "cpu")
    off, pos = torch.zeros(3, dtype=torch.int64), torch.zeros(6, dtype=torch.int32)
    with pytest.raises(ValueError, match="v has shape"):
        c.append(torch.zeros(5, 2, 64), torch.zeros(6, 2, 64), off, pos)
    assert stub.calls == []


def test_binding_refuses_a_cache_of_other_sizes(stub):
    c = pipeline.PagedCache(torch.float32, 4, 16, 2, 64, 2, 3, "cpu")
    off, pos = torch.zeros(3, dtype=torch.int64), torch.zeros(5, dtype=torch.int32)
    x = torch.zeros(5, 2, 64)
    c.append(x, x, off, pos)
    with pytest.raises(ValueError, match="k has shape"):
        c.append(torch.zeros(5, 3, 64), x, off, pos)
    with pytest.raises(ValueError, match="v has shape"):
        c.append(x, x[:4], off, pos)
    with pytest.raises(ValueError, match="tok_offsets"):
        c.append(x, x, off[:2], pos)
    att = pipeline.TreeAttention(torch.float32, 3, 4, 4, 2, 64, 0, 3, 16, "cpu")
    with pytest.raises(ValueError, match="the cache holds"):
        att(torch.zeros(5, 4, 64), off, c)
    assert [n for n, _ in stub.calls] == ["msa_paged_append", "msa_tree_attn_workspace_size"]


def test_attention_refuses_memory_of_other_sizes(stub):
    """Read as [B][m_cap] rows, or left out with m_cap = 0, it would answer for
    another memory."""
    c = pipeline.PagedCache(torch.float32, 4, 16, 2, 64, 2, 3, "cpu")
    q, off = torch.zeros(5, 4, 64), torch.zeros(3, dtype=torch.int64)
    ml = torch.zeros(2, dtype=torch.int32)
    rows = {m: torch.zeros(2, m, 2, 64) for m in (0, 6, 7)}
    none, six = (pipeline.TreeAttention(torch.float32, 2, 4, 4, 2, 64, m, 3, 16, "cpu")
                 for m in (0, 6))
    stub.calls.clear()
    none(q, off, c)
    none(q, off, c, k_mem=rows[0], v_mem=rows[0], mem_len=ml)
    six(q, off, c, k_mem=rows[6], v_mem=rows[6], mem_len=ml)
    assert len(stub.calls) == 3
    for att, k, v, what in ((none, 6, 6, "k_mem"), (six, 7, 7, "k_mem"), (six, None, 6, "k_mem"),
                            (six, 6, 0, "v_mem"), (six, 6, 7, "v_mem"), (six, 6, None, "v_mem")):
        with pytest.raises(ValueError, match=f"{what} has shape"):
            att(q, off, c, k_mem=rows.get(k), v_mem=rows.get(v), mem_len=ml)
    assert len(stub.calls) == 3


def test_a_compiler_that_rejects_the_marshalling_leaves_the_python_path(tmp_path, monkeypatch,
                                                                        capfd):
    """build_marshal says so, takes an older build away and goes on; a working
    compiler's output is put in place whole."""
    import shutil as sh

    from latent_memory_routing_b200 import build

    so, src = tmp_path / "_marshal.so", tmp_path / "marshal.cpp"
    include = tmp_path / "include"
    include.mkdir()
    (include / "Python.h").touch()
    src.write_text("not C++")
    so.write_text("older")
    os.utime(so, (1, 1))
    cxx = tmp_path / "g++"
    monkeypatch.setattr(build, "MARSHAL", str(so))
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(include)})
    monkeypatch.setattr(sh, "which", lambda name: str(cxx))

    def compiler(script):
        cxx.write_text("#!/bin/sh\n" + script)
        cxx.chmod(0o755)

    compiler("echo no such thing >&2\nexit 1\n")
    assert build.build_marshal() is None
    assert "no such thing" in capfd.readouterr().err and not so.exists()
    # the last argument but one is the output
    compiler('while [ "$1" != -o ]; do shift; done\necho built > "$2"\necho "$2" >&2\nexit 0\n')
    assert build.build_marshal() == str(so) and so.read_text() == "built\n"
    assert sorted(p.name for p in tmp_path.iterdir()) == ["_marshal.so", "g++", "include",
                                                          "marshal.cpp"]


# --------------------------------------------------------------- page lists

def test_paged_cache_hands_out_and_takes_back_pages():
    c = pipeline.PagedCache(torch.float32, 5, 16, 1, 64, 2, 3, "cpu")
    c.reserve(0, 17)
    c.reserve(0, 32)                      # already there
    c.reserve(1, 1)
    assert c.block_table[0, :2].tolist() == [0, 1] and c.block_table[1, 0].item() == 2
    with pytest.raises(msa.MsaError) as e:
        c.reserve(1, 49)                  # more than max_pages
    assert e.value.status == -3
    c.reserve(1, 48)
    with pytest.raises(msa.MsaError):
        c.reserve(0, 33)                  # the pool is empty
    c.cache_len[0] = 20
    c.release(0)
    assert c.cache_len[0].item() == 0
    c.reserve(0, 1)
    assert c.block_table[0, 0].item() == 0
    assert sorted(c.owned[0] + c.owned[1] + c.free) == list(range(5))


def test_paged_cache_names_no_page_that_a_sequence_does_not_own():
    """Entries without a page are -1, from the start and after a release."""
    c = pipeline.PagedCache(torch.float32, 5, 16, 1, 64, 2, 3, "cpu")
    assert bool((c.block_table == -1).all())
    c.reserve(0, 17)
    assert c.block_table.tolist() == [[0, 1, -1], [-1, -1, -1]]
    c.release(0)
    assert bool((c.block_table == -1).all())
    c.reserve(1, 33)                      # the released pages are sequence 1's now
    assert c.block_table[0].tolist() == [-1] * 3 and c.owned[1] == [0, 1, 2]


# ------------------------------------------------- the tcgen05 kernel's flags

def _flag_overwritten(n_flags, n_sched, items=9, warps=2):
    """Whether some order of the tcgen05 tree attention's steps lets an item
    write its flag, bad[item % n_flags], before a warp has read that of an
    earlier item.  The roles are those of csrc/tree_attn_tc.cu with one query
    tile and items of one key tile: the MMA thread issues S(v) once the item is
    published and P V(v - 2) has been issued, P V(v) once every warp of stream
    v & 1 has written P(v) and left O(v - 2); a warp takes note of every item,
    and of its stream's own writes the flag between S and P and reads it after
    P V.  All orders are tried."""
    start = (((0, 0),) * (2 * warps), 0, 0)  # (item, step) of a warp; S, P V issued
    seen, todo = {start}, [start]
    while todo:
        ws, vs, vp = todo.pop()
        of = [i // warps for i in range(2 * warps)]

        def past(k, step, stream=None):
            return all(w >= (k, step) for i, w in enumerate(ws) if stream in (None, of[i]))

        def published(k):
            return k < n_sched or (past(k - n_sched, 1) and vp > k - n_sched)

        after = []
        if vs < min(items, vp + 2) and published(vs):
            after.append((ws, vs + 1, vp))
        if vp < vs and past(vp, 2, vp & 1) and (vp < 2 or past(vp - 1, 0, vp & 1)):
            after.append((ws, vs, vp + 1))
        for i, (k, step) in enumerate(ws):
            to = None
            if k < items and step == 0 and published(k):
                to = (k, 1) if k & 1 == of[i] else (k + 1, 0)
            elif step == 1 and vs > k:
                if any(j & 1 == of[x] and j < k and j % n_flags == k % n_flags and s > 0
                       for x, (j, s) in enumerate(ws)):
                    return True
                to = (k, 2)
            elif step == 2 and vp > k:
                to = (k + 1, 0)
            if to:
                after.append((ws[:i] + (to,) + ws[i + 1:], vs, vp))
        todo += [a for a in after if a not in seen]
        seen.update(after)
    return False


def test_tree_attention_flags_outlive_their_readers():
    import re
    path = os.path.join(msa.PKG, "csrc", "tree_attn_tc.cu")
    with open(path, encoding="utf-8") as f:
        text = f.read()
    n_sched = int(re.search(r"constexpr int kSched = (\d+);", text).group(1))
    extra = int(re.search(r"constexpr int kBad = kSched \+ (\d+);", text).group(1))
    assert "int bad[kBad];" in text and text.count("aux.bad[k % kBad]") == 2
    assert _flag_overwritten(n_sched, n_sched)
    assert not _flag_overwritten(n_sched + extra, n_sched)
