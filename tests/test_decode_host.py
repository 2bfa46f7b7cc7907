"""Decoding without a GPU: the oracle's pins, and what the C ABI and the binding refuse
before they touch the device."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import learned_token_pruning_gate_b200 as tg
from learned_token_pruning_gate_b200 import build as tgbuild
from learned_token_pruning_gate_b200 import inputs as gen
from oracle import decode as do
from oracle import delta as dd
from oracle import stack as so

OK, INVALID, SHAPE, DTYPE, ALIGN, UNSUP, WORKSPACE = 0, 1, 2, 3, 4, 5, 8


def _p(n):
    """A pointer that is aligned and never dereferenced; different n do not overlap."""
    return ctypes.c_void_p((n + 1) << 40)


ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    tgbuild.build()
    return tg.library()


# ---- the oracle's pins -------------------------------------------------------------------------


def test_paged_attention_is_the_last_row_of_causal_attention():
    lens, Hq, Hkv, d, page = [5, 33, 16], 4, 2, 64, 16
    p = gen.paged_inputs(lens, Hq, Hkv, d, page, 1, "fp32")
    out, _, _ = do.paged_attention(*[p[n].numpy() for n in ("q", "k_pages", "v_pages", "table", "lens",
                                                             "logsig_pages", "gain", "temp")])
    for b, n in enumerate(lens):
        at = [(int(p["table"][b, j // page]), j % page) for j in range(n)]
        k = np.stack([p["k_pages"].numpy()[i, :, o] for i, o in at])
        v = np.stack([p["v_pages"].numpy()[i, :, o] for i, o in at])
        ls = np.array([p["logsig_pages"].numpy()[i, o] for i, o in at])
        q = np.zeros((n, Hq, d))
        q[-1] = p["q"][b].numpy()
        want = so.gated_attention(q, k, v, [0, n], ls, p["gain"].numpy(), p["temp"].numpy())[-1]
        assert np.allclose(out[b], want, rtol=1e-12, atol=1e-12)


def test_paged_attention_leaves_masked_tokens_out():
    p = gen.paged_inputs([20], 2, 1, 64, 16, 2, "fp32")
    a = {n: t.numpy().copy() for n, t in p.items()}
    names = ("q", "k_pages", "v_pages", "table", "lens", "logsig_pages", "gain", "temp")
    a["logsig_pages"][a["table"][0, 1], :4] = -np.inf  # the last four tokens
    out, lse, _ = do.paged_attention(*[a[n] for n in names])
    a["lens"][0] = 16
    short, slse, _ = do.paged_attention(*[a[n] for n in names])
    assert np.array_equal(out, short) and np.array_equal(lse, slse)
    a["logsig_pages"][:] = -np.inf
    out, lse, _ = do.paged_attention(*[a[n] for n in names])
    assert not out.any() and (lse == -np.inf).all()


def test_delta_step_is_the_scan():
    cu, q, k, v, la, beta = gen.delta_inputs([6], 2, 16, 3, "fp32")
    a = [x.numpy() for x in (q, k, v, la, beta)]
    o, s = dd.scan(*a, cu)
    state = np.zeros((1, 2, 16, 16))
    for t in range(6):
        out, state = do.delta_step(*[x[t:t + 1] for x in a], state)
        assert np.allclose(out[0], o[t], rtol=1e-12, atol=1e-12)
    assert np.allclose(state, s, rtol=1e-12, atol=1e-12)
    out, new = do.delta_step(*[x[:2] for x in a], state, parent=[0, -1])
    fresh, _ = do.delta_step(*[x[1:2] for x in a], np.zeros((1, 2, 16, 16)))
    assert np.array_equal(out[1], fresh[0]) and new.shape[0] == 2


def test_beam_select_is_brute_force():
    rng = np.random.default_rng(2)
    x, s = rng.standard_normal((6, 9)), rng.standard_normal((2, 3))
    best, parent, token = do.beam_select(x, s, 4)
    for g in range(2):
        every = []
        for b, t in itertools.product(range(3), range(9)):
            row = x[g * 3 + b]
            every.append((-(s[g, b] + np.log(np.exp(row[t]) / np.exp(row).sum())), g * 3 + b, t))
        every.sort()
        assert [(p, t) for p, t in zip(parent[g], token[g])] == [(p, t) for _, p, t in every[:4]]
        assert np.allclose(best[g], [-e[0] for e in every[:4]])


def test_cache_update_keeps_every_sequence_its_own_tokens():
    """A hundred steps of random forks and growth, tokens tracked one by one: no sequence ever reads
    another's, counts equal the tables' entries, and compaction changes nothing of that."""
    rng = np.random.default_rng(7)
    page, P, width, B = 4, 24, 6, 5
    # (the oracle takes any page size; the tokens are numbers in place of k and v)
    table, lens, refs = np.full((B, width), -1), np.zeros(B, int), np.zeros(P, int)
    pool = np.zeros((P, page), int)
    owned = [[] for _ in range(B)]
    token, refused = 1, 0
    for step in range(100):
        parent = rng.integers(-1 if step % 3 == 0 else 0, B, B)
        new = rng.integers(0, 4, B)
        cu = np.concatenate([[0], np.cumsum(new)])
        table, lens, refs, start, src, dst = do.cache_update(table, lens, refs, page, parent, cu)
        for a, b in zip(src, dst):
            if b >= 0:
                pool[b] = pool[a]
        owned = [list(owned[p]) if p >= 0 else [] for p in parent]
        for i in range(B):
            refused += start[i] < 0
            for j in range(new[i] if start[i] >= 0 else 0):
                pos = start[i] + j
                pool[table[i, pos // page], pos % page] = token
                owned[i].append(token)
                token += 1
        if step % 10 == 9:
            table, refs, _, src, dst, counts = do.cache_compact(table, lens, refs, page)
            for a, b in zip(src, dst):
                if b >= 0:
                    pool[b] = pool[a]
            assert (refs[:counts[0]] > 0).all() and not refs[counts[0]:].any()
        held = np.zeros(P, int)
        for i in range(B):
            assert [pool[table[i, j // page], j % page] for j in range(lens[i])] == owned[i]
            for p in table[i, :do.pages_for(lens[i], page)]:
                held[p] += 1
        assert np.array_equal(held, refs)
    assert refused > 0


# ---- refusals of the C ABI ---------------------------------------------------------------------


def test_paged_attention_refusals(L):
    def call(q=_p(0), k=_p(1), v=_p(2), dt=0, B=2, Hq=4, Hkv=2, d=64, P=8, page=16, table=_p(3), mp=4, lens=_p(4),
             gain=_p(5), temp=_p(6), out=_p(7), ws=None, nb=0):
        return L.tg_paged_attention(q, k, v, dt, B, Hq, Hkv, d, P, page, table, mp, lens, None, gain, temp, out, None,
                                    ws, nb, None)
    assert call(dt=5) == DTYPE
    assert call(Hq=5) == SHAPE and call(Hkv=0) == SHAPE
    for kw in (dict(d=96), dict(d=256), dict(page=8), dict(page=48), dict(page=256), dict(B=1025), dict(P=2 ** 20 + 1),
               dict(mp=2 ** 20 + 1), dict(Hq=2048, Hkv=1024)):
        assert call(**kw) == UNSUP, kw
    for kw in (dict(B=-1), dict(P=-1), dict(mp=-1), dict(q=None), dict(lens=None), dict(gain=None), dict(temp=None),
               dict(out=None), dict(table=None), dict(k=None), dict(v=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(out=ODD)):
        assert call(**kw) == ALIGN, kw
    assert call(B=0, q=None) == OK
    assert call(B=1024, page=128, mp=2 ** 20) == UNSUP
    n = ctypes.c_size_t(7)
    assert L.tg_paged_attention_workspace_bytes(0, 2, 5, 2, 64, ctypes.byref(n)) == SHAPE and n.value == 0
    assert L.tg_paged_attention_workspace_bytes(0, 2, 4, 2, 64, None) == INVALID
    assert L.tg_paged_attention_workspace_bytes(0, 0, 4, 2, 64, ctypes.byref(n)) == OK and n.value == 0
    assert L.tg_paged_attention_workspace_bytes(0, 2, 4, 2, 64, ctypes.byref(n)) == OK
    if n.value:
        assert call(ws=_p(8), nb=n.value - 1) == WORKSPACE
        assert call(ws=ODD, nb=n.value) == ALIGN


def test_cache_refusals(L):
    def update(ti=_p(0), li=_p(1), Bi=2, ri=_p(2), P=8, page=16, mp=4, parent=_p(3), Bo=2, cu=_p(4), to=_p(5), lo=_p(6),
               ro=_p(7), st=_p(8), cs=_p(9), cd=_p(10)):
        return L.tg_cache_update(ti, li, Bi, ri, P, page, mp, parent, Bo, cu, to, lo, ro, st, cs, cd, None)
    assert update(parent=None, Bo=3) == SHAPE
    for kw in (dict(Bi=1025), dict(Bo=1025), dict(page=20), dict(P=2 ** 20 + 1), dict(mp=2 ** 20 + 1)):
        assert update(**kw) == UNSUP, kw
    for kw in (dict(Bi=-1), dict(Bo=-1), dict(P=-1), dict(mp=-1), dict(ti=None), dict(li=None), dict(ri=None),
               dict(to=None), dict(lo=None), dict(ro=None), dict(st=None), dict(cs=None), dict(cd=None)):
        assert update(**kw) == INVALID, kw
    # a table or lengths in place are for calls without parents; nothing else may overlap
    for kw in (dict(to=_p(0)), dict(lo=_p(1)), dict(st=_p(8), cs=_p(8)), dict(cu=_p(5)), dict(parent=_p(6)),
               dict(ro=_p(0)), dict(ro=ctypes.c_void_p(_p(2).value + 4)),
               dict(parent=None, to=ctypes.c_void_p(_p(0).value + 16))):
        assert update(**kw) == INVALID, kw
        assert b"overlap" in L.tg_last_error_message()

    def compact(t=_p(0), ln=_p(1), B=2, r=_p(2), P=8, page=16, mp=4, to=_p(3), ro=_p(4), pm=_p(5), cs=_p(6), cd=_p(7), n=_p(8)):
        return L.tg_cache_compact(t, ln, B, r, P, page, mp, to, ro, pm, cs, cd, n, None)
    for kw in (dict(t=None), dict(ln=None), dict(r=None), dict(to=None), dict(ro=None), dict(pm=None), dict(cs=None),
               dict(cd=None), dict(n=None), dict(B=-1), dict(pm=_p(2)), dict(cs=_p(7)), dict(to=_p(1))):
        assert compact(**kw) == INVALID, kw
    assert compact(page=0) == UNSUP and compact(B=2000) == UNSUP

    pool = (tg.PagePool * 9)()
    for x in pool:
        x.base, x.page_bytes, x.layers = 1 << 40, 4096, 2
    copy = lambda n_pools=1, P=8, src=_p(0), dst=_p(1), n=4: L.tg_cache_copy_pages(pool, n_pools, P, src, dst, n, None, None)  # noqa: E731
    assert copy(n_pools=9) == UNSUP
    for kw in (dict(n_pools=-1), dict(P=-1), dict(n=-1), dict(src=None), dict(dst=None)):
        assert copy(**kw) == INVALID, kw
    assert L.tg_cache_copy_pages(None, 1, 8, _p(0), _p(1), 4, None, None) == INVALID
    assert copy(n=0) == OK and copy(P=0) == OK and copy(n_pools=0) == OK
    pool[0].page_bytes = 24
    assert copy() == ALIGN
    pool[0].page_bytes, pool[0].base = 4096, (1 << 40) + 8
    assert copy() == ALIGN
    pool[0].base, pool[0].page_bytes = 1 << 40, 0
    assert copy() == SHAPE
    pool[0].page_bytes = 1 << 31
    assert copy() == UNSUP

    def append(k=_p(0), v=_p(1), dt=0, rows=3, B=2, cu=_p(2), st=_p(3), Hkv=2, d=64, P=8, page=16, t=_p(4), mp=4, kp=_p(5),
               vp=_p(6)):
        return L.tg_cache_append(k, v, None, dt, rows, B, cu, st, Hkv, d, P, page, t, mp, kp, vp, None, None)
    assert append(dt=3) == DTYPE and append(Hkv=0) == SHAPE and append(d=0) == SHAPE and append(d=4) == ALIGN
    for kw in (dict(k=None), dict(v=None), dict(cu=None), dict(st=None), dict(t=None), dict(kp=None), dict(vp=None),
               dict(rows=-1), dict(rows=2 ** 31)):
        assert append(**kw) == INVALID, kw
    for kw in (dict(kp=_p(0)), dict(vp=_p(1)), dict(vp=_p(5)), dict(vp=ctypes.c_void_p(_p(0).value + 256))):
        assert append(**kw) == INVALID and b"overlap" in L.tg_last_error_message(), kw
    assert append(kp=ODD) == ALIGN and append(page=100) == UNSUP and append(rows=0) == OK


def test_delta_step_refusals(L):
    def call(q=_p(0), k=_p(1), v=_p(2), dt=0, la=_p(3), be=_p(4), B=2, H=2, d=64, eps=1e-6, s=_p(5), S=2, parent=None,
             so_=_p(6), out=_p(7)):
        return L.tg_gated_delta_step(q, k, v, dt, la, be, B, H, d, eps, s, S, parent, so_, out, None)
    assert call(dt=9) == DTYPE and call(H=0) == SHAPE and call(S=1) == SHAPE and call(d=32) == UNSUP
    assert call(B=2 ** 20, H=2 ** 10, S=2 ** 20) == UNSUP
    for kw in (dict(B=-1), dict(S=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(q=None), dict(k=None), dict(v=None),
               dict(la=None), dict(be=None), dict(s=None), dict(so_=None), dict(out=None), dict(parent=_p(8), so_=_p(5)),
               dict(so_=ctypes.c_void_p(_p(5).value + 16))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(out=_p(0)), dict(out=_p(2)), dict(out=_p(5)), dict(out=_p(6)), dict(so_=_p(1)), dict(parent=_p(7))):
        assert call(**kw) == INVALID and b"overlap" in L.tg_last_error_message(), kw
    assert call(q=ODD) == ALIGN and call(s=ODD) == ALIGN and call(so_=ODD) == ALIGN
    assert call(B=0, q=None) == OK


def test_beam_select_refusals(L):
    def call(x=_p(0), dt=0, s=_p(1), G=2, beams=3, V=100, n=4, so_=_p(2), p=_p(3), t=_p(4), ws=_p(5), nb=1 << 30):
        return L.tg_beam_select(x, dt, s, G, beams, V, n, so_, p, t, ws, nb, None)
    assert call(dt=2) == DTYPE
    assert call(beams=0) == SHAPE and call(V=0) == SHAPE and call(n=0) == SHAPE and call(G=-1) == INVALID
    assert call(beams=33) == UNSUP and call(n=65) == UNSUP and call(V=2 ** 20 + 1) == UNSUP and call(G=2 ** 20) == UNSUP
    for kw in (dict(x=None), dict(s=None), dict(so_=None), dict(p=None), dict(t=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(so_=_p(1)), dict(p=_p(2)), dict(t=_p(0)), dict(ws=_p(0)), dict(ws=_p(3))):
        assert call(**kw) == INVALID and b"overlap" in L.tg_last_error_message(), kw
    assert call(ws=None) == WORKSPACE and call(nb=16) == WORKSPACE
    assert call(x=ODD) == ALIGN and call(ws=ODD) == ALIGN
    assert call(G=0, x=None) == OK
    n = ctypes.c_size_t(7)
    assert L.tg_beam_select_workspace_bytes(2, 0, 100, 4, ctypes.byref(n)) == SHAPE and n.value == 0
    assert L.tg_beam_select_workspace_bytes(2, 3, 100, 4, None) == INVALID
    assert L.tg_beam_select_workspace_bytes(2, 3, 100, 4, ctypes.byref(n)) == OK and n.value > 0


# ---- refusals of the binding -------------------------------------------------------------------


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match) as e:
        fn(*a, **kw)
    assert "CUDA tensors only" not in str(e.value)


def test_binding_rejects_mismatched_operands():
    p = gen.paged_inputs([20, 3], 4, 2, 64, 16, 1, fill=0.0)
    a = [p[n] for n in ("q", "k_pages", "v_pages", "table", "lens")]

    def attn(i=None, x=None, **kw):
        b = list(a)
        if i is not None:
            b[i] = x
        return tg.paged_attention, *b

    for match, i, x in (("q must be", 0, a[0][0]), ("k_pages", 0, a[0].float()), ("k_pages must", 1, a[1][0]),
                        ("v_pages: shape", 2, a[2][1:]), ("v_pages: dtype", 2, a[2].float()),
                        ("table must", 3, a[3][0]), ("table: dtype", 3, a[3].long()), ("lens: shape", 4, a[4][:1]),
                        ("lens: dtype", 4, a[4].long()), ("q must be contiguous", 0, a[0].transpose(0, 1).contiguous().transpose(0, 1)),
                        ("k_pages must be contiguous", 1, a[1].transpose(1, 2).contiguous().transpose(1, 2)),
                        ("k_pages", 0, torch.zeros(2, 4, 128, dtype=torch.bfloat16)),
                        ("multiple", 0, torch.zeros(2, 3, 64, dtype=torch.bfloat16)),
                        ("table: 2 sequences", 0, torch.zeros(3, 4, 64, dtype=torch.bfloat16))):
        fn, *b = attn(i, x)
        _raises(match, fn, *b)
    for match, kw in (("logsig_pages: shape", dict(logsig_pages=p["logsig_pages"][1:])), ("gain: shape", dict(gain=torch.ones(3))),
                      ("temp: dtype", dict(temp=torch.ones(4).double())), ("out: shape", dict(out=a[0][:1])),
                      ("lse: shape", dict(lse=torch.zeros(2, 4))), ("workspace", dict(workspace=torch.zeros(8)))):
        _raises(match, tg.paged_attention, *a, **kw)
    t, ln, r = p["table"], p["lens"], torch.zeros(9, dtype=torch.int32)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for match, kw in (("parent: dtype", dict(parent=torch.zeros(2).long())), ("cu_new: shape", dict(cu_new=i32(2))),
                      ("table_out: shape", dict(table_out=i32(2, 9))), ("refs_out", dict(refs_out=i32(8))),
                      ("lens_out", dict(lens_out=i32(3))), ("start", dict(start=i32(1))),
                      ("copy_dst", dict(parent=i32(3), copy_dst=i32(2)))):
        _raises(match, tg.cache_update, t, ln, r, 16, **kw)
    _raises("refs: dtype", tg.cache_update, t, ln, r.float(), 16)
    _raises("refs: dtype", tg.cache_compact, t, ln, r.long(), 16)
    _raises("refs_out", tg.cache_compact, t, ln, r, 16, refs_out=i32(3))
    pool = torch.zeros(2, 5, 16)
    _raises("too many", tg.cache_copy_pages, [pool] * 9, i32(1), i32(1))
    _raises("copy_dst", tg.cache_copy_pages, [pool], i32(2), i32(1))
    _raises("count", tg.cache_copy_pages, [pool], i32(1), i32(1), i32(2))
    _raises("pools: ", tg.cache_copy_pages, [pool, torch.zeros(2, 6, 16)], i32(1), i32(1))
    _raises("pools: ", tg.cache_copy_pages, [torch.zeros(5)], i32(1), i32(1))
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    args = lambda **kw: [kw.get(n, x) for n, x in dict(k=k, v=k, cu=i32(3), st=i32(2), t=t, kp=a[1], vp=a[2]).items()]  # noqa: E731
    for match, kw in (("k: dtype", dict(k=k.float())), ("v: shape", dict(v=k[:2])), ("cu_new", dict(cu=i32(2))),
                      ("start", dict(st=i32(3))), ("v_pages", dict(vp=a[2][1:]))):
        _raises(match, tg.cache_append, *args(**kw))
    _raises("logsig without", tg.cache_append, *args(), logsig=torch.zeros(3))
    q, st, g = torch.zeros(2, 3, 64), torch.zeros(2, 3, 64, 64), torch.zeros(2, 3)
    for match, b in (("k: shape", (q, q[:1], q, g, g, st)), ("log_alpha", (q, q, q, g[:1], g, st)),
                     ("beta: dtype", (q, q, q, g, g.double(), st)), ("state: shape", (q, q, q, g, g, st[:, :2])),
                     ("1 states", (q, q, q, g, g, st[:1])), ("must be", (q[0], q, q, g, g, st))):
        _raises(match, tg.gated_delta_step, *b)
    _raises("parent", tg.gated_delta_step, q, q, q, g, g, st, parent=i32(3))
    _raises("state_out", tg.gated_delta_step, q, q, q, g, g, st, state_out=st[:1])
    x, s = torch.zeros(6, 10), torch.zeros(2, 3)
    _raises("logits: shape", tg.beam_select, x[:5], s)
    _raises("scores: dtype", tg.beam_select, x, s.double())
    _raises("workspace", tg.beam_select, x, s, 2, torch.zeros(4))


# ---- the decoder's host side -------------------------------------------------------------------


def test_forked_positions_stay_in_range():
    """Parents outside the batch index nothing: such a sequence starts over, as in the cache."""
    from learned_token_pruning_gate_b200.pipeline import _forked

    pos = torch.tensor([7, 9, 4], dtype=torch.int32)
    for parent, want in (([2, 0, 0], [4, 7, 7]), ([-1, 1, -1], [0, 9, 0]), ([3, 2 ** 31 - 1, 2], [0, 0, 4]),
                         ([-2, -2 ** 31, 1], [0, 0, 9])):
        got = _forked(pos, torch.tensor(parent, dtype=torch.int32))
        assert got.tolist() == want and got.dtype == torch.int32


def test_decoder_refuses_a_cache_too_small_for_its_prefill():
    """Pages and tables are counted against the kept rows before anything is allocated."""
    from types import SimpleNamespace

    from learned_token_pruning_gate_b200.pipeline import GatedDecoder

    ck = np.array([0, 33, 33, 49], np.int32)  # pages of 16: 3, 0 and 1
    stack = SimpleNamespace(ck=ck, cu=4 * ck, layers=[None], Hq=2, Hkv=1, dh=64,
                            cache_k=torch.zeros((1, 49, 1, 64)))
    for pages, max_pages in ((3, 3), (4, 2), (0, 0)):
        with pytest.raises(ValueError, match="take 4 pages, 3 of one prompt"):
            GatedDecoder(stack, pages, 16, max_pages, beams=2)
    d = GatedDecoder(stack, 4, 16, 3, beams=2)
    assert d.cu_prefill.tolist() == [0, 33, 33, 33, 33, 49, 49] and d.cache.k.shape == (1, 4, 1, 16, 64)
    none = SimpleNamespace(**dict(vars(stack), ck=np.zeros(1, np.int32), cu=np.zeros(1, np.int32)))
    assert GatedDecoder(none, 1, 16, 1).batch == 0


def test_paged_attention_refuses_overlap(L):
    """Outputs and workspace in one another or in an input, but for out == q."""
    def call(q=_p(0), k=_p(1), v=_p(2), B=2, Hq=4, Hkv=2, d=64, P=8, page=16, table=_p(3), mp=4, lens=_p(4), ls=_p(9),
             gain=_p(5), temp=_p(6), out=_p(7), lse=_p(8), ws=None, nb=0):
        return L.tg_paged_attention(q, k, v, 0, B, Hq, Hkv, d, P, page, table, mp, lens, ls, gain, temp, out, lse, ws, nb,
                                    None)
    at = lambda n, off: ctypes.c_void_p(_p(n).value + off)  # noqa: E731
    # (q and out: 1024 bytes; k and v: 32768; table 32, lens 8, log-gates 512, gain and temp 16, lse 32)
    refused = [dict(out=at(0, 16)), dict(out=at(1, 32752)), dict(out=at(2, 0)), dict(out=at(3, 16)), dict(out=at(4, 0)),
               dict(out=at(9, 496)), dict(out=at(5, 0)), dict(out=at(6, 0)), dict(out=at(8, 16)), dict(lse=at(0, 1020)),
               dict(lse=at(1, 4)), dict(lse=at(3, 28)), dict(lse=at(4, 4)), dict(lse=at(9, 508)), dict(lse=at(5, 12)),
               dict(lse=at(6, 0)), dict(lse=at(7, 1020)), dict(out=_p(0), lse=at(0, 0))]
    n = ctypes.c_size_t(0)
    assert L.tg_paged_attention_workspace_bytes(0, 2, 4, 2, 64, ctypes.byref(n)) == OK and n.value > 0
    refused += [dict(ws=at(i, 0), nb=n.value) for i in range(10)]
    for kw in refused:
        assert call(**kw) == INVALID and b"overlap" in L.tg_last_error_message(), kw
    assert call(B=0, out=at(0, 16)) == OK  # (nothing is read or written)
