"""Decoding calls run together: a stack's prefill and single steps against the whole
stack in fp64, and a beam search over a paged cache and delta-rule states against every
hypothesis computed from its own history."""
import numpy as np
import pytest
import torch

import learned_token_pruning_gate_b200 as tg
from learned_token_pruning_gate_b200 import inputs as gen
from learned_token_pruning_gate_b200.pipeline import GatedDecoder, GatedStack, PagedCache
from oracle import decode as do
from oracle import delta as dd
from oracle import stack as so
from tests.parity_utils import assert_close, dev, host_f32

pytestmark = pytest.mark.gpu


def _decoder(lens, new, n_layers, dm, Hq, Hkv, dh, inter, dtype, page, beams=1, seed=7):
    """A decoder behind a prefill of `lens` kept rows, and the residuals of `new` more tokens each."""
    cu, pos, x0, ls, layers = gen.stack_inputs(lens, n_layers, dm, Hq, Hkv, dh, inter, seed, dtype)
    span = 4 * np.asarray(lens)
    cu_seq = np.concatenate([[0], np.cumsum(span)]).astype(np.int32)
    kept = (np.repeat(cu_seq[:-1], lens) + pos).astype(np.int32)
    st = GatedStack([{k: dev(v) for k, v in ly.items()} for ly in layers], Hq, Hkv, dh, cu_seq, cu,
                    dev(torch.from_numpy(kept)), dev(ls))
    width = max(do.pages_for(n + new, page) for n in lens)
    pages = sum(do.pages_for(n + new, page) for n in lens) * beams + 2
    g = torch.Generator().manual_seed(seed)
    fresh = torch.randn((new, len(lens) * beams, dm), generator=g).to(x0.dtype)
    return GatedDecoder(st, pages, page, width, beams), cu, pos, x0, ls, layers, fresh


def _whole(lens, cu, pos, x0, ls, layers, fresh, Hq, Hkv, dh):
    """The stack in fp64 over each prompt's kept rows and its new tokens behind them."""
    lay = [{k: host_f32(v).astype(np.float64) for k, v in ly.items()} for ly in layers]
    x, p, gates, cu2 = [], [], [], [0]
    for b, n in enumerate(lens):
        x += [host_f32(x0)[cu[b]:cu[b + 1]], host_f32(fresh)[:, b]]
        p += [pos[cu[b]:cu[b + 1]], 4 * n + np.arange(len(fresh))]
        gates += [ls.numpy()[cu[b]:cu[b + 1]], np.zeros(len(fresh))]
        cu2.append(cu2[-1] + n + len(fresh))
    out, _, _ = so.stack(np.concatenate(x), np.concatenate(p), np.array(cu2), np.concatenate(gates), lay, Hq, Hkv, dh)
    return [out[cu2[b] + n:cu2[b + 1]] for b, n in enumerate(lens)]


@pytest.mark.parametrize("lens,new,n_layers,dm,Hq,Hkv,dh,inter,dtype,page", [
    ([30, 0, 17], 5, 2, 256, 4, 2, 64, 512, "bf16", 16),
    ([64, 129], 3, 1, 512, 8, 1, 128, 512, "bf16", 64),
    ([20, 45], 14, 2, 128, 4, 4, 64, 256, "fp32", 32),
])
def test_steps_continue_the_stack(lens, new, n_layers, dm, Hq, Hkv, dh, inter, dtype, page):
    """Per element 2e-2 rms + 2e-2 |ref| in bf16: the budget of the stack's own parity test, whose
    roundings a step shares (bf16 residual, eight intermediates per layer).  fp32: the GEMMs and
    sums of at most 512 terms, 2^-24 each, over two layers: 1e-4 rms + 1e-4."""
    d, cu, pos, x0, ls, layers, fresh = _decoder(lens, new, n_layers, dm, Hq, Hkv, dh, inter, dtype, page)
    want = _whole(lens, cu, pos, x0, ls, layers, fresh, Hq, Hkv, dh)
    d.prefill(dev(x0).clone())
    d.step(dev(fresh[0]).clone())
    d.prefill(dev(x0).clone())  # starts over
    tol = 2e-2 if dtype == "bf16" else 1e-4
    for t in range(new):
        got = host_f32(d.step(dev(fresh[t]).clone()))
        assert tg.device_status() == 0
        for b in range(len(lens)):
            ref = want[b][t]
            assert_close(f"prompt {b} token {t}", got[b], ref, tol * np.sqrt(np.mean(ref ** 2)), tol)
    assert d.cache.lens.tolist() == [n + new for n in lens]
    pos, held = d.pos.clone(), d.cache.lens.clone()
    for x, parent in ((dev(fresh[0])[:, :-1].contiguous(), None), (dev(fresh[0]).double(), None),
                      (dev(fresh[0]), torch.zeros(len(lens), dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):  # refused before anything moves on
            d.step(x, parent)
    assert torch.equal(d.pos, pos) and torch.equal(d.cache.lens, held)


def test_forked_steps_and_replay():
    """Beams that fork from one another see their own history, and a captured pair of forked steps
    replays to the same result."""
    lens, new, beams, page = [21, 40], 6, 3, 16
    args = (1, 128, 4, 2, 64, 256)
    d, cu, pos, x0, ls, layers, fresh = _decoder(lens, new, *args, "fp32", page, beams=beams)
    parents = [np.repeat(np.arange(2) * beams, beams), np.array([0, 0, 2, 5, 4, 3]), np.array([1, 0, 0, 3, 3, 3]),
               np.array([2, 1, 0, 3, 4, 4]), None, np.array([0, 0, 0, 5, 5, 5])]
    parents = [None if p is None else dev(torch.tensor(p, dtype=torch.int32)) for p in parents]

    def search():
        d.prefill(dev(x0).clone())
        outs = []
        for t in range(new):
            outs.append(d.step(dev(fresh[t]).clone(), parents[t]))
        return torch.stack(outs)
    outs = search()
    torch.cuda.synchronize()
    assert tg.device_status() == 0
    # each beam's own history of new tokens, run through the whole stack
    hist = [[] for _ in range(2 * beams)]
    for t in range(new):
        if parents[t] is not None:
            hist = [list(hist[p]) for p in parents[t].tolist()]
        for i in range(2 * beams):
            hist[i].append((t, i))
    for i in range(2 * beams):
        b = i // beams
        mine = torch.stack([fresh[t][j] for t, j in hist[i]])[:, None]
        want = _whole([lens[b]], np.array([0, lens[b]]), pos[cu[b]:cu[b + 1]], x0[cu[b]:cu[b + 1]], ls[cu[b]:cu[b + 1]],
                      layers, mine, 4, 2, 64)[0][-1]
        assert_close(f"beam {i}", host_f32(outs[-1])[i], want, 1e-4 * np.sqrt(np.mean(want ** 2)), 1e-4)
    refs = np.zeros(d.cache.refs.shape[0], np.int32)
    for row, n in zip(d.cache.table.tolist(), d.cache.lens.tolist()):
        for p in row[:do.pages_for(n, page)]:
            refs[p] += 1
    assert np.array_equal(refs, d.cache.refs.cpu().numpy())

    # compaction changes no sequence's tokens; freeing all of them frees every page
    counts = d.cache.compact()
    q = torch.randn((2 * beams, 4, 64), device="cuda")
    live, moved = counts.tolist()
    assert live == int((refs > 0).sum()) and not d.cache.refs[live:].any()
    before = [d.cache.attend(0, q).clone()]
    keep = torch.full((2 * beams,), -1, dtype=torch.int32, device="cuda")
    keep[1] = 1
    d.cache.free(keep)
    assert torch.equal(d.cache.attend(0, q)[1], before[0][1])
    keep[1] = -1
    d.cache.free(keep)
    assert not d.cache.refs.any() and not d.cache.attend(0, q).any()

    # the same search again on the freed cache, its last two forked steps captured and replayed
    d2, *_ = _decoder(lens, new, *args, "fp32", page, beams=beams)
    d2.prefill(dev(x0).clone())
    for t in range(4):
        d2.step(dev(fresh[t]).clone(), parents[t])
    c = d2.cache
    saved = [x.clone() for x in (c.k, c.v, c.logsig, *c._tables, *c._lens, c.refs, d2.pos)]
    xs = [dev(fresh[t]).clone() for t in (4, 5)]
    ident = dev(torch.arange(2 * beams, dtype=torch.int32))

    def pair(x4, x5):
        d2.step(x4, ident)
        d2.step(x5, parents[5])

    def restore():
        for x, s in zip((c.k, c.v, c.logsig, *c._tables, *c._lens, c.refs, d2.pos), saved):
            x.copy_(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pair(xs[0].clone(), xs[1].clone())  # warm
    torch.cuda.synchronize()
    restore()
    graph = torch.cuda.CUDAGraph()
    x4, x5 = xs[0].clone(), xs[1].clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        pair(x4, x5)
    for _ in range(2):
        restore()
        x4.copy_(xs[0])
        x5.copy_(xs[1])
        graph.replay()
        torch.cuda.synchronize()
        assert_close("replayed", host_f32(x5), host_f32(outs[-1]), 1e-6, 1e-6)


def test_beam_search_with_delta_states():
    """selection -> fork of pages and states -> one attention and one delta-rule step, for 7 tokens;
    every beam against its own history from scratch."""
    groups, beams, V, H, d, page, T = 2, 4, 301, 2, 64, 16, 7
    n = groups * beams
    rng = np.random.default_rng(3)
    f32 = lambda *s: rng.standard_normal(s, dtype=np.float32)  # noqa: E731
    emb = {x: torch.from_numpy(f32(V, H, d)).cuda() for x in ("q", "k", "v")}
    head = torch.from_numpy(f32(2 * H * d, V) * 0.3).cuda()
    la, be = torch.full((n, H), -0.05, device="cuda"), torch.full((n, H), 0.7, device="cuda")
    gain, temp = torch.rand(H, device="cuda"), torch.full((H,), 0.9, device="cuda")
    cache = PagedCache(1, 40, H, page, d, n, 4, torch.float32)
    states = [torch.zeros((n, H, d, d), device="cuda") for _ in range(2)]
    tokens = torch.arange(groups, device="cuda").repeat_interleave(beams) + 5
    scores = torch.full((groups, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    parent = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    hist = [[] for _ in range(n)]
    want_scores = np.where(np.arange(n) % beams == 0, 0.0, -np.inf)
    ws = tg.beam_select_workspace(groups, beams, V, beams)
    for t in range(T):
        cache.grow(parent=parent)
        q, k, v = (emb[x][tokens].contiguous() for x in ("q", "k", "v"))
        cache.append(0, k, v)
        o = cache.attend(0, q, gain, temp)
        y, _ = tg.gated_delta_step(q, k, v, la, be, states[t % 2], parent=parent, state_out=states[1 - t % 2])
        logits = torch.cat([o.reshape(n, -1), y.reshape(n, -1)], 1) @ head
        hist = [(list(hist[p]) if p >= 0 else []) + [int(x)] for p, x in zip(parent.tolist(), tokens.tolist())]
        for i in range(n):
            ids = hist[i]
            qs, ks, vs = (emb[x][torch.tensor(ids)].cpu().numpy().astype(np.float64) for x in ("q", "k", "v"))
            ref = so.gated_attention(qs, ks, vs, [0, len(ids)], np.zeros(len(ids)), gain.cpu().numpy(), temp.cpu().numpy())
            assert_close("attention", host_f32(o)[i], ref[-1], 2e-5, 1e-5)
            ry, _ = dd.scan(qs, ks, vs, np.full((len(ids), H), np.float32(-0.05)), np.full((len(ids), H), np.float32(0.7)),
                            [0, len(ids)])
            assert_close("delta rule", host_f32(y)[i], ry[-1], 2e-5, 1e-5)
        scores, parent, token = tg.beam_select(logits, scores, workspace=ws)
        _, wp, wt = do.beam_select(logits.cpu().numpy(), want_scores.reshape(groups, beams), beams)
        assert np.array_equal(parent.cpu().numpy(), wp) and np.array_equal(token.cpu().numpy(), wt)
        want_scores = scores.cpu().numpy().astype(np.float64).reshape(-1)
        parent, tokens = parent.reshape(-1).contiguous(), token.reshape(-1).long()
    assert tg.device_status() == 0
    assert all(len(h) == T for h in hist)


def test_out_of_pages_keeps_the_others():
    """A sequence that finds no page keeps its tokens and reads them; the others go on."""
    cache = PagedCache(1, 3, 1, 16, 64, 2, 4, torch.float32)
    cache.grow(dev(torch.tensor([0, 32, 48], dtype=torch.int32)))
    assert cache.start.tolist() == [0, 0]
    g = torch.Generator("cuda").manual_seed(0)
    k, v = (torch.randn((48, 1, 64), generator=g, device="cuda") for _ in range(2))
    cache.append(0, k, v)
    q = torch.randn((2, 2, 64), generator=g, device="cuda")
    before = cache.attend(0, q).clone()
    cache.grow()  # both need a page, there is none
    assert cache.start.tolist() == [-1, -1] and cache.lens.tolist() == [32, 16]
    cache.append(0, k[:2].contiguous(), v[:2].contiguous())
    assert torch.equal(cache.attend(0, q), before)
    cache.free(dev(torch.tensor([-1, 1], dtype=torch.int32)))
    cache.grow(dev(torch.tensor([0, 0, 1], dtype=torch.int32)))
    assert cache.start.tolist() == [0, 16] and cache.lens.tolist() == [0, 17]
    assert tg.device_status() == 0


def test_step_with_parents_outside_the_batch():
    """Parents that no sequence has: bit 64 of the status, those sequences start over, the others go on."""
    lens = [21, 40]
    d, cu, pos, x0, ls, layers, fresh = _decoder(lens, 3, 1, 128, 4, 2, 64, 256, "fp32", 16)
    i32 = lambda *p: dev(torch.tensor(p, dtype=torch.int32))  # noqa: E731
    d.prefill(dev(x0).clone())
    d.step(dev(fresh[0]).clone())
    want = d.pos.tolist()
    d.step(dev(fresh[1]).clone(), i32(10 ** 6, 1))
    torch.cuda.synchronize()
    assert tg.device_status() == 64
    assert d.cache.lens.tolist() == [1, 42] and d.pos.tolist() == [1, want[1] + 1]
    d.step(dev(fresh[2]).clone(), i32(0, -7))
    torch.cuda.synchronize()
    assert tg.device_status() == 64
    assert d.cache.lens.tolist() == [2, 1] and d.pos.tolist() == [2, 1]


def test_replayed_steps_after_an_odd_number_of_forks():
    """A step captured once is replayed behind later prefills and forks, however many: the same as eager."""
    lens, new, beams = [21, 40], 4, 2
    d, cu, pos, x0, ls, layers, fresh = _decoder(lens, new, 1, 128, 4, 2, 64, 256, "fp32", 16, beams=beams)
    e, *_ = _decoder(lens, new, 1, 128, 4, 2, 64, 256, "fp32", 16, beams=beams)
    fork = dev(torch.tensor([0, 0, 2, 2], dtype=torch.int32))
    swap = dev(torch.tensor([1, 0, 3, 3], dtype=torch.int32))
    d.prefill(dev(x0).clone())
    x = dev(fresh[0]).clone()
    d.step(x)  # (its buffers are allocated)
    graph, forked = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        d.step(x)
    with torch.cuda.graph(forked):
        d.step(x, swap)
    for turn in range(3):
        x1 = dev(x0) * (1.0 + turn)
        d.prefill(x1.clone())
        e.prefill(x1.clone())
        for t, (g, parent) in enumerate(((None, fork), (graph, None), (forked, swap), (graph, None))):
            x.copy_(dev(fresh[t]))
            if g is None:
                d.step(x, parent)
            else:
                g.replay()
            want = e.step(dev(fresh[t]).clone(), parent)
            assert_close(f"prefill {turn} step {t}", host_f32(x), host_f32(want), 1e-6, 1e-6)
            assert torch.equal(d.cache.lens, e.cache.lens) and torch.equal(d.cache.refs, e.cache.refs)
    assert tg.device_status() == 0
