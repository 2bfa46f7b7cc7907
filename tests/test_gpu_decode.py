"""GPU parity of the decoding calls (attention over a paged cache, the cache's pages,
the delta-rule step, beam selection) against the oracle (oracle/decode.py) on the
same inputs.

Error budgets, per element, u = half a step of the output type (2^-8 bf16, 2^-24 fp32):
  attention   A logit is a d-term fp32 sum of exact products: off by at most
              (d + 4) 2^-24 sum |q_i k_i| / (sqrt(d) tau) <= 1.3e-4 for the draws here
              (|q| |k| <= 2.5 d at d <= 128 with tau >= 0.8), typically a tenth of it;
              ex2.approx adds 2^-22.  A relative error e of the weights moves the output by
              at most 2 e sum_j w_j |v_j| (the oracle's magnitude), so fp32: 3e-4 magnitude.
              bf16 kernels may round each weight to bf16 (2^-8) and do round the output
              (2^-8 |out|): 2^-8 (|out| + magnitude) + 3e-4 magnitude.  lse: 2e-4.
  delta step  d-term fp32 sums of values of size |S| <= ~4: 1e-5 absolute + 1e-5 relative on
              the state; the output is rounded once (bf16: 2^-8 relative).
  beams       the score's 32-bit storage: 2^-24 relative, plus 1e-6 for the chunk sums.
Integers and copied bytes are equal."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import learned_token_pruning_gate_b200 as tg
from learned_token_pruning_gate_b200 import inputs as gen
from oracle import decode as do
from tests.parity_utils import assert_close, dev, host_f32

pytestmark = pytest.mark.gpu
PAGE_BIT = 64


@pytest.fixture(autouse=True)
def clean_status():
    yield
    torch.cuda.synchronize()
    assert tg.device_status() == 0


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ---- attention ---------------------------------------------------------------------------------


def _attend(p, workspace="auto", **kw):
    d = {n: dev(t) for n, t in p.items()}
    return tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"],
                              logsig_pages=d["logsig_pages"], gain=d["gain"], temp=d["temp"],
                              want_lse=True, workspace=workspace, **kw)


def _wide(p, entries=8192):
    """The same cache with room for more pages in the table: the kernel is chosen by what a table can hold."""
    t = torch.full((p["table"].shape[0], entries), -1, dtype=torch.int32)
    t[:, :p["table"].shape[1]] = p["table"]
    return dict(p, table=t)


def _check_attention(p, got, lse, what=""):
    h = {n: host_f32(t) if t.is_floating_point() else t.numpy() for n, t in p.items()}
    ref, rlse, mag = do.paged_attention(h["q"], h["k_pages"], h["v_pages"], h["table"], h["lens"],
                                        h["logsig_pages"], h["gain"], h["temp"])
    out = host_f32(got).astype(np.float64)
    bound = 3e-4 * mag + 1e-6
    if p["q"].dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + mag)
    assert bool(np.isfinite(out).all()), f"{what}: not finite"
    worst = (np.abs(out - ref) / bound).max(initial=0.0)
    assert worst <= 1.0, f"{what}: off by {worst:.2f} of the bound"
    lse = lse.cpu().numpy()
    empty = rlse == -np.inf
    assert np.array_equal(lse == -np.inf, empty)
    assert_close("lse", lse[~empty], rlse[~empty], 2e-4, 1e-6)


@pytest.mark.parametrize("lens,Hq,Hkv,d,page", [
    ([1], 4, 2, 64, 16),
    ([0], 4, 2, 64, 16),
    ([0, 1, 15, 16, 17, 0, 33], 4, 2, 64, 16),
    ([63, 64, 65, 127, 128, 129, 2], 16, 8, 128, 64),
    ([700, 3, 0, 1025], 16, 8, 128, 128),
    ([300, 31], 32, 4, 64, 32),       # 8 query heads to a kv head
    ([257, 5], 16, 1, 128, 16),       # one kv head for 16
    ([129, 40], 24, 1, 64, 32),       # more than 16 to a kv head
    ([77], 6, 2, 128, 64),            # a group of 3
    ([5000], 8, 8, 64, 16),           # no groups
    ([2304] * 2 + [1] * 30, 4, 2, 128, 64),
])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_matches_oracle(lens, Hq, Hkv, d, page, dtype):
    p = gen.paged_inputs(lens, Hq, Hkv, d, page, 3, dtype)
    _check_attention(p, *_attend(p), "as it is")
    _check_attention(p, *_attend(p, workspace=None), "without a workspace")
    _check_attention(p, *_attend(_wide(p)), "wide table")
    _check_attention(p, *_attend(_wide(p), workspace=None), "wide table, one SM")


@pytest.mark.parametrize("entries", [1, 2, 3, 5, 8, 9, 31, 32, 33, 100])
@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("bf16", 4, 2, 128), ("bf16", 24, 1, 64), ("fp32", 8, 2, 64)])
def test_attention_every_cluster_size(entries, dtype, Hq, Hkv, d):
    """Tables of 64 to 6400 tokens: a unit on one CTA, on clusters of two to eight, and on the list."""
    full = entries * 64
    lens = sorted({full, full - 1, max(full - 65, 0), full // 2, 1, 0})
    p = gen.paged_inputs(lens, Hq, Hkv, d, 64, entries, dtype, max_pages=entries)
    _check_attention(p, *_attend(p), "few")
    many = gen.paged_inputs([full] + [1] * 40, Hq, Hkv, d, 64, entries, dtype, max_pages=entries)
    _check_attention(many, *_attend(many), "many")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_masked_tokens(dtype):
    """Log-gates of -inf leave a token out, NaN or infinity in its k and v included; a sequence
    with nothing left has output 0; gates of the type's lowest value stay finite."""
    lens = [100, 40, 64, 33, 50]
    p = gen.paged_inputs(lens, 8, 4, 64, 32, 5, dtype)
    t, ls = p["table"], p["logsig_pages"]
    for b, gone in enumerate([range(0, 100, 3), range(40), range(16, 64), range(32), ()]):
        for j in gone:
            page, off = int(t[b, j // 32]), j % 32
            ls[page, off] = -float("inf")
            p["k_pages"][page, :, off] = float("nan")
            p["v_pages"][page, :, off] = float("nan") if j % 2 else float("inf")
    p["gain"][0] = 0.0  # 0 x -inf is still out
    p["gain"][1] = -0.5
    for j in range(0, 50, 2):  # lowest value on some tokens of the last: no weight under a positive gain
        ls[int(t[4, j // 32]), j % 32] = torch.finfo(torch.float32).min
    p["gain"][1:] = p["gain"][1:].abs()
    out, lse = _attend(p)
    h = {n: host_f32(x) if x.is_floating_point() else x.numpy() for n, x in p.items()}
    assert not host_f32(out)[1].any()
    _check_attention(p, out, lse, "masked")
    _check_attention(p, *_attend(p, workspace=None), "masked, without a workspace")
    _check_attention(p, *_attend(_wide(p)), "masked, wide table")
    assert h["gain"][0] == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_all_gates_lowest(dtype):
    """Every gate at the lowest fp32 value: q . k is below its last place, so all weights are equal."""
    p = gen.paged_inputs([70], 4, 2, 64, 16, 6, dtype)
    p["logsig_pages"][:] = torch.finfo(torch.float32).min
    p["gain"][:] = torch.tensor([1.0, 0.5, 0.9, 0.25])
    out, lse = _attend(p)
    v = host_f32(p["v_pages"])
    at = [(int(p["table"][0, j // 16]), j % 16) for j in range(70)]
    for h in range(4):
        x = np.stack([v[pg, h // 2, o] for pg, o in at])
        bound = 2.0 ** -8 * (np.abs(x).mean(0) + np.abs(x.mean(0))) + 1e-6 if dtype == "bf16" else 1e-5
        assert (np.abs(host_f32(out)[0, h] - x.mean(0)) <= bound).all()
    assert np.isfinite(lse.cpu().numpy()).all()


@pytest.mark.parametrize("widen", [lambda p: p, _wide])
def test_attention_defaults_and_workspace_reuse(widen):
    """No gates, gains or temperatures; one workspace over calls of different lengths and shapes."""
    p = widen(gen.paged_inputs([900, 20, 0, 411], 16, 8, 128, 64, 7))
    h = {n: host_f32(t) if t.is_floating_point() else t.numpy() for n, t in p.items()}
    ref, _, mag = do.paged_attention(h["q"], h["k_pages"], h["v_pages"], h["table"], h["lens"])
    d = {n: dev(t) for n, t in p.items()}
    ws = tg.paged_attention_workspace(4, 16, 8, 128)
    for _ in range(3):
        out, lse = tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"],
                                      workspace=ws)
        assert lse is None
        assert (np.abs(host_f32(out) - ref) <= 2.0 ** -8 * (np.abs(ref) + mag) + 3e-4 * mag + 1e-6).all()
        short = dev(torch.tensor([3, 0, 0, 1], dtype=torch.int32))
        tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], short, workspace=ws)
        alone = tg.paged_attention(d["q"][:1], d["k_pages"], d["v_pages"], d["table"][:1], d["lens"][:1],
                                   workspace=ws)[0]
        assert_close("one sequence alone", host_f32(alone), host_f32(out[:1]), 1e-5, 2.0 ** -7)
    inplace = d["q"].clone()
    tg.paged_attention(inplace, d["k_pages"], d["v_pages"], d["table"], d["lens"], workspace=ws, out=inplace)
    assert torch.equal(inplace, out)
    first = tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], workspace=ws)[0]
    assert torch.equal(first, out)


def test_attention_bad_table_and_lengths():
    """A page outside the pool is left out, a length outside the table is cut: bit 64 of the status."""
    p = gen.paged_inputs([64, 64], 4, 2, 64, 16, 8, max_pages=4)
    bad = dict(p, table=p["table"].clone())
    bad["table"][0, 1] = 10 ** 6
    bad["table"][1, 2] = -5
    out, _ = _attend(bad)
    torch.cuda.synchronize()
    assert tg.device_status() == PAGE_BIT
    for b, gone in ((0, 1), (1, 2)):  # the same as leaving the page's tokens out
        masked = dict(p, logsig_pages=p["logsig_pages"].clone())
        masked["logsig_pages"][int(p["table"][b, gone])] = -float("inf")
        h = {n: host_f32(t) if t.is_floating_point() else t.numpy() for n, t in masked.items()}
        ref, _, mag = do.paged_attention(h["q"], h["k_pages"], h["v_pages"], h["table"], h["lens"],
                                         h["logsig_pages"], h["gain"], h["temp"])
        assert (np.abs(host_f32(out)[b] - ref[b]) <= (2.0 ** -8 * (np.abs(ref) + mag) + 3e-4 * mag + 1e-6)[b]).all()
    cut = dict(p, lens=torch.tensor([10 ** 9, -3], dtype=torch.int32))
    out, _ = _attend(cut)
    torch.cuda.synchronize()
    assert tg.device_status() == PAGE_BIT
    whole = dict(p, lens=torch.tensor([64, 0], dtype=torch.int32))
    assert torch.equal(out, _attend(whole)[0])


@pytest.mark.parametrize("widen,longest", [(lambda p: p, 3000), (_wide, 3000), (lambda p: p, 900)])
def test_attention_repeats_and_replays(widen, longest):
    """The same bits every time, eagerly, from another stream and from a captured graph."""
    p = widen(gen.paged_inputs([longest, 1, 777, 0, 64], 16, 8, 128, 64, 9))
    d = {n: dev(t) for n, t in p.items()}
    ws = tg.paged_attention_workspace(5, 16, 8, 128)
    out, lse = torch.empty_like(d["q"]), torch.empty((16, 5), device="cuda")

    def call():
        tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], d["logsig_pages"],
                           d["gain"], d["temp"], out=out, lse=lse, workspace=ws)
    call()
    want, want_lse = out.clone(), lse.clone()
    _check_attention(p, want, want_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(5):
            out.zero_()
            call()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
        call()
    for _ in range(3):
        out.zero_()
        g.replay()
    assert torch.equal(out, want)
    d["lens"].copy_(_i32([5, 900, 0, 1, 33]))  # lengths are read at run time: the graph follows
    d["table"].copy_(d["table"].roll(1, 0))
    d["lens"].clamp_(max=1)
    g.replay()
    eager = tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], d["logsig_pages"],
                               d["gain"], d["temp"], workspace=None)[0]
    torch.cuda.synchronize()
    bits = tg.device_status()  # the rolled table has -1 where a length of 1 now points
    assert bits in (0, PAGE_BIT)
    assert_close("replayed", host_f32(out), host_f32(eager), 1e-6, 2.0 ** -7)


def test_attention_on_two_streams():
    """Two calls at once, each with its own workspace, beside a third one's kernels."""
    ps = [_wide(gen.paged_inputs(lens, 16, 8, 128, 64, 20 + i)) for i, lens in enumerate(([2000, 33, 900], [5, 3000]))]
    ds = [{n: dev(t) for n, t in p.items()} for p in ps]
    wss = [tg.paged_attention_workspace(len(p["lens"]), 16, 8, 128) for p in ps]
    outs = [[torch.empty_like(d["q"]) for _ in range(20)] for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for i in range(20):
        for d, ws, o, s in zip(ds, wss, outs, streams):
            with torch.cuda.stream(s):
                tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], d["logsig_pages"],
                                   d["gain"], d["temp"], out=o[i], workspace=ws)
    torch.cuda.synchronize()
    for p, d, o in zip(ps, ds, outs):
        want, lse = tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], d["logsig_pages"],
                                       d["gain"], d["temp"], want_lse=True)
        _check_attention(p, want, lse)
        assert all(torch.equal(x, want) for x in o)


def test_two_graphs_share_a_workspace():
    """Two captured calls of different shapes on one workspace, replayed in turn with eager calls between."""
    ps = [_wide(gen.paged_inputs(lens, 16, 8, 128, 64, 30 + i)) for i, lens in enumerate(([1500, 700], [64, 2500, 9]))]
    ds = [{n: dev(t) for n, t in p.items()} for p in ps]
    ws = tg.paged_attention_workspace(3, 16, 8, 128)
    outs = [torch.empty_like(d["q"]) for d in ds]

    def call(i):
        d = ds[i]
        tg.paged_attention(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], d["logsig_pages"], d["gain"],
                           d["temp"], out=outs[i], workspace=ws)
    want, graphs = [], []
    for i in range(2):
        call(i)
        want.append(outs[i].clone())
        _check_attention(ps[i], *_attend(ps[i]))
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[i]):
            call(i)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        call(1 - i)
        graphs[i].replay()
        assert torch.equal(outs[i], want[i]) and torch.equal(outs[1 - i], want[1 - i])


def test_attention_far_pages():
    """Offsets past 2^31 elements and 2^32 bytes: the last pages of a pool of 5 GB."""
    P, Hkv, page, d = 9000, 8, 128, 128
    k = torch.zeros((P, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator("cuda").manual_seed(1)
    rows = torch.randn((3, Hkv, page, d), generator=g, device="cuda").bfloat16()
    k[P - 3:], v[P - 3:] = rows, rows.flip(0)
    q = torch.randn((1, 16, d), generator=g, device="cuda").bfloat16()
    table = _i32([[P - 1, P - 3, P - 2]])
    out, _ = tg.paged_attention(q, k, v, table, _i32([300]))
    near, _ = tg.paged_attention(q, k[P - 3:].clone(), v[P - 3:].clone(), _i32([[2, 0, 1]]), _i32([300]))
    assert torch.equal(out, near) and out.abs().sum() > 0


# ---- the cache's pages -------------------------------------------------------------------------


def _random_cache(rng, B, page, P, longest, width, share=0.5):
    """Sequences that share whole prefixes of pages (and sometimes a partly filled last one)."""
    free = list(rng.permutation(P))
    rows, lens = [], []
    for b in range(B):
        n = int(rng.integers(0, longest + 1))
        row = []
        if rows and rng.random() < share:
            o = int(rng.integers(0, len(rows)))
            if rng.random() < 0.5:
                row, n = list(rows[o]), lens[o]
            else:
                row = list(rows[o][:int(rng.integers(0, min(len(rows[o]), n // page) + 1))])
        while len(row) < do.pages_for(n, page) and free:
            row.append(int(free.pop()))
        n = min(n, len(row) * page)
        rows.append(row[:do.pages_for(n, page)])
        lens.append(n)
    table = np.full((B, width), -1, np.int32)
    refs = np.zeros(P, np.int32)
    for b, row in enumerate(rows):
        table[b, :len(row)] = row
        for p in row:
            refs[p] += 1
    return table, np.array(lens, np.int32), refs


def _check_update(got, want):
    for name, g, w in zip(got._fields, got, want):
        assert np.array_equal(g.cpu().numpy(), w), f"{name}: {g.cpu().numpy()} for {w}"


@pytest.mark.parametrize("B,page,P,longest,Bo", [
    (1, 16, 4, 40, 1), (5, 16, 40, 100, 7), (32, 16, 300, 200, 32), (200, 32, 3000, 500, 333),
    (1024, 16, 20000, 200, 1024), (7, 128, 11, 300, 3), (3, 64, 1, 64, 2),
])
@pytest.mark.parametrize("new", [0, 1, 37])
def test_cache_update_matches_oracle(B, page, P, longest, Bo, new):
    rng = np.random.default_rng(B * 1000 + new)
    width = longest // page + 2
    for trial in range(3):
        table, lens, refs = _random_cache(rng, B, page, P, longest, width)
        parent = rng.integers(-1, B, Bo).astype(np.int32) if trial else None
        n = B if parent is None else Bo
        cu = np.concatenate([[0], np.cumsum(rng.integers(0, new + 1, n))]).astype(np.int32) if new else None
        want = do.cache_update(table, lens, refs, page, parent, cu)
        dp, dc = (None if x is None else _i32(x) for x in (parent, cu))
        t, ln, rf = _i32(table), _i32(lens), _i32(refs)
        _check_update(tg.cache_update(t, ln, rf, page, dp, dc), want)
        assert np.array_equal(rf.cpu().numpy(), refs)
        _check_update(tg.cache_update(t, ln, rf, page, dp, dc, refs_out=rf), want)  # counts in place
        if parent is None:  # all in place
            rf = _i32(refs)
            got = tg.cache_update(t, ln, rf, page, None, dc, table_out=t, lens_out=ln, refs_out=rf)
            full = np.array(table)
            for i, n_i in enumerate(want[1]):
                k = do.pages_for(n_i, page)
                full[i, :k] = want[0][i, :k]
            _check_update(got, (full,) + want[1:])


def test_cache_update_copies_before_it_writes():
    """Three holders of a partly filled page grow: two copy, the last keeps it; a fourth that does
    not grow makes the third copy too."""
    table = _i32([[5, 2, -1]] * 4)
    refs = torch.zeros(8, dtype=torch.int32, device="cuda")
    refs[5] = refs[2] = 3
    u = tg.cache_update(table[:3].contiguous(), _i32([20, 20, 20]), refs, 16, cu_new=_i32([0, 1, 2, 3]))
    assert u.copy_src.tolist() == [2, 2, -1] and u.copy_dst.tolist() == [0, 1, -1]
    assert u.table[:, 1].tolist() == [0, 1, 2] and u.refs.tolist() == [1, 1, 1, 0, 0, 3, 0, 0]
    refs[5] = refs[2] = 4
    u = tg.cache_update(table, _i32([20] * 4), refs, 16, cu_new=_i32([0, 1, 2, 3, 3]))
    assert u.copy_dst.tolist() == [0, 1, 3, -1] and u.refs.tolist() == [1, 1, 1, 1, 0, 4, 0, 0]
    assert u.start.tolist() == [20] * 4 and u.lens.tolist() == [21, 21, 21, 20]


def test_cache_update_runs_out_of_pages():
    """The first sequence that lacks a page, and later ones that need or share one, stay as they are."""
    table = _i32([[0, -1], [1, -1], [2, -1], [2, -1], [3, -1]])
    refs = _i32([1, 1, 2, 1, 0])
    lens = _i32([16, 16, 10, 10, 5])
    u = tg.cache_update(table, lens, refs, 16, cu_new=_i32([0, 1, 2, 3, 4, 5]))
    assert u.start.tolist() == [16, -1, -1, -1, 5]
    assert u.lens.tolist() == [17, 16, 10, 10, 6]
    assert u.table.tolist()[0] == [0, 4] and u.refs.tolist() == [1, 1, 2, 1, 1]
    assert u.copy_dst.tolist() == [-1] * 5
    # too long for the table: refused by itself, the others are served
    u = tg.cache_update(table, lens, refs, 16, cu_new=_i32([0, 17, 18, 18, 18, 18]))
    assert u.start.tolist() == [-1, 16, 10, 10, 5] and u.lens.tolist() == [16, 17, 10, 10, 5]
    # freed pages are handed out in the same call
    u = tg.cache_update(table, lens, refs, 16, parent=_i32([0, 1, 1]), cu_new=_i32([0, 1, 2, 3]))
    assert u.table.tolist() == [[0, 2], [1, 3], [1, 4]] and u.refs.tolist() == [1, 2, 1, 1, 1]


def test_cache_update_bad_entries():
    """Parents and pages outside their range are skipped; nothing outside the buffers is touched."""
    table, lens, refs = _i32([[0, 9999], [1, -7]]), _i32([20, 20]), _i32([1, 1, 0, 0])
    u = tg.cache_update(table, lens, refs, 16, parent=_i32([0, 0, 7, -9]), cu_new=_i32([0, 1, 2, 3, 4]))
    torch.cuda.synchronize()
    assert tg.device_status() == PAGE_BIT
    assert u.start.tolist() == [-1, -1, 0, 0] and u.refs.tolist() == [2, 1, 1, 0]
    u = tg.cache_update(table, _i32([-4, 10 ** 9]), refs, 16, cu_new=_i32([5, 1, 2]))
    torch.cuda.synchronize()
    assert tg.device_status() == PAGE_BIT
    assert u.lens.tolist()[0] == 0


@pytest.mark.parametrize("B,page,P,longest", [(1, 16, 3, 20), (6, 16, 200, 300), (64, 64, 5000, 2000),
                                              (3, 128, 1, 100), (0, 16, 9, 10)])
def test_cache_compact_matches_oracle(B, page, P, longest):
    rng = np.random.default_rng(P)
    table, lens, refs = _random_cache(rng, B, page, P, longest, longest // page + 2)
    want = do.cache_compact(table, lens, refs, page)
    t, ln, rf = _i32(table), _i32(lens), _i32(refs)
    _check_update(tg.cache_compact(t, ln, rf, page), want)
    got = tg.cache_compact(t, ln, rf, page, table_out=t, refs_out=rf)
    _check_update(got, want)
    again = tg.cache_compact(t, ln, rf, page)  # already compact
    assert again.counts.tolist() == [int(want[5][0]), 0]
    assert torch.equal(again.refs, rf)


@pytest.mark.parametrize("B,P", [(64, 4096), (65, 4096), (64, 4097), (1, 4097), (1024, 3000), (3, 65536)])
def test_cache_compact_on_a_cluster(B, P):
    """Both sides of the sizes from which a cluster of CTAs renumbers, many times in a row: every launch's
    CTAs must all run before one writes another's shared memory."""
    rng = np.random.default_rng(B + P)
    table, lens, refs = _random_cache(rng, B, 16, P, 16 * (P // B) // 2, P // B)
    want = do.cache_compact(table, lens, refs, 16)
    t, ln, rf = _i32(table), _i32(lens), _i32(refs)
    _check_update(tg.cache_compact(t, ln, rf, 16), want)
    got = [tg.cache_compact(t, ln, rf, 16) for _ in range(50)]
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, got[0]))
    _check_update(got[-1], want)


@pytest.mark.parametrize("shape,dtype", [((3, 40, 2, 16, 64), torch.bfloat16), ((1, 40, 16), torch.float32),
                                         ((2, 40, 8, 64, 128), torch.float32), ((1, 40, 5, 48), torch.uint8)])
def test_cache_copy_pages(shape, dtype):
    g = torch.Generator("cuda").manual_seed(2)
    bits = torch.randint(-120, 120, shape, generator=g, device="cuda")
    pool, other = bits.to(dtype), bits.flip(0).to(dtype)
    want, want_other = pool.clone(), other.clone()
    src, dst = [3, -1, 7, 7, 5, 39, 0], [4, 6, -1, 8, 5, 1, 38]
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            want[:, b], want_other[:, b] = want[:, a].clone(), want_other[:, a].clone()
    tg.cache_copy_pages([pool, other], _i32(src), _i32(dst))
    assert torch.equal(pool, want) and torch.equal(other, want_other)
    before = pool.clone()
    tg.cache_copy_pages([pool], _i32([9, 10]), _i32([20, 21]), _i32([1]))
    assert torch.equal(pool[:, 20], before[:, 9]) and torch.equal(pool[:, 21], before[:, 21])
    tg.cache_copy_pages([pool], _i32([9, 10]), _i32([22, 23]), _i32([0]))
    assert torch.equal(pool[:, 22], before[:, 22])
    tg.cache_copy_pages([pool], _i32([40, 2]), _i32([1, 99]))  # outside the pool
    torch.cuda.synchronize()
    assert tg.device_status() == PAGE_BIT


@pytest.mark.parametrize("new,start,Hkv,d,page,dtype", [
    ([1, 1, 1], [0, 15, 16], 2, 64, 16, "bf16"),
    ([0, 37, 0, 130, 1], [5, 0, 3, 60, 127], 8, 128, 64, "bf16"),
    ([200, 3], [0, 0], 1, 64, 128, "fp32"),
    ([3, 5, 2], [-1, 7, -1], 3, 128, 32, "fp32"),
])
def test_cache_append(new, start, Hkv, d, page, dtype):
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    rng = np.random.default_rng(4)
    g = torch.Generator().manual_seed(4)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    ends = [max(s, 0) + n for s, n in zip(start, new)]
    width = max(do.pages_for(e, page) for e in ends)
    P = sum(do.pages_for(e, page) for e in ends) + 2
    perm = list(rng.permutation(P))
    table = np.full((len(new), width), -1, np.int32)
    for b, e in enumerate(ends):
        for j in range(do.pages_for(e, page)):
            table[b, j] = perm.pop()
    rows = int(cu[-1]) + 3  # three rows behind the last sequence belong to nobody
    k, v = (torch.randn((rows, Hkv, d), generator=g).to(t) for _ in range(2))
    ls = torch.randn(rows, generator=g)
    kp, vp = (torch.randn((P, Hkv, page, d), generator=g).to(t) for _ in range(2))
    lp = torch.randn((P, page), generator=g)
    for gates in (ls, None):
        wk, wv, wl = host_f32(kp).copy(), host_f32(vp).copy(), lp.numpy().copy()
        do.cache_append(host_f32(k), host_f32(v), cu, start, table, wk, wv, None if gates is None else ls.numpy(), wl)
        gk, gv, gl = dev(kp).clone(), dev(vp).clone(), dev(lp).clone()
        tg.cache_append(dev(k), dev(v), _i32(cu), _i32(start), _i32(table), gk, gv, dev(gates), gl)
        assert np.array_equal(host_f32(gk), wk) and np.array_equal(host_f32(gv), wv)
        assert np.array_equal(gl.cpu().numpy(), wl)
    gk2, gv2 = dev(kp).clone(), dev(vp).clone()
    tg.cache_append(dev(k), dev(v), _i32(cu), _i32(start), _i32(table), gk2, gv2)
    assert torch.equal(gk2, gk) and torch.equal(gv2, gv)
    # a row that no page holds
    tg.cache_append(dev(k), dev(v), _i32(cu), _i32([10 ** 6] * len(new)), _i32(table), gk2, gv2)
    torch.cuda.synchronize()
    assert tg.device_status() == PAGE_BIT
    assert torch.equal(gk2, gk)


# ---- the delta rule ----------------------------------------------------------------------------


@pytest.mark.parametrize("B,H,d", [(1, 1, 64), (1, 16, 128), (7, 3, 64), (33, 4, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("forked", [False, True])
def test_delta_step_matches_oracle(B, H, d, dtype, forked):
    _, q, k, v, la, beta = gen.delta_inputs([B], H, d, 3, dtype)
    g = torch.Generator().manual_seed(5)
    S = B + 2
    state = torch.randn((S, H, d, d), generator=g)
    parent = torch.randint(-1, S, (B,), generator=g).to(torch.int32) if forked else None
    if B > 2:
        la[1] = -float("inf")
        beta[2] = 0.0
    out, new = tg.gated_delta_step(dev(q), dev(k), dev(v), dev(la), dev(beta), dev(state), parent=dev(parent))
    ro, rs = do.delta_step(host_f32(q), host_f32(k), host_f32(v), host_f32(la), host_f32(beta), state.numpy(),
                           None if parent is None else parent.numpy())
    assert_close("state", new.cpu().numpy(), rs, 1e-5, 1e-5)
    assert_close("out", host_f32(out), ro, 1e-5, 2.0 ** -8 if dtype == "bf16" else 1e-5)
    if not forked:  # in place
        st = dev(state).clone()
        out2, _ = tg.gated_delta_step(dev(q), dev(k), dev(v), dev(la), dev(beta), st, state_out=st[:B])
        assert torch.equal(st[:B], new) and torch.equal(out2, out) and torch.equal(st[B:].cpu(), state[B:])


def test_delta_steps_continue_the_scan():
    """A scan over a prompt and steps over the rest give the scan over all of it."""
    T, n, H, d = 40, 33, 2, 128
    cu, q, k, v, la, beta = gen.delta_inputs([T], H, d, 8, "fp32")
    o, s = tg.gated_delta_scan(dev(q), dev(k), dev(v), cu, dev(la), dev(beta), algo="recurrent")
    rows = lambda t, a, b: dev(t[a:b])  # noqa: E731
    _, state = tg.gated_delta_scan(rows(q, 0, n), rows(k, 0, n), rows(v, 0, n), np.array([0, n], np.int32),
                                   rows(la, 0, n), rows(beta, 0, n), algo="recurrent")
    for t in range(n, T):
        out, _ = tg.gated_delta_step(*[rows(x, t, t + 1) for x in (q, k, v, la, beta)], state, state_out=state)
        assert_close(f"token {t}", host_f32(out)[0], host_f32(o)[t], 2e-6, 1e-5)
    assert_close("state", host_f32(state), host_f32(s), 5e-6, 1e-5)


def test_delta_step_bad_parent():
    _, q, k, v, la, beta = gen.delta_inputs([2], 2, 64, 3, "fp32")
    state = torch.ones((2, 2, 64, 64), device="cuda")
    args = [dev(x) for x in (q, k, v, la, beta)]
    _, new = tg.gated_delta_step(*args, state, parent=_i32([99, -2]))
    torch.cuda.synchronize()
    assert tg.device_status() == PAGE_BIT
    assert torch.equal(new, tg.gated_delta_step(*args, state, parent=_i32([-1, -1]))[1])


# ---- beams -------------------------------------------------------------------------------------


def _check_beams(logits, scores, n_out, got):
    best, parent, token = do.beam_select(host_f32(logits), scores.numpy(), n_out)
    assert np.array_equal(got[1].cpu().numpy(), parent)
    assert np.array_equal(got[2].cpu().numpy(), token)
    assert np.array_equal(got[0].cpu().numpy() == -np.inf, best == -np.inf)
    fin = best > -np.inf
    assert_close("scores", got[0].cpu().numpy()[fin], best[fin], 1e-6, 2.0 ** -23)


@pytest.mark.parametrize("G,beams,V,n_out", [
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 4), (1, 4, 32000, 8), (3, 5, 8191, 5), (2, 4, 8193, 4),
    (2, 2, 8200, 64), (1, 32, 1000, 64), (5, 8, 50001, 16), (1, 2, 131071, 1),
])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_beam_select_matches_oracle(G, beams, V, n_out, dtype):
    g = torch.Generator().manual_seed(V + n_out)
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    logits = (3.0 * torch.randn((G * beams, V), generator=g)).to(t)
    scores = -5.0 * torch.rand((G, beams), generator=g)
    _check_beams(logits, scores, n_out, tg.beam_select(dev(logits), dev(scores), n_out))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_beam_select_ties_and_missing(dtype):
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    V, beams = 20000, 4
    flat = torch.zeros((beams, V), dtype=t)
    scores = torch.zeros((1, beams))
    _check_beams(flat, scores, 8, tg.beam_select(dev(flat), dev(scores), 8))  # everything equal
    scores = torch.tensor([[0.0, -float("inf"), -float("inf"), -float("inf")]])
    _check_beams(flat, scores, 8, tg.beam_select(dev(flat), dev(scores), 8))  # the first step of a search
    x = (2.0 * torch.randn((beams, V), generator=torch.Generator().manual_seed(1))).to(t)
    x[1] = x[0]  # two beams with the same continuations
    x[2, 100:] = -float("inf")
    x[3] = -float("inf")
    x[3, 17] = 2.0  # a finished beam: one token, at no cost
    scores = torch.tensor([[-1.0, -1.0, -0.5, -3.0]])
    _check_beams(x, scores, 64, tg.beam_select(dev(x), dev(scores), 64))
    x[0, 19999] = float("nan")
    x[1, 5] = float("inf")
    x[3] = -float("inf")
    _check_beams(x, scores, 64, tg.beam_select(dev(x), dev(scores), 64))
    x[2] = -float("inf")
    x[2, 7] = -1.0
    x[2, 3] = 0.0
    x[2, 4] = -0.0
    got = tg.beam_select(dev(x), dev(scores), 5)
    _check_beams(x, scores, 5, got)
    assert got[2].tolist() == [[3, 4, 7, -1, -1]]
    scores[:] = float("nan")
    assert tg.beam_select(dev(x), dev(scores), 2)[1].tolist() == [[-1, -1]]


def test_beam_select_one_workspace():
    """One workspace over calls of different shapes and types, eager and replayed: always the same result."""
    shapes = [(1, 4, 32000, 8, torch.float32), (300, 1, 40, 3, torch.bfloat16), (5, 8, 50001, 16, torch.bfloat16),
              (2, 3, 7, 4, torch.float32)]
    g = torch.Generator().manual_seed(5)
    ws = tg.beam_select_workspace(5, 8, 50001, 16)
    calls = []
    for G, beams, V, n, t in shapes:
        x, s = (2.0 * torch.randn((G * beams, V), generator=g)).to(t), -torch.rand((G, beams), generator=g)
        calls.append((x, s, n, dev(x), dev(s), tg.beam_select(dev(x), dev(s), n)))
        _check_beams(x, s, n, calls[-1][5])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = [tg.beam_select(x, s, n, workspace=ws) for _, _, n, x, s, _ in calls]
    for i in (0, 2, 1, 3, 3, 2, 0):
        _, _, n, x, s, want = calls[i]
        got = tg.beam_select(x, s, n, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph.replay()
        for got, (_, _, _, _, _, want) in zip(captured, calls):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_beam_select_largest():
    """The largest sizes: 32 beams of 2^20 logits, 64 candidates; and many groups of one beam."""
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((32, 2 ** 20), generator=g, device="cuda") * 2.0
    scores = -torch.rand((1, 32), generator=g, device="cuda")
    best, parent, token = tg.beam_select(x, scores, 64)
    total = (x.double() - torch.logsumexp(x.double(), 1, keepdim=True) + scores.double().T).reshape(-1)
    want = torch.topk(total, 64)
    assert torch.equal(parent[0].long() * 2 ** 20 + token[0], want.indices)  # (random fp32: no two are equal)
    assert_close("scores", best[0].cpu().numpy(), want.values.cpu().numpy(), 1e-6, 2.0 ** -23)
    x = torch.randn((3000, 33), generator=g, device="cuda").bfloat16()
    best, parent, token = tg.beam_select(x, torch.zeros((3000, 1), device="cuda"), 1)
    assert torch.equal(parent[:, 0].cpu(), torch.arange(3000, dtype=torch.int32))
    first = (x == x.amax(1, keepdim=True)).float().argmax(1)
    assert torch.equal(x.gather(1, token.long()), x.amax(1, keepdim=True))
    assert (token[:, 0] <= first).all()


def test_beam_select_sorted_rows():
    """Rising and falling logits: the best all lie in one chunk, and in one thread's part of it."""
    V = 30000
    up = torch.arange(V, dtype=torch.float32) * 1e-3
    x = torch.stack([up, up.flip(0), up.roll(100), -up])
    scores = torch.tensor([[0.0, -0.25, -0.5, -40.0]])
    _check_beams(x, scores, 64, tg.beam_select(dev(x), dev(scores), 64))
    spikes = torch.zeros((1, V))
    spikes[0, 256 * 4:256 * 4 + 64] = torch.arange(64).float() + 1
    _check_beams(spikes, torch.zeros((1, 1)), 64, tg.beam_select(dev(spikes), torch.zeros((1, 1), device="cuda"), 64))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", ["lowest", -1e10, -1e30])
def test_beam_select_masked_chunks(dtype, mask):
    """A mask of finite values over whole chunks (16384 logits in bf16, 8192 in fp32), the last, ragged one
    among them, over all but a few tokens, and over a whole row, whose tokens are then all alike."""
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    low = torch.finfo(t).min if mask == "lowest" else mask
    V, beams = 40003, 5
    x = (2.0 * torch.randn((beams, V), generator=torch.Generator().manual_seed(4))).to(t)
    x[0, 8192:32768] = low
    x[1, 32768:] = low
    keep = x[2, [3, 20000, 39999]].clone()
    x[2] = low
    x[2, [3, 20000, 39999]] = keep
    x[3] = low
    scores = torch.tensor([[-1.0, -1.5, -0.5, 6.0, -2.0]])
    for n_out in (5, 64):
        got = tg.beam_select(dev(x), dev(scores), n_out)
        _check_beams(x, scores, n_out, got)
        assert set(range(5)) >= set(got[1].tolist()[0]) and 2 in got[1].tolist()[0]
    alone = tg.beam_select(dev(x[3:4].clone()), torch.zeros((1, 1), device="cuda"), 3)
    assert alone[2].tolist() == [[0, 1, 2]]
    assert_close("even", alone[0].cpu().numpy(), np.full((1, 3), -np.log(V)), 1e-6, 2.0 ** -23)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_beam_select_largest_values(dtype):
    """A logit of 3e38: no other token has a weight, and all have finite scores."""
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    V = 20000
    x = (2.0 * torch.randn((2, V), generator=torch.Generator().manual_seed(5))).to(t)
    x[0, 17000] = 3e38
    x[1, 100:20000] = -1e38
    scores = torch.tensor([[-3.0, -1.0]])
    got = tg.beam_select(dev(x), dev(scores), 4)
    _check_beams(x, scores, 4, got)
    assert 17000 in got[2].tolist()[0]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [33, 1001, 8195, 50257, 131071])
def test_beam_select_equal_beams_at_odd_vocabularies(V, dtype):
    """Beams of the same logits and the same score: every token's beams come in their order.  With an odd
    vocabulary the rows start at every offset from a 16-byte boundary, which the rows' sums may not show."""
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    beams, n_out = 8, 24
    for seed in range(4):
        row = 2.0 * torch.randn((2, 1, V), generator=torch.Generator().manual_seed(100 * V + seed))
        x = row.expand(2, beams, V).reshape(2 * beams, V).to(t).contiguous()
        scores = torch.tensor([[-1.25] * beams, [-0.5] * beams])
        _check_beams(x, scores, n_out, tg.beam_select(dev(x), dev(scores), n_out))
    flat = torch.full((beams, V), -3.0, dtype=t)
    _check_beams(flat, scores[:1], n_out, tg.beam_select(dev(flat), dev(scores[:1]), n_out))


@pytest.mark.parametrize("dtype,Vs", [("bf16", (16383, 16385, 16386, 16391, 7)), ("fp32", (8191, 8193, 8194, 8195, 3))])
def test_beam_select_row_ends(dtype, Vs):
    """Rows that end just before or behind a chunk's end, the last row at every offset from a 16-byte
    boundary; the first and last tokens, and those at the chunk's end, are the best."""
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    for V in Vs:
        for beams in range(1, 10):
            x = torch.randn((beams, V), generator=torch.Generator().manual_seed(V + beams)).to(t)
            marked = sorted({at for at in (0, 1, V // 2 // 8 * 8 - 1, V - 9, V - 8, V - 7, V - 6, V - 5, V - 4, V - 3,
                                           V - 2, V - 1) if 0 <= at < V})
            for b in range(beams):
                x[b, marked] = (6.0 + torch.arange(len(marked)).roll(b) + 0.25 * b).to(t)
            scores = torch.linspace(-1.0, -0.25, beams)[None]
            _check_beams(x, scores, 64, tg.beam_select(dev(x), dev(scores), 64))


def test_beam_select_merge_memory():
    """Sizes whose merge takes just under 48 KB of dynamic shared memory, in a process that has launched
    no larger one: the kernel's own few hundred bytes count too."""
    code = """if 1:
        import torch
        import learned_token_pruning_gate_b200 as tg
        g = torch.Generator("cuda").manual_seed(6)
        for V in (500000, 503000):
            x = torch.randn((32, V), generator=g, device="cuda") * 2.0
            scores = -torch.rand((1, 32), generator=g, device="cuda")
            _, parent, token = tg.beam_select(x, scores, 64)
            total = (x.double() - torch.logsumexp(x.double(), 1, keepdim=True) + scores.double().T).reshape(-1)
            assert torch.equal(parent[0].long() * V + token[0], torch.topk(total, 64).indices)
        print("equal")
    """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.split() == ["equal"], run.stderr[-2000:]


@pytest.mark.parametrize("B,P", [(4, 40), (70, 5000)])
def test_cache_update_to_no_sequences(B, P):
    """A fork into no sequences (no parents at all, which is not the absence of parents) frees every page."""
    table, lens, refs = _random_cache(np.random.default_rng(3), B, 16, P, 100, 8)
    got = tg.cache_update(_i32(table), _i32(lens), _i32(refs), 16, parent=_i32([]))
    assert refs.any() and not got.refs.any() and got.table.shape == (0, 8) and got.lens.shape == (0,)
    none = tg.cache_update(got.table, got.lens, got.refs, 16, cu_new=_i32([0]))
    assert not none.refs.any() and none.start.shape == (0,)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gain", [1.5, 64.0, -2.0])
def test_attention_gates_whose_bias_overflows(dtype, gain):
    """gain x the lowest gate is beyond fp32 where the formula's softmax is not: such tokens alone share
    their weight evenly; beside others they have none (all of it, under a negative gain)."""
    p = gen.paged_inputs([40, 300], 4, 2, 64, 16, 9, dtype)
    p["gain"][:] = gain
    low = torch.finfo(torch.float32).min
    ls, t = p["logsig_pages"], p["table"]
    ls[t[0, :3].long()] = low
    for j in range(0, 300, 3):
        ls[int(t[1, j // 16]), j % 16] = low
    for q in (p, _wide(p)):
        for workspace in ("auto", None):
            out, lse = _attend(q, workspace)
            h = {n: host_f32(x) if x.is_floating_point() else x.numpy() for n, x in q.items()}
            ref, _, mag = do.paged_attention(*[h[n] for n in ("q", "k_pages", "v_pages", "table", "lens", "logsig_pages",
                                                              "gain", "temp")])
            bound = 3e-4 * mag + 1e-6 + (2.0 ** -8 * (np.abs(ref) + mag) if dtype == "bf16" else 0.0)
            assert (np.abs(host_f32(out) - ref) <= bound).all()
            assert bool(torch.isfinite(lse).all())  # (of the lowest value's size: no fp32 number is the formula's)


def test_attention_weights_keep_their_bits():
    """What is left when all but the last bits of a weight cancel.  Of three tokens two weigh 1 and have
    v = -hi and -lo, the first 16 bits of the third's weight w, as two bf16 numbers, and the third has v = 1:
    out = (w - hi - lo) / (2 + w), about 2^-19.5.  q = 0, so logits are gain x gate to half a place.
    The numerator may be off by w's errors (ex2.approx 2^-22, its argument below 1 rounded twice, 2^-23 in
    all) and three fp32 additions of sums below 1, truncated: 2^-22 + 2^-23 + 3 x 2^-23 < 8e-7; the weights'
    first 16 bits alone would be off by 3.8e-6 here."""
    H, d, page = 8, 64, 16
    bf = lambda x: torch.tensor(x).to(torch.bfloat16).double().numpy()  # noqa: E731
    gain = np.random.default_rng(1).uniform(0.05, 0.6, 200000).astype(np.float32)
    w = np.exp(-gain.astype(np.float64))
    hi = bf(w)
    lo = bf(w - hi)
    best = np.argsort(-np.abs(w - hi - lo))[:H]
    gain, w, hi, lo = gain[best], w[best], hi[best], lo[best]
    assert (np.abs(w - hi - lo) > 3.8e-6).all()
    p = gen.paged_inputs([3], H, H, d, page, 1, "bf16", fill=0.0)
    at = int(p["table"][0, 0])
    p["q"].zero_()
    p["gain"], p["temp"] = torch.from_numpy(gain), torch.ones(H)
    p["logsig_pages"][at, :3] = torch.tensor([0.0, 0.0, -1.0])
    for h in range(H):
        for j, x in enumerate((-hi[h], -lo[h], 1.0)):
            p["v_pages"][at, h, j] = float(x)
    want = ((w - hi - lo) / (2.0 + w))[:, None]
    for q in (p, _wide(p)):
        for workspace in ("auto", None):
            out, _ = _attend(q, workspace)
            assert (np.abs(host_f32(out)[0] - want) <= 8e-7 / (2.0 + w[:, None]) + 2.0 ** -9 * np.abs(want)).all()
