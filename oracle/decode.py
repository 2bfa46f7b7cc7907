"""Plain fp64 / integer oracle of decoding from a gated prefill (test infrastructure).

Everything is written out from the definitions, sequence by sequence and page by
page; nothing is blocked, vectorised over pages, or shared with the CUDA library:

    paged_attention   softmax over a sequence's cached tokens with the gate's bias
    cache_update      a step of the page tables as a loop over sequences
    cache_compact     live pages into the lowest numbers
    cache_append      rows into pages
    delta_step        one token of the gated delta rule
    beam_select       the best continuations over beams and vocabulary

A token's k and v are found through its sequence's table; a token whose log-gate
is -inf is left out, and a sequence with no token left has output 0 and lse -inf.
"""
from __future__ import annotations

import numpy as np


def paged_attention(q, k_pages, v_pages, table, lens, logsig_pages=None, gain=None, temp=None):
    """q [B, Hq, d], pages [P, Hkv, page, d]; returns (out, lse [Hq, B], magnitude), where
    magnitude is sum_j w_j |v_j|, the size that a relative error of the weights acts on."""
    q, kp, vp = (np.asarray(a, np.float64) for a in (q, k_pages, v_pages))
    B, Hq, d = q.shape
    Hkv, page = kp.shape[1], kp.shape[2]
    gain = np.ones(Hq) if gain is None else np.asarray(gain, np.float64)
    temp = np.ones(Hq) if temp is None else np.asarray(temp, np.float64)
    out, mag, lse = np.zeros_like(q), np.zeros_like(q), np.full((Hq, B), -np.inf)
    for b in range(B):
        tokens = [(int(table[b][j // page]), j % page) for j in range(int(lens[b]))]
        ls = np.array([0.0 if logsig_pages is None else logsig_pages[p][o] for p, o in tokens])
        seen = [i for i in range(len(tokens)) if ls[i] != -np.inf]
        if not seen:
            continue
        at = [tokens[i] for i in seen]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k = np.stack([kp[p, g, o] for p, o in at])
            v = np.stack([vp[p, g, o] for p, o in at])
            x = k @ q[b, h] / (np.sqrt(d) * temp[h]) + gain[h] * ls[seen]
            w = np.exp(x - x.max())
            lse[h, b] = x.max() + np.log(w.sum())
            w /= w.sum()
            out[b, h], mag[b, h] = w @ v, w @ np.abs(v)
    return out, lse, mag


def pages_for(n, page):
    return -(-int(n) // page)


def cache_update(table, lens, refs, page, parent=None, cu_new=None, table_out=None):
    """Returns (table, lens, refs, start, copy_src, copy_dst) as integer arrays."""
    lens, refs = [int(n) for n in lens], [int(r) for r in refs]
    max_pages = len(table[0]) if len(table) else 0
    parent = list(range(len(lens))) if parent is None else [int(p) for p in parent]
    rows, held = [], []
    for p in parent:
        rows.append([] if p < 0 else [int(x) for x in table[p][:pages_for(lens[p], page)]])
        held.append(0 if p < 0 else lens[p])
    for b, n in enumerate(lens):
        for p in table[b][:pages_for(n, page)]:
            refs[int(p)] += parent.count(b) - 1
    at_entry = list(refs)
    free = [p for p, r in enumerate(refs) if r <= 0]
    start, src, dst, out_of_pages = [], [], [], False
    grows = [0 if cu_new is None else int(cu_new[i + 1]) - int(cu_new[i]) for i in range(len(rows))]
    for i, pages in enumerate(rows):
        n = grows[i]
        more = pages_for(held[i] + n, page) - len(pages)
        writes_into = pages[-1] if n > 0 and held[i] % page else None
        start.append(-1)
        src.append(-1)
        dst.append(-1)
        if len(pages) + more > max_pages:
            continue
        copies = writes_into is not None and refs[writes_into] > 1
        if more + copies > len(free):
            out_of_pages = True
        if out_of_pages and (more + copies or (writes_into is not None and at_entry[writes_into] > 1)):
            continue
        start[i] = held[i]
        held[i] += n
        if copies:
            src[i], dst[i] = writes_into, free.pop(0)
            refs[src[i]] -= 1
            refs[dst[i]] = 1
            pages[-1] = dst[i]
        for _ in range(more):
            pages.append(free.pop(0))
            refs[pages[-1]] = 1
    out = np.full((len(rows), max_pages), -1, np.int32) if table_out is None else np.array(table_out)
    for i, pages in enumerate(rows):
        out[i, :len(pages)] = pages
    return out, np.array(held, np.int32), np.array(refs, np.int32), np.array(start, np.int32), \
        np.array(src, np.int32), np.array(dst, np.int32)


def cache_compact(table, lens, refs, page):
    """Returns (table, refs, page_map, copy_src, copy_dst, counts)."""
    live = [p for p, r in enumerate(refs) if r > 0]
    n = len(live)
    holes, movers = [p for p in range(n) if refs[p] <= 0], [p for p in live if p >= n]
    page_map = np.full(len(refs), -1, np.int32)
    for p in live:
        page_map[p] = p
    src, dst = np.full(len(refs), -1, np.int32), np.full(len(refs), -1, np.int32)
    for i, (a, b) in enumerate(zip(movers, holes)):
        page_map[a], src[i], dst[i] = b, a, b
    out = np.full_like(np.asarray(table, np.int32), -1)
    for b, length in enumerate(lens):
        for j in range(pages_for(length, page)):
            out[b, j] = page_map[table[b][j]]
    new = np.zeros(len(refs), np.int32)
    for p in live:
        new[page_map[p]] = refs[p]
    return out, new, page_map, src, dst, np.array([n, len(movers)], np.int32)


def cache_append(k, v, cu_new, start, table, k_pages, v_pages, logsig=None, logsig_pages=None):
    """Writes into the given (host) pages."""
    page = k_pages.shape[2]
    for b in range(len(start)):
        for i in range(int(cu_new[b]), int(cu_new[b + 1])):
            if start[b] < 0:
                continue
            pos = int(start[b]) + i - int(cu_new[b])
            p, o = int(table[b][pos // page]), pos % page
            k_pages[p, :, o], v_pages[p, :, o] = k[i], v[i]
            if logsig_pages is not None:
                logsig_pages[p, o] = 0.0 if logsig is None else logsig[i]


def delta_step(q, k, v, log_alpha, beta, state, parent=None, eps=1e-6):
    """Returns (out [B, H, d], state [B, H, d, d])."""
    q, k, v, state = (np.asarray(a, np.float64) for a in (q, k, v, state))
    B, H, d = q.shape
    out, new = np.zeros((B, H, d)), np.zeros((B, H, d, d))
    for b in range(B):
        p = b if parent is None else int(parent[b])
        for h in range(H):
            kn = k[b, h] / np.sqrt(k[b, h] @ k[b, h] + eps)
            qn = q[b, h] / np.sqrt(q[b, h] @ q[b, h] + eps) / np.sqrt(d)
            old = np.zeros((d, d)) if p < 0 else np.exp(float(log_alpha[b, h])) * state[p, h]
            new[b, h] = old + float(beta[b, h]) * np.outer(v[b, h] - old @ kn, kn)
            out[b, h] = new[b, h] @ qn
    return out, new


def beam_select(logits, scores, n_out):
    """Returns (scores [G, n_out], parent, token)."""
    logits, scores = np.asarray(logits, np.float64), np.asarray(scores, np.float64)
    G, beams = scores.shape
    V = logits.shape[1]
    best = np.full((G, n_out), -np.inf)
    parent, token = np.full((G, n_out), -1, np.int32), np.full((G, n_out), -1, np.int32)
    for g in range(G):
        found = []
        for b in range(beams):
            x = logits[g * beams + b]
            if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
                continue
            # (the maximum first: the log of the sum is below the last place of, say, -3e38)
            total = scores[g, b] + ((x - x.max()) - np.log(np.exp(x - x.max()).sum()))
            order = np.lexsort((np.arange(V), -total))[:n_out]
            found += [(-total[t], b, int(t)) for t in order if np.isfinite(total[t])]
        for i, (s, b, t) in enumerate(sorted(found)[:n_out]):
            best[g, i], parent[g, i], token[g, i] = -s, g * beams + b, t
    return best, parent, token
