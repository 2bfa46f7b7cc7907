"""Decoding after a gated prefill: the cases that its operators are measured on.

A gated prefill leaves, per prompt, the kept rows' k, v and log-gates and (in a
hybrid backbone) one delta-rule state per head.  Decoding reads them one token
at a time, as a single sequence or as the beams of a search:

    attention   gated attention of one new token per sequence over a paged cache
    fork        one step of a page cache under a beam search: every sequence takes
                its parent's pages, shared ones are counted, a shared last page is
                copied before it is written, pages for the new token are handed out
    compact     the live pages of a cache move to its lowest page numbers
    append      rows of k, v and log-gates go into their sequences' pages
    delta       one token of the gated delta rule, state in, state out
    beam        the best continuations over beams and vocabulary

`own` chooses between the plain torch form of an operator and the package's call.
"""
import math

import torch

own = False

F32, F64, I32, I64 = torch.float32, torch.float64, torch.int32, torch.int64
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases -------------------------------------------------------------------------------------


def listed():
    return [
        # one user, a short prompt pruned to a few hundred rows: latency is all there is
        dict(name="attention_one_short", op="attention", dtype="bf16", hq=16, hkv=8, d=128, page=16,
             batch=1, shortest=320, longest=320),
        # a serving batch behind the 16k workload: 2304 kept rows and some generated tokens each
        dict(name="attention_batch_2k", op="attention", dtype="bf16", hq=16, hkv=8, d=128, page=64,
             batch=16, shortest=2304, longest=2817),
        # the ragged workload with one prompt that was not pruned: very unequal lengths
        dict(name="attention_ragged_long", op="attention", dtype="bf16", hq=16, hkv=8, d=128, page=128,
             batch=7, shortest=1151, longest=131073),
        # many short chats on a model with eight query heads to a key head, odd lengths from one token on
        dict(name="attention_wide_groups", op="attention", dtype="bf16", hq=32, hkv=4, d=64, page=32,
             batch=61, shortest=1, longest=4353),
        # the small fp32 configuration, as a test or a reference run decodes it
        dict(name="attention_fp32", op="attention", dtype="fp32", hq=4, hkv=2, d=64, page=16,
             batch=33, shortest=256, longest=1024),
        # a step of a beam search, 8 requests of 4 beams: most beams share their prompt's pages
        dict(name="fork_beams", op="fork", dtype="bf16", layers=4, hkv=8, d=128, page=16, groups=8,
             beams=4, prompt=1200, tail=75, pool=2048),
        # a long-running server's pool, a third of it in use in scattered pages, before it is shrunk
        dict(name="compact_pool", op="compact", dtype="bf16", layers=2, hkv=8, d=128, page=64, batch=24,
             longest=3000, pool=1500),
        # the kept rows of a ragged prefill batch on their way into pages
        dict(name="append_prefill", op="append", dtype="bf16", hkv=8, d=128, page=64, batch=4,
             shortest=1152, longest=8704),
        # one user's token in a hybrid layer
        dict(name="delta_one", op="delta", dtype="bf16", heads=16, d=128, batch=1, beams=0),
        # 48 beams of a hybrid layer, each reading its parent's state
        dict(name="delta_beams", op="delta", dtype="bf16", heads=32, d=128, batch=48, beams=1),
        # one request of 4 beams
        dict(name="beam_one", op="beam", dtype="fp32", groups=1, beams=4, vocab=32000, n_out=8),
        # a serving batch, odd vocabulary
        dict(name="beam_batch", op="beam", dtype="bf16", groups=12, beams=8, vocab=131071, n_out=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "fork", "compact", "append", "delta", "beam", "beam"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "attention":
        hq, hkv, d = rng.choice([(16, 8, 128), (4, 2, 64), (32, 4, 64), (32, 4, 128), (8, 8, 64), (16, 1, 128), (12, 4, 128)])
        batch = _log_int(rng, 1, 96)
        # the plain form pads to the longest, so that batch x longest bounds its memory
        longest = _log_int(rng, 1, min(131072, max(2, (1 << 27) // (batch * hkv * d))))
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128]), batch=batch,
                    shortest=rng.choice([1, longest, max(1, longest // 3)]), longest=longest)
    if op == "fork":
        page = rng.choice([16, 32, 64])
        groups, beams, prompt, tail = _log_int(rng, 1, 12), _log_int(rng, 1, 8), _log_int(rng, 1, 1500), _log_int(rng, 1, 100)
        need = groups * (prompt // page + 1) + 2 * groups * beams * (tail // page + 2)
        return dict(op=op, dtype=dtype, layers=rng.choice([1, 2, 4]), hkv=rng.choice([2, 4, 8]), d=rng.choice([64, 128]),
                    page=page, groups=groups, beams=beams, prompt=prompt, tail=tail, pool=need + rng.randint(0, 200))
    if op == "compact":
        page, batch, longest = rng.choice([16, 32, 64]), _log_int(rng, 1, 24), _log_int(rng, 10, 2000)
        need = batch * (longest // page + 1)
        return dict(op=op, dtype=dtype, layers=rng.choice([1, 2]), hkv=rng.choice([2, 8]), d=rng.choice([64, 128]), page=page,
                    batch=batch, longest=longest, pool=need + rng.randint(0, need))
    if op == "append":
        batch = _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, 20000 // batch)
        return dict(op=op, dtype=dtype, hkv=rng.choice([2, 8]), d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                    batch=batch, shortest=rng.choice([1, longest]), longest=longest)
    if op == "delta":
        return dict(op=op, dtype=dtype, heads=rng.choice([3, 4, 16, 32]), d=rng.choice([64, 128]), batch=_log_int(rng, 1, 48),
                    beams=rng.choice([0, 1]))
    beams = rng.choice([1, 2, 4, 5, 8, 16])
    groups = _log_int(rng, 1, 96 // beams)
    return dict(op=op, dtype=dtype, groups=groups, beams=beams, vocab=_log_int(rng, 1000, 131072 if dtype == "bf16" else 60000),
                n_out=rng.choice([beams, 2 * beams]))


# ---- inputs ------------------------------------------------------------------------------------


def _lengths(case, gen):
    """Sequence lengths, spread evenly over the logarithm from shortest to longest, in a random order."""
    lo, hi, n = case["shortest"], case["longest"], case["batch"]
    u = torch.rand(n, generator=gen, dtype=F64)
    if n > 1:
        u[0], u[1] = 0.0, 1.0
    lens = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo))).round().long().clamp(lo, hi)
    return lens[torch.randperm(n, generator=gen)]


def _attention_lengths(case, gen):
    if case.get("name") == "attention_ragged_long" or case["longest"] > 20000:
        return _lengths(case, gen)
    n = case["batch"]
    return torch.randint(case["shortest"], case["longest"] + 1, (n,), generator=gen)


def _randn(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return x if scale == 1.0 else x * scale


def _log_gates(shape, seed):
    """Log-gates of kept rows: log sigmoid of scores; the protected (question and generated) rows have 0."""
    z = _randn(shape, seed, F32, 2.0)
    return torch.where(_randn(shape, seed + 1) < -1.0, torch.zeros_like(z), torch.nn.functional.logsigmoid(z))


def _table(lens, page, pages, gen, width):
    """A table of random distinct pages for sequences of these lengths, -1 behind them."""
    counts = [(int(n) + page - 1) // page for n in lens]
    perm = torch.randperm(pages, generator=gen)
    table = torch.full((len(counts), width), -1, dtype=I32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c].to(I32)
        at += c
    return table


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed * 7919 + 17)
    s = dict(case, dtype=DTYPES[case["dtype"]])
    return globals()["_prepare_" + case["op"]](s, seed * 1000, gen)


def _prepare_attention(s, seed, gen):
    lens = _attention_lengths(s, gen)
    page = s["page"]
    pages = sum((int(n) + page - 1) // page for n in lens) + 3
    shape = (pages, s["hkv"], page, s["d"])
    s.update(q=_randn((s["batch"], s["hq"], s["d"]), seed + 1, s["dtype"]), k_pages=_randn(shape, seed + 2, s["dtype"]),
             v_pages=_randn(shape, seed + 3, s["dtype"]), logsig_pages=_log_gates((pages, page), seed + 4),
             gain=torch.rand(s["hq"], generator=gen).cuda(), temp=(0.8 + 0.4 * torch.rand(s["hq"], generator=gen)).cuda(),
             table=_table(lens, page, pages, gen, (s["longest"] + page - 1) // page + 2).cuda(), lens=lens.to(I32).cuda())
    if own:
        import learned_token_pruning_gate_b200 as tg

        s["workspace"] = tg.paged_attention_workspace(s["batch"], s["hq"], s["hkv"], s["d"], s["dtype"])
    return s


def _prepare_pools(s, seed, pages):
    shape = (s["layers"], pages, s["hkv"], s["page"], s["d"])
    s["pools"] = [_randn(shape, seed + 2, s["dtype"]), _randn(shape, seed + 3, s["dtype"]),
                  _log_gates((1, pages, s["page"]), seed + 4)]


def _prepare_fork(s, seed, gen):
    """Beams that share their prompt's whole pages and own a tail each; some share the tail's pages too."""
    page, groups, beams, pages = s["page"], s["groups"], s["beams"], s["pool"]
    perm = torch.randperm(pages, generator=gen).tolist()
    rows, lens = [], []
    for _ in range(groups):
        prompt = max(1, s["prompt"] - int(torch.randint(0, s["prompt"] // 4 + 1, (1,), generator=gen)))
        whole = [perm.pop() for _ in range(prompt // page)]
        n = prompt + int(torch.randint(1, s["tail"] + 1, (1,), generator=gen))
        tail = None
        for _ in range(beams):
            if tail is None or torch.rand(1, generator=gen) < 0.5:
                tail = [perm.pop() for _ in range((n + page - 1) // page - len(whole))]
            rows.append(whole + tail)
            lens.append(n)
    width = (s["prompt"] + s["tail"]) // page + 3
    table = torch.full((len(rows), width), -1, dtype=I32)
    refs = torch.zeros(pages, dtype=I32)
    for i, r in enumerate(rows):
        table[i, :len(r)] = torch.tensor(r, dtype=I32)
        refs[r] += 1
    n = groups * beams
    parent = torch.randint(0, beams, (n,), generator=gen) + torch.arange(n) // beams * beams
    s.update(table=table.cuda(), lens=torch.tensor(lens, dtype=I32).cuda(), refs=refs.cuda(), parent=parent.to(I32).cuda(),
             cu_new=torch.arange(n + 1, dtype=I32).cuda(), table_out=torch.full((n, width), -1, dtype=I32).cuda())
    _prepare_pools(s, seed, pages)
    return s


def _prepare_compact(s, seed, gen):
    lens = torch.randint(1, s["longest"] + 1, (s["batch"],), generator=gen)
    table = _table(lens, s["page"], s["pool"], gen, s["longest"] // s["page"] + 3)
    refs = torch.zeros(s["pool"], dtype=I32)
    refs[table[table >= 0].long()] = 1
    s.update(table=table.cuda(), lens=lens.to(I32).cuda(), refs=refs.cuda(), table_out=torch.full_like(table, -1).cuda())
    _prepare_pools(s, seed, s["pool"])
    return s


def _prepare_append(s, seed, gen):
    new = _lengths(s, gen)
    page = s["page"]
    start = torch.randint(0, 2 * page, (s["batch"],), generator=gen)
    lens = start + new
    width = s["longest"] // page + 3
    pages = s["batch"] * width
    rows = int(new.sum())
    shape = (pages, s["hkv"], page, s["d"])
    s.update(k=_randn((rows, s["hkv"], s["d"]), seed + 1, s["dtype"]), v=_randn((rows, s["hkv"], s["d"]), seed + 2, s["dtype"]),
             logsig=_log_gates((rows,), seed + 3), cu_new=torch.cat([torch.zeros(1, dtype=I64), new.cumsum(0)]).to(I32).cuda(),
             start=start.to(I32).cuda(), table=_table(lens, page, pages, gen, width).cuda(), k_pages=_randn(shape, seed + 4, s["dtype"]),
             v_pages=_randn(shape, seed + 5, s["dtype"]), logsig_pages=_log_gates((pages, page), seed + 6))
    return s


def _prepare_delta(s, seed, gen):
    b, h, d = s["batch"], s["heads"], s["d"]
    rows = (b, h, d)
    s.update(q=_randn(rows, seed + 1, s["dtype"]), k=_randn(rows, seed + 2, s["dtype"]), v=_randn(rows, seed + 3, s["dtype"]),
             log_alpha=-0.1 * _randn((b, h), seed + 4).abs(), beta=torch.sigmoid(_randn((b, h), seed + 5)),
             state=_randn((b, h, d, d), seed + 6, F32, 0.3), state_out=torch.zeros((b, h, d, d), device="cuda"),
             parent=torch.randint(0, b, (b,), generator=gen).to(I32).cuda() if s["beams"] else None)
    return s


def _prepare_beam(s, seed, gen):
    rows = s["groups"] * s["beams"]
    # a few likely tokens over a broad floor, as a language model's logits are
    logits = _randn((rows, s["vocab"]), seed + 1, F32, 2.0)
    logits[:, ::97] += _randn((rows, (s["vocab"] + 96) // 97), seed + 2, F32, 4.0)
    s.update(logits=logits.to(s["dtype"]), scores=-30.0 * torch.rand((s["groups"], s["beams"]), generator=gen).cuda() ** 2)
    if own:
        import learned_token_pruning_gate_b200 as tg

        s["workspace"] = tg.beam_select_workspace(s["groups"], s["beams"], s["vocab"], s["n_out"])
    return s


# ---- one pass ----------------------------------------------------------------------------------


def run(s):
    return globals()[("_own_" if own else "_plain_") + s["op"]](s)


def _own_attention(s):
    import learned_token_pruning_gate_b200 as tg

    return tg.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], logsig_pages=s["logsig_pages"],
                              gain=s["gain"], temp=s["temp"], want_lse=True, workspace=s["workspace"])


def _own_fork(s):
    import learned_token_pruning_gate_b200 as tg

    u = tg.cache_update(s["table"], s["lens"], s["refs"], s["page"], parent=s["parent"], cu_new=s["cu_new"],
                        table_out=s["table_out"])
    tg.cache_copy_pages(s["pools"], u.copy_src, u.copy_dst)
    return [u.table, u.lens, u.refs, u.start, u.copy_src, u.copy_dst] + s["pools"]


def _own_compact(s):
    import learned_token_pruning_gate_b200 as tg

    c = tg.cache_compact(s["table"], s["lens"], s["refs"], s["page"], table_out=s["table_out"])
    tg.cache_copy_pages(s["pools"], c.copy_src, c.copy_dst, c.counts[1:])
    return [c.table, c.refs, c.page_map, c.counts] + s["pools"]


def _own_append(s):
    import learned_token_pruning_gate_b200 as tg

    tg.cache_append(s["k"], s["v"], s["cu_new"], s["start"], s["table"], s["k_pages"], s["v_pages"], logsig=s["logsig"],
                    logsig_pages=s["logsig_pages"])
    return [s["k_pages"], s["v_pages"], s["logsig_pages"]]


def _own_delta(s):
    import learned_token_pruning_gate_b200 as tg

    return tg.gated_delta_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["state"], parent=s["parent"],
                               state_out=s["state_out"])


def _own_beam(s):
    import learned_token_pruning_gate_b200 as tg

    return tg.beam_select(s["logits"], s["scores"], s["n_out"], workspace=s["workspace"])


def _plain_attention(s):
    b, hq, d = s["q"].shape
    hkv, page = s["hkv"], s["page"]
    span = s["table"].shape[1] * page
    at = s["table"].clamp(min=0).long()
    k = s["k_pages"][at].float().transpose(1, 2).reshape(b, hkv, span, d)
    v = s["v_pages"][at].float().transpose(1, 2).reshape(b, hkv, span, d)
    gates = s["logsig_pages"][at].reshape(b, 1, 1, span)
    q = s["q"].float().reshape(b, hkv, hq // hkv, d)
    logits = q @ k.transpose(2, 3)
    logits = logits / (math.sqrt(d) * s["temp"].reshape(1, hkv, -1, 1)) + s["gain"].reshape(1, hkv, -1, 1) * gates
    seen = torch.arange(span, device="cuda") < s["lens"][:, None]
    logits = logits.masked_fill(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    out = (e / total) @ v.masked_fill(~seen[:, None, :, None], 0.0)
    lse = (top + torch.log(total)).reshape(b, hq)
    return out.reshape(b, hq, d).to(s["dtype"]), lse.t().contiguous()


def _plain_fork(s):
    table, lens, refs, page = s["table"], s["lens"].long(), s["refs"], s["page"]
    parent = s["parent"].long()
    pages, width = refs.numel(), table.shape[1]
    col = torch.arange(width, device="cuda")
    # fork: every sequence takes its parent's pages; a page's count changes by (children - 1) per holder
    held = lens[parent]
    used = (held + page - 1) // page
    out = torch.where(col < used[:, None], table[parent], s["table_out"])
    children = torch.zeros_like(lens).scatter_add_(0, parent, torch.ones_like(parent))
    before = (lens + page - 1) // page
    listed_pages = torch.where(col < before[:, None], table.long(), pages)
    count = torch.zeros(pages + 1, dtype=I64, device="cuda")
    count[:pages] = refs
    count.scatter_add_(0, listed_pages.reshape(-1), (children - 1)[:, None].expand(-1, width).reshape(-1))
    count = count[:pages]
    # growth: a last page that others hold too is copied by all but the last of its holders that grow
    new = (s["cu_new"][1:] - s["cu_new"][:-1]).long()
    grown = (held + new + page - 1) // page
    fits = grown <= width
    last = out.gather(1, (used - 1).clamp(min=0)[:, None])[:, 0].long()
    partial = (held % page != 0) & (new > 0) & fits
    same = (last[:, None] == last[None]) & partial[:, None] & partial[None]
    rank = same.tril(-1).sum(1)
    shares = partial & (count[last.clamp(min=0)] > 1)
    copies = shares & (count[last.clamp(min=0)] - rank > 1)
    need = torch.where(fits, grown - used + copies, 0)
    prefix = need.cumsum(0)
    free = count == 0
    served = fits & ((prefix <= free.sum()) | ((need == 0) & ~shares))
    order = torch.where(free, free.cumsum(0) - 1, pages)
    handed = torch.empty(pages + 1, dtype=I64, device="cuda")
    handed[order] = torch.arange(pages, device="cuda")
    first = used - copies.long()
    pick = (prefix - need)[:, None] + col - first[:, None]
    takes = (col >= first[:, None]) & (col < grown[:, None]) & served[:, None]
    fresh = handed[pick.clamp(0, pages)]
    out = torch.where(takes, fresh, out.long())
    copies = copies & served
    count = torch.cat([count, count.new_zeros(1)])
    count.scatter_add_(0, torch.where(copies, last, pages), -torch.ones_like(last))
    count.scatter_(0, torch.where(takes, fresh, pages).reshape(-1), 1)
    start = torch.where(served, held, -1)
    src = torch.where(copies, last, -1)
    dst = torch.where(copies, out.gather(1, (used - 1).clamp(min=0)[:, None])[:, 0], -1)
    _plain_copy(s["pools"], src, dst)
    ints = [out, torch.where(served, held + new, held), count[:pages], start, src, dst]
    return [x.to(I32) for x in ints] + s["pools"]


def _plain_copy(pools, src, dst):
    moved = dst >= 0
    src, dst = src[moved], dst[moved]
    for p in pools:
        p[:, dst] = p[:, src]


def _plain_compact(s):
    table, refs, page = s["table"], s["refs"], s["page"]
    pages, width = refs.numel(), table.shape[1]
    live = refs > 0
    n = live.sum()
    at = torch.arange(pages, device="cuda")
    moves, holes = live & (at >= n), ~live & (at < n)
    m = moves.sum()
    move_rank, hole_rank = moves.cumsum(0) - 1, holes.cumsum(0) - 1
    hole = torch.full((pages + 1,), -1, dtype=I64, device="cuda")
    hole[torch.where(holes, hole_rank, pages)] = at
    page_map = torch.where(moves, hole[move_rank.clamp(min=0)], torch.where(live, at, -1))
    src, dst = at[moves], page_map[moves]
    used = (s["lens"].long() + page - 1) // page
    mapped = page_map[table.clamp(min=0).long()]
    out = torch.where(torch.arange(width, device="cuda") < used[:, None], mapped, s["table_out"].long())
    refs_out = torch.zeros(pages + 1, dtype=I64, device="cuda")
    refs_out[torch.where(live, page_map, pages)] = refs.long()
    for p in s["pools"]:
        p[:, dst] = p[:, src]
    return [x.to(I32) for x in (out, refs_out[:pages], page_map, torch.stack([n, m]))] + s["pools"]


def _plain_append(s):
    row = torch.arange(s["k"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu_new"][1:].long(), row, right=True)
    pos = s["start"].long()[seq] + row - s["cu_new"].long()[seq]
    page, off = s["table"][seq, pos // s["page"]].long(), pos % s["page"]
    s["k_pages"][page, :, off] = s["k"]
    s["v_pages"][page, :, off] = s["v"]
    s["logsig_pages"][page, off] = s["logsig"]
    return [s["k_pages"], s["v_pages"], s["logsig_pages"]]


def _plain_delta(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    d = s["d"]
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6) / math.sqrt(d)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    state = s["state"] if s["parent"] is None else s["state"][s["parent"].long()]
    old = torch.exp(s["log_alpha"])[..., None, None] * state
    c = s["beta"][..., None] * (v - (old * k[..., None, :]).sum(-1))
    new = old + c[..., None] * k[..., None, :]
    return (new * q[..., None, :]).sum(-1).to(s["dtype"]), new


def _plain_beam(s):
    groups, beams, vocab = s["groups"], s["beams"], s["vocab"]
    # in 64 bits: beams meet at sums that differ in the last places of 32
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    logp = x - top - torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    total = (s["scores"].double().reshape(-1, 1) + logp).reshape(groups, beams * vocab)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)
    best, at = best[:, :s["n_out"]], at[:, :s["n_out"]]
    parent = at // vocab + torch.arange(groups, device="cuda")[:, None] * beams
    return best.float(), parent.to(I32), (at % vocab).to(I32)


# ---- what one pass cannot do without -------------------------------------------------------------


def work(case):
    e = DTYPES[case["dtype"]].itemsize
    op = case["op"]
    if op == "attention":
        # lengths differ by seed: their expected sum
        lo, hi, n = case["shortest"], case["longest"], case["batch"]
        if case.get("name") == "attention_ragged_long" or hi > 20000:
            rest = (hi - lo) / math.log(hi / lo) if hi > lo else hi
            tokens = lo + hi + (n - 2) * rest if n > 1 else rest
        else:
            tokens = n * (lo + hi) / 2
        row = case["hkv"] * case["d"] * e
        pages = tokens / case["page"] + n
        return {"bytes": int(tokens * (2 * row + 4) + 2 * n * case["hq"] * case["d"] * e + 4 * (n * case["hq"] + pages)),
                "flops": int(4 * tokens * case["hq"] * case["d"])}
    if op == "fork":
        n = case["groups"] * case["beams"]
        used = n * ((case["prompt"] * 7 / 8 + case["tail"] / 2) / case["page"] + 1)
        copied = n / 3 * case["page"] * (2 * case["layers"] * case["hkv"] * case["d"] * e + 4)
        return {"bytes": int(2 * copied + 8 * used + 8 * case["pool"] + 24 * n), "flops": 0}
    if op == "compact":
        live = case["batch"] * (case["longest"] / 2 / case["page"] + 0.5)
        moved = max(0.0, live * (1 - live / case["pool"])) * case["page"] * (2 * case["layers"] * case["hkv"] * case["d"] * e + 4)
        return {"bytes": int(2 * moved + 8 * live + 12 * case["pool"]), "flops": 0}
    if op == "append":
        lo, hi, n = case["shortest"], case["longest"], case["batch"]
        rest = (hi - lo) / math.log(hi / lo) if hi > lo else hi
        rows = lo + hi + (n - 2) * rest if n > 1 else rest
        return {"bytes": int(2 * rows * (2 * case["hkv"] * case["d"] * e + 4)), "flops": 0}
    if op == "delta":
        rows = case["batch"] * case["heads"]
        return {"bytes": rows * (8 * case["d"] ** 2 + 4 * case["d"] * e + 8), "flops": rows * 7 * case["d"] ** 2}
    rows = case["groups"] * case["beams"]
    return {"bytes": rows * case["vocab"] * e + 4 * rows + 12 * case["groups"] * case["n_out"], "flops": 3 * rows * case["vocab"]}


# ---- from the definitions, in 64 bits ------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _exact_attention(s):
    b, hq, d = s["q"].shape
    group = hq // s["hkv"]
    out = torch.zeros((b, hq, d), dtype=F64, device="cuda")
    lse = torch.zeros((hq, b), dtype=F64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        at = s["table"][i, :(n + s["page"] - 1) // s["page"]].long()
        gates = s["logsig_pages"][at].reshape(-1)[:n].double()
        for g in range(s["hkv"]):
            k = s["k_pages"][at, g].reshape(-1, d)[:n].double()
            v = s["v_pages"][at, g].reshape(-1, d)[:n].double()
            heads = slice(g * group, (g + 1) * group)
            scale = (s["temp"][heads].double() * math.sqrt(d))[:, None]
            logit = torch.einsum("hd,nd->hn", s["q"][i, heads].double(), k) / scale + s["gain"][heads].double()[:, None] * gates
            lse[heads, i] = torch.logsumexp(logit, 1)
            out[i, heads] = torch.softmax(logit, 1) @ v
    return out, lse


def _exact_fork(s):
    """The pages as a list of counts and tables, sequence by sequence."""
    page = s["page"]
    lens, rows, refs = s["lens"].tolist(), s["table"].tolist(), s["refs"].tolist()
    parent, cu = s["parent"].tolist(), s["cu_new"].tolist()
    out = s["table_out"].tolist()
    for b, n in enumerate(lens):
        for p in rows[b][:-(-n // page)]:
            refs[p] += parent.count(b) - 1
    kept = [list(rows[p][:-(-lens[p] // page)]) for p in parent]
    held = [lens[p] for p in parent]
    free = [p for p, r in enumerate(refs) if r == 0]
    before = list(refs)
    start, src, dst, full = [], [], [], False
    for i, pages in enumerate(kept):
        n = cu[i + 1] - cu[i]
        more = -(-(held[i] + n) // page) - len(pages)
        partial = n > 0 and held[i] % page != 0
        shared = partial and refs[pages[-1]] > 1
        need = more + shared
        wide = len(pages) + more > len(out[i])
        full = full or (need > len(free) and not wide)
        a = b = -1
        if wide or (full and (need or (partial and before[pages[-1]] > 1))):
            start.append(-1)
        else:
            start.append(held[i])
            if shared:
                a, b = pages[-1], free.pop(0)
                refs[a] -= 1
                refs[b] = 1
                pages[-1] = b
            for _ in range(more):
                pages.append(free.pop(0))
                refs[pages[-1]] = 1
            held[i] += n
        src.append(a)
        dst.append(b)
        out[i][:len(pages)] = pages
    for p in s["pools"]:
        for a, b in zip(src, dst):
            if b >= 0:
                p[:, b].copy_(p[:, a])
    return [torch.tensor(x, dtype=I32) for x in (out, held, refs, start, src, dst)] + s["pools"]


def _exact_compact(s):
    refs, page = s["refs"].tolist(), s["page"]
    live = [p for p, r in enumerate(refs) if r > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] == 0]
    movers = [p for p in live if p >= n]
    page_map = [p if r > 0 else -1 for p, r in enumerate(refs)]
    for a, b in zip(movers, holes):
        page_map[a] = b
    out = s["table_out"].tolist()
    for i, (row, length) in enumerate(zip(s["table"].tolist(), s["lens"].tolist())):
        used = -(-length // page)
        out[i][:used] = [page_map[p] for p in row[:used]]
    new = [0] * len(refs)
    for p in live:
        new[page_map[p]] = refs[p]
    for p in s["pools"]:
        for a, b in zip(movers, holes):
            p[:, b].copy_(p[:, a])
    return [torch.tensor(x, dtype=I32) for x in (out, new, page_map, [n, len(movers)])] + s["pools"]


def _exact_append(s):
    cu, start, table = s["cu_new"].tolist(), s["start"].tolist(), s["table"].tolist()
    for b, first in enumerate(start):
        row, pos = cu[b], first
        while row < cu[b + 1]:
            off = pos % s["page"]
            n = min(s["page"] - off, cu[b + 1] - row)
            at = table[b][pos // s["page"]]
            s["k_pages"][at, :, off:off + n] = s["k"][row:row + n].transpose(0, 1)
            s["v_pages"][at, :, off:off + n] = s["v"][row:row + n].transpose(0, 1)
            s["logsig_pages"][at, off:off + n] = s["logsig"][row:row + n]
            row, pos = row + n, pos + n
    return [s["k_pages"], s["v_pages"], s["logsig_pages"]]


def _exact_delta(s):
    b, h, d = s["q"].shape
    out = torch.empty((b, h, d), dtype=F64, device="cuda")
    new = torch.empty((b, h, d, d), dtype=F64, device="cuda")
    for i in range(b):
        old = s["state"][i if s["parent"] is None else int(s["parent"][i])].double()
        q, k, v = (s[n][i].double() for n in ("q", "k", "v"))
        q = q / torch.sqrt(torch.einsum("hd,hd->h", q, q) + 1e-6)[:, None] / math.sqrt(d)
        k = k / torch.sqrt(torch.einsum("hd,hd->h", k, k) + 1e-6)[:, None]
        old = old * torch.exp(s["log_alpha"][i].double())[:, None, None]
        c = (v - torch.einsum("hij,hj->hi", old, k)) * s["beta"][i].double()[:, None]
        new[i] = old + torch.einsum("hi,hj->hij", c, k)
        out[i] = torch.einsum("hij,hj->hi", new[i], q)
    return out, new


def _exact_beam(s):
    beams, vocab, n = s["beams"], s["vocab"], s["n_out"]
    best, parent, token = [], [], []
    for g in range(s["groups"]):
        found = []
        for b in range(beams):
            x = s["logits"][g * beams + b].double()
            logp = torch.log_softmax(x, 0) + s["scores"][g, b].double()
            # every continuation that can be among this beam's best, the ones equal to its last included
            floor = torch.topk(logp, min(n, vocab)).values[-1]
            for t in (logp >= floor).nonzero()[:, 0].tolist():
                found.append((-float(logp[t]), g * beams + b, t))
        found.sort()
        best.append([-f[0] for f in found[:n]])
        parent.append([f[1] for f in found[:n]])
        token.append([f[2] for f in found[:n]])
    return torch.tensor(best, dtype=F64), torch.tensor(parent, dtype=I32), torch.tensor(token, dtype=I32)
