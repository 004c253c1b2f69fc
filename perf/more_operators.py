"""The paged 8-bit cache as cases: rows appended to pages that hold 8-bit codes with a scale for each page and kv
head (and read back), attention over such pages for single tokens and for prompt rows, and the pages' own upkeep:
freeing, forking and reserving with copies of what is shared, and compacting.  `run` computes a case in its plain
form (torch operations, 32 bits; 64 for norms, angles and what decides a rounding) or, with `own` set, by the
library's calls; `exact` is the definition in 64 bits."""
import math

import numpy as np
import torch

own = False
EPS = 2.0 ** -20
SMALLEST = 2.0 ** -40          # a page's scale below this is stored as 0
TOP = {"i8": 127.0, "e4m3": 448.0}


def _spread(n, lo, hi, turn=7):
    """n lengths from lo to hi, evenly over their logarithm, in a scattered order."""
    at = [(i * turn) % n for i in range(n)]
    return ",".join(str(int(round(lo * (hi / lo) ** (a / max(1, n - 1))))) for a in at)


def _cache(name, op, n_q, n_kv, head_dim, window, rope_dims, theta, k_eq_v, page, codes, past, rows):
    return {"name": name, "op": op, "n_q": n_q, "n_kv": n_kv, "head_dim": head_dim, "window": window,
            "rope_dims": rope_dims, "theta": theta, "k_eq_v": k_eq_v, "page": page, "codes": codes, "past": past,
            "rows": rows}


def _pages(name, op, caches, n_kv, head_dim, page, groups, beams, lo, hi, n_pages):
    return {"name": name, "op": op, "caches": caches, "n_kv": n_kv, "head_dim": head_dim, "page": page,
            "groups": groups, "beams": beams, "lo": lo, "hi": hi, "n_pages": n_pages}


def listed():
    """`past`: tokens that a sequence holds before the new rows (-1: an idle slot of a fixed batch), `rows`: its new
    rows."""
    ones = ",".join(["1"] * 64)
    return [
        # a decode step's new rows of 64 sequences: latency; every row joins a page that is begun, or begins one
        _cache("append-step", "append", 8, 2, 256, 512, 256, 1e4, False, 64, "i8", _spread(64, 100, 8000), ones),
        # prompt chunks of ragged lengths, one that starts inside a page, one of a single row, one of none
        _cache("append-prompt", "append", 32, 8, 128, 0, 128, 1e4, False, 32, "e4m3", "0,77,4000,0,31",
               "4096,2500,1,0,1411"),
        # one short sequence: latency
        _cache("decode-short", "decode", 4, 2, 64, 0, 64, 1e4, False, 16, "i8", "41", "1"),
        # a serving batch of ragged sequences with idle slots
        _cache("decode-ragged", "decode", 32, 8, 128, 0, 128, 1e4, False, 32, "e4m3",
               _spread(62, 500, 16000) + ",-1,-1", ones),
        # the stack's full layer (keys = values, one kv head, partial rotation) over eight sequences of 32k
        _cache("decode-full", "decode", 16, 1, 512, 0, 128, 1e6, True, 64, "i8", ",".join(["32700"] * 8),
               ",".join(["1"] * 8)),
        # verify windows of four drafted rows on the stack's sliding layer
        _cache("verify-sliding", "prefill", 8, 2, 256, 512, 256, 1e4, False, 64, "i8", _spread(16, 40, 6000),
               ",".join(["4"] * 16)),
        # whole prompts of different lengths in one call, one row and none among them
        _cache("prompt-packed", "prefill", 32, 8, 128, 0, 128, 1e4, False, 32, "e4m3", "0,0,0,0,0",
               "4096,1500,777,1,0"),
        # a prompt's later chunk over what is cached already: few rows, many keys
        _cache("chunk-long", "prefill", 8, 2, 256, 0, 256, 1e4, False, 64, "i8", "16300", "500"),
        # a step of beam search on one cache: dropped beams freed, others forked, a token reserved for each
        _pages("beams-one", "fork", 1, 2, 64, 16, 4, 4, 30, 300, 512),
        # the same on the stack's 20 sliding donors, whose pages are copied together
        _pages("beams-stack", "fork", 20, 2, 256, 64, 24, 4, 200, 1500, 1024),
        # a pool with holes made dense: one cache, and the stack's donors
        _pages("compact-one", "compact", 1, 2, 64, 16, 8, 2, 30, 300, 600),
        _pages("compact-stack", "compact", 20, 2, 256, 64, 40, 2, 100, 1500, 900),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    head_dim = rng.choice([64, 128, 128, 256, 512])
    n_kv = rng.choice([1, 2, 4, 8])
    while n_kv * head_dim > 1024:
        n_kv //= 2
    page = rng.choice([16, 32, 64, 128])
    what = rng.random()
    if what < 0.24:
        beams = rng.choice([2, 3, 4, 6])
        groups = _log(rng, 1, 96 // beams)
        hi = _log(rng, 2 * page, 24 * page)
        n_pages = groups * beams * (hi // page + 3) + rng.randint(0, 200)
        caches = _log(rng, 1, 20)
        while caches * n_pages * page * n_kv * head_dim * 2 > (1 << 30) and caches > 1:
            caches //= 2
        c = _pages("", rng.choice(["fork", "compact"]), caches, n_kv, head_dim, page, groups, beams,
                   rng.randint(1, page), hi, n_pages)
        return {k: v for k, v in c.items() if k != "name"}
    group = rng.choice([1, 2, 4, 8, 16, 3])
    while n_kv * group * head_dim > 8192:
        group = max(1, group // 2)
    codes, window = rng.choice(["i8", "e4m3"]), rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    rope = rng.choice([0, head_dim // 4, head_dim // 2, head_dim])
    k_eq_v = rng.random() < 0.25
    if what < 0.44:
        n = _log(rng, 1, 64)
        rows = [_log(rng, 1, 4096 // n) if rng.random() < 0.9 else 0 for _ in range(n - 1)] + [_log(rng, 1, 64)]
        past = [rng.choice([0, _log(rng, 1, 8000)]) for _ in range(n)]
        op = "append"
    elif what < 0.74:
        n = _log(rng, 1, 96)
        top = max(64, min(32000, 32000 * 8 * 512 // (n * n_kv * head_dim)))
        past = [_log(rng, 1, top) if rng.random() < 0.95 else -1 for _ in range(n - 1)] + [_log(rng, 1, top)]
        rows, op = [1] * n, "decode"
    else:
        n = _log(rng, 1, 8)
        rows = [_log(rng, 1, 2048 // n) if rng.random() < 0.9 else 0 for _ in range(n - 1)] + [_log(rng, 1, 1024)]
        past = [rng.choice([0, _log(rng, 1, 8000 // n)]) for _ in range(n)]
        while sum(_seen(p, r, window) for p, r in zip(past, rows)) * n_kv * group * head_dim > 4e10:
            past, rows = [p // 2 for p in past], [-(-r // 2) for r in rows]
        op = "prefill"
    c = _cache("", op, n_kv * group, n_kv, head_dim, window, rope, rng.choice([1e4, 1e6]), k_eq_v, page, codes,
               ",".join(map(str, past)), ",".join(map(str, rows)))
    return {k: v for k, v in c.items() if k != "name"}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _seen(past, rows, window):
    """(row, key) pairs of one sequence: a row at p sees min(p + 1, window) keys."""
    if past < 0:
        return 0
    ends = range(past + 1, past + rows + 1)
    return sum(min(e, window) if window > 0 else e for e in ends)


def work(case):
    if case["op"] in ("fork", "compact"):
        moved, entries = _counts(case)
        page = case["page"] * case["n_kv"] * case["head_dim"] * 2 + case["n_kv"] * 8
        return {"bytes": 2.0 * moved * case["caches"] * page + 4 * (entries + case["n_pages"]), "flops": 0.0}
    past, rows, d, n_kv, n_q = _ints(case["past"]), _ints(case["rows"]), case["head_dim"], case["n_kv"], case["n_q"]
    if case["op"] == "append":
        new = sum(rows)
        again = sum(r + p % case["page"] for p, r in zip(past, rows) if r)
        raw = 1 if case["k_eq_v"] else 2
        return {"bytes": new * n_kv * d * (2 * raw + 2) + again * n_kv * d * 2 * (1 + 2), "flops": 20.0 * new * n_kv * d}
    keys = 0
    for p, r in zip(past, rows):
        if p >= 0 and r:
            first = max(0, p - case["window"] + 1) if case["window"] > 0 else 0
            keys += p + r - first
    pairs = sum(_seen(p, r, case["window"]) for p, r in zip(past, rows))
    return {"bytes": keys * n_kv * d * 2 + sum(rows) * n_q * d * 4, "flops": 4.0 * pairs * n_q * d}


# ---- inputs ---------------------------------------------------------------------------------------------------------


def _codes(g, shape, kind):
    """Codes as quantized rows have them: values about a quarter of the largest."""
    x = torch.randn(shape, generator=g, device="cuda") * (TOP[kind] / 4)
    x = x.clamp_(-TOP[kind], TOP[kind])
    return x.round_().to(torch.int8) if kind == "i8" else x.to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("fork", "compact"):
        return _prepare_pages(case, seed, g)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    past, rows, page, n_kv, d = _ints(case["past"]), _ints(case["rows"]), case["page"], case["n_kv"], case["head_dim"]
    n, dev = len(past), {"device": "cuda", "dtype": torch.int32}
    # pages in scattered order, a tenth of the pool free
    held = [max(0, -(-(max(p, 0) + r) // page)) if p >= 0 else 0 for p, r in zip(past, rows)]
    n_pages = sum(held) + max(1, sum(held) // 10)
    order = np.random.RandomState(seed).permutation(n_pages)
    tables, at = np.full((n, max(1, max(held))), -1, np.int32), 0
    for s, h in enumerate(held):
        tables[s, :h] = order[at:at + h]
        at += h
    offs = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    state = {"case": dict(case), "n_rows": int(offs[-1]), "max_rows": max(1, max(rows)), "n_pages": n_pages,
             "tables": torch.tensor(tables, **dev), "start": torch.tensor(past, **dev),
             "offs": torch.tensor(offs, **dev), "max_pos": max(0, max(p + max(r, 1) - 1 for p, r in zip(past, rows)))}
    shape = (n_pages, n_kv, page, d)
    state["k"], state["v"] = _codes(g, shape, case["codes"]), _codes(g, shape, case["codes"])
    unit = 4 / TOP[case["codes"]]
    scales = lambda: unit * (0.7 + 0.6 * torch.rand(n_pages, n_kv, generator=g, device="cuda"))  # noqa: E731
    state["ks"], state["vs"] = scales(), scales()
    total = state["n_rows"]
    if case["op"] == "append":
        state["k_raw"] = rnd(total, n_kv, d).bfloat16()
        state["v_raw"] = None if case["k_eq_v"] else rnd(total, n_kv, d).bfloat16()
        state["k_w"] = (1 + 0.1 * rnd(d)).bfloat16()
        # what is read back: each sequence from the first row of the page that its new rows begin in
        first = [p // page * page for p in past]
        back = [p + r - f if r else 0 for p, r, f in zip(past, rows, first)]
        boffs = np.concatenate([[0], np.cumsum(back)]).astype(np.int32)
        state["back_start"], state["back_offs"] = torch.tensor(first, **dev), torch.tensor(boffs, **dev)
        state["n_back"] = int(boffs[-1])
    else:
        state["q"] = rnd(total, case["n_q"], d).bfloat16()
        # scores of deviation about 3: rows with a few large weights and many small ones
        state["q_w"] = ((1 + 0.1 * rnd(d)) * 3 / math.sqrt(d)).bfloat16()
    return state


def _beams(case):
    """Tokens and shared prompt pages of the groups: (length of the prompt, length of each beam's own tail)."""
    n = case["groups"]
    whole = _ints(_spread(n, case["lo"] + 1, case["hi"], turn=5))
    return [(w * 2 // 3, w - w * 2 // 3) for w in whole]


def _counts(case):
    """Pages that one pass moves, and the table entries that it reads or writes."""
    page, moved, entries, live = case["page"], 0, 0, 0
    for prompt, tail in _beams(case):
        beams, full = case["beams"], prompt // page
        length = prompt + tail
        entries += beams * -(-length // page)
        if case["op"] == "fork":
            survivors, shared = max(1, beams // 2), min(max(1, beams // 2), beams - max(1, beams // 2))
            if length % page:
                moved += beams - (survivors - shared)     # forks and the beams that they were forked from
        else:
            live += full + beams * (-(-length // page) - full)
    if case["op"] == "compact":
        moved = int(round(live * (1 - live / max(live, case["n_pages"]))))
    return moved, entries


def _prepare_pages(case, seed, g):
    groups, beams, page, n_kv, d = case["groups"], case["beams"], case["page"], case["n_kv"], case["head_dim"]
    n_seqs, n_pages = groups * beams, case["n_pages"]
    max_pages = -(-(case["hi"] + 2) // page) + 1
    order = list(np.random.RandomState(seed).permutation(n_pages))
    # tables, lengths and references in one buffer, as a pool keeps them
    tables, lens, refs = np.full((n_seqs, max_pages), -1, np.int32), np.zeros(n_seqs, np.int32), np.zeros(n_pages, np.int32)
    for b, (prompt, tail) in enumerate(_beams(case)):
        shared = [order.pop() for _ in range(prompt // page)]     # the prompt's whole pages, held by every beam
        for i in range(beams):
            s = b * beams + i
            mine = shared + [order.pop() for _ in range(-(-(prompt + tail) // page) - len(shared))]
            tables[s, :len(mine)], lens[s] = mine, prompt + tail
            refs[mine] += 1
    first = torch.tensor(np.concatenate([tables.ravel(), lens, refs]), device="cuda")
    state = {"case": dict(case), "first": first, "now": first.clone(), "n_seqs": n_seqs, "n_pages": n_pages,
             "max_pages": max_pages}
    cut = [n_seqs * max_pages, n_seqs, n_pages]
    state["tables"], state["lens"], state["refs"] = torch.split(state["now"], cut)
    state["tables"] = state["tables"].view(n_seqs, max_pages)
    # [cache and kind][page][head][token][dim]: k of cache c at 2 c, v at 2 c + 1
    state["codes"] = torch.randint(-127, 128, (2 * case["caches"], n_pages, n_kv, page, d), generator=g, device="cuda",
                                   dtype=torch.int8)
    state["scales"] = 0.03 * (0.7 + 0.6 * torch.rand(2 * case["caches"], n_pages, n_kv, generator=g, device="cuda"))
    if case["op"] == "fork":
        # of each group the later beams are dropped and the earlier ones forked in their place, in turn
        keep = max(1, beams // 2)
        child = [b * beams + i for b in range(groups) for i in range(keep, beams)]
        parent = [b * beams + (i - keep) % keep for b in range(groups) for i in range(keep, beams)]
        state["child"] = torch.tensor(child, device="cuda", dtype=torch.int32)
        state["parent"] = torch.tensor(parent, device="cuda", dtype=torch.int32)
        state["n_new"] = torch.ones(n_seqs, device="cuda", dtype=torch.int32)
    return state


# ---- the plain forms ------------------------------------------------------------------------------------------------


def _to_bf16(x):
    """64 bits to bf16 in one rounding: a value that 32 bits round onto a tie is moved off it first."""
    f = x.float()
    rest = x - f.double()
    tie = (f.view(torch.int32) & 0xFFFF) == 0x8000
    f = torch.where(tie & (rest != 0), torch.nextafter(f, f + torch.sign(rest).float()), f)
    return f.bfloat16()


def _norm(x, w):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _to_bf16(y if w is None else y * w.double())


def _rotate(x, pos, rope_dims, theta):
    """Pairs (j, j + rope_dims / 2) of rows [rows, heads, D] at their positions."""
    if rope_dims == 0:
        return x
    h, d = rope_dims // 2, x.shape[-1]
    f = theta ** (-2.0 * torch.arange(h, dtype=torch.float64, device=x.device) / d)
    a = pos.double()[:, None, None] * f
    c, s, lo, hi = a.cos(), a.sin(), x[..., :h].double(), x[..., h:rope_dims].double()
    return torch.cat([_to_bf16(lo * c - hi * s), _to_bf16(hi * c + lo * s), x[..., rope_dims:]], -1)


def _places(offs, start, n):
    """Sequence and position of each of n packed rows."""
    row = torch.arange(n, device=offs.device, dtype=torch.int32)
    seq = torch.searchsorted(offs[1:].contiguous(), row, right=True)
    return seq, (start[seq] + row - offs[seq]).long()


def _encode(x, kind):
    if kind == "i8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _append_kind(x, codes, scales, state, seq, pos):
    """Quantize the rows x [rows, n_kv, D] into their pages."""
    kind, size = state["case"]["codes"], state["case"]["page"]
    page, slot = state["tables"][seq, pos // size].long(), pos % size
    most = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax")
    new = most / TOP[kind]
    new = torch.where(new < SMALLEST, torch.zeros_like(new), new)
    # pages that already hold rows keep a scale at least as large, and their rows move to it
    start, offs = state["start"].long(), state["offs"]
    begun = (offs[1:] > offs[:-1]) & (start % size > 0)
    old_page = state["tables"].gather(1, (start // size).clamp(max=state["tables"].shape[1] - 1)[:, None])[:, 0].long()
    old_page = torch.where(begun, old_page, -1)
    has_old = torch.zeros(scales.shape[0] + 1, device=x.device, dtype=torch.bool)
    has_old[old_page] = True
    has_old[-1] = False
    has_old = has_old[:-1]
    scale = torch.where(has_old[:, None], torch.maximum(new, scales), new)
    touched = torch.zeros(scales.shape[0], device=x.device, dtype=torch.bool)
    touched[page] = True
    at = old_page.clamp(min=0)
    was, now = scales[at][:, :, None, None], scale[at][:, :, None, None]
    old = codes.view(torch.int8)[at]
    moved = _encode(old.view(codes.dtype).float() * was / torch.where(now > 0, now, torch.ones_like(now)), kind)
    grown = begun[:, None, None, None] & (now > was)
    grown = grown & (torch.arange(size, device=x.device)[None, None, :, None] < (start % size)[:, None, None, None])
    # a sequence without such a page writes what its page 0 holds to a row that nothing reads
    raw = torch.where(grown, moved.view(torch.int8), old)
    keep = torch.where(begun, old_page, codes.shape[0])
    padded = torch.cat([codes.view(torch.int8), codes.view(torch.int8)[:1]])
    padded[keep] = raw
    s = scale[page][..., None]
    y = _encode(torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x)), kind)
    padded[page, :, slot] = y.view(torch.int8)
    codes.view(torch.int8).copy_(padded[:-1])
    scales.copy_(torch.where(touched[:, None], scale, scales))


def _read_back(state):
    seq, pos = _places(state["back_offs"], state["back_start"], state["n_back"])
    size = state["case"]["page"]
    page, slot = state["tables"][seq, pos // size].long(), pos % size
    take = lambda c, s: (c.view(torch.int8)[page, :, slot].view(c.dtype).float() * s[page][..., None]).bfloat16()  # noqa: E731
    return take(state["k"], state["ks"]), take(state["v"], state["vs"])


def _append_plain(state):
    case = state["case"]
    seq, pos = _places(state["offs"], state["start"], state["n_rows"])
    k = _rotate(_norm(state["k_raw"], state["k_w"]), pos, case["rope_dims"], case["theta"])
    v = _norm(state["k_raw"] if case["k_eq_v"] else state["v_raw"], None)
    _append_kind(k.float(), state["k"], state["ks"], state, seq, pos)
    _append_kind(v.float(), state["v"], state["vs"], state, seq, pos)
    k_back, v_back = _read_back(state)
    return {"k": k_back, "v": v_back, "k_scales": state["ks"], "v_scales": state["vs"]}


def _attend_plain(state):
    case = state["case"]
    n_kv, d, size = case["n_kv"], case["head_dim"], case["page"]
    offs, start, total = state["offs"], state["start"], state["n_rows"]
    seq, pos = _places(offs, start, total)
    q = _rotate(_norm(state["q"], state["q_w"]), pos, case["rope_dims"], case["theta"]).float()
    n, most = start.shape[0], state["max_rows"]
    group = case["n_q"] // n_kv
    # rows padded to [sequence, kv head, head of the group, row]
    padded = torch.zeros(n, most, case["n_q"], d, device=q.device)
    t = torch.arange(total, device=q.device) - offs[seq]
    padded[seq, t] = q
    padded = padded.view(n, most, n_kv, group, d).permute(0, 2, 3, 1, 4).reshape(n, n_kv, group * most, d)
    held = state["tables"].clamp(min=0).long()

    def values(codes, scales):
        x = codes[held].float() if codes.dtype == torch.int8 else codes.view(torch.int8)[held].view(codes.dtype).float()
        x = x * scales[held][..., None, None]             # [n, pages, n_kv, page, D]
        return x.permute(0, 2, 1, 3, 4).reshape(n, n_kv, -1, d)

    s = padded @ values(state["k"], state["ks"]).transpose(2, 3)
    key = torch.arange(s.shape[-1], device=q.device)
    at = start.long()[:, None] + torch.arange(most, device=q.device)
    see = key <= at[..., None]
    if case["window"] > 0:
        see &= key > at[..., None] - case["window"]
    see &= (start >= 0)[:, None, None]
    s = s.view(n, n_kv, group, most, -1).masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    p /= p.sum(-1, keepdim=True).clamp_(min=1e-30)
    o = p.view(n, n_kv, group * most, -1) @ values(state["v"], state["vs"])
    o = o.view(n, n_kv, group, most, d).permute(0, 3, 1, 2, 4).reshape(n, most, case["n_q"], d)
    return {"out": o[seq, t].bfloat16()}


def _reset(state):
    """The pool as it was before the step, so that every pass does the same work."""
    state["now"].copy_(state["first"])


def _freed(state, which):
    """All pages of the sequences `which` given back."""
    page, held = state["case"]["page"], state["tables"][which.long()]
    used = torch.arange(held.shape[1], device=held.device)[None] < (-(-state["lens"][which.long()] // page))[:, None]
    state["refs"].index_add_(0, torch.where(used, held, 0).view(-1).long(), -used.view(-1).to(torch.int32))
    state["tables"][which.long()] = -1
    state["lens"][which.long()] = 0


def _fork_plain(state):
    _reset(state)
    page, tables, lens, refs = state["case"]["page"], state["tables"], state["lens"], state["refs"]
    child, parent = state["child"].long(), state["parent"].long()
    _freed(state, state["child"])
    # the children hold their parents' pages
    tables[child] = tables[parent]
    lens[child] = lens[parent]
    used = torch.arange(tables.shape[1], device=lens.device)[None] < (-(-lens[child] // page))[:, None]
    refs.index_add_(0, torch.where(used, tables[child], 0).view(-1).long(), used.view(-1).to(torch.int32))
    # room for n_new tokens: a shared page that would be written is copied, then new pages follow
    new = lens + state["n_new"]
    has, want = -(-lens // page), -(-new // page)
    last = tables.gather(1, (has - 1).clamp(min=0)[:, None].long())[:, 0]
    copy = (state["n_new"] > 0) & (lens % page > 0) & (refs[last.clamp(min=0).long()] > 1)
    need = want - has + copy.to(torch.int32)
    upto = torch.cumsum(need, 0)
    free = torch.argsort((refs > 0).to(torch.int32), stable=True).to(torch.int32)
    granted = (need == 0) | (upto <= (refs == 0).sum())
    start = lens.clone()
    first = (upto - need).long()
    fill = first + copy.long()                            # where a sequence's new pages begin in the list
    i = torch.arange(tables.shape[1], device=lens.device)[None]
    fresh = granted[:, None] & (i >= has[:, None]) & (i < want[:, None])
    copied = granted & copy
    n_pages = refs.shape[0]
    took = free[(fill[:, None] + i - has[:, None]).clamp(0, n_pages - 1)]
    into = free[first.clamp(0, n_pages - 1)]
    tables.copy_(torch.where(fresh, took, tables))
    tables.scatter_(1, (has - 1).clamp(min=0)[:, None].long(),
                    torch.where(copied, into, tables.gather(1, (has - 1).clamp(min=0)[:, None].long())[:, 0])[:, None])
    src, dst = last[copied].long(), into[copied].long()
    state["codes"][:, dst] = state["codes"][:, src]
    state["scales"][:, dst] = state["scales"][:, src]
    refs.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    refs.index_add_(0, torch.cat([dst, took[fresh].long()]), torch.ones(1, device=refs.device, dtype=torch.int32).expand(dst.numel() + int(fresh.sum())))
    lens.copy_(torch.where(granted, new, lens))
    return {"tables": tables, "lens": lens, "refs": refs, "granted": granted.to(torch.int32), "start": start,
            "codes": state["codes"], "scales": state["scales"]}


def _compact_plain(state):
    _reset(state)
    tables, refs, n_pages = state["tables"], state["refs"], state["n_pages"]
    live = refs > 0
    n_live = live.sum()
    ids = torch.arange(n_pages, device=refs.device)
    hole, late = ids[~live & (ids < n_live)], ids[live & (ids >= n_live)]
    moved = torch.where(live, ids, -1).to(torch.int32)
    moved[late] = hole.to(torch.int32)
    state["codes"][:, hole] = state["codes"][:, late]
    state["scales"][:, hole] = state["scales"][:, late]
    refs[hole] = refs[late]
    refs[late] = 0
    tables.copy_(torch.where(tables >= 0, moved[tables.clamp(min=0).long()], tables))
    return {"tables": tables, "lens": state["lens"], "refs": refs, "page_map": moved,
            "n_live": n_live.to(torch.int32).view(1), "codes": state["codes"], "scales": state["scales"]}


# ---- the library's calls --------------------------------------------------------------------------------------------


def _one_cache(kvq, state, k, v, ks, vs):
    case = state["case"]
    kind = kvq.KVQ_CODE_E4M3 if k.dtype == torch.float8_e4m3fn else kvq.KVQ_CODE_I8
    return kvq.paged_cache(k, v, ks, vs, state["n_pages"], case["page"], case["n_kv"], case["head_dim"], kind)


def _own_layer(kvq, state):
    case = state["case"]
    state["layer"] = kvq.layer(case["n_q"], case["n_kv"], case["head_dim"], case["window"], case["rope_dims"],
                               case["theta"], EPS, case["k_eq_v"])
    state["cache"] = _one_cache(kvq, state, state["k"], state["v"], state["ks"], state["vs"])


def _append_own(state):
    import quantized_kv_attention_quant_gb300 as kvq
    if "layer" not in state:
        _own_layer(kvq, state)
        shape = (state["n_back"],) + tuple(state["k_raw"].shape[1:])
        state["back"] = [torch.empty(shape, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    n, most = state["tables"].shape
    kvq.kvq_paged_append(state["layer"], state["cache"], state["tables"], most, n, state["offs"], state["start"],
                         state["n_rows"], state["k_raw"], state["v_raw"], state["k_w"])
    kvq.kvq_paged_gather(state["cache"], state["tables"], most, n, state["back_offs"], state["back_start"],
                         state["n_back"], state["back"][0], state["back"][1])
    return {"k": state["back"][0], "v": state["back"][1], "k_scales": state["ks"], "v_scales": state["vs"]}


def _attend_own(state):
    import quantized_kv_attention_quant_gb300 as kvq
    n, most = state["tables"].shape
    decode = state["case"]["op"] == "decode"
    if "layer" not in state:
        _own_layer(kvq, state)
        if decode:
            state["ws_bytes"] = kvq.attn_paged_decode_workspace_bytes(state["layer"], state["cache"], n, state["max_pos"])
        else:
            state["ws_bytes"] = kvq.attn_paged_prefill_workspace_bytes(state["layer"], state["cache"], n,
                                                                       state["n_rows"], state["max_rows"],
                                                                       state["max_pos"])
        state["ws"] = torch.empty(state["ws_bytes"], dtype=torch.uint8, device="cuda")
        state["out"] = torch.empty_like(state["q"])
    if decode:
        kvq.attn_paged_decode(state["layer"], state["cache"], state["tables"], most, n, state["start"],
                              state["max_pos"], state["q"], state["q_w"], state["out"], 0, None, state["ws"],
                              state["ws_bytes"])
    else:
        kvq.attn_paged_prefill(state["layer"], state["cache"], state["tables"], most, n, state["offs"], state["start"],
                               state["n_rows"], state["max_rows"], state["max_pos"], state["q"], state["q_w"],
                               state["out"], 0, None, state["ws"], state["ws_bytes"])
    return {"out": state["out"]}


def _pages_own(state):
    import quantized_kv_attention_quant_gb300 as kvq
    case, n_seqs = state["case"], state["n_seqs"]
    fork = case["op"] == "fork"
    if "pool" not in state:
        state["pool"] = kvq.page_pool(state["tables"], state["lens"], state["refs"], n_seqs, state["max_pages"],
                                      state["n_pages"], case["page"])
        c, s = state["codes"], state["scales"]
        state["caches"] = kvq.paged_caches([_one_cache(kvq, state, c[2 * i], c[2 * i + 1], s[2 * i], s[2 * i + 1])
                                            for i in range(case["caches"])])
        state["ws_bytes"] = kvq.kvq_pages_workspace_bytes(state["pool"])
        state["ws"] = torch.empty(state["ws_bytes"], dtype=torch.uint8, device="cuda")
        ints = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        state["granted"], state["started"] = ints(n_seqs), ints(n_seqs)
        state["page_map"], state["n_live"] = ints(state["n_pages"]), ints(1)
    pool, ws = state["pool"], (state["ws"], state["ws_bytes"])
    _reset(state)
    got = {"tables": state["tables"], "lens": state["lens"], "refs": state["refs"], "codes": state["codes"],
           "scales": state["scales"]}
    if fork:
        n = state["child"].shape[0]
        kvq.kvq_pages_free(pool, state["child"], None, n)
        kvq.kvq_pages_fork(pool, state["parent"], state["child"], n, None)
        kvq.kvq_pages_reserve(pool, state["caches"], state["n_new"], state["started"], state["granted"], *ws)
        return got | {"granted": state["granted"], "start": state["started"]}
    kvq.kvq_pages_compact(pool, state["caches"], state["page_map"], state["n_live"], *ws)
    return got | {"page_map": state["page_map"], "n_live": state["n_live"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return _append_own(state) if op == "append" else _pages_own(state) if op in ("fork", "compact") else _attend_own(state)
    if op == "append":
        return _append_plain(state)
    return _fork_plain(state) if op == "fork" else _compact_plain(state) if op == "compact" else _attend_plain(state)


# ---- the definition in 64 bits --------------------------------------------------------------------------------------


def _nearest_bf16(x):
    """bf16 nearest to values in 64 bits, ties to even, as 64-bit values."""
    m, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 8).clamp(min=-133))
    return torch.round(x / step) * step


def _turned(x, w, at, case):
    """The normed row, turned as complex pairs, with the two roundings to bf16 that the cache's rows have."""
    size = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    y = _nearest_bf16(x / size * w)
    half = case["rope_dims"] // 2
    if half:
        rate = torch.tensor([case["theta"] ** (-2.0 * j / x.shape[-1]) for j in range(half)], dtype=torch.float64,
                            device=x.device)
        z = torch.complex(y[..., :half], y[..., half:2 * half]) * torch.exp(1j * at[:, None, None] * rate)
        y = y.clone()
        y[..., :half], y[..., half:2 * half] = _nearest_bf16(z.real), _nearest_bf16(z.imag)
    return y


def _nearest_code(x, kind):
    if kind == "i8":
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))     # three bits behind the leading one, 2^-9 at least
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(case, state):
    past, rows, size, kind = _ints(case["past"]), _ints(case["rows"]), case["page"], case["codes"]
    tables = state["tables"].cpu().tolist()
    one = torch.ones(case["head_dim"], dtype=torch.float64, device="cuda")
    scales = {"k": state["ks"].double(), "v": state["vs"].double()}
    got, at = {"k": [], "v": []}, 0
    for s, (p, r) in enumerate(zip(past, rows)):
        if not r:
            continue
        raw = state["k_raw"][at:at + r].double()
        place = torch.arange(p, p + r, device="cuda").double()
        fresh = {"k": _turned(raw, state["k_w"].double(), place, case),
                 "v": _turned(raw if case["k_eq_v"] else state["v_raw"][at:at + r].double(), one, place,
                              {**case, "rope_dims": 0})}
        at += r
        for i in range(p // size, (p + r - 1) // size + 1):
            page = tables[s][i]
            lo, hi = max(p, i * size), min(p + r, (i + 1) * size)
            for kind_of in "kv":
                x = fresh[kind_of][lo - p:hi - p]                     # [rows, n_kv, D]
                scale = x.abs().amax((0, 2)) / TOP[kind]
                scale = torch.where(scale < SMALLEST, 0.0, scale)
                out = []
                if lo > i * size:
                    was = scales[kind_of][page].clone()
                    scale = torch.maximum(scale, was)
                    old = state[kind_of].view(torch.int8)[page][:, :lo - i * size].view(state[kind_of].dtype).double()
                    ratio = torch.where(scale > 0, was / scale, 0.0)[:, None, None]
                    old = torch.where(ratio == 1, old, _nearest_code(old * ratio, kind)).transpose(0, 1)
                    out.append(old * scale[:, None])
                safe = torch.where(scale > 0, scale, 1.0)[:, None]
                out.append(torch.where(scale[:, None] > 0, _nearest_code(x / safe, kind), 0.0) * scale[:, None])
                scales[kind_of][page] = scale
                got[kind_of].append(torch.cat(out))
    return {"k": torch.cat(got["k"]), "v": torch.cat(got["v"]), "k_scales": scales["k"], "v_scales": scales["v"]}


def _exact_attend(case, state):
    past, rows, size, n_kv = _ints(case["past"]), _ints(case["rows"]), case["page"], case["n_kv"]
    group, out, at = case["n_q"] // n_kv, torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda"), 0
    for s, (p, r) in enumerate(zip(past, rows)):
        if not r or p < 0:
            at += r
            continue
        place = torch.arange(p, p + r, device="cuda")
        q = _turned(state["q"][at:at + r].double(), state["q_w"].double(), place.double(), case)
        first = max(0, p - case["window"] + 1) if case["window"] > 0 else 0
        keys = torch.arange(first, p + r, device="cuda")
        page, slot = state["tables"][s][keys // size].long(), keys % size
        hide = keys[None, :] > place[:, None]
        if case["window"] > 0:
            hide |= keys[None, :] <= place[:, None] - case["window"]
        for h in range(n_kv):
            k, v = (state[c].view(torch.int8)[page, h, slot].view(state[c].dtype).double() * state[c + "s"][page, h].double()[:, None]
                    for c in "kv")
            for j in range(h * group, (h + 1) * group):
                score = torch.einsum("id,jd->ij", q[:, j], k).masked_fill(hide, -math.inf)
                out[at:at + r, j] = torch.einsum("ij,jd->id", torch.softmax(score, 1), v)
        at += r
    return {"out": out}


def _exact_pages(case, state):
    """The pool's bookkeeping, one sequence and one page after another."""
    size, tables = case["page"], state["first"][:state["n_seqs"] * state["max_pages"]].view(state["n_seqs"], -1).tolist()
    rest = state["first"][state["n_seqs"] * state["max_pages"]:].tolist()
    lens, refs = rest[:state["n_seqs"]], rest[state["n_seqs"]:]
    holds = lambda s: -(-lens[s] // size)  # noqa: E731
    codes, scales = state["codes"].clone(), state["scales"].double()
    src, dst, more = [], [], {}
    if case["op"] == "fork":
        child, parent = state["child"].tolist(), state["parent"].tolist()
        for c in child:
            for i in range(holds(c)):
                refs[tables[c][i]] -= 1
            tables[c], lens[c] = [-1] * len(tables[c]), 0
        for c, p in zip(child, parent):
            tables[c], lens[c] = list(tables[p]), lens[p]
            for i in range(holds(p)):
                refs[tables[p][i]] += 1
        free, before, asked = [i for i, r in enumerate(refs) if r == 0], list(refs), 0
        more = {"granted": [], "start": list(lens)}
        for s in range(len(lens)):
            have, want = holds(s), -(-(lens[s] + 1) // size)
            shared = lens[s] % size and before[tables[s][have - 1]] > 1
            need = want - have + bool(shared)
            mine = free[asked:asked + need]
            asked += need
            more["granted"].append(int(len(mine) == need))
            if len(mine) < need:
                continue
            if shared:
                src.append(tables[s][have - 1])
                dst.append(mine.pop(0))
                refs[src[-1]] -= 1
                tables[s][have - 1] = dst[-1]
                refs[dst[-1]] += 1
            for i, page in zip(range(have, want), mine):
                tables[s][i] = page
                refs[page] += 1
            lens[s] += 1
    else:
        n_live = sum(r > 0 for r in refs)
        dst = [i for i in range(n_live) if refs[i] == 0]
        src = [i for i in range(n_live, len(refs)) if refs[i] > 0]
        moved = [i if r > 0 else -1 for i, r in enumerate(refs)]
        for a, b in zip(src, dst):
            moved[a], refs[b], refs[a] = b, refs[a], 0
        tables = [[moved[p] if p >= 0 else p for p in t] for t in tables]
        more = {"page_map": moved, "n_live": [n_live]}
    for a, b in zip(src, dst):
        codes[:, b], scales[:, b] = codes[:, a].clone(), scales[:, a].clone()
    ints = {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in {"tables": tables, "lens": lens, "refs": refs, **more}.items()}
    return ints | {"codes": codes, "scales": scales}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, state)
    return _exact_pages(case, state) if case["op"] in ("fork", "compact") else _exact_attend(case, state)
