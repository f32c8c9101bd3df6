"""Measured cases of the paged-cache operators: the page plan, the append, the attention of one
new token over a paged cache, and the attention over selected pages.

A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` takes one pass
through the operator (in elementary torch operations, or with `own` through the framework),
`exact` computes the same outputs from the definitions in 64 bits, `work` counts the bytes and
operations a pass cannot do without.

The cache holds pages of P tokens, [n_pages][P][n_kv][d]; a slot is page * P + offset. The
sequences' pages are a random permutation, rows of the cache that hold no token are NaN. Every
buffer's size is its pool's, whatever the lengths.
"""
import math

import numpy as np
import torch

own = False

INV127 = np.float32(1.0) / np.float32(127.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a round of 8 sequences after verification: each keeps 1 to 7 tokens of its draft block
        {"name": "plan, round of 8", "op": "plan", "B": 8, "P": 32, "lo": 4096, "hi": 32768, "grow": 7,
         "admit": 0.0, "shrink": 0.0, "spare": 1.5, "tokens": 56},
        # a busy server's step: 1000 sequences, some admitted with their prompts, some ended
        # (all pages returned) and a pool that runs out before the last of them
        {"name": "plan, 1000 sequences", "op": "plan", "B": 1000, "P": 16, "lo": 1, "hi": 32768, "grow": 9,
         "admit": 0.1, "shrink": 0.1, "spare": 0.9, "tokens": 2000000},
        # the keys of one verification step of 64 sequences, 9 tokens each, with page summaries
        {"name": "append, verified step", "op": "append", "B": 64, "new": 9, "ctx": 2048, "P": 32, "n_kv": 1,
         "d": 512, "dtype": "bf16", "v": False, "sums": True},
        # two prompts of 32768 tokens into the full-attention cache, with page summaries
        {"name": "append, prompts", "op": "append", "B": 2, "new": 32768, "ctx": 0, "P": 64, "n_kv": 1, "d": 512,
         "dtype": "bf16", "v": False, "sums": True},
        # a sliding layer of a one-sequence draft: the smallest call
        {"name": "attention, one window", "op": "attention", "B": 1, "lo": 4096, "hi": 4096, "P": 16, "n_head": 4,
         "n_kv": 1, "d": 256, "window": 512, "dtype": "bf16", "v": False},
        # the full layer of a batch of ragged long contexts
        {"name": "attention, ragged long", "op": "attention", "B": 8, "lo": 4096, "hi": 32768, "P": 64, "n_head": 4,
         "n_kv": 1, "d": 512, "window": 0, "dtype": "bf16", "v": False},
        # grouped heads of dim 128 over two KV heads, an even batch
        {"name": "attention, 32 x 8192", "op": "attention", "B": 32, "lo": 8192, "hi": 8192, "P": 32, "n_head": 8,
         "n_kv": 2, "d": 128, "window": 0, "dtype": "bf16", "v": False},
        # a cache with its own V, groups of eight heads, many short ragged sequences, some empty
        {"name": "attention, short with V", "op": "attention", "B": 61, "lo": 0, "hi": 4095, "P": 16, "n_head": 16,
         "n_kv": 2, "d": 128, "window": 0, "dtype": "bf16", "v": True},
        # an fp32 model's cache with small heads
        {"name": "attention, fp32", "op": "attention", "B": 16, "lo": 100, "hi": 8000, "P": 16, "n_head": 4,
         "n_kv": 2, "d": 64, "window": 0, "dtype": "f32", "v": True},
        # one sequence that attends 64 pages of its 32768 keys
        {"name": "selected, one sequence", "op": "selected", "B": 1, "lo": 32768, "hi": 32768, "P": 32, "n_head": 4,
         "n_kv": 1, "d": 512, "n_select": 64},
        # the ragged long batch with 32 pages each
        {"name": "selected, ragged long", "op": "selected", "B": 8, "lo": 4096, "hi": 32768, "P": 64, "n_head": 4,
         "n_kv": 1, "d": 512, "n_select": 32},
        # very long contexts: 16 sequences of 131072 keys, 128 pages each
        {"name": "selected, 16 x 131072", "op": "selected", "B": 16, "lo": 131072, "hi": 131072, "P": 64, "n_head": 4,
         "n_kv": 1, "d": 512, "n_select": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "selected"])
    P = rng.choice([16, 32, 64, 128])
    if op == "plan":
        hi = _log(rng, 16, 32768)
        B, grow, admit = _log(rng, 1, 1000), rng.randint(1, 17), rng.choice([0.0, 0.1, 0.7])
        tokens = min(1900000, B * grow + int(rng.choice([0.5, 2.0]) * admit * B * hi))
        return {"op": op, "B": B, "P": P, "lo": rng.choice([1, hi // 2 + 1]), "hi": hi, "grow": grow, "admit": admit,
                "shrink": rng.choice([0.0, 0.3]), "spare": rng.choice([0.5, 1.5]), "tokens": tokens}
    d = rng.choice([64, 128, 256, 512])
    if op == "append":
        n_kv, total = rng.choice([1, 2, 4]), _log(rng, 1, 60000)
        B = max(1, min(total, _log(rng, 1, 200)))
        new = max(1, total * 128 // (n_kv * d) // B)
        return {"op": op, "B": B, "new": new, "ctx": _log(rng, 1, 4096) - 1, "P": P, "n_kv": n_kv, "d": d,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "v": rng.choice([False, True]),
                "sums": rng.choice([False, True])}
    if op == "selected":
        d = rng.choice([128, 256, 512])
        B, hi = _log(rng, 1, 32), _log(rng, 500, 131072)
        hi = max(1, min(hi, 2000000 // B))
        n_kv = rng.choice([1, 1, 2])
        return {"op": op, "B": B, "lo": rng.choice([hi, 1 + hi // 8]), "hi": hi, "P": P, "n_head": 4 * n_kv,
                "n_kv": n_kv, "d": d, "n_select": rng.randint(3, 128 * 64 // P)}
    n_kv, dtype = rng.choice([1, 2, 3]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    B = _log(rng, 1, 256)
    hi = _log(rng, 1, 32768)
    size = n_kv * d * (4 if dtype == "f32" else 2)
    hi = max(1, min(hi, 200000000 // (B * size)))
    return {"op": op, "B": B, "lo": rng.choice([0, hi // 2, hi]), "hi": hi, "P": P,
            "n_head": n_kv * rng.choice([1, 2, 4, 8]), "n_kv": n_kv, "d": d, "window": rng.choice([0, 0, 512, 1024]),
            "dtype": dtype, "v": rng.choice([False, True])}


# ---------------------------------------------------------------- inputs


def _lengths(rs, c):
    return rs.randint(c["lo"], c["hi"] + 1, c["B"]).astype(np.int64)


def _tables(rs, lengths, P, cols, n_pages):
    """Random pages for every sequence: block table [B][cols] (-1 behind each sequence's pages)
    and the pages left over."""
    need = -(-lengths // P)
    perm = rs.permutation(n_pages)
    table = np.full((len(lengths), cols), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, perm[at:].astype(np.int32)


def _normal(g, shape, dtype):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(generator=g)


def _unwritten(x, table, lengths, P):
    """NaN in every row of the cache that holds no token."""
    held = np.zeros((x.shape[0], P), bool)
    for b, n in enumerate(lengths):
        full, rest = divmod(int(n), P)
        held[table[b, :full]] = True
        if rest:
            held[table[b, full], :rest] = True
    x.view(x.shape[0], P, -1)[torch.from_numpy(~held).cuda()] = float("nan")


def _summaries(k, chunk=2048):
    """Codes and scales of the mean key of every page (any page of a cache, complete or not)."""
    n, P = k.shape[:2]
    codes = torch.empty((n,) + tuple(k.shape[2:]), dtype=torch.int8, device="cuda")
    scales = torch.empty((n, k.shape[2]), dtype=torch.float32, device="cuda")
    for i in range(0, n, chunk):
        codes[i:i + chunk], scales[i:i + chunk] = _quantised(k[i:i + chunk])
    return codes, scales


def prepare(case, seed):
    c = case
    rs = np.random.RandomState(seed % (1 << 32))
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    P = c["P"]
    s = dict(c)
    if c["op"] == "plan":
        B = c["B"]
        old = _lengths(rs, c)
        new = old + rs.randint(1, c["grow"] + 1, B)
        what = rs.uniform(size=B)
        admitted, ended = what < c["admit"], what > 1 - c["shrink"]
        new[ended] = rs.choice([0, 1], ended.sum()) * rs.randint(0, old[ended] + 1)
        new[admitted], old[admitted] = old[admitted], 0
        cols = -(-(c["hi"] + c["grow"]) // P)
        want = np.maximum(-(-new // P) - -(-old // P), 0)
        n_pages = 2 * B * cols
        table, left = _tables(rs, old, P, cols, n_pages)
        left = left[:max(1, int(c["spare"] * want.sum()))]
        ring = np.full(n_pages, -1, np.int32)
        head = rs.randint(n_pages)
        ring[(head + np.arange(len(left))) % n_pages] = left
        s.update(old=i32(old), new=i32(new), table=i32(table), ring=i32(ring), state=i32([head, len(left)]),
                 max_tokens=c["tokens"])
        return s
    dtype = TYPES[c.get("dtype", "bf16")]
    if c["op"] == "append":
        B, new, ctx = c["B"], c["new"], c["ctx"]
        old = rs.randint(0, ctx + 1, B)
        cols = -(-(ctx + new) // P)
        n_pages = B * cols + 1
        table, _ = _tables(rs, old + new, P, cols, n_pages)
        pos = old[:, None] + np.arange(new)[None]
        slots = table[np.arange(B)[:, None], pos // P].astype(np.int64) * P + pos % P
        shape = (n_pages, P, c["n_kv"], c["d"])
        s.update(k=_normal(g, shape, dtype), slots=i32(slots.reshape(-1)),
                 k_new=_normal(g, (B * new,) + shape[2:], dtype), vc=None, v_new=None, codes=None, scales=None)
        if c["v"]:
            s.update(vc=_normal(g, shape, dtype), v_new=_normal(g, (B * new,) + shape[2:], dtype))
        if c["sums"]:
            s["codes"], s["scales"] = _summaries(s["k"])
        return s
    lengths = _lengths(rs, c)
    cols = max(1, -(-c["hi"] // P))
    n_pages = c["B"] * cols + 1
    table, _ = _tables(rs, lengths, P, cols, n_pages)
    shape = (n_pages, P, c["n_kv"], c["d"])
    s.update(k=_normal(g, shape, dtype), table=i32(table), lens=i32(lengths),
             q=_normal(g, (c["B"], c["n_head"], c["d"]), torch.float32), vc=None, codes=None, scales=None)
    if c["op"] == "selected":
        # pages differ in what they hold: a direction of their own on top of each key
        s["k"] += _normal(g, (n_pages, 1) + shape[2:], dtype)
        s["codes"], s["scales"] = _summaries(s["k"])
    _unwritten(s["k"], table, lengths, P)
    if c.get("v"):
        s["vc"] = _normal(g, shape, dtype)
        _unwritten(s["vc"], table, lengths, P)
    return s


# ---------------------------------------------------------------- the plain forms


def _quantised(pages):
    """Mean key of each page, as int8 codes and one fp32 scale per KV head."""
    mean = pages.double().mean(1).float()
    scale = mean.abs().amax(-1) * torch.tensor(INV127, device=pages.device)
    code = torch.where(scale[..., None] > 0, torch.round(mean / scale[..., None]), 0.0)
    return code.to(torch.int8), scale


def _plain_plan(s):
    P, T, table, ring = s["P"], s["max_tokens"], s["table"], s["ring"]
    n_pages, (B, cols) = ring.numel(), table.shape
    old, new = s["old"].long(), s["new"].long()
    head, count = s["state"].long()
    n0, n1 = (old + P - 1) // P, (new + P - 1) // P
    fits = (new >= 0) & (new <= cols * P)
    grow, shrink = (new > old) & fits, (new < old) & fits
    need, tok = torch.where(grow, n1 - n0, 0), torch.where(grow, new - old, 0)
    cp, ct = need.cumsum(0), tok.cumsum(0)
    granted = grow & (cp <= count) & (ct <= T)
    free = torch.where(shrink, n0 - n1, 0)
    cf = free.cumsum(0)
    len_out = torch.where(granted | shrink, new, old)
    cu = torch.cat([cp.new_zeros(1), torch.where(granted, ct, 0).cummax(0).values])
    taken, freed, total = torch.where(granted, cp, 0).max(), cf[-1], cu[-1]
    col = torch.arange(cols, device=table.device)
    give = granted[:, None] & (col >= n0[:, None]) & (col < n1[:, None])
    at = (head + (cp - need)[:, None] + col - n0[:, None]) % n_pages
    take = shrink[:, None] & (col >= n1[:, None]) & (col < n0[:, None])
    to = torch.where(take, (head + count + (cf - free)[:, None] + col - n1[:, None]) % n_pages, n_pages)
    longer = torch.cat([ring, ring.new_zeros(1)])
    longer[to.reshape(-1)] = table.reshape(-1)
    table.copy_(torch.where(give, ring[at], table))
    ring.copy_(longer[:n_pages])
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    pos = (old[b] + t - cu[b]).clamp(0, cols * P - 1)
    slots = torch.where(t < total, table[b, pos // P].long() * P + pos % P, -1)
    state = torch.stack([(head + taken) % n_pages, count - taken + freed])
    denied = ((grow & ~granted) | ~fits).sum()
    status = torch.stack([total, taken, freed, denied])
    return [x.to(torch.int32) for x in (len_out, slots, cu, state, status)] + [table, ring]


def _plain_append(s):
    slots = s["slots"].long()
    P = s["P"]
    for cache, rows in ((s["k"], s["k_new"]), (s["vc"], s["v_new"])):
        if cache is not None:
            cache.view((-1,) + tuple(cache.shape[2:]))[slots] = rows
    out = [s["k"], s["vc"]]
    if s["codes"] is not None:
        done = slots[slots % P == P - 1] // P
        s["codes"][done], s["scales"][done] = _quantised(s["k"][done])
        out.append(s["codes"] * s["scales"][..., None])
    return out


def _plain_attend(s, pages, token):
    """Attention over the keys of the logical pages [B][n_kv][n] (-1: none); token: the keys'
    positions that may be attended, as a function of the position."""
    k, table, q = s["k"], s["table"].long(), s["q"]
    B, n_kv, n = pages.shape
    P, d = s["P"], q.shape[-1]
    pos = pages[..., None] * P + torch.arange(P, device=q.device)
    keep = ((pages[..., None] >= 0) & token(pos)).reshape(B, n_kv, 1, n * P)
    page = torch.gather(table, 1, pages.clamp(min=0).reshape(B, -1)).reshape(B, n_kv, n)
    page = page.clamp(min=0)
    heads = torch.arange(n_kv, device=q.device)[None, :, None]
    hold = keep.reshape(B, n_kv, n * P, 1)
    read = lambda x: x.transpose(1, 2)[page, heads].reshape(B, n_kv, n * P, d).float().masked_fill(~hold, 0)  # noqa: E731
    kk = read(k)
    vv = kk if s["vc"] is None else read(s["vc"])
    x = torch.matmul(q.reshape(B, n_kv, -1, d), kk.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = x.masked_fill(~keep, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, vv) / torch.where(total > 0, total, 1.0)
    return out.reshape(q.shape), (m + torch.log(total)).reshape(q.shape[:2])


def _plain_attention(s):
    L = s["lens"].long()[:, None, None, None]
    W, n_kv = s["window"], s["n_kv"]
    lo = (L - W).clamp(min=0) if W else torch.zeros_like(L)
    n = s["table"].shape[1] if not W else min(s["table"].shape[1], -(-W // s["P"]) + 1)
    pages = lo[..., 0] // s["P"] + torch.arange(n, device=L.device)
    pages = torch.where(pages * s["P"] < L[..., 0], pages, -1).expand(-1, n_kv, -1)
    return _plain_attend(s, pages, lambda pos: (pos >= lo) & (pos < L))


def _plain_selected(s):
    q, table, L, P, k = s["q"], s["table"].long(), s["lens"].long(), s["P"], s["n_select"]
    B, cols = table.shape
    d, n_kv = q.shape[-1], s["n_kv"]
    qs = q.abs().amax(-1) * torch.tensor(INV127, device=q.device)
    qc = torch.where(qs[..., None] > 0, torch.round(q / qs[..., None]), 0.0)
    page = table.clamp(min=0)
    codes = s["codes"][page].permute(0, 2, 1, 3).float()
    # whole numbers below 2^24: exact in fp32 in any order
    dots = torch.matmul(qc.reshape(B, n_kv, -1, d), codes.transpose(2, 3))
    score = dots * qs.reshape(B, n_kv, -1, 1) * s["scales"][page].permute(0, 2, 1)[:, :, None]
    score = score.amax(2)
    n = ((L + P - 1) // P)[:, None, None]
    col = torch.arange(cols, device=q.device)
    score = torch.where((col < 1) | (col >= n - 1), math.inf, score).masked_fill(col >= n, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    order = torch.where(order < n, order, cols).sort(-1).values
    sel = torch.full((B, n_kv, k), -1, dtype=torch.long, device=q.device)
    sel[..., :order.shape[-1]] = torch.where(order < cols, order, -1)
    out, lse = _plain_attend(s, sel, lambda pos: pos < L[:, None, None, None])
    return sel.to(torch.int32), out, lse


# ---------------------------------------------------------------- one pass


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention,
                "selected": _plain_selected}[op](s)
    import mtp_speculative_decoding_gemma4_gb300 as mtp
    if op == "plan":
        return mtp.page_plan(s["old"], s["new"], s["table"], s["ring"], s["state"], s["P"], s["max_tokens"]) + (
            s["table"], s["ring"])
    if "kv" not in s:  # the cache's descriptor, which a program keeps as long as the cache
        s["kv"] = mtp.PagedKV(s["k"], s.get("table"), s.get("lens"), v=s["vc"], codes=s["codes"], scales=s["scales"])
    kv = s["kv"]
    if op == "append":
        mtp.page_append(kv, s["k_new"], s["slots"], v_new=s["v_new"])
        return [s["k"], s["vc"]] + ([] if s["codes"] is None else [s["codes"] * s["scales"][..., None]])
    if op == "attention":
        return mtp.paged_attention(s["q"], kv, window=s["window"], want_lse=True)
    sel = mtp.page_select(s["q"], kv, s["n_select"], keep_first=1, keep_last=1)
    return (sel,) + mtp.paged_attention(s["q"], kv, pages=sel, want_lse=True)


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "plan":
        return None
    P = c["P"]
    if c["op"] == "append":
        if s["codes"] is None:
            return None
        slot_of = s["slots"].cpu().numpy()
        s["k"].view((-1,) + tuple(s["k"].shape[2:]))[s["slots"].long()] = s["k_new"]
        value = s["codes"].double() * s["scales"].double()[..., None]
        for done in np.array_split(slot_of[slot_of % P == P - 1] // P, 64):
            done = torch.from_numpy(done.astype(np.int64)).cuda()
            # the codes are defined by the means and steps as fp32 numbers
            mean = (s["k"][done].double().sum(1) / P).cpu().numpy().astype(np.float32)
            step = np.abs(mean).max(-1, keepdims=True) * INV127
            code = np.rint(mean / step).astype(np.float64)
            value[done] = torch.from_numpy(code * step.astype(np.float64)).cuda()
        return [None, None, value]
    B, H, d = s["q"].shape
    n_kv, G = c["n_kv"], H // c["n_kv"]
    out = torch.zeros((B, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].cpu().numpy()
    for b in range(B):
        L = int(lens[b])
        if not L:
            continue
        pages = s["table"][b, :-(-L // P)].long()
        for g in range(n_kv):
            q = s["q"][b, g * G:(g + 1) * G]
            lo = max(0, L - c["window"]) if c.get("window") else 0
            at = torch.arange(lo, L, device="cuda")
            if c["op"] == "selected":
                n = len(pages)
                step = (q.abs().max(-1).values.cpu().numpy() * INV127)[:, None]
                code = np.rint(q.cpu().numpy() / step).astype(np.float64)
                dots = (torch.from_numpy(code).cuda() @ s["codes"][pages, g].double().T).cpu().numpy()
                score = (dots.astype(np.float32) * step * s["scales"][pages, g].cpu().numpy()[None]).max(0)
                score[0] = score[n - 1] = np.inf
                best = np.sort(np.argsort(-score, kind="stable")[:c["n_select"]])
                at = (torch.from_numpy(best).cuda()[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)
                at = at[at < L]
            rows = s["k"][pages[at // P], at % P, g].double()
            x = (q.double() @ rows.T) / math.sqrt(d)
            if s["vc"] is not None:
                rows = s["vc"][pages[at // P], at % P, g].double()
            lse[b, g * G:(g + 1) * G] = torch.logsumexp(x, -1)
            out[b, g * G:(g + 1) * G] = torch.softmax(x, -1) @ rows
    return [None, out, lse] if c["op"] == "selected" else [out, lse]


def work(case):
    c, P = case, case["P"]
    size = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "plan":
        mean = (c["lo"] + c["hi"]) / 2
        stay = 1 - c["admit"] - c["shrink"]
        tokens = c["B"] * (stay * (c["grow"] + 1) / 2 + c["admit"] * mean)
        moved = c["B"] * (stay * (c["grow"] + 1) / 2 + c["admit"] * mean + c["shrink"] * mean * 0.75) / P
        return {"bytes": 4 * (4 * c["B"] + tokens + 2 * moved), "flops": tokens}
    if c["op"] == "append":
        rows, width = c["B"] * c["new"], c["n_kv"] * c["d"]
        n = rows * width * size * 2 * (2 if c["v"] else 1) + 4 * rows
        return {"bytes": n + (rows // P * width if c["sums"] else 0), "flops": rows * width if c["sums"] else 0}
    mean, q = (c["lo"] + c["hi"]) / 2, c["B"] * c["n_head"] * c["d"] * 4
    if c["op"] == "attention":
        if c["window"]:
            mean = min(mean, c["window"])
        keys = c["B"] * mean
        return {"bytes": keys * c["n_kv"] * c["d"] * size * (2 if c["v"] else 1) + 2 * q,
                "flops": 4 * keys * c["n_head"] * c["d"]}
    keys = c["B"] * min(mean, c["n_select"] * P)
    pages = c["B"] * mean / P
    return {"bytes": keys * c["n_kv"] * c["d"] * size + pages * c["n_kv"] * (c["d"] + 4) + 2 * q,
            "flops": 4 * keys * c["n_head"] * c["d"] + 2 * pages * c["n_head"] * c["d"]}
