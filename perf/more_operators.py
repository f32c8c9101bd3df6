"""Measured cases of the operators around a verification step: attention of a chunk of new tokens
over a paged cache, log probabilities of given tokens with entropy and top alternatives, forking
sequences over shared pages, and collecting (or compacting) the pages that sequences hold.

A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` takes one pass
through the operator (in elementary torch operations, or with `own` through the framework),
`exact` computes the same outputs from the definitions in 64 bits, `work` counts the bytes and
operations a pass cannot do without.

The cache holds pages of P tokens, [n_pages][P][n_kv][d]; the sequences' pages are a random
permutation. New tokens are the last ones of their sequences, packed sequence after sequence; how
many there are in all is the case's, how they fall to the sequences is the seed's. Every buffer's
size is its pool's, whatever the lengths.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence's draft block of 4 and the token before it, a sliding layer: the smallest call
        {"name": "chunk, one window", "op": "chunk", "B": 1, "new_lo": 5, "new": 5, "lo": 4096, "hi": 4096, "P": 16,
         "n_head": 4, "n_kv": 1, "d": 256, "window": 512, "dtype": "bf16", "v": False},
        # a verification step's full layer: 8 ragged long contexts, 7 tokens each (a draft block of 6)
        {"name": "chunk, verified long", "op": "chunk", "B": 8, "new_lo": 7, "new": 7, "lo": 4096, "hi": 32768, "P": 64,
         "n_head": 4, "n_kv": 1, "d": 512, "window": 0, "dtype": "bf16", "v": False},
        # two slices of 2048 prompt tokens against long contexts, full layer
        {"name": "chunk, prompt slices", "op": "chunk", "B": 2, "new_lo": 2048, "new": 2048, "lo": 16384, "hi": 32768,
         "P": 64, "n_head": 8, "n_kv": 1, "d": 512, "window": 0, "dtype": "bf16", "v": False},
        # the same slices and two more in a sliding layer
        {"name": "chunk, sliding slices", "op": "chunk", "B": 4, "new_lo": 1024, "new": 2048, "lo": 4096, "hi": 16384,
         "P": 32, "n_head": 8, "n_kv": 1, "d": 256, "window": 512, "dtype": "bf16", "v": False},
        # whole ragged prompts with a V of its own, grouped heads of dim 128
        {"name": "chunk, prompts with V", "op": "chunk", "B": 8, "new_lo": 1, "new": 4096, "lo": 0, "hi": 0, "P": 32,
         "n_head": 8, "n_kv": 2, "d": 128, "window": 0, "dtype": "bf16", "v": True},
        # an fp32 model: ragged draft blocks over short contexts
        {"name": "chunk, fp32", "op": "chunk", "B": 16, "new_lo": 1, "new": 17, "lo": 100, "hi": 4000, "P": 16,
         "n_head": 4, "n_kv": 2, "d": 64, "window": 0, "dtype": "f32", "v": True},
        # the target's rows of one sequence's verified draft block
        {"name": "scores, one draft block", "op": "scores", "rows": 5, "V": 262144, "dtype": "bf16", "top": 5,
         "temperature": 1.0, "skip": 0},
        # a verification step of 64 sequences, 9 rows each, with 20 alternatives
        {"name": "scores, 64 x 9 rows", "op": "scores", "rows": 576, "V": 262144, "dtype": "bf16", "top": 20,
         "temperature": 0.8, "skip": 0},
        # one prompt continued by 64 samples
        {"name": "fork, 64 samples", "op": "fork", "B": 65, "n": 64, "fan": 65, "lo": 8001, "hi": 8001, "P": 64,
         "n_kv": 1, "d": 512, "v": False, "spare": 80},
        # every second sequence replaced by a copy of another one (a beam search's step), a cache with V
        {"name": "fork, 256 beams", "op": "fork", "B": 512, "n": 256, "fan": 2, "lo": 1, "hi": 2048, "P": 16,
         "n_kv": 2, "d": 128, "v": True, "spare": 300},
        # a server's pool of two million tokens after a round that ended many of 1000 sequences
        {"name": "collect, 1000 sequences", "op": "collect", "B": 1000, "lo": 0, "hi": 3000, "P": 16, "n_kv": 1,
         "d": 64, "v": False, "pages": 131072, "shared": 0.3, "compact": False, "sums": False},
        # a pool half in use that is packed into its front, so that the rest can be given back
        {"name": "collect, compaction", "op": "collect", "B": 61, "lo": 0, "hi": 4095, "P": 32, "n_kv": 2, "d": 128,
         "v": True, "pages": 8192, "shared": 0.2, "compact": True, "sums": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "scores", "scores", "fork", "collect"])
    P = rng.choice([16, 32, 64, 128])
    if op == "scores":
        V = _log(rng, 50, 262144)
        rows = max(1, min(_log(rng, 1, 5000), 576 * 262144 // V // 2))
        return {"op": op, "rows": rows, "V": V, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "top": min(V, rng.choice([0, 1, 5, 20, 32])), "temperature": rng.choice([1.0, 0.7, 1.5]),
                "skip": rng.choice([0, 0, 3])}
    if op == "chunk":
        d, dtype, v = rng.choice([64, 128, 128, 256, 512]), rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.choice([False, True])
        n_kv = rng.choice([1, 2, 3])
        nh = n_kv * rng.choice([1, 2, 4, 5, 8])
        B, hi = _log(rng, 1, 100), _log(rng, 64, 32768)
        new = min(hi, _log(rng, 1, 2048))
        tc = dtype == "bf16" and d >= 128
        while 4 * B * new * nh * d * hi > (4e11 if tc else 2e10) or B * new * nh * hi > 5e8 or B * hi * n_kv * d > 2e8:
            B, new, hi = (B + 1) // 2 if B > 1 else 1, (new + 1) // 2, max(1, hi * 3 // 4)
        return {"op": op, "B": B, "new_lo": rng.choice([0, new // 2, new]), "new": new, "lo": rng.choice([0, hi // 2, hi]),
                "hi": hi, "P": P, "n_head": nh, "n_kv": n_kv, "d": d, "window": rng.choice([0, 0, 512, 1024]),
                "dtype": dtype, "v": v}
    n_kv, d, hi = rng.choice([1, 2]), rng.choice([64, 128, 256]), _log(rng, 20, 8192)
    if op == "fork":
        B = _log(rng, 2, 400)
        hi = max(1, min(hi, 100000000 // (B * n_kv * d)))
        fan = rng.choice([2, 2, 4, B])
        n = max(1, B - -(-B // fan))
        return {"op": op, "B": B, "n": n, "fan": fan, "lo": rng.choice([0, hi // 2, hi]), "hi": hi, "P": P, "n_kv": n_kv,
                "d": d, "v": rng.choice([False, True]), "spare": rng.choice([B, n // 2])}
    B = _log(rng, 1, 500)
    hi = max(1, min(hi, 100000000 // (B * n_kv * d)))
    return {"op": op, "B": B, "lo": rng.choice([0, hi // 2]), "hi": hi, "P": P, "n_kv": n_kv, "d": d,
            "v": rng.choice([False, True]), "pages": B * -(-hi // P) + _log(rng, 1, 2000),
            "shared": rng.choice([0.0, 0.3]), "compact": rng.choice([False, True]), "sums": rng.choice([False, True])}


# ---------------------------------------------------------------- inputs


def _normal(g, shape, dtype, by=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, by, generator=g)


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


def _tokens(c):
    """New tokens of a chunk case."""
    return max(1, c["B"] * (c["new_lo"] + c["new"]) // 2)


def _sum_to(rs, x, lo, hi, total):
    """x with entries moved within [lo, hi] until they add up to total."""
    for b in rs.permutation(len(x)):
        x[b] = np.clip(x[b] + total - x.sum(), lo, hi)
    return x


def prepare(case, seed):
    c = case
    rs = np.random.RandomState(seed % (1 << 32))
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()  # noqa: E731
    s = dict(c)
    if c["op"] == "scores":
        dtype = TYPES[c["dtype"]]
        rows, V = c["rows"], c["V"]
        # rows of a wider tensor where `skip` says so; logits as a language model's: a few large ones
        x = _normal(g, (rows, V + c["skip"]), dtype, 2.0)
        hot = torch.randint(0, V, (rows, 8), generator=g, device="cuda")
        x.scatter_(1, hot, _normal(g, (rows, 8), dtype, 4.0) + 8)
        token = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, hot[:, 0],
                            torch.randint(0, V, (rows,), generator=g, device="cuda"))
        s.update(logits=x[:, :V], token=token.to(torch.int32))
        return s
    P, B = c["P"], c["B"]
    row = (c["n_kv"], c["d"])
    if c["op"] == "chunk":
        dtype = TYPES[c["dtype"]]
        new = _sum_to(rs, rs.randint(c["new_lo"], c["new"] + 1, B), c["new_lo"], c["new"], _tokens(c))
        lengths = np.maximum(rs.randint(c["lo"], c["hi"] + 1, B), new)
        most = max(c["hi"], c["new"])
        cols = max(1, -(-most // P))
        table, _ = _tables(rs, lengths, P, cols, B * cols + 1)
        cu = np.concatenate([[0], np.cumsum(new)])
        shape = (B * cols + 1, P) + row
        # queries of twice the size of the keys: attention that prefers some of them
        s.update(k=_normal(g, shape, dtype), vc=_normal(g, shape, dtype) if c["v"] else None, table=i32(table),
                 lens=i32(lengths), cu=i32(cu), q=_normal(g, (_tokens(c), c["n_head"], c["d"]), dtype, 2.0),
                 codes=None, scales=None)
        return s
    dtype = torch.bfloat16
    lengths = rs.randint(c["lo"], c["hi"] + 1, B)
    cols = max(1, -(-c["hi"] // P))
    if c["op"] == "fork":
        # destinations hold nothing; every source is forked `fan` - 1 times
        dst = np.array([b for b in range(B) if b % c["fan"]][:c["n"]])
        src = dst // c["fan"] * c["fan"]
        lengths[dst] = 0
        cut = lengths[src] - rs.randint(0, np.minimum(lengths[src], 9) + 1)
        n_pages = (B - len(dst)) * cols + c["spare"] + 1
        table, left = _tables(rs, lengths, P, cols, n_pages)
        ring = np.full(n_pages, -1, np.int32)
        head = rs.randint(n_pages)
        ring[(head + np.arange(c["spare"])) % n_pages] = left[:c["spare"]]
        s.update(src=i32(src), dst=i32(dst), cut=i32(cut), ring=i32(ring), state=i32([head, c["spare"]]))
    else:
        n_pages = c["pages"]
        table, left = _tables(rs, lengths, P, cols, n_pages)
        # some sequences share the first pages of the one before them
        for b in np.nonzero(rs.uniform(size=B) < c["shared"])[0]:
            if b:
                n = min(lengths[b], lengths[b - 1]) // P // 2
                table[b, :n] = table[b - 1, :n]
        s.update(ring=i32(np.full(n_pages, -1)))
    shape = (n_pages, P) + row
    s.update(k=_normal(g, shape, dtype), vc=_normal(g, shape, dtype) if c["v"] else None, table=i32(table),
             lens=i32(lengths), codes=None, scales=None)
    if c.get("sums"):
        s.update(codes=torch.randint(-127, 128, (n_pages,) + row, dtype=torch.int8, generator=g, device="cuda"),
                 scales=torch.rand((n_pages, c["n_kv"]), generator=g, device="cuda"))
    return s


# ---------------------------------------------------------------- the plain forms


def _plain_chunk(s):
    k, table, q, P, W = s["k"], s["table"].long(), s["q"], s["P"], s["window"]
    (T, nh, d), (B, cols), n_kv, M = q.shape, table.shape, s["n_kv"], s["new"]
    G, dev = nh // n_kv, q.device
    cu, L = s["cu"].long(), s["lens"].long()
    new, first = cu[1:] - cu[:-1], L - (cu[1:] - cu[:-1])
    # the pages that the sequences' first tokens can reach back to, and all behind them
    n = cols if not W else min(cols, (W + M - 2) // P + 2)
    page0 = (first - W + 1).clamp(min=0) // P if W else torch.zeros_like(first)
    lp = page0[:, None] + torch.arange(n, device=dev)
    page = torch.gather(table, 1, lp.clamp(max=cols - 1)).clamp(min=0)
    key = (lp[:, :, None] * P + torch.arange(P, device=dev)).reshape(B, n * P)
    hold = (key < L[:, None])[:, None, :, None]
    read = lambda x: x[page].permute(0, 3, 1, 2, 4).reshape(B, n_kv, n * P, d).float().masked_fill(~hold, 0)  # noqa: E731
    kk = read(k)
    vv = kk if s["vc"] is None else read(s["vc"])
    at = torch.arange(M, device=dev)
    token = (cu[:-1, None] + at).clamp(max=T - 1)
    qq = q[token].reshape(B, M, n_kv, G, d).permute(0, 2, 1, 3, 4).reshape(B, n_kv, M * G, d).float()
    pos = first[:, None] + at
    keep = (key[:, None] <= pos[:, :, None]) & (key < L[:, None])[:, None]
    if W:
        keep = keep & (key[:, None] > pos[:, :, None] - W)
    keep = keep[:, None, :, None].expand(B, n_kv, M, G, n * P).reshape(B, n_kv, M * G, n * P)
    x = torch.matmul(qq, kk.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = x.masked_fill(~keep, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, vv) / torch.where(total > 0, total, 1.0)
    out = out.reshape(B, n_kv, M, G, d).permute(0, 2, 1, 3, 4).reshape(B * M, nh, d)
    lse = (m + torch.log(total)).reshape(B, n_kv, M, G).permute(0, 2, 1, 3).reshape(B * M, nh)
    # token t is number t - cu[b] of its sequence b
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    from_ = b * M + (t - cu[b]).clamp(max=M - 1)
    held = t < cu[-1]
    return (torch.where(held[:, None, None], out[from_], 0).to(q.dtype),
            torch.where(held[:, None], lse[from_], 0))


def _plain_scores(s):
    x = s["logits"].float() / s["temperature"]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    lse = m + torch.log(total)
    out = (torch.gather(x, 1, s["token"].long()[:, None]) - m - torch.log(total))[:, 0]
    entropy = (torch.log(total) - (e * (x - m)).sum(-1, keepdim=True) / total)[:, 0]
    if not s["top"]:
        return out, entropy
    ids = torch.sort(s["logits"], dim=-1, descending=True, stable=True).indices[:, :s["top"]]
    return out, entropy, ids.to(torch.int32), torch.gather(x, 1, ids) - lse


def _plain_fork(s):
    P, table, ring, k, lens = s["P"], s["table"], s["ring"], s["k"], s["lens"].long()
    (B, cols), n_pages, dev = table.shape, ring.numel(), table.device
    src, dst, cut = s["src"].long(), s["dst"].long(), s["cut"].long()
    head, count = s["state"].long()
    i = torch.arange(len(src), device=dev)
    ok = (src >= 0) & (src < B) & (dst >= 0) & (dst < B)
    a, z = src.clamp(0, B - 1), dst.clamp(0, B - 1)
    owner = torch.full((B,), len(src), device=dev).scatter_reduce_(0, z, torch.where(ok, i, len(src)), "amin")
    ok = ok & (owner[z] == i) & ((owner[a] == len(src)) | (a == z)) & (cut >= 0) & (cut <= lens[a])
    need = (ok & (cut % P > 0)).long()
    take = need.cumsum(0)
    ok = ok & (take <= count)
    taken = (need * ok).sum()
    fresh = ring[(head + take - need) % n_pages]
    whole = cut // P
    old = torch.gather(table[a], 1, whole.clamp(max=cols - 1)[:, None])[:, 0].long()
    # rows of the partial pages
    at = torch.arange(P, device=dev)
    copy = (ok & (need > 0) & (old >= 0) & (old < n_pages))[:, None] & (at < (cut % P)[:, None])
    f, r = copy.nonzero(as_tuple=True)
    for x in (k, s["vc"]):
        if x is not None:
            x[fresh[f].long(), r] = x[old[f], r]
    col = torch.arange(cols, device=dev)
    rows = torch.where(col < whole[:, None], table[a], torch.where((col == whole[:, None]) & (need > 0)[:, None],
                                                                   fresh[:, None], table[z]))
    longer = torch.cat([table, table.new_zeros(1, cols)])
    longer[torch.where(ok, z, B)] = rows
    table.copy_(longer[:B])
    out = torch.cat([s["lens"], s["lens"].new_zeros(1)])
    out[torch.where(ok, z, B)] = s["cut"]
    state = torch.stack([(head + taken) % n_pages, count - taken])
    status = torch.stack([ok.sum(), taken, (whole * ok).sum(), (~ok).sum()])
    return out[:B], state.to(torch.int32), status.to(torch.int32), table, k, s["vc"]


def _plain_collect(s):
    P, table, ring, lens = s["P"], s["table"].long(), s["ring"], s["lens"].long()
    (B, cols), n, dev = table.shape, ring.numel(), table.device
    held = torch.arange(cols, device=dev) < ((lens.clamp(0, cols * P) + P - 1) // P)[:, None]
    good = held & (table >= 0) & (table < n)
    mark = torch.zeros(n + 1, dtype=torch.bool, device=dev)
    mark[torch.where(good, table, n).reshape(-1)] = True
    mark = mark[:n]
    used = mark.sum()
    order = torch.sort(mark.to(torch.int8), stable=True).indices
    i = torch.arange(n, device=dev)
    status = [used, n - used, torch.zeros_like(used), (held & ~good).sum()]
    table_out = None
    if s["compact"]:
        high = (mark & (i >= used)).nonzero()[:, 0]
        low = order[:len(high)]
        for x in (s["k"], s["vc"], s["codes"], s["scales"]):
            if x is not None:
                x[low] = x[high]
        to = i.clone()
        to[high] = low
        status[2] = torch.full_like(used, len(high))
        table_out = torch.where(good, to[table.clamp(0, n - 1)], -1).to(torch.int32)
        order = (i + used) % n
    ring.copy_(torch.where(i < n - used, order, ring))
    state = torch.stack([torch.zeros_like(used), n - used])
    moved = (s["k"], s["vc"], s["codes"], s["scales"]) if s["compact"] else (None,) * 4
    return (table_out, state.to(torch.int32), torch.stack(status).to(torch.int32), ring) + moved


# ---------------------------------------------------------------- one pass


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"chunk": _plain_chunk, "scores": _plain_scores, "fork": _plain_fork, "collect": _plain_collect}[op](s)
    import mtp_speculative_decoding_gemma4_gb300 as mtp
    if op == "scores":
        got = mtp.token_logprobs(s["logits"], s["token"], temperature=s["temperature"], top_k=s["top"])
        return got if s["top"] else got[:2]
    if "kv" not in s:  # the cache's descriptor, which a program keeps as long as the cache
        s["kv"] = mtp.PagedKV(s["k"], s["table"], s["lens"], v=s["vc"], codes=s["codes"], scales=s["scales"])
    kv = s["kv"]
    if op == "chunk":
        return mtp.paged_attention_chunk(s["q"], kv, s["cu"], window=s["window"], want_lse=True)
    if op == "fork":
        return mtp.page_fork(kv, s["src"], s["dst"], s["cut"], s["ring"], s["state"]) + (s["table"], s["k"], s["vc"])
    got = mtp.page_collect(kv, s["ring"], compact=s["compact"])
    return got + (s["ring"],) + ((s["k"], s["vc"], s["codes"], s["scales"]) if s["compact"] else (None,) * 4)


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    c = case
    if c["op"] in ("fork", "collect"):
        return None
    s = prepare(c, seed)
    if c["op"] == "scores":
        n, k = c["rows"], c["top"]
        out = torch.zeros(n, dtype=torch.float64, device="cuda")
        entropy, best = torch.zeros_like(out), torch.zeros((n, k), dtype=torch.float64, device="cuda")
        for i in range(0, n, 64):
            lp = torch.log_softmax(s["logits"][i:i + 64].double() / c["temperature"], -1)
            out[i:i + 64] = torch.gather(lp, 1, s["token"][i:i + 64].long()[:, None])[:, 0]
            entropy[i:i + 64] = -(lp.exp() * lp).sum(-1)
            if k:
                best[i:i + 64] = torch.topk(lp, k).values
        return (out, entropy, None, best) if k else (out, entropy)
    T, H, d = s["q"].shape
    n_kv, G, P = c["n_kv"], H // c["n_kv"], c["P"]
    out = torch.zeros((T, H, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    for b in range(c["B"]):
        pages = s["table"][b].long()
        for t0 in range(cu[b], cu[b + 1], 256):
            t1 = min(cu[b + 1], t0 + 256)
            pos = torch.arange(t0, t1, device="cuda") - cu[b + 1] + lens[b]
            hi = lens[b] - cu[b + 1] + t1
            lo = max(0, hi - (t1 - t0) - c["window"] + 1) if c["window"] else 0
            at = torch.arange(lo, hi, device="cuda")
            off = at > pos[:, None]
            if c["window"]:
                off = off | (at <= pos[:, None] - c["window"])
            for h in range(n_kv):
                keys = s["k"][pages[at // P], at % P, h].double()
                vals = keys if s["vc"] is None else s["vc"][pages[at // P], at % P, h].double()
                for i in range(h * G, h * G + G):
                    x = (s["q"][t0:t1, i].double() @ keys.T / math.sqrt(d)).masked_fill(off, -math.inf)
                    lse[t0:t1, i] = torch.logsumexp(x, -1)
                    out[t0:t1, i] = torch.softmax(x, -1) @ vals
    return out, lse


def work(case):
    c = case
    if c["op"] == "scores":
        size = 4 if c["dtype"] == "f32" else 2
        n = c["rows"] * c["V"]
        return {"bytes": n * size + c["rows"] * (12 + 8 * c["top"]), "flops": 4 * n}
    P, row = c["P"], c["n_kv"] * c["d"] * (2 if c["v"] else 1)
    if c["op"] == "chunk":
        size = 4 if c["dtype"] == "f32" else 2
        new = _tokens(c) / c["B"]
        keys = max((c["lo"] + c["hi"]) / 2, new)
        mean = keys - new / 2  # keys of a token
        if c["window"]:
            mean, keys = min(mean, c["window"]), min(keys, c["window"] + new)
        rows = c["B"] * new * c["n_head"]
        return {"bytes": c["B"] * keys * row * size + rows * (2 * c["d"] * size + 4), "flops": 4 * rows * mean * c["d"]}
    mean = (c["lo"] + c["hi"]) / 2
    if c["op"] == "fork":
        tables = 2 * c["n"] * mean / P * 4
        return {"bytes": tables + c["n"] * (P / 2 * row * 2 * 2 + 24) + 8 * c["B"], "flops": c["n"]}
    used = c["B"] * mean / P
    bytes_ = 4 * used + 4 * (c["pages"] - used)
    if c["compact"]:
        moved = used * max(0.0, 1 - used / c["pages"])
        bytes_ += 4 * used + moved * (P * row * 2 + (c["n_kv"] * (c["d"] + 4) if c["sums"] else 0)) * 2
    return {"bytes": bytes_, "flops": used}
