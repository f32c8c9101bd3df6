"""Forks of sequences over shared pages and the collection (and compaction) of a cache's pages, against
plain NumPy forms; refusals without a device; a run of the paged operators together."""
import ctypes

import numpy as np
import pytest
import torch

from mtp_speculative_decoding_gemma4_gb300 import binding as B
from mtp_speculative_decoding_gemma4_gb300 import build as build_mod

gpu = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- plain forms


def plain_fork(lens, table, pages, src, dst, cut, ring, state):
    """Fork by fork. `pages`: arrays [n_pages][P]... of rows. Returns (len_out, state, status), table and
    pages changed in place."""
    n_seq, cols = table.shape
    n, P = len(ring), pages[0].shape[1]
    lens = np.clip(lens, 0, cols * P)
    head, count = int(state[0]) % n, min(max(int(state[1]), 0), n)
    fits = [0 <= s < n_seq and 0 <= d < n_seq for s, d in zip(src, dst)]
    first = {}
    for i, d in enumerate(dst):
        if fits[i]:
            first.setdefault(int(d), i)
    out, before, old = lens.copy(), table.copy(), [x.copy() for x in pages]
    granted = taken = shared = want = 0
    for i, (s, d, m) in enumerate(zip(src.tolist(), dst.tolist(), cut.tolist())):
        if not fits[i] or first[d] != i or (s != d and s in first) or not 0 <= m <= lens[s]:
            continue
        want += m % P > 0
        if want > count:
            continue
        whole = m // P
        table[d, :whole] = before[s, :whole]
        if m % P:
            fresh, was = ring[(head + taken) % n], before[s, whole]
            taken += 1
            table[d, whole] = fresh
            if 0 <= was < n and 0 <= fresh < n:
                for x, y in zip(pages, old):
                    x[fresh, :m % P] = y[was, :m % P]
        out[d] = m
        granted += 1
        shared += whole
    return out, np.array([(head + taken) % n, count - taken]), np.array([granted, taken, shared, len(src) - granted])


def plain_collect(lens, table, n, P, compact):
    """(table_out, the ring's entries, state, status, moves from -> to)."""
    need = -(-np.clip(lens, 0, table.shape[1] * P) // P)
    held = np.arange(table.shape[1]) < need[:, None]
    good = held & (table >= 0) & (table < n)
    pages = np.unique(table[good])
    used = len(pages)
    free = np.setdiff1d(np.arange(n), pages)
    to = np.arange(n)
    high = pages[pages >= used]
    if compact:
        to[high] = free[:len(high)]
        free = np.arange(used, n)
    table_out = np.where(good, to[np.clip(table, 0, n - 1)], -1)
    moves = {int(p): int(to[p]) for p in high} if compact else {}
    return table_out, free, [0, n - used], [used, n - used, len(moves), int((held & ~good).sum())], moves


# ---------------------------------------------------------------- refusals (no device)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


FAKE = 1 << 20


def _kv(**over):
    c = B.mtp_paged_kv()
    for f in ("k", "block_table", "ctx_len"):
        setattr(c, f, FAKE)
    for f, x in dict(stride_page=16 * 64, stride_t=64, stride_h=64, table_stride=8, n_pages=32, page_size=16,
                     max_pages=8, n_kv_head=1, head_dim=64, dtype=B.MTP_DTYPE_BF16).items():
        setattr(c, f, x)
    for f, x in over.items():
        setattr(c, f, x)
    return c


@pytest.mark.parametrize("args", [
    dict(B=0), dict(B=8193), dict(n=-1), dict(n=8193), dict(src=None), dict(dst=None), dict(length=None), dict(ring=None),
    dict(state=None), dict(len_out=None), dict(state_out=None), dict(status=None), dict(src=FAKE + 2), dict(len_out=FAKE),
    dict(len_out=3 * FAKE), dict(state_out=5 * FAKE), dict(kv=dict(block_table=None)), dict(kv=dict(ctx_len=None)),
    dict(kv=dict(k=None)), dict(kv=dict(table_stride=7))])
def test_bad_forks_are_refused_before_the_device(lib, args):
    a = dict(B=4, src=2 * FAKE, dst=3 * FAKE, length=4 * FAKE, n=3, ring=FAKE, state=5 * FAKE, len_out=6 * FAKE,
             state_out=7 * FAKE, status=8 * FAKE, kv={})
    a.update(args)
    assert lib.mtp_page_fork(_kv(**a["kv"]), a["B"], a["src"], a["dst"], a["length"], a["n"], a["ring"], a["state"],
                             a["len_out"], a["state_out"], a["status"], None) == B.MTP_ERR_INVALID_ARG
    assert B.mtp_last_error()


@pytest.mark.parametrize("args", [
    dict(B=0), dict(B=(1 << 20) + 1), dict(ring=None), dict(ring=FAKE + 2), dict(state=None), dict(status=None),
    dict(stride=7), dict(table=FAKE + 32), dict(table=FAKE, stride=9), dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=15),
    dict(kv=dict(block_table=None)), dict(kv=dict(n_pages=0))])
def test_bad_collections_are_refused_before_the_device(lib, args):
    a = dict(B=4, ring=2 * FAKE, table=3 * FAKE, stride=8, state=4 * FAKE, status=5 * FAKE, ws=6 * FAKE, ws_bytes=1 << 30, kv={})
    a.update(args)
    assert lib.mtp_page_collect(_kv(**a["kv"]), a["B"], a["ring"], a["table"], a["stride"], a["state"], a["status"],
                                a["ws"], a["ws_bytes"], None) == B.MTP_ERR_INVALID_ARG
    assert B.mtp_last_error()


def test_the_collection_s_workspace(lib):
    n = ctypes.c_int64()
    assert lib.mtp_page_collect_workspace(_kv(), 0, ctypes.byref(n)) == 0 and 0 < n.value < 64
    assert lib.mtp_page_collect_workspace(_kv(), 1, None) == B.MTP_ERR_INVALID_ARG


# ---------------------------------------------------------------- a cache


class Cache:
    def __init__(self, seed, lengths, P, n_kv, d, dtype="bf16", own_v=False, layout="token", spare=40, sums=False, share=0.0):
        self.rs = rs = np.random.RandomState(seed)
        self.L, self.P = np.asarray(lengths, np.int32), P
        self.cols = max(1, int(-(-self.L.max() // P)) + 1)
        held = -(-np.clip(self.L, 0, None) // P)
        self.n = n = int(held.sum()) + spare
        perm = rs.permutation(n)
        self.table = np.full((len(self.L), self.cols), -7, np.int32)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = perm[at:at + h]
            at += h
            if b and rs.uniform() < share:
                s = min(self.L[b], self.L[b - 1]) // P
                self.table[b, :s] = self.table[b - 1, :s]
        self.left = perm[at:].astype(np.int32)
        g = torch.Generator().manual_seed(seed)
        dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.rows = [torch.randn((n, P, n_kv, d), generator=g).to(dt) for _ in range(2 if own_v else 1)]
        lay = {"token": lambda x: x.cuda(), "head": lambda x: x.transpose(1, 2).contiguous().cuda().transpose(1, 2),
               "wide": lambda x: torch.cat([x, x], 3).cuda()[..., :d]}[layout]
        self.dev = [lay(x) for x in self.rows]
        self.codes = torch.randint(-127, 128, (n, n_kv, d), generator=g, dtype=torch.int8) if sums else None
        self.scales = torch.rand((n, n_kv), generator=g) if sums else None

    def kv(self):
        from mtp_speculative_decoding_gemma4_gb300 import PagedKV
        self.dtable = _dev(self.table)
        self.sums = (self.codes.cuda(), self.scales.cuda()) if self.codes is not None else (None, None)
        return PagedKV(self.dev[0], self.dtable, _dev(self.L), v=self.dev[1] if len(self.dev) > 1 else None,
                       codes=self.sums[0], scales=self.sums[1])

    def ring(self, count):
        ring = np.full(self.n, -9, np.int32)
        head = int(self.rs.randint(self.n))
        ring[(head + np.arange(count)) % self.n] = self.left[:count]
        return ring, np.array([head, count], np.int32)


def _equal(dev, want):
    assert torch.equal(dev.cpu(), torch.as_tensor(want).to(dev.dtype)), (dev.cpu(), want)


def _rows_np(c):
    return [x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32).numpy().copy() for x in c.rows]


def _rows_equal(c, pages):
    for dev, p in zip(c.dev, pages):
        got = dev.cpu().contiguous().view(torch.int16 if dev.dtype == torch.bfloat16 else torch.int32).numpy()
        np.testing.assert_array_equal(got, p)


def _fork(c, src, dst, cut, count, times=2):
    from mtp_speculative_decoding_gemma4_gb300 import page_fork
    src, dst, cut = (np.asarray(x, np.int32) for x in (src, dst, cut))
    ring, state = c.ring(count)
    kv, pages, table = c.kv(), _rows_np(c), c.table.copy()
    want = plain_fork(c.L, table, pages, src, dst, cut, ring, state)
    dr, ds = _dev(ring), _dev(state)
    for _ in range(times):  # (the inputs stay as they were: the call can be repeated)
        got = page_fork(kv, _dev(src), _dev(dst), _dev(cut), dr, ds)
        for g, w in zip(got, want):
            _equal(g, w)
        _equal(c.dtable, table)
        _rows_equal(c, pages)
    _equal(dr, ring)
    _equal(ds, state)
    return want


@gpu
@pytest.mark.parametrize("P", [1, 2, 8, 16, 64, 256])
@pytest.mark.parametrize("dtype,n_kv,d,own_v,layout", [
    ("bf16", 1, 64, False, "token"), ("bf16", 3, 40, True, "head"), ("f32", 2, 20, True, "wide"), ("bf16", 1, 512, False, "wide")])
def test_forks(P, dtype, n_kv, d, own_v, layout):
    c = Cache(P + d, [3 * P + P // 2, 0, 0, P, 0, 5 * P - 1, 0, 1], P, n_kv, d, dtype, own_v, layout)
    w = _fork(c, [0, 0, 3, 5, 7], [1, 2, 4, 6, 7], [3 * P + P // 2, 2 * P + 1, P, P - 1, 1], 20)
    assert w[2][0] == 5


@gpu
def test_a_prompt_forked_many_times_and_the_largest_call():
    c = Cache(1, [1000] + [0] * 299, 16, 1, 64, spare=400)
    assert _fork(c, [0] * 299, list(range(1, 300)), [1000] * 299, 400)[2][0] == 299
    c = Cache(2, [33, 20] + [0] * 8190, 16, 1, 8, spare=8200)
    src = np.arange(8190) % 2
    assert _fork(c, src, np.arange(2, 8192), np.where(src, 20, 33), 8190)[2][0] == 8190


@gpu
@pytest.mark.parametrize("count", [0, 1, 3, 7])
def test_forks_that_are_denied(count):
    c = Cache(3, [40, 50, 64, 0, 0, 0, 10, 0, 0], 16, 1, 64)
    #      ok  none left?  whole   dst twice  src is a dst  range of src, dst, length           self
    src = [0, 1, 2, 0, 4, 9, 0, -1, 0, 0, 6, 2]
    dst = [3, 4, 5, 3, 7, 8, 9, 8, -1, 8, 6, 8]
    cut = [40, 37, 64, 5, 3, 3, 3, 3, 3, 41, 7, 33]
    w = _fork(c, src, dst, cut, count)
    assert w[2][0] + w[2][3] == 12 and w[2][1] <= count
    # the dst of a denied fork still keeps others from being granted: fork 11 has fork 9's destination
    assert w[0][8] == 0


@gpu
def test_forks_of_bad_pages_and_odd_lengths():
    c = Cache(4, [40, 0, 0, 30], 16, 1, 64)
    c.table[0, 1], c.table[0, 2] = -1, 1 << 20  # copied as they are; no row is read from them
    c.L[3] = 1 << 30
    _fork(c, [0, 3], [1, 2], [40, 17], 5)


@gpu
def test_no_forks_and_streams():
    from mtp_speculative_decoding_gemma4_gb300 import page_fork
    c = Cache(5, [40, 17, 0], 16, 1, 64)
    w = _fork(c, [], [], [], 5)
    assert list(w[2]) == [0, 0, 0, 0]
    ring, state = c.ring(5)
    kv = c.kv()
    args = [_dev(np.array(x, np.int32)) for x in ([0], [2], [40])] + [_dev(ring), _dev(state)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = page_fork(kv, *args, stream=s.cuda_stream)
    s.synchronize()
    assert got[0].tolist() == [40, 17, 40]
    for bad in (args[0].long(), args[0][:0], args[0].cpu()):
        with pytest.raises(ValueError):
            page_fork(kv, args[0], bad, *args[2:])
    with pytest.raises(ValueError):
        page_fork(kv, *args[:3], args[3][:4], args[4])


# ---------------------------------------------------------------- collection


def _collect(c, compact, n_times=2):
    from mtp_speculative_decoding_gemma4_gb300 import page_collect
    kv = c.kv()
    ring = _dev(np.full(c.n, -3, np.int32))
    table, free, state, status, moves = plain_collect(c.L, c.table, c.n, c.P, compact)
    pages = _rows_np(c)
    for a, b in moves.items():
        for x in pages:
            x[b] = x[a]
    for _ in range(n_times):
        got = page_collect(kv, ring, compact=compact)
        if compact:
            _equal(got[0], table)
        else:
            assert got[0] is None
        _equal(got[1], state)
        _equal(got[2], status)
        _equal(ring, np.concatenate([free, np.full(c.n - len(free), -3)]))
        _rows_equal(c, pages)
        if c.codes is not None:
            codes, scales = c.codes.clone(), c.scales.clone()
            for a, b in moves.items():
                codes[b], scales[b] = codes[a], scales[a]
            assert torch.equal(c.sums[0].cpu(), codes) and torch.equal(c.sums[1].cpu(), scales)
        assert torch.equal(c.dtable.cpu(), torch.from_numpy(c.table))
    return status


@gpu
@pytest.mark.parametrize("compact", [False, True])
@pytest.mark.parametrize("dtype,n_kv,d,own_v,layout,sums", [
    ("bf16", 1, 64, False, "token", True), ("bf16", 3, 40, True, "head", True), ("f32", 2, 20, True, "wide", True),
    ("bf16", 1, 512, False, "wide", False)])
@pytest.mark.parametrize("spare", [0, 1, 31, 700])
def test_collections(compact, dtype, n_kv, d, own_v, layout, sums, spare):
    rs = np.random.RandomState(spare)
    c = Cache(spare + d, np.maximum(rs.randint(-5, 300, 23), 0), 16, n_kv, d, dtype, own_v, layout, spare, sums, share=0.4)
    moved = _collect(c, compact)[2]
    assert moved > 0 if compact and spare >= 31 else moved == 0 or compact


@gpu
@pytest.mark.parametrize("compact", [False, True])
@pytest.mark.parametrize("n_pages", [1, 31, 32, 33, 1024, 40000, 200000])
def test_pool_sizes(n_pages, compact):
    rs = np.random.RandomState(n_pages)
    c = Cache(n_pages, [0], 8, 1, 8, spare=n_pages)
    assert c.n == n_pages
    rows = max(1, min(40, n_pages // 3))
    c.cols = 700
    c.L = rs.randint(0, 700 * 8, rows).astype(np.int32)
    c.table = rs.randint(0, n_pages, (rows, 700)).astype(np.int32)  # (shared at random)
    _collect(c, compact)


@gpu
@pytest.mark.parametrize("compact", [False, True])
def test_full_empty_and_bad_tables(compact):
    c = Cache(1, [160] * 3, 16, 1, 64, spare=0)
    assert _collect(c, compact) == [30, 0, 0, 0]
    c = Cache(1, [0] * 3, 16, 1, 64, spare=50)
    assert _collect(c, compact) == [0, 50, 0, 0]
    c = Cache(2, [100, 37, 64], 16, 1, 64)
    c.table[0, 1], c.table[1, 2], c.table[2, 0] = -1, 1 << 20, c.n
    c.L = np.array([100, 1 << 30, -4], np.int32)  # clamped to the table's width and to 0
    assert _collect(c, compact)[3] >= 2


@gpu
def test_a_compaction_into_the_table_itself(lib):
    c = Cache(7, [100, 37, 64, 0, 250], 16, 1, 64, spare=60)
    kv = c.kv()
    table, free, state, status, moves = plain_collect(c.L, c.table, c.n, 16, True)
    ring, out = _dev(np.full(c.n, -3, np.int32)), torch.empty(6, dtype=torch.int32, device="cuda")
    n = B.mtp_page_collect_workspace(kv.p, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert lib.mtp_page_collect(kv.p, 5, ring.data_ptr(), c.dtable.data_ptr(), c.cols, out.data_ptr(), out.data_ptr() + 8,
                                ws.data_ptr(), n, None) == 0
    torch.cuda.synchronize()
    _equal(c.dtable, table)
    _equal(out, state + status)
    assert moves


@gpu
def test_pages_farther_apart_than_32_bits():
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_collect, page_fork
    n, P, d = 12, 16, 64
    step = (3 << 30) // n // 8 * 8
    k = torch.empty(step * n, dtype=torch.bfloat16, device="cuda").as_strided((n, P, 1, d), (step, d, d, 1))
    rows = torch.randn(n, P, 1, d).bfloat16()
    k.copy_(rows)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kv = PagedKV(k, i32([[11, 10], [0, 0]]), i32([20, 0]))
    ring, state = i32([9] + [0] * 11), i32([0, 1])
    page_fork(kv, i32([0]), i32([1]), i32([20]), ring, state)
    assert kv.block_table.tolist() == [[11, 10], [11, 9]] and torch.equal(k[9, :4].cpu(), rows[10, :4])
    kv.ctx_len.copy_(i32([20, 20]))
    table, state, status = page_collect(kv, ring, compact=True)
    assert table.tolist() == [[2, 1], [2, 0]] and status.tolist() == [3, 9, 3, 0]
    assert torch.equal(k[2].cpu(), rows[11]) and torch.equal(k[1].cpu(), rows[10]) and torch.equal(k[0, :4].cpu(), rows[10, :4])


# ---------------------------------------------------------------- together


@gpu
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f32")])
def test_samples_of_a_prompt_from_plan_to_compaction(d, dtype):
    """A prompt is planned, appended and attended in slices, forked into samples, each sample appends and
    attends tokens of its own, some end, the pages are collected and compacted, and attention over the
    compacted cache is what it was; also as one captured graph."""
    from mtp_speculative_decoding_gemma4_gb300 import (PagedKV, page_append, page_collect, page_fork, page_plan,
                                                       paged_attention, paged_attention_chunk)
    P, cols, n_pages, nh, S = 16, 12, 200, 4, 5
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(d)
    rows = lambda n, h: torch.randn((n, h, d), generator=g).to(dt).cuda()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.zeros((n_pages, P, 1, d), dtype=dt, device="cuda")
    table, ring = torch.full((S, cols), -1, dtype=torch.int32, device="cuda"), i32(list(range(n_pages)))
    state, lens = i32([0, n_pages]), i32([0] * S)
    kv = PagedKV(k, table, lens)
    prompt, q, keys = rows(70, 1), rows(70, nh), []

    def plan_and_append(new, data):
        len_out, slots, cu, state_out, status = page_plan(lens, i32(new), table, ring, state, P, data.shape[0])
        page_append(kv, data, slots)
        lens.copy_(len_out), state.copy_(state_out)
        return cu

    # the prompt in two slices; together they are what one slice gives
    parts = []
    for a, b in ((0, 33), (33, 70)):
        cu = plan_and_append([b] + [0] * (S - 1), prompt[a:b])
        parts.append(paged_attention_chunk(q[a:b].contiguous(), kv, cu))
    whole = paged_attention_chunk(q, kv, i32([0] + [70] * S))
    tol = 2 * torch.finfo(dt).eps if dt == torch.bfloat16 else 4e-5
    assert float((torch.cat(parts).float() - whole.float()).abs().max()) <= tol * 4
    # four samples of it: 4 whole pages shared, 6 rows copied each
    len_out, state_out, status = page_fork(kv, i32([0] * 4), i32([1, 2, 3, 4]), i32([70] * 4), ring, state)
    lens.copy_(len_out), state.copy_(state_out)
    assert status.tolist() == [4, 4, 16, 0] and lens.tolist() == [70] * 5
    own = rows(5 * 7, 1)
    cu = plan_and_append([77] * 5, own)
    qs = rows(5 * 7, nh)
    got = paged_attention_chunk(qs, kv, cu)
    for s in range(S):
        all_keys = torch.cat([prompt, own[7 * s:7 * s + 7]])[:, 0].double()
        x = qs[7 * s:7 * s + 7].double() @ all_keys.T / d ** 0.5
        x = x.masked_fill(torch.arange(77, device="cuda") > torch.arange(70, 77, device="cuda")[:, None, None], float("-inf"))
        p = torch.softmax(x, -1)
        want, most = p @ all_keys, p @ all_keys.abs()
        u = torch.finfo(torch.bfloat16).eps / 2 if dt == torch.bfloat16 else 0
        assert ((got[7 * s:7 * s + 7].double() - want).abs() <= u * (want.abs() + most * (1 + u)) + 2e-5).all()
    # samples 1 and 3 end; what no one holds is free again, then the rest is packed
    lens.copy_(i32([77, 0, 77, 0, 77]))
    one = rows(5, nh).float()
    before = paged_attention(one, kv)
    _, state_out, status = page_collect(kv, ring)
    held = 4 + 3 * 1  # the shared pages, and each one's own
    assert status.tolist()[:2] == [held, n_pages - held]
    state.copy_(state_out)
    table_out, state_out, status = page_collect(kv, ring, compact=True)
    table.copy_(table_out), state.copy_(state_out)
    assert int(table_out.max()) == held - 1 and state_out.tolist() == [0, n_pages - held]
    assert torch.equal(paged_attention(one, kv), before)
    # and on from there: a round that forks a survivor onto a free sequence, planned, appended and attended
    # in one graph
    data, qg = rows(4 * 3, 1), rows(4 * 3, nh)
    src, dst, cut, new, cu_all = i32([2]), i32([1]), i32([75]), i32([80, 78, 80, 0, 80]), None
    saved = [x.clone() for x in (k, table, lens, state, ring)]

    def round_():
        len_out, state_out, _ = page_fork(kv, src, dst, cut, ring, state)
        lens.copy_(len_out), state.copy_(state_out)
        len_out, slots, cu, state_out, _ = page_plan(lens, new, table, ring, state, P, 12)
        page_append(kv, data, slots)
        lens.copy_(len_out), state.copy_(state_out)
        return paged_attention_chunk(qg, kv, cu, want_lse=True)

    want = [x.clone() for x in round_()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = round_()
    for _ in range(2):
        for x, y in zip((k, table, lens, state, ring), saved):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
