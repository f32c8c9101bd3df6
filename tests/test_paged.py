"""Paged-cache operators: the page plan, the append with page summaries, the selection of pages
and the attention of one new token, against the NumPy forms; refusals without a device."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from mtp_speculative_decoding_gemma4_gb300 import binding as B
from mtp_speculative_decoding_gemma4_gb300 import build as build_mod
from oracle import paged as OP

gpu = pytest.mark.gpu

# Attention in fp32 against fp64, N(0, 1) queries and keys, scale 1 / sqrt(d). A key enters
# exactly; each of the d additions of a score rounds a partial sum of size <= sqrt(d) by at most
# 2^-24 relative (2^-23 where the adder truncates), so the score's error is about
# 2^-23 sqrt(d) sqrt(d / 2) scale = 2^-23 sqrt(d / 2) = 1.9e-6 at d = 512, added as independent
# errors. Every probability is off by its score's error, relative, and an output, a mean of values
# of size 1, by no more; a maximum over 10^4..10^6 outputs is some 5 such errors (1e-5), the sums
# over the keys add less. lse moves with the scores. 2e-5 is twice that.
ATT_TOL = 2e-5


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- refusals (no device)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


FAKE = 4096  # an aligned address that is never used: validation fails first


def _kv(**over):
    c = B.mtp_paged_kv()
    for f in ("k", "block_table", "ctx_len", "codes", "scales"):
        setattr(c, f, FAKE)
    for f, x in dict(stride_page=16 * 64, stride_t=64, stride_h=64, table_stride=8, n_pages=32, page_size=16,
                     max_pages=8, n_kv_head=1, head_dim=64, dtype=B.MTP_DTYPE_BF16, **{}).items():
        setattr(c, f, x)
    for f, x in over.items():
        setattr(c, f, x)
    return c


BAD_KV = [
    (dict(k=None), B.MTP_ERR_INVALID_ARG), (dict(k=FAKE + 8), B.MTP_ERR_INVALID_ARG),
    (dict(v=FAKE + 2), B.MTP_ERR_INVALID_ARG), (dict(dtype=2), B.MTP_ERR_INVALID_ARG),
    (dict(page_size=24), B.MTP_ERR_UNSUPPORTED_SHAPE), (dict(page_size=512), B.MTP_ERR_UNSUPPORTED_SHAPE),
    (dict(page_size=0), B.MTP_ERR_UNSUPPORTED_SHAPE), (dict(page_size=-16), B.MTP_ERR_UNSUPPORTED_SHAPE),
    (dict(head_dim=60), B.MTP_ERR_UNSUPPORTED_SHAPE), (dict(head_dim=520), B.MTP_ERR_UNSUPPORTED_SHAPE),
    (dict(n_kv_head=0), B.MTP_ERR_UNSUPPORTED_SHAPE), (dict(n_pages=0), B.MTP_ERR_INVALID_ARG),
    (dict(n_pages=1 << 27), B.MTP_ERR_INVALID_ARG), (dict(stride_t=60), B.MTP_ERR_INVALID_ARG),
    (dict(stride_t=68), B.MTP_ERR_INVALID_ARG), (dict(stride_page=-1024), B.MTP_ERR_INVALID_ARG),
    (dict(scales=None), B.MTP_ERR_INVALID_ARG), (dict(codes=FAKE + 4), B.MTP_ERR_INVALID_ARG),
]
BAD_TABLE = [(dict(block_table=None), B.MTP_ERR_INVALID_ARG), (dict(ctx_len=None), B.MTP_ERR_INVALID_ARG),
             (dict(max_pages=0), B.MTP_ERR_INVALID_ARG), (dict(table_stride=7), B.MTP_ERR_INVALID_ARG),
             (dict(max_pages=1 << 27, table_stride=1 << 27), B.MTP_ERR_INVALID_ARG)]


@pytest.mark.parametrize("over,code", BAD_KV + BAD_TABLE)
def test_bad_caches_are_refused_before_the_device(lib, over, code):
    kv, n = _kv(**over), ctypes.c_int64()
    assert lib.mtp_paged_attention_workspace(kv, 1, 4, 0, ctypes.byref(n)) == code, B.mtp_last_error()
    assert B.mtp_last_error()
    assert lib.mtp_paged_attention(kv, FAKE, 1, 4, 0, 0.0, None, 0, 2 * FAKE, None, FAKE, 1 << 30, None) == code
    assert lib.mtp_page_select(kv, FAKE, 1, 4, 4, 1, 1, FAKE, FAKE, 1 << 30, None) == code
    if (over, code) in BAD_KV:
        assert lib.mtp_page_append(kv, FAKE, None, 64, 64, FAKE, 1, None) == code


@pytest.mark.parametrize("args", [
    dict(q=None), dict(q=FAKE + 4), dict(out=None), dict(out=FAKE + 8), dict(B=0), dict(nh=0), dict(nh=3, n_kv=2),
    dict(window=-1), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(pages=FAKE, n_list=0),
    dict(n_list=4), dict(pages=FAKE, n_list=-1), dict(ws_bytes=0), dict(ws=FAKE + 8), dict(ws=None)])
def test_bad_attention_arguments_are_refused_before_the_device(lib, args):
    a = dict(q=FAKE, B=1, nh=4, window=0, scale=0.0, pages=None, n_list=0, out=2 * FAKE, lse=None, ws=FAKE,
             ws_bytes=1 << 40, n_kv=1)
    a.update(args)
    # long contexts, so that a workspace is needed
    kv = _kv(max_pages=4096, table_stride=4096, n_kv_head=a["n_kv"], stride_t=64 * a["n_kv"])
    rc = lib.mtp_paged_attention(kv, a["q"], a["B"], a["nh"], a["window"], a["scale"], a["pages"], a["n_list"],
                                 a["out"], a["lse"], a["ws"], a["ws_bytes"], None)
    assert rc == B.MTP_ERR_INVALID_ARG
    assert B.mtp_last_error()


@pytest.mark.parametrize("args,code", [
    (dict(codes=None, scales=None), B.MTP_ERR_INVALID_ARG), (dict(q=None), B.MTP_ERR_INVALID_ARG),
    (dict(sel=None), B.MTP_ERR_INVALID_ARG), (dict(k=1), B.MTP_ERR_INVALID_ARG), (dict(first=-1), B.MTP_ERR_INVALID_ARG),
    (dict(last=0), B.MTP_ERR_INVALID_ARG), (dict(first=3, last=2), B.MTP_ERR_INVALID_ARG),
    (dict(nh=33), B.MTP_ERR_UNSUPPORTED_SHAPE), (dict(ws_bytes=31), B.MTP_ERR_INVALID_ARG)])
def test_bad_selections_are_refused_before_the_device(lib, args, code):
    a = dict(q=FAKE, nh=4, k=4, first=1, last=1, sel=FAKE, ws_bytes=1 << 30)
    over = {f: a_ for f, a_ in args.items() if f in ("codes", "scales")}
    a.update({f: x for f, x in args.items() if f not in over})
    if a["k"] == 1:
        a["first"] = 1  # keep_first + keep_last > n_select
    assert lib.mtp_page_select(_kv(**over), a["q"], 1, a["nh"], a["k"], a["first"], a["last"], a["sel"], FAKE,
                               a["ws_bytes"], None) == code
    assert B.mtp_last_error()


@pytest.mark.parametrize("args", [dict(k_new=None), dict(slots=None), dict(T=-1), dict(row=56), dict(row=68),
                                  dict(v=FAKE, v_new=None), dict(v_new=2 * FAKE), dict(k_new=FAKE + 2)])
def test_bad_appends_are_refused_before_the_device(lib, args):
    a = dict(k_new=FAKE, v_new=None, row=64, slots=FAKE, T=3, v=None)
    a.update(args)
    assert lib.mtp_page_append(_kv(v=a["v"] and 2 * a["v"]), a["k_new"], a["v_new"], a["row"], a["row"], a["slots"],
                               a["T"], None) == B.MTP_ERR_INVALID_ARG
    assert B.mtp_last_error()


@pytest.mark.parametrize("args,code", [
    (dict(P=12), B.MTP_ERR_UNSUPPORTED_SHAPE), (dict(P=0), B.MTP_ERR_UNSUPPORTED_SHAPE),
    (dict(B=0), B.MTP_ERR_INVALID_ARG), (dict(B=8193), B.MTP_ERR_INVALID_ARG), (dict(cols=0), B.MTP_ERR_INVALID_ARG),
    (dict(stride=3), B.MTP_ERR_INVALID_ARG), (dict(n_pages=0), B.MTP_ERR_INVALID_ARG),
    (dict(T=-1), B.MTP_ERR_INVALID_ARG), (dict(slots=None), B.MTP_ERR_INVALID_ARG),
    (dict(slots=FAKE + 4), B.MTP_ERR_INVALID_ARG), (dict(len_out=FAKE), B.MTP_ERR_INVALID_ARG),
    (dict(state_out=FAKE), B.MTP_ERR_INVALID_ARG), (dict(cols=1 << 27, stride=1 << 27), B.MTP_ERR_INVALID_ARG),
    (dict(old=None), B.MTP_ERR_INVALID_ARG), (dict(status=None), B.MTP_ERR_INVALID_ARG)])
def test_bad_plans_are_refused_before_the_device(lib, args, code):
    a = dict(old=FAKE, B=2, cols=4, stride=4, n_pages=8, P=16, T=8, len_out=2 * FAKE, slots=FAKE, state_out=2 * FAKE,
             status=FAKE)
    a.update(args)
    assert lib.mtp_page_plan(a["old"], FAKE, a["B"], FAKE, a["stride"], a["cols"], FAKE, a["n_pages"], FAKE, a["P"],
                             a["T"], a["len_out"], a["slots"], FAKE, a["state_out"], a["status"], None) == code
    assert B.mtp_last_error()


def test_workspaces_need_no_device(lib):
    n = ctypes.c_int64(-1)
    assert lib.mtp_page_select_workspace(_kv(), 3, ctypes.byref(n)) == 0 and n.value == 4 * 3 * 8
    assert lib.mtp_paged_attention_workspace(_kv(), 3, 4, 0, ctypes.byref(n)) == 0 and n.value >= 0
    assert lib.mtp_paged_attention_workspace(_kv(), 3, 4, 0, None) == B.MTP_ERR_INVALID_ARG


# ---------------------------------------------------------------- the plan


def _plan_case(seed, Bn, P, cols, spare, kind):
    rs = np.random.RandomState(seed)
    old = rs.randint(0, cols * P + 1, Bn)
    new = rs.randint(0, cols * P + 1, Bn)
    if kind == "grow":
        new = np.minimum(old + rs.randint(0, 10, Bn), cols * P)
    elif kind == "fresh":
        old[:] = 0
    elif kind == "end":
        new[:] = 0
    elif kind == "odd":
        new[rs.randint(0, Bn, 3)] = [-1, cols * P + 1, 2 ** 31 - 1]
        old[0] = -5
    held = -(-np.maximum(old, 0) // P)
    n_pages = int(held.sum()) + spare
    perm = rs.permutation(n_pages).astype(np.int32)
    table = np.full((Bn, cols + 3), -7, np.int32)  # three columns that are not the table's
    at = 0
    for b in range(Bn):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    ring = np.full(n_pages, -9, np.int32)
    head = rs.randint(n_pages)
    ring[(head + np.arange(spare)) % n_pages] = perm[at:]
    return old.astype(np.int32), new.astype(np.int32), table, ring, np.array([head, spare], np.int32)


@gpu
@pytest.mark.parametrize("kind", ["any", "grow", "fresh", "end", "odd"])
@pytest.mark.parametrize("Bn,P,cols,spare,tokens", [(1, 1, 1, 1, 1), (1, 16, 7, 9, 200), (5, 16, 9, 11, 301),
                                                     (33, 32, 4, 200, 3000), (700, 8, 5, 900, 9001),
                                                     (1025, 64, 3, 1, 50), (8192, 4, 3, 9000, 40000)])
def test_plan_matches_the_plain_form(kind, Bn, P, cols, spare, tokens):
    from mtp_speculative_decoding_gemma4_gb300 import page_plan
    old, new, table, ring, state = _plan_case(17 * Bn + P, Bn, P, cols, spare, kind)
    want = OP.page_plan(old, new, table[:, :cols], ring, state, P, tokens)
    d_table, d_ring = _dev(table), _dev(ring)
    for _ in range(2):  # the inputs stay, so a second call gives the same again
        got = page_plan(_dev(old), _dev(new), d_table[:, :cols], d_ring, _dev(state), P, tokens)
        for name, g, w in zip(("len", "slots", "cu", "state", "status"), got, want):
            np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
        t = d_table.cpu().numpy()
        np.testing.assert_array_equal(t[:, :cols], want[5])
        assert (t[:, cols:] == -7).all()  # columns behind the table's stay as they were
        np.testing.assert_array_equal(d_ring.cpu().numpy(), want[6])


@gpu
def test_plan_without_slots_counts_and_denies():
    from mtp_speculative_decoding_gemma4_gb300 import page_plan
    old, new, table, ring, state = _plan_case(3, 6, 16, 5, 9, "any")
    got = page_plan(_dev(old), _dev(new), _dev(table[:, :5]), _dev(ring), _dev(state), 16, 0)
    want = OP.page_plan(old, new, table[:, :5], ring, state, 16, 0)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)


# ---------------------------------------------------------------- cache cases


class Case:
    """A paged cache with random pages: NaN wherever no token lives."""

    def __init__(self, seed, lengths, P, n_head, n_kv, d, dtype, cols=None, own_v=False, layout="token", spare=3):
        rs = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        self.L = np.asarray(lengths, np.int32)
        Bn = len(self.L)
        self.P, self.n_kv, self.d, self.n_head = P, n_kv, d, n_head
        self.cols = cols or max(1, int(-(-self.L.max() // P)))
        held = -(-np.clip(self.L, 0, self.cols * P) // P)
        n_pages = int(held.sum()) + spare
        perm = rs.permutation(n_pages)
        self.table = np.full((Bn, self.cols), -1, np.int32)
        at = 0
        for b in range(Bn):
            self.table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        keep = np.zeros((n_pages, P), bool)
        for b in range(Bn):
            for t in range(min(max(int(self.L[b]), 0), self.cols * P)):
                keep[self.table[b, t // P], t % P] = True
        dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]

        def cache():
            x = torch.randn((n_pages, P, n_kv, d), generator=g).to(dt)
            x[torch.from_numpy(~keep)] = float("nan")
            return x

        self.k = cache()
        self.v = cache() if own_v else None
        self.q = torch.randn((Bn, n_head, d), generator=g)
        dev = (lambda x: x.transpose(1, 2).contiguous().cuda().transpose(1, 2)) if layout == "head" else (
            lambda x: x.cuda())
        if layout == "both":  # K and V of a page side by side in one allocation
            kv = torch.stack([self.k, self.v], 1).cuda()
            self.dk, self.dv = kv[:, 0], kv[:, 1]
        else:
            self.dk, self.dv = dev(self.k), None if self.v is None else dev(self.v)

    def kv(self, **more):
        from mtp_speculative_decoding_gemma4_gb300 import PagedKV
        return PagedKV(self.dk, _dev(self.table), _dev(self.L), v=self.dv, **more)

    def want(self, scale=0.0, window=0, pages=None):
        k = self.k.double().numpy()
        v = k if self.v is None else self.v.double().numpy()
        s = scale or 1 / np.sqrt(self.d)
        r = [OP.paged_attention(self.q[b].numpy(), k, v, self.table[b], self.L[b], s, window,
                                None if pages is None else pages[b]) for b in range(len(self.L))]
        return np.stack([x[0] for x in r]), np.stack([x[1] for x in r])


def _close(got, want, tol=ATT_TOL):
    out, lse = (x.cpu().numpy() for x in got)
    assert np.isfinite(out).all()
    assert np.max(np.abs(out - want[0]), initial=0) <= tol
    empty = np.isneginf(want[1])
    assert (np.isneginf(lse) == empty).all() and (out[empty] == 0).all()
    assert np.max(np.abs(lse[~empty] - want[1][~empty]), initial=0) <= tol


SHAPES = [  # n_head, n_kv, d, dtype
    (4, 1, 256, "bf16"), (4, 1, 512, "bf16"), (8, 2, 128, "bf16"), (16, 2, 128, "bf16"), (3, 3, 128, "bf16"),
    (5, 1, 256, "bf16"), (20, 2, 128, "bf16"), (7, 1, 512, "bf16"), (2, 1, 384, "bf16"), (2, 1, 32, "f32"),
    (4, 2, 64, "f32"), (6, 2, 64, "bf16"), (9, 1, 80, "bf16"), (4, 1, 512, "f32"), (12, 4, 200, "f32"), (1, 1, 8, "bf16")]


@gpu
@pytest.mark.parametrize("own_v", [False, True])
@pytest.mark.parametrize("n_head,n_kv,d,dtype", SHAPES)
def test_attention_matches_the_plain_form(n_head, n_kv, d, dtype, own_v):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(n_head + d, [1, 0, 16, 17, 127, 128, 129, 300, 1000], 16, n_head, n_kv, d, dtype, own_v=own_v)
    _close(paged_attention(c.q.cuda(), c.kv(), want_lse=True), c.want())


@gpu
@pytest.mark.parametrize("window", [1, 15, 16, 100, 128, 513])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_window_edges(d, window):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(d + window, [1, 0, 15, 16, 100, 128, 129, 511, 512, 513, 900], 32, 4, 1, d, "bf16", own_v=d == 128)
    _close(paged_attention(c.q.cuda(), c.kv(), window=window, want_lse=True), c.want(window=window))


@gpu
@pytest.mark.parametrize("P", [1, 2, 4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,n_head", [(64, 2), (128, 4), (256, 8), (512, 4)])
def test_page_sizes(P, d, n_head):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(P + d, [700, 3, 257], P, n_head, 1, d, "bf16")
    _close(paged_attention(c.q.cuda(), c.kv(), want_lse=True), c.want())


@gpu
@pytest.mark.parametrize("layout", ["token", "head", "both"])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_layouts(layout, dtype, d):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(5, [70, 3, 257], 32, 6, 3, d, dtype, own_v=True, layout=layout)
    _close(paged_attention(c.q.cuda(), c.kv(), want_lse=True), c.want())


@gpu
@pytest.mark.parametrize("d", [128, 512, 64])
def test_long_and_ragged(d):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(d, [20001, 1, 0, 4096, 12345, 37], 64, 4, 1, d, "bf16")
    _close(paged_attention(c.q.cuda(), c.kv(), want_lse=True), c.want())


@gpu
@pytest.mark.parametrize("Bn", [1, 2, 151, 700])
def test_batches(Bn):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    L = np.random.RandomState(Bn).randint(0, 400, Bn)
    c = Case(Bn, np.maximum(L, L == L.max()), 16, 4, 1, 128, "bf16", cols=40)
    _close(paged_attention(c.q.cuda(), c.kv(), want_lse=True), c.want())


@gpu
def test_large_scores_do_not_overflow():
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    for d in (64, 256):
        c = Case(9, [500, 40], 16, 4, 1, d, "bf16")
        c.q *= 300
        # scores reach 1e3, so the error of one (2^-24 relative) is 1e-4 in the exponent
        _close(paged_attention(c.q.cuda(), c.kv(), want_lse=True), c.want(), 2e-3)


@gpu
def test_lengths_past_the_table_and_bad_pages_are_left_out():
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    for d in (64, 128):
        c = Case(4, [160, 100, 33, 64], 16, 4, 1, d, "bf16")
        c.L = np.array([2 ** 31 - 1, 100, -3, 64], np.int32)
        c.table[1, 2], c.table[1, 4], c.table[3] = 2 ** 31 - 1, -2 ** 31, -1
        _close(paged_attention(c.q.cuda(), c.kv(), want_lse=True), c.want())


@gpu
@pytest.mark.parametrize("d,dtype,n_kv", [(512, "bf16", 1), (128, "bf16", 2), (64, "f32", 2), (256, "bf16", 1)])
@pytest.mark.parametrize("P", [8, 16, 64])
def test_listed_pages(d, dtype, n_kv, P):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(d + P, [5 * P + 3, 9 * P, 1, 0, 30 * P + 1], P, 4 * n_kv, n_kv, d, dtype)
    rs = np.random.RandomState(P)
    pages = rs.randint(-2, c.cols + 2, (5, n_kv, 11)).astype(np.int32)  # some twice, some no page
    pages[2] = -1
    pages[4, :, 0] = 30
    _close(paged_attention(c.q.cuda(), c.kv(), pages=_dev(pages), want_lse=True), c.want(pages=pages))
    _close(paged_attention(c.q.cuda(), c.kv(), pages=_dev(pages), window=3 * P + 1, want_lse=True),
           c.want(pages=pages, window=3 * P + 1))


@gpu
def test_scale_and_given_output():
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(1, [77, 5], 16, 4, 2, 128, "bf16")
    out = torch.full((2, 4, 128), float("nan"), device="cuda")
    r = paged_attention(c.q.cuda(), c.kv(), scale=0.3, out=out)
    assert r is out and np.max(np.abs(out.cpu().numpy() - c.want(scale=0.3)[0])) <= ATT_TOL


# ---------------------------------------------------------------- append and summaries


def _rows(rs, shape, dtype):
    return torch.from_numpy(rs.standard_normal(shape).astype(np.float32)).to(
        {"bf16": torch.bfloat16, "f32": torch.float32}[dtype])


def _bits(x):
    return x.cpu().contiguous().view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32).numpy()


@gpu
@pytest.mark.parametrize("T", [0, 1, 7, 300, 2049])
@pytest.mark.parametrize("n_kv,d,dtype,own_v,layout,P", [
    (1, 512, "bf16", False, "token", 32), (2, 128, "bf16", True, "head", 16), (3, 64, "f32", True, "both", 8),
    (1, 8, "bf16", False, "token", 1), (4, 200, "f32", False, "head", 64), (1, 256, "bf16", True, "token", 256)])
def test_append_writes_its_rows_and_nothing_else(T, n_kv, d, dtype, own_v, layout, P):
    from mtp_speculative_decoding_gemma4_gb300 import page_append
    rs = np.random.RandomState(T + d)
    c = Case(T + d, [1], P, n_kv, n_kv, d, dtype, own_v=own_v, layout=layout, spare=2 + 2 * T // P)
    n = c.k.shape[0]
    slots = rs.permutation(n * P)[:T].astype(np.int32)
    slots[rs.uniform(size=T) < 0.1] = -1
    if T > 5:
        slots[3], slots[4] = n * P, 2 ** 31 - 1
    k_new, v_new = _rows(rs, (T, n_kv, d), dtype), _rows(rs, (T, n_kv, d), dtype) if own_v else None
    codes = torch.randint(-127, 128, (n, n_kv, d), dtype=torch.int8)
    scales = torch.rand(n, n_kv)
    dc, ds = codes.cuda(), scales.cuda()
    page_append(c.kv(codes=dc, scales=ds), k_new.cuda(), _dev(slots), v_new=None if v_new is None else v_new.cuda())
    for cache, rows, dev in ((c.k, k_new, c.dk), (c.v, v_new, c.dv)):
        if cache is None:
            continue
        for t, s in enumerate(slots):
            if 0 <= s < n * P:
                cache[s // P, s % P] = rows[t]
        np.testing.assert_array_equal(_bits(dev), _bits(cache))
    k = c.k.float().numpy()
    for s in slots:
        if 0 <= s < n * P and s % P == P - 1:
            for g in range(n_kv):
                a, b = OP.page_summary(k[s // P, :, g])
                codes[s // P, g], scales[s // P, g] = torch.from_numpy(a), float(b)
    np.testing.assert_array_equal(dc.cpu().numpy(), codes.numpy())
    np.testing.assert_array_equal(ds.cpu().numpy(), scales.numpy())


@gpu
def test_append_takes_strided_rows():
    from mtp_speculative_decoding_gemma4_gb300 import page_append
    rs = np.random.RandomState(0)
    c = Case(2, [40], 16, 2, 2, 64, "bf16", own_v=True)
    both = _rows(rs, (5, 2, 2, 64), "bf16").cuda()  # rows of K and V interleaved
    slots = np.array([3, 17, 40, 2, 33], np.int32)
    page_append(c.kv(), both[:, 0], _dev(slots), v_new=both[:, 1])
    for i, s in enumerate(slots):
        assert torch.equal(c.dk[s // 16, s % 16], both[i, 0]) and torch.equal(c.dv[s // 16, s % 16], both[i, 1])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_summaries_of_odd_pages(dtype):
    # all zero, one huge row, values that cancel, infinities and NaN
    from mtp_speculative_decoding_gemma4_gb300 import page_append
    P, d = 16, 64
    c = Case(2, [1], P, 1, 1, d, dtype, spare=8)
    rs = np.random.RandomState(1)
    rows = _rows(rs, (6 * P, 1, d), dtype)
    rows[:P] = 0
    rows[P] *= 1e30
    rows[2 * P:3 * P:2] = -rows[2 * P + 1:3 * P:2]
    rows[2 * P] += 1e-3
    rows[3 * P + 5, 0, 7] = float("inf")
    rows[4 * P + 5, 0, 7] = float("nan")
    n = c.k.shape[0]
    codes, scales = torch.zeros((n, 1, d), dtype=torch.int8).cuda(), torch.zeros((n, 1)).cuda()
    page_append(c.kv(codes=codes, scales=scales), rows.cuda(), _dev(np.arange(6 * P, dtype=np.int32)))
    for p in range(6):
        a, b = OP.page_summary(rows[p * P:(p + 1) * P, 0].float().numpy())
        np.testing.assert_array_equal(codes[p, 0].cpu().numpy(), a)
        np.testing.assert_array_equal(scales[p].cpu().numpy(), [b])


# ---------------------------------------------------------------- selection


def _summarised(c, seed):
    rs = np.random.RandomState(seed)
    n = c.k.shape[0]
    codes = rs.randint(-127, 128, (n, c.n_kv, c.d)).astype(np.int8)
    scales = (rs.uniform(size=(n, c.n_kv)) * 0.02).astype(np.float32)
    return codes, scales


def _check_select(c, codes, scales, k, first=1, last=1):
    from mtp_speculative_decoding_gemma4_gb300 import page_select
    kv = c.kv(codes=_dev(codes), scales=_dev(scales))
    got = page_select(c.q.cuda(), kv, k, keep_first=first, keep_last=last).cpu().numpy()
    for b, L in enumerate(c.L):
        L = min(max(int(L), 0), c.cols * c.P)
        want = OP.page_select(c.q[b].numpy(), codes, scales, c.table[b], L, c.P, len(codes), k, first, last)
        np.testing.assert_array_equal(got[b], want, err_msg=f"sequence {b}")
    return kv, got


@gpu
@pytest.mark.parametrize("n_head,n_kv,d,dtype", [(4, 1, 512, "bf16"), (8, 2, 128, "bf16"), (2, 2, 64, "f32"),
                                                 (12, 1, 256, "bf16"), (32, 1, 128, "bf16"), (1, 1, 8, "bf16"),
                                                 (6, 3, 200, "bf16")])
@pytest.mark.parametrize("P,k", [(16, 5), (8, 64), (4, 33)])
def test_selection_matches_the_plain_form(n_head, n_kv, d, dtype, P, k):
    c = Case(d + P, [1, 0, 5 * P, k * P, k * P + 1, 40 * P + 3, 300 * P + 1, 257 * P], P, n_head, n_kv, d, dtype)
    codes, scales = _summarised(c, d)
    _check_select(c, codes, scales, k)
    _check_select(c, codes, scales, k, first=0, last=3)


@gpu
def test_selection_of_many_pages():
    # more pages than one pass holds, few distinct scores
    c = Case(1, [20000, 9999, 4097], 1, 2, 1, 16, "bf16")
    codes, scales = _summarised(c, 1)
    codes[:] = codes[:, :, :1] // 64
    scales[:] = 0.5
    for k in (2, 100, 5000):
        _check_select(c, codes, scales, k)


@gpu
def test_ties_go_to_the_lower_page_and_odd_scores():
    c = Case(6, [64 * 16, 50 * 16 + 1], 16, 4, 2, 128, "bf16")
    codes, scales = _summarised(c, 6)
    _check_select(c, np.zeros_like(codes), scales, 9)              # every score 0
    s2 = scales.copy()
    s2[::3] = np.nan                                               # pages that are always read
    _check_select(c, codes, s2, 30)
    c.table[0, 5:40] = -1                                          # entries that are no page
    _check_select(c, codes, scales, 9)
    c.q[0, 1] = 0                                                  # a head without a direction
    c.q[1, 0, 3] = float("inf")                                    # and one that is not finite
    c.q[1, 2, 3] = float("nan")
    _check_select(c, codes, scales, 9)


# ---------------------------------------------------------------- together


@gpu
def test_serving_rounds():
    """Rounds of plan, append, select and attend with growing, rolled back, ended and new
    sequences, against the same tokens kept in plain rows."""
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_append, page_plan, page_select, paged_attention
    rs = np.random.RandomState(0)
    Bn, P, d, nh, cols, n_pages, T, k = 7, 16, 128, 4, 24, 80, 400, 5
    cache = torch.full((n_pages, P, 1, d), float("nan"), dtype=torch.bfloat16).cuda()
    codes, scales = torch.zeros((n_pages, 1, d), dtype=torch.int8).cuda(), torch.zeros((n_pages, 1)).cuda()
    table = torch.full((Bn, cols), -1, dtype=torch.int32).cuda()
    ring, state = torch.arange(n_pages, dtype=torch.int32).cuda(), _dev(np.array([0, n_pages], np.int32))
    lens = torch.zeros(Bn, dtype=torch.int32).cuda()
    rows = [np.zeros((0, d), np.float32) for _ in range(Bn)]
    for step in range(12):
        old = lens.cpu().numpy()
        new = old + rs.randint(0, 30, Bn)
        if step % 3 == 2:
            new[rs.randint(Bn)] = 0
            b = rs.randint(Bn)
            new[b] = max(0, old[b] - rs.randint(0, 20))
        new = np.minimum(new, cols * P).astype(np.int32)
        lens, slots, cu, state, status = page_plan(lens, _dev(new), table, ring, state, P, T)
        out, cu, status = lens.cpu().numpy(), cu.cpu().numpy(), status.cpu().numpy()
        new_rows = _rows(rs, (T, 1, d), "bf16")
        kv = PagedKV(cache, table, lens, codes=codes, scales=scales)
        page_append(kv, new_rows.cuda(), slots)
        assert cu[Bn] == status[0] and int(state[1]) + sum(-(-out // P)) == n_pages
        for b in range(Bn):
            rows[b] = rows[b][:out[b]]
            if out[b] > old[b]:
                rows[b] = np.concatenate([rows[b], new_rows[cu[b]:cu[b + 1], 0].float().numpy()])
            assert len(rows[b]) == out[b]
        held = np.concatenate([table[b, :-(-out[b] // P)].cpu().numpy() for b in range(Bn)])
        assert len(set(held)) == len(held)
        q = torch.randn((Bn, nh, d), generator=torch.Generator().manual_seed(step))
        sel = page_select(q.cuda(), kv, k)
        for pages in (None, sel):
            got = paged_attention(q.cuda(), kv, pages=pages, want_lse=True)
            want = []
            for b in range(Bn):
                n = -(-out[b] // P)
                plain = np.zeros((max(n, 1), P, 1, d))
                plain.reshape(-1, d)[:out[b]] = rows[b]
                at = None
                if pages is not None:
                    sums = [OP.page_summary(plain[p, :, 0].astype(np.float32)) for p in range(max(n, 1))]
                    at = OP.page_select(q[b].numpy(), np.stack([s[0] for s in sums])[:, None],
                                        np.stack([s[1] for s in sums])[:, None], np.arange(n), out[b], P, max(n, 1), k,
                                        1, 1)
                    np.testing.assert_array_equal(sel[b].cpu().numpy(), at)
                want.append(OP.paged_attention(q[b].numpy(), plain, plain, np.arange(max(n, 1)), out[b],
                                               1 / np.sqrt(d), pages=at))
            _close(got, (np.stack([w[0] for w in want]), np.stack([w[1] for w in want])))


@gpu
def test_captured_calls_on_a_side_stream_read_new_contents():
    from mtp_speculative_decoding_gemma4_gb300 import page_select, paged_attention
    c = Case(3, [900, 20, 333], 16, 4, 1, 256, "bf16")
    codes, scales = _summarised(c, 3)
    kv, q = c.kv(codes=_dev(codes), scales=_dev(scales)), c.q.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        paged_attention(q, kv, pages=page_select(q, kv, 4))
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):  # two graphs, replayed one after the other and at the same time
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            sel = page_select(q, kv, 4)
            r = [paged_attention(q, kv, want_lse=True), paged_attention(q, kv, pages=sel, want_lse=True)]
        graphs.append((g, sel, r))
    for turn in range(3):
        c.L = np.array([[900, 20, 333], [17, 0, 320], [5, 20, 1]][turn], np.int32)
        c.q = torch.randn(c.q.shape, generator=torch.Generator().manual_seed(turn))
        kv.ctx_len.copy_(_dev(c.L))
        q.copy_(c.q)
        torch.cuda.synchronize()
        for (g, _, _), st in zip(graphs, (side, torch.cuda.Stream())):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, sel, r in graphs:
            at = sel.cpu().numpy()
            _close(r[0], c.want())
            _close(r[1], c.want(pages=at))


@gpu
def test_explicit_stream_and_argument_checks():
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_append, page_plan, page_select, paged_attention
    c = Case(3, [90, 20], 16, 4, 1, 128, "bf16")
    kv, q = c.kv(), c.q.cuda()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = paged_attention(q, kv, want_lse=True, stream=st.cuda_stream)
    st.synchronize()
    _close(got, c.want())
    _close(paged_attention(q, kv, want_lse=True, stream=0), c.want())
    with pytest.raises(ValueError):
        paged_attention(q.cpu(), kv)
    with pytest.raises(ValueError):
        paged_attention(q[:1], kv)
    with pytest.raises(ValueError):
        paged_attention(q.bfloat16(), kv)
    with pytest.raises(ValueError):
        paged_attention(q, kv, pages=torch.zeros((2, 1, 0), dtype=torch.int32).cuda())
    with pytest.raises(ValueError):
        paged_attention(q, kv, out=torch.empty(3).cuda())
    with pytest.raises(B.MtpError):
        paged_attention(q, kv, window=-1)
    with pytest.raises(B.MtpError):
        page_select(q, kv, 3)  # no summaries
    with pytest.raises(ValueError):
        page_select(q, kv, 0)
    with pytest.raises(ValueError):
        page_append(kv, torch.zeros((2, 1, 64), dtype=torch.bfloat16).cuda(), _dev(np.zeros(2, np.int32)))
    with pytest.raises(ValueError):
        PagedKV(c.dk, _dev(c.table))
    with pytest.raises(ValueError):
        PagedKV(c.dk.half())
    with pytest.raises(ValueError):
        page_plan(_dev(c.L), _dev(c.L), _dev(c.table[:1]), _dev(c.L), _dev(c.L), 16, 4)


@gpu
def test_calls_of_several_threads_and_streams_keep_apart():
    # two host threads on the default stream and two on streams of their own, over one descriptor
    import threading
    from mtp_speculative_decoding_gemma4_gb300 import page_select, paged_attention
    c = Case(11, [3000, 4096, 777, 1], 16, 4, 1, 128, "bf16")
    codes, scales = _summarised(c, 11)
    kv = c.kv(codes=_dev(codes), scales=_dev(scales))
    qs = [torch.randn(c.q.shape, generator=torch.Generator().manual_seed(i)) for i in range(4)]
    want = []
    for q in qs:
        c.q = q
        want.append((c.want(), np.stack([OP.page_select(q[b].numpy(), codes, scales, c.table[b], int(c.L[b]), 16,
                                                        len(codes), 9, 1, 1) for b in range(4)])))
    got, streams, errors = [[] for _ in qs], [None, None, torch.cuda.Stream(), torch.cuda.Stream()], []
    dq = [q.cuda() for q in qs]
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(20):
                    got[i].append((paged_attention(dq[i], kv, want_lse=True), page_select(dq[i], kv, 9)))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(4):
        for att, sel in got[i]:
            _close(att, want[i][0])
            np.testing.assert_array_equal(sel.cpu().numpy(), want[i][1])


@gpu
@pytest.mark.parametrize("n_nan", [5, 9, 10, 64])
def test_kept_pages_come_before_pages_that_are_not_finite(n_nan):
    c = Case(8, [64 * 16], 16, 4, 1, 128, "bf16")
    codes, scales = _summarised(c, 8)
    nan = np.random.RandomState(n_nan).permutation(64)[:n_nan]
    scales[c.table[0, nan]] = np.nan
    _check_select(c, codes, scales, 10)
    _check_select(c, codes, scales, 10, first=3, last=7)
    _, got = _check_select(c, codes, scales, 10, first=0, last=2)
    assert {62, 63} <= set(got[0, 0].tolist())


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_the_widest_window_is_every_key(d):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(d, [100, 1], 16, 4, 1, d, "bf16")
    _close(paged_attention(c.q.cuda(), c.kv(), window=2 ** 31 - 1, want_lse=True), c.want())


def test_outputs_over_inputs_are_refused_before_the_device(lib):
    kv = _kv()
    for q, out, lse in ((FAKE, FAKE, None), (FAKE, 2 * FAKE, 2 * FAKE)):
        assert lib.mtp_paged_attention(kv, q, 1, 4, 0, 0.0, None, 0, out, lse, FAKE, 1 << 30,
                                       None) == B.MTP_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("d,n_head", [(128, 4), (128, 8), (256, 3), (256, 8), (512, 4), (512, 7)])
@pytest.mark.parametrize("P,window", [(8, 0), (32, 100), (128, 0), (256, 333)])
def test_many_ragged_sequences(d, n_head, P, window):
    # more units than clusters fit: the keys of all sequences dealt evenly over the SMs
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    L = np.random.RandomState(d + P).randint(0, 900, 47)
    L[[0, 5, 46]] = 0
    c = Case(d + P + n_head, L, P, n_head, 1, d, "bf16", own_v=P == 32)
    _close(paged_attention(c.q.cuda(), c.kv(), window=window, want_lse=True), c.want(window=window))
    pages = np.random.RandomState(P).randint(-1, c.cols, (47, 1, 7)).astype(np.int32)
    _close(paged_attention(c.q.cuda(), c.kv(), window=window, pages=_dev(pages), want_lse=True),
           c.want(window=window, pages=pages))


@gpu
@pytest.mark.parametrize("d,n_head", [(128, 4), (256, 8), (512, 4), (512, 8)])
def test_one_sequence_over_all_sms(d, n_head):
    # a unit in as many parts as there are SMs
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(d + n_head, [40000], 64, n_head, 1, d, "bf16", own_v=d == 128)
    _close(paged_attention(c.q.cuda(), c.kv(), want_lse=True), c.want())


@gpu
def test_plans_of_two_threads_with_different_batches():
    # calls that need different amounts of shared memory, side by side
    import threading
    from mtp_speculative_decoding_gemma4_gb300 import page_plan
    cases, errors = [], []
    for Bn in (8192, 4097):
        old, new, table, ring, state = _plan_case(Bn, Bn, 4, 3, 9000, "any")
        cases.append((OP.page_plan(old, new, table[:, :3], ring, state, 4, 40000),
                      [_dev(x) for x in (old, new, np.ascontiguousarray(table[:, :3]), ring, state)], torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(want, dev, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(200):
                    got = page_plan(*dev, 4, 40000)
                for name, g, w in zip(("len", "slots", "cu", "state", "status"), got, want):
                    np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P", [1, 4, 64, 256])
def test_summaries_of_the_largest_values(dtype, P):
    # rows at the ends of the type's range: the sums would leave it, the mean does not
    from mtp_speculative_decoding_gemma4_gb300 import page_append
    d, n = 64, 4
    c = Case(2, [1], P, 1, 1, d, dtype, spare=8)
    rs, most = np.random.RandomState(P), torch.finfo(c.k.dtype).max
    rows = torch.full((n * P, 1, d), most, dtype=c.k.dtype)
    rows[P:2 * P] = -most
    rows[2 * P:3 * P, 0, : d // 2] *= -1
    # the last page in runs: half of the sum's weight on either side
    rows[3 * P:] *= torch.from_numpy(np.where(rs.uniform(size=(P, 1, d)) < 0.75, 1.0, -1.0)).to(c.k.dtype)
    m = c.k.shape[0]
    for cut in (0, P // 2):  # in one call, and the pages in two
        codes, scales = torch.zeros((m, 1, d), dtype=torch.int8).cuda(), torch.zeros((m, 1)).cuda()
        slots = np.arange(n * P, dtype=np.int32)
        first = slots % P < cut
        kv = c.kv(codes=codes, scales=scales)
        for part in (first, ~first):
            page_append(kv, rows[torch.from_numpy(part)].contiguous().cuda(), _dev(slots[part]))
        for p in range(n):
            a, b = OP.page_summary(rows[p * P:(p + 1) * P, 0].float().numpy())
            np.testing.assert_array_equal(codes[p, 0].cpu().numpy(), a)
            np.testing.assert_array_equal(scales[p].cpu().numpy(), [b])


def test_sizes_past_the_limits_are_refused_before_the_device(lib):
    kv = _kv()
    assert lib.mtp_page_append(kv, FAKE, None, 64, 64, FAKE, (1 << 30) + 1, None) == B.MTP_ERR_INVALID_ARG
    assert lib.mtp_page_append(kv, FAKE, None, 1 << 41, 64, FAKE, 2, None) == B.MTP_ERR_INVALID_ARG
    # outputs that begin inside the queries [4][64]; a scale that is infinite in base 2
    for q, out, lse, scale in ((2 * FAKE, 2 * FAKE + 512, None, 0.0), (2 * FAKE, 2 * FAKE - 512, None, 0.0),
                               (FAKE, 2 * FAKE, FAKE + 1020, 0.0), (FAKE, 2 * FAKE, 2 * FAKE - 4, 0.0),
                               (FAKE, 2 * FAKE, None, 3e38)):
        assert lib.mtp_paged_attention(kv, q, 1, 4, 0, scale, None, 0, out, lse, FAKE, 1 << 30,
                                       None) == B.MTP_ERR_INVALID_ARG
        assert B.mtp_last_error()


# ---------------------------------------------------------------- summaries of pages of large spread


def _cancelling(rs, P, d):
    """Rows of values of size 2^-3 to 4 and, in about half of the places, pairs of -2^20 and 2^20:
    a spread below 2^24, so that a mean is the rounded sum, whatever its order."""
    x = rs.choice([-1, 1], (P, d)) * 2.0 ** rs.uniform(-2.9, 2, (P, d))
    for j in range(d):
        at = rs.permutation(P)[:2 * (P // 4)]
        x[at[::2], j], x[at[1::2], j] = 2.0 ** 20, -2.0 ** 20
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


@gpu
@pytest.mark.parametrize("n_kv,d", [(1, 512), (1, 64), (2, 128), (3, 200)])
@pytest.mark.parametrize("P", [4, 16, 32, 256])
def test_summaries_where_large_values_cancel(P, n_kv, d):
    # the mean rounded once: exact sums in 64 bits have one value, so codes and scales are equal
    # bit by bit, for pages written whole, in two calls, and row by row in any order of one call
    from mtp_speculative_decoding_gemma4_gb300 import page_append
    rs = np.random.RandomState(P + d)
    n = 3
    c = Case(1, [1], P, n_kv, n_kv, d, "bf16", spare=n + 1)
    m = c.k.shape[0]
    rows = _cancelling(rs, n * P, n_kv * d).view(n * P, n_kv, d)
    want = [[OP.page_summary(rows[p * P:(p + 1) * P, g].float().numpy()) for g in range(n_kv)] for p in range(n)]
    slots = np.arange(n * P, dtype=np.int32)
    cut = slots % P < max(1, P // 3)
    for how in ("whole", "two calls", "any order"):
        parts = {"whole": [slots], "two calls": [slots[cut], slots[~cut]], "any order": [rs.permutation(slots)]}[how]
        codes, scales = torch.zeros((m, n_kv, d), dtype=torch.int8).cuda(), torch.zeros((m, n_kv)).cuda()
        kv = c.kv(codes=codes, scales=scales)
        for at in parts:
            page_append(kv, rows[torch.from_numpy(at.astype(np.int64))].contiguous().cuda(), _dev(at))
        for p in range(n):
            for g in range(n_kv):
                np.testing.assert_array_equal(codes[p, g].cpu().numpy(), want[p][g][0], err_msg=f"{how}, page {p}")
                np.testing.assert_array_equal(scales[p, g].cpu().numpy(), want[p][g][1], err_msg=f"{how}, page {p}")


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P", [8, 32, 256])
def test_summaries_of_any_spread_stay_within_the_bound(dtype, P):
    # beyond that spread a mean is off by at most 2^-24 of itself and P^2 2^-48 of the largest
    # value (the sum's running errors, each 2^-24 of a partial sum, are summed in fp32). One
    # dimension of a page holds values, so the scale is |m| / 127, rounded twice more.
    from mtp_speculative_decoding_gemma4_gb300 import page_append
    rs = np.random.RandomState(P)
    n, d = 200, 8
    c = Case(1, [1], P, 1, 1, d, dtype, spare=n)
    rows = torch.zeros((n * P, 1, d))
    rows[:, 0, 0] = torch.from_numpy((rs.choice([-1, 1], n * P) * 2.0 ** rs.uniform(-30, 30, n * P)).astype(np.float32))
    rows = rows.to(c.k.dtype)
    for p in range(n):  # the largest values come in pairs that cancel
        x = rows[p * P:(p + 1) * P, 0, 0]
        order = x.abs().argsort(descending=True)
        x[order[1:P // 2:2]] = -x[order[0:P // 2:2]][:len(order[1:P // 2:2])]
    codes, scales = torch.zeros((n + 1, 1, d), dtype=torch.int8).cuda(), torch.zeros((n + 1, 1)).cuda()
    page_append(c.kv(codes=codes, scales=scales), rows.cuda(), _dev(np.arange(n * P, dtype=np.int32)))
    got = scales.cpu().double().numpy()[:, 0] * 127
    for p in range(n):
        x = rows[p * P:(p + 1) * P, 0, 0].double().tolist()
        mean, most = math.fsum(x) / P, max(map(abs, x))
        assert abs(got[p] - abs(mean)) <= 4 * 2.0 ** -24 * abs(mean) + P * P * 2.0 ** -48 * most, p


# ---------------------------------------------------------------- scores below the range of fp32


@gpu
@pytest.mark.parametrize("own_v", [False, True])
@pytest.mark.parametrize("n_kv,d,dtype,cols", [(1, 64, "bf16", 8), (2, 32, "f32", 8), (1, 64, "f32", 600),
                                               (1, 128, "bf16", 8), (2, 256, "bf16", 300), (1, 512, "bf16", 8)])
def test_keys_of_score_minus_infinity_are_not_an_empty_sequence(n_kv, d, dtype, cols, own_v):
    # every attended key scores -inf (0 / 0): NaN, not the 0 and -inf of nothing to attend; the
    # other sequences keep their values
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    P = 16
    c = Case(d, [0, 3, 40, min(cols * P, 5000)], P, 2 * n_kv, n_kv, d, dtype, cols=cols, own_v=own_v)
    want = c.want()
    for b in (1, 3):
        c.q[b, :, 0] = 1 + 2.0 ** -9 + 2.0 ** -18  # three terms of one sign
        for lp in range(-(-int(c.L[b]) // P)):
            c.dk[int(c.table[b, lp]), :, :, 0] = float("-inf")
    for window in (0, 2):
        out, lse = (x.cpu() for x in paged_attention(c.q.cuda(), c.kv(), window=window, want_lse=True))
        for b in (1, 3):
            assert not torch.isfinite(out[b, :, 0]).any() and torch.isnan(lse[b]).all()
            if own_v:
                assert torch.isnan(out[b]).all()
        if window == 0:
            assert np.max(np.abs(out[2].numpy() - want[0][2])) <= ATT_TOL
            assert np.max(np.abs(lse[2].numpy() - want[1][2])) <= ATT_TOL
        assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


@gpu
def test_one_key_of_score_minus_infinity_has_no_weight():
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(1, [50], 16, 2, 1, 64, "f32", own_v=True)
    c.q[0, :, 0] = 1
    page = int(c.table[0, 0])
    c.dk[page, 3, 0, 0] = float("-inf")
    k = c.k.double().numpy()
    keep = [t for t in range(50) if t != 3]
    s = c.q[0].double().numpy() @ np.stack([k[c.table[0, t // 16], t % 16, 0] for t in keep]).T / 8
    v = np.stack([c.v[int(c.table[0, t // 16]), t % 16, 0].double().numpy() for t in keep])
    p = np.exp(s - s.max(1, keepdims=True))
    out, lse = paged_attention(c.q.cuda(), c.kv(), want_lse=True)
    assert np.max(np.abs(out[0].cpu().numpy() - p @ v / p.sum(1, keepdims=True))) <= ATT_TOL
    assert np.max(np.abs(lse[0].cpu().numpy() - (s.max(1) + np.log(p.sum(1))))) <= ATT_TOL


# ---------------------------------------------------------------- the three terms


def _terms(x):
    """The three bf16 terms of fp32 values."""
    hi = x.bfloat16().float()
    mid = (x - hi).bfloat16().float()
    return hi, mid, x - hi - mid


@gpu
@pytest.mark.parametrize("n_head", [4, 8])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_the_last_bits_of_a_query_count(d, n_head):
    # two dims whose keys are equal and whose query values differ in the third bf16 term alone: the
    # first two terms' products cancel exactly in any order, so a score is the third term's
    # product, about 8, rounded twice (it and its scale): 2^-22 of 8. Without it every score is 0.
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(d, [40, 300, 16], 16, n_head, 1, d, "bf16", own_v=True)
    g = torch.Generator().manual_seed(d)
    x = (1 + torch.rand((3, n_head), generator=g)) * 2.0 ** 20 * math.sqrt(d)
    hi, mid, lo = _terms(x)
    c.q.zero_()
    at = 3 * (d // 4)
    c.q[:, :, at], c.q[:, :, 5] = x, -(hi + mid)
    assert lo.abs().max() >= 2.0 ** 3
    for kk in (c.k, c.dk):
        kk[..., at] = kk[..., 5]
    out, lse = paged_attention(c.q.cuda(), c.kv(), want_lse=True)
    want = c.want()
    # |k| <= 5 and |lo| <= 2^-17 x <= 2^4 sqrt(d): scores up to 80, off by 2^-22 of that
    tol = ATT_TOL + 80 * 2.0 ** -22 * 4
    assert np.max(np.abs(out.cpu().numpy() - want[0])) <= tol
    assert np.max(np.abs(lse.cpu().numpy() - want[1])) <= tol


@gpu
@pytest.mark.parametrize("n_head", [4, 8])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_the_last_bits_of_a_probability_count(d, n_head):
    # two keys of values 1 and -1 and scores s in (-1, 0) and 0: out = (p - 1) / (p + 1) at p = e^s. p is
    # off by its exponent's two roundings and exp2f's 2 units (3 2^-23 in all), the sums and the
    # quotient by 3 2^-24: below 2^-20. Without the third term p is off by up to 2^-17.
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    Bn = 64
    c = Case(d, [2] * Bn, 16, n_head, 1, d, "bf16", own_v=True)
    c.q.zero_()
    c.q[:, :, 9] = -torch.rand((Bn, n_head), generator=torch.Generator().manual_seed(d))
    for b in range(Bn):
        page = int(c.table[b, 0])
        for kk in (c.k, c.dk):
            kk[page, :2] = 0
            kk[page, 0, 0, 9] = 1
        for vv in (c.v, c.dv):
            vv[page, 0], vv[page, 1] = 1, -1
    out, _ = paged_attention(c.q.cuda(), c.kv(), scale=1.0, want_lse=True)
    p = np.exp(c.q[:, :, 9].double().numpy())
    assert np.max(np.abs(out.cpu().numpy() - ((p - 1) / (p + 1))[..., None])) <= 2.0 ** -20


# ---------------------------------------------------------------- loads of what earlier kernels write


def test_paged_kernels_do_not_use_the_read_only_path():
    # they are programmatic dependents, resident while an earlier kernel may still write the block
    # table, the lengths, the pages and the summaries; ld.global.nc asks that nothing does
    csrc = os.path.join(os.path.dirname(B.__file__), "csrc")
    names = [n for n in sorted(os.listdir(csrc)) if n.startswith(("mtp_paged", "mtp_page"))]
    assert len(names) >= 7
    for name in names:
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        assert "__ldg(" not in text and "global.nc" not in text and "__restrict__" not in text, name


@gpu
def test_attention_right_behind_the_plan_that_writes_its_table():
    # a plan, an attention of other sequences and an attention over the plan's table, queued
    # together many times: the second attention is launched while the plan may still run
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_plan, paged_attention
    P, d, cols, n_pages = 16, 128, 64, 200
    rs = np.random.RandomState(3)
    cache = _rows(rs, (n_pages, P, 1, d), "bf16")
    dk, q = cache.cuda(), torch.randn((2, 4, d), generator=torch.Generator().manual_seed(3))
    zero, lens = torch.zeros(2, dtype=torch.int32).cuda(), _dev(np.array([1000, 333], np.int32))
    state, dq = _dev(np.array([0, n_pages], np.int32)), q.cuda()
    other = PagedKV(dk, torch.zeros((2, 1), dtype=torch.int32).cuda(), _dev(np.array([1, 2], np.int32)))
    rings = [rs.permutation(n_pages).astype(np.int32) for _ in range(40)]
    held = [(torch.full((2, cols), -1, dtype=torch.int32).cuda(), _dev(r)) for r in rings]
    kvs, got = [PagedKV(dk, t, lens) for t, _ in held], []
    torch.cuda.synchronize()
    for kv, (table, ring) in zip(kvs, held):
        page_plan(zero, lens, table, ring, state, P, 1400)
        paged_attention(dq, other)
        got.append(paged_attention(dq, kv, want_lse=True))
    torch.cuda.synchronize()
    k = cache.double().numpy()
    for ring, r in zip(rings, got):
        table = np.full((2, cols), -1, np.int32)
        table[0, :63], table[1, :21] = ring[:63], ring[63:84]
        want = [OP.paged_attention(q[b].numpy(), k, k, table[b], L, 1 / np.sqrt(d)) for b, L in enumerate((1000, 333))]
        _close(r, (np.stack([w[0] for w in want]), np.stack([w[1] for w in want])))


# ---------------------------------------------------------------- rounds, far rows, rows alone


@gpu
def test_a_captured_round_over_a_kept_descriptor():
    # plan, append, selection and attention of a round in one graph: the descriptor keeps its
    # length tensor, into which the round copies the plan's lengths
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_append, page_plan, page_select, paged_attention
    rs = np.random.RandomState(4)
    Bn, P, d, nh, cols, n_pages, T, k = 5, 16, 128, 4, 12, 60, 128, 4
    cache = torch.full((n_pages, P, 1, d), float("nan"), dtype=torch.bfloat16).cuda()
    codes, scales = torch.zeros((n_pages, 1, d), dtype=torch.int8).cuda(), torch.zeros((n_pages, 1)).cuda()
    table = torch.full((Bn, cols), -1, dtype=torch.int32).cuda()
    ring, state = torch.arange(n_pages, dtype=torch.int32).cuda(), _dev(np.array([0, n_pages], np.int32))
    lens, new = torch.zeros(Bn, dtype=torch.int32).cuda(), torch.zeros(Bn, dtype=torch.int32).cuda()
    rows, q = torch.zeros((T, 1, d), dtype=torch.bfloat16).cuda(), torch.zeros((Bn, nh, d)).cuda()
    kv = PagedKV(cache, table, lens, codes=codes, scales=scales)

    def turn():
        len_out, slots, cu, state_out, status = page_plan(lens, new, table, ring, state, P, T)
        page_append(kv, rows, slots)
        lens.copy_(len_out)
        state.copy_(state_out)
        sel = page_select(q, kv, k)
        return cu, sel, paged_attention(q, kv, want_lse=True), paged_attention(q, kv, pages=sel, want_lse=True)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        turn()  # nothing grows: no lengths, no rows
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            cu, sel, full, some = turn()
    torch.cuda.synchronize()
    kept = [np.zeros((0, d), np.float32) for _ in range(Bn)]
    for step in range(8):
        old = lens.cpu().numpy()
        grow = old + rs.randint(0, 25, Bn)
        if step % 3 == 2:
            grow[rs.randint(Bn)] = 0
            b = rs.randint(Bn)
            grow[b] = max(0, old[b] - 17)
        new.copy_(_dev(np.minimum(grow, cols * P).astype(np.int32)))
        fresh = _rows(rs, (T, 1, d), "bf16")
        rows.copy_(fresh)
        hq = torch.randn((Bn, nh, d), generator=torch.Generator().manual_seed(step))
        q.copy_(hq)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        out, at = lens.cpu().numpy(), cu.cpu().numpy()
        assert int(state[1]) + sum(-(-out // P)) == n_pages
        for pages, got in ((None, full), (sel.cpu().numpy(), some)):
            want = []
            for b in range(Bn):
                if pages is None:
                    kept[b] = kept[b][:out[b]]
                    if out[b] > old[b]:
                        kept[b] = np.concatenate([kept[b], fresh[at[b]:at[b + 1], 0].float().numpy()])
                    assert len(kept[b]) == out[b]
                n = max(1, -(-out[b] // P))
                plain = np.zeros((n, P, 1, d))
                plain.reshape(-1, d)[:out[b]] = kept[b]
                if pages is not None:
                    sums = [OP.page_summary(plain[p, :, 0].astype(np.float32)) for p in range(n)]
                    np.testing.assert_array_equal(pages[b], OP.page_select(
                        hq[b].numpy(), np.stack([s[0] for s in sums])[:, None], np.stack([s[1] for s in sums])[:, None],
                        np.arange(-(-out[b] // P)), out[b], P, n, k, 1, 1))
                want.append(OP.paged_attention(hq[b].numpy(), plain, plain, np.arange(n), out[b], 1 / np.sqrt(d),
                                               pages=None if pages is None else pages[b]))
            _close(got, (np.stack([w[0] for w in want]), np.stack([w[1] for w in want])))


@gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_pages_farther_apart_than_32_bits(dtype, d):
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_append, page_select, paged_attention
    P, n, far = 16, 3, (1 << 31) + 64
    c = Case(d, [40], P, 4, 1, d, dtype, spare=0)
    c.table[0] = [2, 0, 1]
    rows = _rows(np.random.RandomState(1), (n * P, 1, d), dtype)
    buf = torch.zeros((n - 1) * far + P * d, dtype=rows.dtype, device="cuda")
    k = buf.as_strided((n, P, 1, d), (far, d, d, 1))
    codes, scales = torch.zeros((n, 1, d), dtype=torch.int8).cuda(), torch.zeros((n, 1)).cuda()
    kv = PagedKV(k, _dev(c.table), _dev(c.L), codes=codes, scales=scales)
    slots = (c.table[0][:, None] * P + np.arange(P)).reshape(-1).astype(np.int32)
    page_append(kv, rows.cuda(), _dev(slots))
    c.k = torch.zeros((n, P, 1, d), dtype=rows.dtype)
    for i, s in enumerate(slots):
        c.k[s // P, s % P] = rows[i]
        assert torch.equal(k[s // P, s % P].cpu(), rows[i])
    for p in range(n):
        np.testing.assert_array_equal(codes[p, 0].cpu().numpy(), OP.page_summary(c.k[p, :, 0].float().numpy())[0])
    _close(paged_attention(c.q.cuda(), kv, want_lse=True), c.want())
    sel = page_select(c.q.cuda(), kv, 2)
    assert sel.tolist() == [[[0, 2]]]
    _close(paged_attention(c.q.cuda(), kv, pages=sel, want_lse=True), c.want(pages=sel.cpu().numpy()))
    # rows alone, from a source whose rows are as far apart
    src = torch.zeros(far + d, dtype=rows.dtype, device="cuda").as_strided((2, 1, d), (far, d, 1))
    src.copy_(rows[:2])
    page_append(PagedKV(k), src, _dev(np.array([2 * P + 7, 2 * P + 9], np.int32)))
    assert torch.equal(k[2, 7].cpu(), rows[0]) and torch.equal(k[2, 9].cpu(), rows[1])


@gpu
def test_summaries_past_32_bits():
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_append, page_select
    d, n, cols = 512, (1 << 23) + 40, 90
    k = torch.empty((n, 1, 1, d), dtype=torch.bfloat16, device="cuda")
    codes, scales = torch.empty((n, 1, d), dtype=torch.int8, device="cuda"), torch.empty((n, 1), device="cuda")
    rs = np.random.RandomState(0)
    table = (n - 1 - rs.permutation(cols)).astype(np.int32)[None]
    rows, q = _rows(rs, (cols, 1, d), "bf16"), torch.randn((1, 4, d), generator=torch.Generator().manual_seed(1))
    kv = PagedKV(k, _dev(table), _dev(np.array([cols], np.int32)), codes=codes, scales=scales)
    page_append(kv, rows.cuda(), _dev(table[0]))
    sums = [OP.page_summary(rows[i].float().numpy()) for i in range(cols)]
    got = codes[torch.from_numpy(table[0].astype(np.int64)).cuda(), 0].cpu().numpy()
    np.testing.assert_array_equal(got, np.stack([s[0] for s in sums]))
    want = OP.page_select(q[0].numpy(), np.stack([s[0] for s in sums])[:, None], np.stack([s[1] for s in sums])[:, None],
                          np.arange(cols), cols, 1, cols, 7, 1, 1)
    np.testing.assert_array_equal(page_select(q.cuda(), kv, 7).cpu().numpy()[0], want)


@gpu
@pytest.mark.parametrize("T", [0, 1, 7, 300, 2049])
@pytest.mark.parametrize("n_kv,d,dtype,own_v,layout,P", [
    (1, 512, "bf16", False, "token", 32), (2, 128, "bf16", True, "head", 16), (3, 64, "f32", True, "both", 8),
    (1, 8, "bf16", False, "token", 1), (4, 200, "f32", False, "head", 64), (1, 256, "bf16", True, "token", 256)])
def test_append_of_rows_alone(T, n_kv, d, dtype, own_v, layout, P):
    # a cache without summaries: every row in its slot, everything else as it was
    from mtp_speculative_decoding_gemma4_gb300 import page_append
    rs = np.random.RandomState(T + d)
    c = Case(T + d, [1], P, n_kv, n_kv, d, dtype, own_v=own_v, layout=layout, spare=2 + 2 * T // P)
    n = c.k.shape[0]
    slots = rs.permutation(n * P)[:T].astype(np.int32)
    slots[rs.uniform(size=T) < 0.1] = -1
    if T > 5:
        slots[3], slots[4], slots[5] = n * P, 2 ** 31 - 1, -2 ** 31
    k_new, v_new = _rows(rs, (T, n_kv, d), dtype), _rows(rs, (T, n_kv, d), dtype) if own_v else None
    page_append(c.kv(), k_new.cuda(), _dev(slots), v_new=None if v_new is None else v_new.cuda())
    for cache, rows, dev in ((c.k, k_new, c.dk), (c.v, v_new, c.dv)):
        if cache is None:
            continue
        for t, s in enumerate(slots):
            if 0 <= s < n * P:
                cache[s // P, s % P] = rows[t]
        np.testing.assert_array_equal(_bits(dev), _bits(cache))


@gpu
@pytest.mark.parametrize("n_kv,d,dtype", [(1, 8, "bf16"), (2, 64, "bf16"), (1, 16, "f32")])
@pytest.mark.parametrize("how", ["any order", "from inside a page", "runs of nine"])
def test_appends_of_many_rows_in_any_order(n_kv, d, dtype, how):
    # more rows than one launch sums: pages written whole, completed by a later run of the call, by
    # rows in any order, or behind older rows; the bound of the sums is the one of small calls
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_append
    T, P = 70001, 16
    n = T // 8 // P * 16 + 40
    rs = np.random.RandomState(d)
    cache = _rows(rs, (n, P, n_kv, d), dtype)
    rows = _rows(rs, (T, n_kv, d), dtype)
    if how == "any order":
        slots = rs.permutation(n * P)[:T]
    elif how == "from inside a page":
        slots = 7 + np.arange(T)
    else:
        start = rs.permutation(n * P // 9)[:T // 9 + 1]
        slots = (start[:, None] * 9 + np.arange(9)).reshape(-1)[:T]
    slots = slots.astype(np.int32)
    dk, codes, scales = cache.cuda(), torch.zeros((n, n_kv, d), dtype=torch.int8).cuda(), torch.zeros((n, n_kv)).cuda()
    page_append(PagedKV(dk, codes=codes, scales=scales), rows.cuda(), _dev(slots))
    cache.view(n * P, n_kv, d)[torch.from_numpy(slots.astype(np.int64))] = rows
    np.testing.assert_array_equal(_bits(dk), _bits(cache))
    done = slots[slots % P == P - 1] // P
    mean = (cache.double().sum(1) / P).float().numpy()
    scale = np.abs(mean).max(-1) * OP.INV127
    code = np.clip(np.rint(mean / scale[..., None]), -127, 127)
    want_codes, want_scales = np.zeros((n, n_kv, d), np.int8), np.zeros((n, n_kv), np.float32)
    want_codes[done], want_scales[done] = code[done], scale[done]
    np.testing.assert_array_equal(codes.cpu().numpy(), want_codes)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_scales)


@gpu
def test_the_time_of_an_append_grows_with_its_rows():
    # 2^20 rows in any order: some 5 ms, with every page looked up among all rows 50 ms
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, page_append
    T, P, d = 1 << 20, 16, 8
    k, rows = torch.zeros((T // P, P, 1, d), dtype=torch.bfloat16).cuda(), torch.zeros((T, 1, d), dtype=torch.bfloat16).cuda()
    codes, scales = torch.zeros((T // P, 1, d), dtype=torch.int8).cuda(), torch.zeros((T // P, 1)).cuda()
    kv, slots = PagedKV(k, codes=codes, scales=scales), _dev(np.random.RandomState(0).permutation(T).astype(np.int32))
    times = []
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        page_append(kv, rows, slots)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert min(times) <= 15
