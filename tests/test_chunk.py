"""Attention of a chunk of new tokens over a paged cache against a plain form in 64 bits; refusals
without a device."""
import ctypes

import numpy as np
import pytest
import torch

from mtp_speculative_decoding_gemma4_gb300 import binding as B
from mtp_speculative_decoding_gemma4_gb300 import build as build_mod

gpu = pytest.mark.gpu

# fp32 models, N(0, 1) queries and keys, scale 1 / sqrt(d): each of the d additions of a score rounds
# a partial sum of size <= sqrt(d) by at most 2^-24 relative, so a score is off by some 2^-24 sqrt(d) *
# sqrt(d / 2) / sqrt(d) = 2^-24 sqrt(d / 2) = 1e-6 at d = 512 (independent errors), a probability by as
# much, relative, and an output, a mean of values of size 1, by no more; a maximum over 10^4..10^6
# outputs is some 5 such errors, the sums over the keys add less. lse moves with the scores. 2e-5 is
# four times that, for truncating adders as well.
TOL = 2e-5
# bf16: an output is rounded to it (2^-8 of itself), and on tensor cores every probability is (2^-8 of
# itself, so an output by at most 2^-8 sum_j p_j |v_j|).
HALF = torch.finfo(torch.bfloat16).eps / 2


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- refusals (no device)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


FAKE = 1 << 20  # an aligned address that is never used: validation fails first


def _kv(**over):
    c = B.mtp_paged_kv()
    for f in ("k", "block_table", "ctx_len"):
        setattr(c, f, FAKE)
    for f, x in dict(stride_page=16 * 64, stride_t=64, stride_h=64, table_stride=4096, n_pages=32, page_size=16,
                     max_pages=4096, n_kv_head=1, head_dim=64, dtype=B.MTP_DTYPE_BF16).items():
        setattr(c, f, x)
    for f, x in over.items():
        setattr(c, f, x)
    return c


@pytest.mark.parametrize("args,code", [
    (dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(out=None), 1), (dict(out=FAKE + 2), 1), (dict(cu=None), 1),
    (dict(cu=FAKE + 2), 1), (dict(lse=FAKE + 1), 1), (dict(B=0), 1), (dict(B=(1 << 20) + 1), 1), (dict(T=-1), 1),
    (dict(T=(1 << 24) + 1), 1), (dict(T=1 << 24, nh=8), 1), (dict(nh=0), 1), (dict(nh=3, kv=dict(n_kv_head=2)), 1),
    (dict(stride=255), 1), (dict(stride=260), 1), (dict(stride=1 << 41), 1), (dict(window=-1), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 8), 1), (dict(ws_bytes=0), 1), (dict(out=FAKE), 1), (dict(lse=FAKE), 1), (dict(lse=2 * FAKE), 1),
    (dict(kv=dict(block_table=None)), 1), (dict(kv=dict(ctx_len=None)), 1), (dict(kv=dict(dtype=2)), 1),
    (dict(kv=dict(head_dim=60)), 2), (dict(kv=dict(page_size=24)), 2)])
def test_bad_arguments_are_refused_before_the_device(lib, args, code):
    a = dict(q=FAKE, stride=256, cu=FAKE, B=1, T=4, nh=4, window=0, scale=0.0, out=2 * FAKE, lse=None, ws=4 * FAKE,
             ws_bytes=1 << 40, kv={})
    a.update(args)
    rc = lib.mtp_paged_attention_chunk(_kv(**a["kv"]), a["q"], a["stride"], a["cu"], a["B"], a["T"], a["nh"],
                                       a["window"], a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)
    assert rc == code
    assert B.mtp_last_error()


def test_the_workspace_call_refuses_what_the_call_does_and_no_token_needs_none(lib):
    n = ctypes.c_int64(-1)
    for args in ((0, 4, 4), (1, -1, 4), (1, 4, 0)):
        assert lib.mtp_paged_attention_chunk_workspace(_kv(), *args, ctypes.byref(n)) == B.MTP_ERR_INVALID_ARG
    assert lib.mtp_paged_attention_chunk_workspace(_kv(), 1, 4, 4, None) == B.MTP_ERR_INVALID_ARG
    assert lib.mtp_paged_attention_chunk_workspace(_kv(), 1, 0, 4, ctypes.byref(n)) == 0 and n.value == 0
    # no tokens: nothing is launched, so no device is needed either
    assert lib.mtp_paged_attention_chunk(_kv(), None, 0, FAKE, 1, 0, 4, 0, 0.0, None, None, None, 0, None) == 0


# ---------------------------------------------------------------- cases


class Case:
    """A paged cache with random pages, NaN wherever no token lives, and the sequences' last tokens
    as new ones. `pad` rows of q belong to no sequence."""

    def __init__(self, seed, lengths, new, P, n_head, n_kv, d, dtype="bf16", own_v=False, layout="token", pad=0,
                 q_by=1.0, q_skip=0):
        rs, g = np.random.RandomState(seed), torch.Generator().manual_seed(seed)
        self.L, self.new = np.asarray(lengths, np.int32), np.asarray(new, np.int32)
        Bn = len(self.L)
        self.P, self.n_kv, self.d, self.n_head, self.bf16 = P, n_kv, d, n_head, dtype == "bf16"
        self.cols = max(1, int(-(-self.L.max() // P)))
        held = -(-np.clip(self.L, 0, None) // P)
        n_pages = int(held.sum()) + 3
        perm = rs.permutation(n_pages)
        self.table = np.full((Bn, self.cols), -1, np.int32)
        keep, at = np.zeros((n_pages, P), bool), 0
        for b in range(Bn):
            self.table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
            t = np.arange(self.L[b])
            keep[self.table[b, t // P], t % P] = True
        dt = torch.bfloat16 if self.bf16 else torch.float32

        def cache():
            x = torch.randn((n_pages, P, n_kv, d), generator=g).to(dt)
            x[torch.from_numpy(~keep)] = float("nan")
            return x

        self.k, self.v = cache(), cache() if own_v else None
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad
        self.q = (torch.randn((self.T, n_head, d), generator=g) * q_by).to(dt)
        if pad:
            self.q[self.cu[-1]:] = float("nan")
        dev = (lambda x: x.transpose(1, 2).contiguous().cuda().transpose(1, 2)) if layout == "head" else (
            lambda x: x.cuda())
        self.dk, self.dv = dev(self.k), None if self.v is None else dev(self.v)
        wide = torch.full((self.T, n_head * d + q_skip), float("nan"), dtype=dt, device="cuda")
        wide[:, :n_head * d] = self.q.reshape(self.T, -1).cuda()
        self.dq = wide[:, :n_head * d].unflatten(1, (n_head, d))

    def kv(self):
        from mtp_speculative_decoding_gemma4_gb300 import PagedKV
        return PagedKV(self.dk, _dev(self.table), _dev(self.L), v=self.dv)

    def run(self, window=0, scale=0.0, **more):
        from mtp_speculative_decoding_gemma4_gb300 import paged_attention_chunk
        return paged_attention_chunk(self.dq, self.kv(), _dev(self.cu), window=window, scale=scale, want_lse=True, **more)

    def want(self, window=0, scale=0.0):
        """out, lse and sum_j p_j |v_j| in fp64, NaN in rows of no sequence."""
        dev = "cuda" if torch.cuda.is_available() else "cpu"
        k, q = self.k.to(dev), self.q.to(dev)
        v = k if self.v is None else self.v.to(dev)
        G, s = self.n_head // self.n_kv, scale or self.d ** -0.5
        out = torch.full((self.T, self.n_head, self.d), float("nan"), dtype=torch.float64, device=dev)
        mean, lse = out.clone(), out[..., 0].clone()
        for b, (L, n) in enumerate(zip(self.L.tolist(), self.new.tolist())):
            t = torch.arange(max(L, 0), device=dev)
            page = torch.from_numpy(self.table[b]).to(dev).long()[t // self.P]
            pos = (L - n + torch.arange(n, device=dev))[:, None]
            on = (t <= pos) & (page >= 0)
            if window:
                on = on & (t > pos - window)
            rows = slice(int(self.cu[b]), int(self.cu[b + 1]))
            some = on.any(-1)
            for h in range(self.n_head):
                keys, vals = (x[page.clamp(min=0), t % self.P, h // G].double() for x in (k, v))
                used = on.any(0)
                keys, vals = (x.masked_fill(~used[:, None], 0.0) for x in (keys, vals))
                x = (q[rows, h].double() @ keys.T * s).masked_fill(~on, float("-inf"))
                p = torch.where(some[:, None], torch.softmax(x, -1), 0.0)
                out[rows, h], mean[rows, h] = p @ vals, p @ vals.abs()
                lse[rows, h] = torch.logsumexp(x, -1) if L > 0 else float("-inf")
        return out, lse, mean

    def check(self, window=0, scale=0.0, tol=TOL, got=None):
        out, lse = got or self.run(window, scale)
        want, wl, mean = (x[:self.cu[-1]].cuda() for x in self.want(window, scale))
        out, lse = out[:self.cu[-1]], lse[:self.cu[-1]]
        assert out.dtype == (torch.bfloat16 if self.bf16 else torch.float32) and torch.isfinite(out).all()
        most = tol + (HALF * (want.abs() + mean * (1 + HALF)) if self.bf16 else 0)
        over = (out.double() - want).abs() - most
        assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())
        empty = torch.isneginf(wl)
        assert torch.equal(torch.isneginf(lse), empty) and (out[empty] == 0).all()
        off = (lse.double() - wl)[~empty].abs()
        assert off.numel() == 0 or float(off.max()) <= tol * (1 + scale), float(off.max())


# ---------------------------------------------------------------- against 64 bits


SHAPES = [  # n_head, n_kv, d, dtype
    (4, 1, 256, "bf16"), (4, 1, 512, "bf16"), (8, 2, 128, "bf16"), (16, 2, 128, "bf16"), (3, 3, 128, "bf16"),
    (5, 1, 256, "bf16"), (40, 2, 128, "bf16"), (7, 1, 512, "bf16"), (72, 1, 256, "bf16"), (130, 1, 128, "bf16"),
    (2, 1, 384, "bf16"), (2, 1, 32, "f32"), (4, 2, 64, "f32"), (6, 2, 64, "bf16"), (9, 1, 80, "bf16"),
    (4, 1, 512, "f32"), (12, 4, 200, "f32"), (1, 1, 8, "bf16"), (70, 1, 64, "f32")]


@gpu
@pytest.mark.parametrize("own_v", [False, True])
@pytest.mark.parametrize("n_head,n_kv,d,dtype", SHAPES)
def test_matches_the_plain_form(n_head, n_kv, d, dtype, own_v):
    c = Case(n_head + d, [1, 0, 16, 17, 127, 128, 129, 300, 1000, 5], [1, 0, 16, 5, 1, 0, 129, 33, 7, 5], 16, n_head,
             n_kv, d, dtype, own_v=own_v)
    c.check()


@gpu
@pytest.mark.parametrize("window", [1, 15, 16, 100, 128, 513, 100000])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_window_edges(d, window):
    Case(d + window, [1, 0, 15, 16, 100, 128, 129, 511, 512, 513, 900], [1, 0, 3, 16, 70, 1, 9, 130, 1, 513, 64], 32, 4,
         1, d, own_v=d == 128).check(window=window)


@gpu
@pytest.mark.parametrize("P", [1, 2, 4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,n_head", [(64, 2), (128, 4), (256, 8), (512, 4)])
def test_page_sizes(P, d, n_head):
    Case(P + d, [700, 3, 257], [65, 3, 9], P, n_head, 1, d).check()


@gpu
@pytest.mark.parametrize("n", [1, 2, 3, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_chunk_lengths(d, n):
    Case(n + d, [n, 1500], [n, min(n, 1500)], 64, 4, 1, d).check()


@gpu
@pytest.mark.parametrize("dtype,d,own_v", [("bf16", 128, True), ("bf16", 64, False), ("f32", 64, True), ("bf16", 512, True)])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_layouts_and_strided_queries(layout, dtype, d, own_v):
    Case(5, [70, 3, 257], [9, 3, 40], 32, 6, 3, d, dtype, own_v=own_v, layout=layout, q_skip=16).check()


@gpu
@pytest.mark.parametrize("d", [128, 256, 512, 64])
@pytest.mark.parametrize("new", [[5, 1, 0, 17, 9, 37], [4000, 1, 0, 4096, 3, 37]])
def test_long_and_ragged(d, new):
    Case(d, [20001, 1, 0, 4096, 12345, 37], new, 64, 4, 1, d).check()


@gpu
@pytest.mark.parametrize("Bn", [1, 2, 151, 700])
@pytest.mark.parametrize("d", [64, 128, 512])
def test_batches(Bn, d):
    rs = np.random.RandomState(Bn)
    L = np.maximum(rs.randint(0, 400, Bn), 1)
    Case(Bn, L, np.minimum(rs.randint(0, 12, Bn), L), 16, 4, 1, d).check()


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (64, "bf16"), (128, "bf16"), (256, "bf16"), (512, "bf16")])
@pytest.mark.parametrize("by", [0.0, 20.0])
def test_flat_and_peaked_scores(d, dtype, by):
    """All scores equal; and scores of size 20 that grow and fall by more than any rescaling step. A
    score's error is `by` times that of an N(0, 1) query."""
    Case(d, [2000, 333], [100, 333], 32, 4, 1, d, dtype, own_v=True, q_by=by).check(tol=TOL * max(by, 1))


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (256, "bf16"), (512, "bf16")])
def test_scores_that_rise_with_the_position(d, dtype):
    """Keys that grow with their position, all along the query: the running maximum moves at every step."""
    c = Case(1, [1500], [90], 16, 2, 1, d, dtype)
    t = torch.arange(1500)
    page = torch.from_numpy(c.table[0]).long()[t // 16]
    rise = (t.double() / 1500 * 40)[:, None, None] * d ** -0.5 * torch.ones(1, 1, d)
    c.k[page, t % 16] = rise.to(c.k.dtype)
    c.q = torch.ones_like(c.q)
    c.dk, c.dq = c.k.cuda(), c.q.cuda()
    c.check(tol=TOL * 40)


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (256, "bf16"), (512, "bf16")])
def test_rows_of_no_sequence_are_left_as_they_were(d, dtype):
    c = Case(2, [40, 300], [7, 5], 16, 4, 1, d, dtype, pad=9)
    out = torch.full_like(c.dq.contiguous(), 7.0)
    got = c.run(out=out)
    c.check(got=got)
    assert (got[0][c.cu[-1]:] == 7.0).all()
    first = got[0].clone()
    # the same where the first rows belong to none: cu begins behind them
    c.cu = c.cu + 4
    out.fill_(7.0)
    c.dq = torch.cat([c.dq[-4:], c.dq[:-4]]).contiguous()
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention_chunk
    more = paged_attention_chunk(c.dq, c.kv(), _dev(c.cu), out=out)
    assert torch.equal(more[4:c.cu[-1]], first[:c.cu[-1] - 4])
    assert (more[:4] == 7.0).all() and (more[c.cu[-1]:] == 7.0).all()


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (64, "bf16"), (128, "bf16"), (256, "bf16"), (512, "bf16")])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("own_v", [False, True])
def test_what_is_not_attended_does_not_reach_a_row(d, dtype, what, own_v):
    """A key (or value) that is not finite reaches the rows that attend it and no others, whether it
    is one of the new tokens or falls out of some rows' window."""
    c = Case(3, [200, 90], [60, 60], 16, 4, 1, d, dtype, own_v=own_v)
    want = {w: c.run(w) for w in (0, 50)}
    bad = {0: 170, 1: 45}  # positions
    x = c.dv if own_v else c.dk
    for b, t in bad.items():
        x[c.table[b, t // 16], t % 16, :, 3] = what
    for w, (clean, _) in want.items():
        out, lse = c.run(w)
        for b, t in bad.items():
            for i in range(60):
                pos, row = c.L[b] - 60 + i, c.cu[b] + i
                if t <= pos and (not w or t > pos - w):
                    # (a key of -inf may score -inf and then has no weight)
                    assert not torch.isfinite(out[row]).all() or what == float("inf") and not own_v
                else:
                    assert torch.equal(out[row], clean[row])


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (512, "bf16")])
def test_pages_that_are_none_and_sequences_shorter_than_their_new_tokens(d, dtype):
    c = Case(4, [100, 64, 5], [10, 3, 5], 16, 4, 1, d, dtype)
    c.table[0, 2], c.table[1, :] = -1, -1  # a hole; a sequence of no page at all
    table = c.table.copy()
    table[1, :] = 1 << 20
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, paged_attention_chunk
    got = paged_attention_chunk(c.dq, PagedKV(c.dk, _dev(table), _dev(c.L)), _dev(c.cu), want_lse=True)
    c.check(got=got)
    assert (got[0][10:13] == 0).all() and torch.isneginf(got[1][10:13]).all()
    # 8 new tokens said of a sequence that holds 5: the first 3 attend nothing
    cu = np.array([0, 10, 10, 18], np.int32)
    got = paged_attention_chunk(c.dq, PagedKV(c.dk, _dev(table), _dev(c.L)), _dev(cu), want_lse=True)
    assert (got[0][10:13] == 0).all() and torch.isneginf(got[1][10:13]).all()
    assert torch.isfinite(got[0]).all() and (got[0][13:] != 0).any(-1).all()


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (256, "bf16"), (512, "bf16")])
def test_the_largest_window_and_sequences_shorter_than_their_new_tokens(d, dtype):
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, paged_attention_chunk
    c = Case(11, [40, 200], [17, 30], 16, 4, 1, d, dtype)
    kv, cu = c.kv(), _dev(c.cu)
    assert torch.equal(paged_attention_chunk(c.dq, kv, cu, window=2 ** 31 - 1), paged_attention_chunk(c.dq, kv, cu))
    # 17 new tokens said of a sequence of 12: the first 5 attend nothing, the others what 12 of 12 do
    short = PagedKV(c.dk, _dev(c.table), _dev(np.array([12, 200], np.int32)))
    for w in (0, 2 ** 31 - 1, 4):
        got = paged_attention_chunk(c.dq, short, cu, window=w)
        want = paged_attention_chunk(c.dq[5:].contiguous(), short, cu - torch.tensor([0, 5, 5], dtype=torch.int32, device="cuda"), window=w)
        assert (got[:5] == 0).all() and (got[5:].float() - want.float()).abs().max() <= 2 * HALF * want.abs().max()


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (64, "bf16"), (128, "bf16"), (512, "bf16")])
def test_pages_farther_apart_than_32_bits(d, dtype):
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, paged_attention_chunk
    c = Case(12, [90, 50], [20, 3], 16, 4, 1, d, dtype)
    want = c.run()[0]
    step = (1 << 32) // (4 if c.bf16 else 8) // c.k.shape[0] * 3 // 8 * 8  # 6 GB in all
    far = torch.empty(step * c.k.shape[0], dtype=c.k.dtype, device="cuda").as_strided(c.k.shape, (step, d, d, 1))
    assert far.stride(0) * (far.shape[0] - 1) * far.element_size() > 1 << 32
    far.copy_(c.dk)
    assert torch.equal(paged_attention_chunk(c.dq, PagedKV(far, _dev(c.table), _dev(c.L)), _dev(c.cu)), want)


@gpu
def test_lengths_and_offsets_out_of_range_are_clamped():
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, paged_attention_chunk
    for d, dtype in ((64, "f32"), (128, "bf16")):
        c = Case(6, [64, 64], [6, 6], 16, 4, 1, d, dtype)
        want = c.run()[0]
        got = paged_attention_chunk(c.dq, PagedKV(c.dk, _dev(c.table), _dev(np.array([1 << 30, 64], np.int32))),
                                    _dev(np.array([-5, 6, 1 << 30], np.int32)))
        assert torch.equal(got, want)


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (256, "bf16"), (512, "bf16")])
def test_one_token_each_equals_the_one_token_attention(d, dtype):
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention
    c = Case(8, [1, 700, 33], [1, 1, 1], 16, 4, 1, d, dtype)
    out, lse = c.run()
    one, one_lse = paged_attention(c.dq.float(), c.kv(), want_lse=True)
    assert float((lse - one_lse).abs().max()) <= 2 * TOL
    want, _, mean = c.want()
    most = 2 * TOL + (HALF * (want.abs() + mean * (1 + HALF)) if c.bf16 else 0)
    assert ((out.double() - one.double()).abs() <= most).all()


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (512, "bf16")])
def test_streams_graphs_and_repeats(d, dtype):
    """The same call on another stream, twice at once on two streams and in a replayed graph whose
    inputs change gives the same bits."""
    from mtp_speculative_decoding_gemma4_gb300 import paged_attention_chunk
    c = Case(9, [3000, 100], [40, 7], 16, 4, 1, d, dtype)
    kv, cu = c.kv(), _dev(c.cu)
    want = paged_attention_chunk(c.dq, kv, cu)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [paged_attention_chunk(c.dq, kv, cu, stream=s.cuda_stream) for s in (a, b) for _ in range(3)]
    torch.cuda.synchronize()
    for x in got:
        assert torch.equal(x, want)
    q = torch.zeros_like(c.dq)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = paged_attention_chunk(q, kv, cu)
    for _ in range(2):
        q.copy_(c.dq)
        g.replay()
        assert torch.equal(out, want)
        q.zero_()
        g.replay()
        torch.cuda.synchronize()


@gpu
def test_python_checks():
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, paged_attention_chunk
    c = Case(1, [20], [4], 16, 4, 2, 64, "bf16")
    kv, cu = c.kv(), _dev(c.cu)
    for q in (c.dq.float(), c.dq[0], c.dq[..., :32], c.dq.cpu(), c.dq.transpose(0, 1)):
        with pytest.raises(ValueError):
            paged_attention_chunk(q, kv, cu)
    for bad in (cu[:1], cu.long(), cu.cpu(), None):
        with pytest.raises(ValueError):
            paged_attention_chunk(c.dq, kv, bad)
    with pytest.raises(ValueError):
        paged_attention_chunk(c.dq, kv, cu, out=torch.empty(4, 4, 64, device="cuda"))
    with pytest.raises(ValueError):
        paged_attention_chunk(c.dq, PagedKV(c.dk), cu)
    with pytest.raises(B.MtpError):
        paged_attention_chunk(c.dq[:, :3].contiguous(), kv, cu)  # 3 heads on 2 KV heads
    empty = paged_attention_chunk(c.dq[:0], kv, torch.zeros_like(cu))
    assert empty.shape == (0, 4, 64)


# ---------------------------------------------------------------- device waits that run out


def test_the_limits_of_the_waits_are_checked(lib):
    for bad in ((-2, 0), (-1, -1)):
        assert lib.mtp_set_chunk_debug(*bad) == B.MTP_ERR_INVALID_ARG and B.mtp_last_error()
    assert lib.mtp_set_chunk_debug(-1, 0) == B.MTP_OK


def _given_up(c, skip, window=0):
    """Outputs of a call whose waits for sequence `skip` run out after some 10 ms, against those of an
    ordinary call: NaN in the rows of the sequence, and in no row or every element of another; the
    rows that have NaN."""
    clean = [x.clone() for x in c.run(window)]
    B.mtp_set_chunk_debug(skip, 20_000_000)
    try:
        out, lse = c.run(window)
        torch.cuda.synchronize()
    finally:
        B.mtp_set_chunk_debug()
    mine = slice(int(c.cu[skip]), int(c.cu[skip + 1]))
    assert torch.isnan(out[mine]).all() and torch.isnan(lse[mine]).all()
    gone = torch.isnan(lse)
    assert torch.equal(torch.isnan(out).any(-1), gone) and torch.equal(torch.isnan(out).all(-1), gone)
    assert torch.equal(out[~gone], clean[0][~gone]) and torch.equal(lse[~gone], clean[1][~gone])
    again = c.run(window)
    assert all(torch.equal(a, b) for a, b in zip(again, clean))
    return gone.any(-1)


@gpu
@pytest.mark.parametrize("skip", [0, 1, 3, 5])
@pytest.mark.parametrize("d,n_head,own_v", [(128, 4, False), (128, 4, True), (256, 4, False), (512, 4, False), (512, 4, True)])
def test_waits_that_run_out_leave_nan(d, n_head, own_v, skip):
    """Few rows and many, in units of one CTA and in units that cross CTAs."""
    L = [300, 5000, 40, 20000, 100, 64]
    for new in ([5, 7, 1, 8, 3, 5], [200, 70, 40, 90, 33, 64]):
        _given_up(Case(d, L, new, 64, n_head, 1, d, own_v=own_v), skip)


@gpu
@pytest.mark.parametrize("d", [128, 256, 512])
def test_waits_that_run_out_reach_the_rows_of_their_own_ctas(d):
    n = 700
    rs = np.random.RandomState(d)
    c = Case(d, rs.randint(20, 400, n), np.full(n, 6), 16, 4, 1, d)
    gone = _given_up(c, 350, window=100).cpu().reshape(n, 6).any(1)
    assert gone[350] and int(gone.sum()) <= 40
    assert int(gone.nonzero().max() - gone.nonzero().min()) <= 40


@gpu
@pytest.mark.parametrize("Bn", [2, 31, 32, 33, 65])
@pytest.mark.parametrize("d", [128, 256])
def test_batches_around_a_warp_s_lanes(Bn, d):
    rs = np.random.RandomState(Bn)
    L = rs.randint(1, 500, Bn)
    Case(Bn + d, L, np.minimum(rs.randint(0, 40, Bn), L), 16, 4, 1, d).check(window=90)


@gpu
@pytest.mark.parametrize("d,own_v", [(512, False), (256, False), (128, True)])
def test_other_tokens_queries_neither_move_a_row_nor_slow_it_down(d, own_v):
    """Sequences of 5 tokens of 4 heads: the other 12 columns of a tile of 32 hold the next tokens' queries,
    here of sequences without a key. Large ones cost no more than zeros (when they counted among the scores
    that move references, 11 to 18 % more), and the rows' bits are the same."""
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, paged_attention_chunk
    Bn, L, P = 16, 16384, 64
    g = torch.Generator(device="cuda").manual_seed(d)
    k = torch.randn((Bn * L // P, P, 1, d), generator=g, device="cuda").bfloat16()
    v = torch.randn(k.shape, generator=g, device="cuda").bfloat16() if own_v else None
    table = torch.full((2 * Bn, L // P), -1, dtype=torch.int32, device="cuda")
    table[::2] = torch.randperm(Bn * L // P, generator=g, device="cuda").int().view(Bn, -1)
    kv = PagedKV(k, table, torch.tensor([L, 0] * Bn, dtype=torch.int32, device="cuda"), v=v)
    cu = torch.tensor(np.concatenate([[0], np.cumsum([5, 3] * Bn)]), dtype=torch.int32, device="cuda")
    q = torch.randn((Bn, 8, 4, d), generator=g, device="cuda").bfloat16()
    calm, loud = q.clone(), q.clone()
    calm[:, 5:], loud[:, 5:] = 0, q[:, 5:] * 30
    calm, loud = calm.view(8 * Bn, 4, d), loud.view(8 * Bn, 4, d)
    out = torch.empty_like(calm)

    def least(x):
        times = []
        for _ in range(40):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            paged_attention_chunk(x, kv, cu, out=out)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert torch.equal(paged_attention_chunk(calm, kv, cu), paged_attention_chunk(loud, kv, cu))
    ratios = []
    for _ in range(6):  # (the first that shows no difference will do)
        ratios.append(least(loud) / least(calm))
        if ratios[-1] < 1.06:
            return
    assert False, ratios


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (64, "bf16"), (200, "f32"), (128, "bf16"), (256, "bf16"), (512, "bf16")])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("n", [3, 150])
def test_a_value_that_is_not_finite_reaches_rows_of_no_weight_for_it(d, dtype, what, n):
    """Key 60 scores so low that its weight is 0 in fp32: its value is attended all the same, by the rows from
    token 60 on (in a window of 100, up to token 159)."""
    c = Case(5, [200], [n], 16, 4, 1, d, dtype, own_v=True)
    c.q = torch.ones_like(c.q)
    c.k = torch.where(torch.isnan(c.k), c.k, 0 * c.k)
    c.k[c.table[0, 3], 12] = -300.0
    c.dk, c.dq = c.k.cuda(), c.q.cuda()
    clean = {w: c.run(w)[0] for w in (0, 100)}
    c.dv[c.table[0, 3], 12, :, 3] = what
    for w in (0, 100):
        out = c.run(w)[0]
        for i in range(n):
            pos = 200 - n + i
            if pos >= 60 and (not w or pos < 160):
                assert not torch.isfinite(out[i]).all(-1).any()
            else:
                assert torch.equal(out[i], clean[w][i])


@gpu
def test_the_most_heads():
    """1024 KV heads of 1024 query heads each, which is more than a grid has rows of 16."""
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, paged_attention_chunk
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((2, 1, 1024, 8), generator=g, device="cuda").bfloat16()
    table, lens = torch.ones((32, 1), dtype=torch.int32, device="cuda"), torch.ones(32, dtype=torch.int32, device="cuda")
    q = torch.randn((1, 1 << 20, 8), generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0] * 8 + [1] * 25, dtype=torch.int32, device="cuda")
    out = paged_attention_chunk(q, PagedKV(k, table, lens), cu)
    assert torch.equal(out.view(1024, 1024, 8), k[1, 0][:, None].expand(1024, 1024, 8))


@gpu
@pytest.mark.parametrize("scale", [1.0, 0.03])
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (64, "bf16"), (512, "f32"), (128, "bf16"), (256, "bf16"), (512, "bf16")])
@pytest.mark.parametrize("new", [[5, 1, 7], [200, 1, 90]])
def test_a_scale_of_the_caller_s(new, d, dtype, scale):
    """Scores of the size that the default scale gives N(0, 1) queries, or smaller, so that the errors are no
    larger either."""
    c = Case(d, [3000, 40, 700], new, 16, 4, 1, d, dtype, own_v=d == 128, q_by=d ** -0.5 if scale == 1.0 else 1.0)
    c.check(scale=scale)
    c.check(window=100, scale=scale)


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (512, "bf16")])
def test_tens_of_thousands_of_short_and_empty_sequences(d, dtype):
    """40000 sequences of at most one page of 16 tokens, of which up to 3 are new and mostly none."""
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV, paged_attention_chunk
    Bn, P, dt = 40000, 16, torch.bfloat16 if dtype == "bf16" else torch.float32
    rs = np.random.RandomState(d)
    L = rs.randint(0, P + 1, Bn).astype(np.int32)
    new = np.minimum(np.where(rs.uniform(size=Bn) < 0.3, rs.randint(1, 4, Bn), 0), L)
    new[:2000], new[-2000:] = 0, 0
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(d)
    k = torch.randn((Bn, P, 1, d), generator=g, device="cuda").to(dt)
    table = torch.randperm(Bn, generator=g, device="cuda").int()[:, None]
    q = torch.randn((int(cu[-1]), 2, d), generator=g, device="cuda").to(dt)
    out, lse = paged_attention_chunk(q, PagedKV(k, table, _dev(L)), _dev(cu), want_lse=True)
    seq = np.repeat(np.arange(Bn), new)
    pos = L[seq] - new[seq] + np.arange(len(seq)) - cu[seq]
    keys = k[table[_dev(seq).long(), 0].long(), :, 0].double()
    x = torch.einsum("thd,tjd->thj", q.double(), keys) * d ** -0.5
    x = x.masked_fill((torch.arange(P, device="cuda") > _dev(pos)[:, None])[:, None], float("-inf"))
    p = torch.softmax(x, -1)
    want, mean = torch.einsum("thj,tjd->thd", p, keys), torch.einsum("thj,tjd->thd", p, keys.abs())
    most = TOL + (HALF * (want.abs() + mean * (1 + HALF)) if dtype == "bf16" else 0)
    assert ((out.double() - want).abs() <= most).all()
    assert ((lse.double() - torch.logsumexp(x, -1)).abs() <= TOL).all()
