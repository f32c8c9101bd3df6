"""Log probabilities of given tokens, entropies and top alternatives against a plain form in 64
bits; refusals without a device."""
import ctypes
import math

import numpy as np
import pytest
import torch

from mtp_speculative_decoding_gemma4_gb300 import binding as B
from mtp_speculative_decoding_gemma4_gb300 import build as build_mod

gpu = pytest.mark.gpu

U = torch.finfo(torch.float32).eps / 2  # 2^-24, half a step relative to a value


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


FAKE = 1 << 20  # an aligned address that is never used: validation fails first


@pytest.mark.parametrize("args", [
    dict(logits=None), dict(logits=FAKE + 1), dict(token=None), dict(token=FAKE + 2), dict(ids=None), dict(best=None),
    dict(best=FAKE + 2), dict(dtype=2), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(V=0), dict(V=(1 << 30) + 1),
    dict(k=-1), dict(k=33), dict(V=8, k=9), dict(stride=99999), dict(stride=1 << 41), dict(T=0.0), dict(T=-1.0),
    dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-38), dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=100),
    dict(logprob=None, entropy=None, k=0), dict(entropy=FAKE + 2)])
def test_bad_arguments_are_refused_before_the_device(lib, args):
    a = dict(logits=FAKE, dtype=0, stride=100000, token=FAKE, rows=3, V=100000, T=1.0, k=5, logprob=FAKE, entropy=FAKE,
             ids=FAKE, best=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(args)
    assert lib.mtp_token_logprobs(a["logits"], a["dtype"], a["stride"], a["token"], a["rows"], a["V"], a["T"], a["k"],
                                  a["logprob"], a["entropy"], a["ids"], a["best"], a["ws"], a["ws_bytes"],
                                  None) == B.MTP_ERR_INVALID_ARG
    assert B.mtp_last_error()


def test_the_workspace_call(lib):
    n = ctypes.c_int64(-1)
    assert lib.mtp_token_logprobs_workspace(0, 0, 100, 5, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.mtp_token_logprobs_workspace(0, 1, 262144, 5, ctypes.byref(n)) == 0 and n.value > 0
    for bad in ((2, 1, 10, 0), (0, -1, 10, 0), (0, 1, 0, 0), (0, 1, 10, 33)):
        assert lib.mtp_token_logprobs_workspace(*bad, ctypes.byref(n)) == B.MTP_ERR_INVALID_ARG
    assert lib.mtp_token_logprobs_workspace(0, 1, 10, 1, None) == B.MTP_ERR_INVALID_ARG
    # no rows: nothing is launched, so no device is needed either
    assert lib.mtp_token_logprobs(None, 0, 0, None, 0, 10, 1.0, 0, None, None, None, None, None, 0, None) == 0


# ---------------------------------------------------------------- against 64 bits


def _check(logits, tokens, temperature=1.0, k=0, stream=None):
    from mtp_speculative_decoding_gemma4_gb300 import token_logprobs
    got = [x.cpu() for x in token_logprobs(logits, tokens, temperature=temperature, top_k=k, stream=stream)]
    V = logits.shape[-1]
    x = logits.cpu().double().reshape(-1, V) / temperature
    raw = logits.cpu().double().reshape(-1, V)
    t = tokens.cpu().long().reshape(-1)
    lp, ent = got[0].reshape(-1), got[1].reshape(-1)
    some = ~(torch.isnan(x).any(-1) | (x == math.inf).any(-1) | (x == -math.inf).all(-1))
    logp = torch.log_softmax(torch.where(some[:, None], x, 0.0), -1)
    # S is a sum of at most V / 512 + 64 positive terms one after the other, each addition off by half
    # a step (an exponential by two steps); an exponent d = (x - m) c by 3 half steps of itself, which
    # the terms of the entropy and the logprob carry as well
    n = V / 512 + 64
    H = -(logp.exp() * torch.where(logp > -math.inf, logp, 0.0)).sum(-1)
    off = (ent.double() - H).abs()
    assert torch.isnan(ent[~some]).all() and (off <= U * ((n + 4) * (2 * H + 1) + 8 * (H + 4)))[some].all(), float(off[some].max())
    inside = (t >= 0) & (t < V)
    want = torch.gather(logp, 1, t.clamp(0, V - 1)[:, None])[:, 0]
    assert torch.isnan(lp[~(some & inside)]).all()
    ok = some & inside
    fine = ok & torch.isfinite(want)
    assert torch.equal(lp[ok & ~fine].double(), want[ok & ~fine])
    # d is (x - m) c, whose size is that of the logprob and of log2 S together
    assert ((lp.double() - want).abs() <= U * (n + 6 * (want.abs() + math.log(V) + 4)))[fine].all()
    if k:
        ids, best = got[2].reshape(-1, k).long(), got[3].reshape(-1, k)
        order = torch.sort(raw, dim=-1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(ids[some], order[some])
        assert (ids[~some] == -1).all() and torch.isnan(best[~some]).all()
        w = torch.gather(logp, 1, order)[some]
        b = best[some].double()
        fin = torch.isfinite(w)
        assert torch.equal(b[~fin], w[~fin])
        assert ((b - w).abs() <= U * (n + 6 * (w.abs() + math.log(V) + 4)))[fin].all()
    return got


def _case(rows, V, dtype, seed=0, by=3.0, skip=0, offset=0):
    g = torch.Generator().manual_seed(seed + rows + V)
    wide = torch.randn((rows, V + skip), generator=g).mul_(by).to(dtype)
    flat = torch.empty(wide.numel() + offset, dtype=dtype, device="cuda")
    flat[offset:] = wide.reshape(-1).cuda()
    logits = flat[offset:].view(rows, V + skip)[:, :V]
    return logits, torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 32, 50, 1000, 4096, 4097, 16384, 16385, 50257, 262144])
@pytest.mark.parametrize("rows", [1, 5, 33])
def test_matches_the_plain_form(rows, V, dtype):
    _check(*_case(rows, V, dtype), k=min(V, 20))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("skip,offset", [(0, 1), (3, 0), (5, 3), (8, 8), (1, 7)])
@pytest.mark.parametrize("rows,V", [(4, 999), (700, 1003), (3, 40001)])
def test_strides_and_alignments(rows, V, skip, offset, dtype):
    """Rows that begin anywhere in a 16-byte vector, between others whose values are all larger."""
    logits, tokens = _case(rows, V, dtype, skip=skip, offset=offset)
    logits._base.view(-1)[:offset] = 1e4
    if skip:
        torch.as_strided(logits, (rows, skip), (V + skip, 1), logits.storage_offset() + V).fill_(1e4)
    _check(logits, tokens, k=9)


@gpu
@pytest.mark.parametrize("k", [0, 1, 2, 31, 32])
@pytest.mark.parametrize("temperature", [0.05, 0.7, 1.0, 30.0])
def test_temperatures_and_counts(k, temperature):
    for rows, V in ((3, 30000), (640, 5000)):
        _check(*_case(rows, V, torch.bfloat16), temperature=temperature, k=k)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V", [(2, 40000), (400, 20000)])
@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "rising", "falling", "one thread", "lowest", "masked", "mostly masked", "all but 3"])
def test_ties_orders_and_masks(kind, rows, V, dtype):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((rows, V), generator=g) * 3
    i = torch.arange(V)
    lowest = torch.finfo(dtype).min
    if kind == "equal":
        x = torch.full_like(x, -2.5)
    elif kind == "few":  # hundreds of equal values at the top
        x = torch.randint(-2, 3, (rows, V), generator=g).float()
    elif kind == "zeros":  # of both signs, which are equal
        x = torch.where(x > 0, 0.0, torch.where(x > -3, -0.0, x))
    elif kind == "rising":
        x = (i * (60.0 / V) - 30).expand(rows, V).clone()
    elif kind == "falling":
        x = (30 - i * (60.0 / V)).expand(rows, V).clone()
    elif kind == "one thread":  # the largest all in vectors that one thread reads
        x[:, (i // 8) % 256 == 77] += 20
    elif kind == "lowest":
        x = torch.full_like(x, lowest)
        x[0, 17:30] = lowest / 2
    elif kind == "masked":
        x[:, torch.rand(V, generator=g) < 0.5] = -math.inf
        x[:, torch.rand(V, generator=g) < 0.3] = lowest
    elif kind == "mostly masked":
        x = torch.full_like(x, -math.inf)
        x[:, V // 2::V // 6] = 1.0
    elif kind == "all but 3":
        x = torch.full_like(x, lowest)
        x[:, [5, V - 1, V // 2]] = 2.0
    _check(x.to(dtype).cuda(), torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda(), k=20)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40, 100000])
def test_rows_without_a_softmax_and_tokens_out_of_range(V, dtype):
    logits, tokens = _case(8, V, dtype)
    logits[1, V // 2] = float("nan")
    logits[2, V - 1] = math.inf
    logits[3] = -math.inf
    logits[4] = float("nan")
    tokens[5], tokens[6], tokens[7] = -1, V, 2 ** 31 - 1
    _check(logits, tokens, k=6)


@gpu
def test_shapes_streams_and_graphs():
    from mtp_speculative_decoding_gemma4_gb300 import token_logprobs
    g = torch.Generator().manual_seed(1)
    logits = torch.randn((4, 6, 3000), generator=g).cuda()
    tokens = torch.randint(0, 3000, (4, 6), generator=g, dtype=torch.int32).cuda()
    got = _check(logits, tokens, k=4)
    assert [tuple(x.shape) for x in got] == [(4, 6), (4, 6), (4, 6, 4), (4, 6, 4)]
    one = _check(logits[0, 0], tokens[0, 0], k=2)
    assert one[0].shape == () and one[2].shape == (2,)
    assert token_logprobs(logits[:0], tokens[:0])[0].shape == (0, 6)
    big = torch.randn((3, 200000), generator=g).cuda()
    t3 = tokens[0, :3].contiguous()
    want = [x.clone() for x in token_logprobs(big, t3, top_k=8)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    many = [token_logprobs(big, t3, top_k=8, stream=s[i % 2].cuda_stream) for i in range(6)]
    torch.cuda.synchronize()
    for m in many:
        assert all(torch.equal(a, b) for a, b in zip(m, want))
    x = torch.zeros_like(big)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token_logprobs(x, t3, top_k=8)
    for _ in range(2):
        x.copy_(big)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        x.zero_()
        graph.replay()
    with pytest.raises(ValueError):
        token_logprobs(big.half(), t3)
    with pytest.raises(ValueError):
        token_logprobs(big, t3.long())
    with pytest.raises(ValueError):
        token_logprobs(big, t3[:2])
    with pytest.raises(ValueError):
        token_logprobs(big.t(), t3)
    with pytest.raises(ValueError):
        token_logprobs(big, t3.cpu())
    with pytest.raises(B.MtpError):
        token_logprobs(big, t3, top_k=40)
    with pytest.raises(B.MtpError):
        token_logprobs(big, t3, temperature=0.0)


@gpu
def test_a_call_without_a_token(lib):
    logits, tokens = _case(3, 5000, torch.bfloat16)
    out = torch.empty(2, 3, device="cuda")
    assert lib.mtp_token_logprobs(logits.data_ptr(), 0, 5000, None, 3, 5000, 1.0, 0, None, out[1].data_ptr(), None, None,
                                  torch.empty(4096, device="cuda").data_ptr(), 16384, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(out[1].cpu(), _check(logits, tokens)[1])


@gpu
def test_after_a_verified_block():
    """The emitted tokens of a greedy verification have the rows' largest probability where the target
    replaced a draft, and -1 behind them."""
    from mtp_speculative_decoding_gemma4_gb300 import token_logprobs, verify_greedy
    g = torch.Generator().manual_seed(5)
    logits = torch.randn((6, 5, 4096), generator=g).bfloat16().cuda()
    best = logits.float().argmax(-1).int()
    drafts = best[:, :4].clone()
    drafts[1, 0] += 1
    drafts[3, 2] = 7
    n, out = verify_greedy(logits, drafts.contiguous())
    lp, _, ids, top = token_logprobs(logits, out, top_k=1)
    for b in range(6):
        m = int(n[b])
        assert torch.equal(lp[b, :m + 1], top[b, :m + 1, 0]) and torch.isnan(lp[b, m + 1:]).all()
    assert torch.equal(ids[..., 0], best)


@gpu
@pytest.mark.parametrize("k", [5, 20, 32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lists_that_fill_between_meetings(dtype, k):
    """Rows of many chunks, of which about 3 k elements enter the list between two meetings, so that what
    it holds lies near the count from which on it is sorted: the same bits at every call, and the right ones."""
    from mtp_speculative_decoding_gemma4_gb300 import token_logprobs
    logits, tokens = _case(640, 150001, dtype)
    want = _check(logits, tokens, k=k)
    for _ in range(8):
        got = token_logprobs(logits, tokens, top_k=k)
        assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V", [(400, 60000), (96, 262144), (700, 50257)])
@pytest.mark.parametrize("kind", ["first masked", "first lower", "rising", "two steps"])
def test_lists_that_overfill_long_before_the_end(kind, rows, V, dtype):
    """Logits of which more exceed the best of the first ids than the list holds, in slices that go on
    for several chunks behind the meeting that finds it out: every chunk enters the sums all the same."""
    g = torch.Generator().manual_seed(7)
    x = torch.randn((rows, V), generator=g) * 2
    i = torch.arange(V)
    if kind == "first masked":
        x[:, :8192] = -math.inf
    elif kind == "first lower":
        x[:, :8192] -= 10
    elif kind == "rising":
        x = (i * (60.0 / V) - 30).expand(rows, V).clone()
    elif kind == "two steps":  # a second time behind a later meeting
        x += 10 * ((i >= 8192).float() + (i >= 8192 * 5).float())
    tokens = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32)
    tokens[:2] = torch.tensor([V - 1, 0])
    _check(x.to(dtype).cuda(), tokens.cuda(), k=20)


@gpu
@pytest.mark.parametrize("V", [40, 70000])
@pytest.mark.parametrize("temperature", [2.0, 7.0, 1e30])
def test_differences_beyond_the_type_s_range(V, temperature):
    """Logits farther apart than fp32's largest value, whose log probabilities at the temperature are not."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn((3, V), generator=g)
    x[0, 3], x[0, 5] = 3e38, -3e38
    x[1] = torch.finfo(torch.float32).min
    x[1, :3] = torch.tensor([3e38, 3e38, -math.inf])
    x[2, 7], x[2, 9] = 2e38, -2e38
    _check(x.cuda(), torch.tensor([5, 30, 9], dtype=torch.int32).cuda(), temperature=temperature, k=20)
