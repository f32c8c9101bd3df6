"""Draft blocks over paged caches against the oracle and against the draft block over one tensor."""
import ctypes
from dataclasses import replace

import numpy as np
import pytest
import torch

import oracle as O
from mtp_speculative_decoding_gemma4_gb300 import binding as B
from mtp_speculative_decoding_gemma4_gb300 import build as build_mod
from mtp_synth import configs as C
from mtp_synth import gen as G

from _util import TOL, compare_block, config_data, inputs_to_device, oracle_block, weights_to_device

gpu = pytest.mark.gpu


def _paged(k, ctx_len, P, seed, spare=2, **more):
    """A right-padded K [B][Lmax][n_kv][d] (device) as a PagedKV with random pages."""
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV
    L = np.asarray(ctx_len)
    Bn, Lmax, n_kv, d = k.shape
    cols = -(-Lmax // P)
    need = -(-L // P)
    perm = np.random.RandomState(seed).permutation(int(need.sum()) + spare)
    cache = torch.full((len(perm), P, n_kv, d), float("nan"), dtype=k.dtype, device=k.device)
    table = np.full((Bn, cols), -1, np.int32)
    at = 0
    for b in range(Bn):
        pages = perm[at:at + need[b]]
        table[b, :need[b]] = pages
        at += need[b]
        rows = torch.full((need[b] * P, n_kv, d), float("nan"), dtype=k.dtype, device=k.device)
        rows[:L[b]] = k[b, :L[b]]
        cache[torch.from_numpy(pages.astype(np.int64)).cuda()] = rows.view(-1, P, n_kv, d)
    return PagedKV(cache, torch.from_numpy(table).cuda(), torch.from_numpy(L.astype(np.int32)).cuda(), **more), table


def _drafter(shape, w, max_batch, max_ctx):
    from mtp_speculative_decoding_gemma4_gb300 import Drafter
    wd, tgt = weights_to_device(w)
    return Drafter(shape, wd, tgt, max_batch=max_batch, max_ctx=max_ctx)


def _run(dr, d, kv_s, kv_f, n, **kw):
    tok, hid = dr.draft_block_paged(d["hidden"], d["last_token"], kv_s, kv_f, d["pos"], n, **kw)
    torch.cuda.synchronize()
    assert dr.status() == 0
    return tok.cpu().numpy(), None if hid is None else hid.cpu().numpy()


@gpu
@pytest.mark.parametrize("path", [0, 1, 5])
@pytest.mark.parametrize("dtype,d,n_head,n_kv,P,max_batch", [
    ("f32", 32, 2, 1, 16, 5), ("bf16", 64, 4, 2, 8, 5), ("bf16", 128, 8, 1, 16, 5), ("bf16", 256, 4, 1, 64, 1)])
def test_paged_block_matches_the_oracle(dtype, d, n_head, n_kv, P, max_batch, path):
    if path == 5 and (dtype == "f32" or max_batch == 1):
        pytest.skip("the tensor-core path serves bf16 batches")
    shape = replace(C.TINY_F32, dtype=dtype, layer_types=("S", "F", "S"), window=24, n_head=n_head, n_kv_head=n_kv,
                    head_dim_swa=d, head_dim_full=d)
    L = np.array([1, 24, 25, 200, 131], np.int32)[-max_batch:]
    wl = C.Workload(batch=len(L), ctx=200, n_draft=3)
    w = G.make_weights(shape, 7 + d)
    inp = G.make_step_inputs(shape, wl, 7 + d, ctx_len=L)
    ref = O.draft_block(O.Shape.of(shape), O.decode_weights(w), inp.hidden, inp.last_token, inp.k_swa, inp.k_full,
                        inp.ctx_len, inp.pos, 3)
    dr = _drafter(shape, w, max_batch, 200)
    dr.set_path(path)
    dd = inputs_to_device(inp, dtype)
    kv_s, _ = _paged(dd["k_swa"], L, P, 1)
    kv_f, _ = _paged(dd["k_full"], L, P, 2)
    for _ in range(2):  # the second call replays the first one's graph
        tok, hid = _run(dr, dd, kv_s, kv_f, 3)
        compare_block(tok, hid, ref, dtype)
    tok2, none = _run(dr, dd, kv_s, kv_f, 3, want_hidden=False)
    assert none is None and np.array_equal(tok2, tok)
    dr.close()


@gpu
@pytest.mark.parametrize("index,P", [(2, 64), (3, 32), (4, 16)])
def test_paged_block_matches_the_block_over_one_tensor(index, P):
    # the benchmark shapes at their sizes: same tokens up to near ties, hidden states within the
    # tolerance of the precision contract
    shape, wl, w, inp = config_data(index)
    dr = _drafter(shape, w, wl.batch, wl.ctx)
    d = inputs_to_device(inp, shape.dtype)
    a, ha = dr.draft_block(d["hidden"], d["last_token"], d["k_swa"], d["k_full"], d["ctx_len"], d["pos"], 2)
    a, ha = a.cpu().numpy(), ha.cpu().numpy()
    kv_s, _ = _paged(d["k_swa"], inp.ctx_len, P, 1)
    kv_f, _ = _paged(d["k_full"], inp.ctx_len, P, 2)
    b, hb = _run(dr, d, kv_s, kv_f, 2)
    assert np.max(np.abs(ha[:, 0] - hb[:, 0])) <= TOL[shape.dtype]
    assert np.mean(a == b) >= 0.98
    dr.close()


@gpu
@pytest.mark.parametrize("dtype,d,path", [("bf16", 128, 5), ("bf16", 128, 1), ("f32", 32, 1), ("bf16", 512, 5)])
def test_selected_pages_match_the_oracle_over_those_keys(dtype, d, path):
    # summaries that decide the selection whatever the query: pages of scale NaN are always
    # selected, every other page scores 0, so the lowest of them fill up
    P, L, k = 16, np.array([16 * 20 + 5, 16 * 9, 33], np.int32), 6
    shape = replace(C.TINY_F32, dtype=dtype, layer_types=("F", "F"), n_head=4, n_kv_head=1, head_dim_swa=d,
                    head_dim_full=d)
    wl = C.Workload(batch=3, ctx=400, n_draft=2)
    w = G.make_weights(shape, 3)
    inp = G.make_step_inputs(shape, wl, 3, ctx_len=L)
    dd = inputs_to_device(inp, dtype)
    kv, table = _paged(dd["k_full"], L, P, 5)
    n = kv.k.shape[0]
    scales = np.ones((n, 1), np.float32)
    always = {0: [7, 12, 19], 1: [3, 4, 5], 2: []}
    for b, pages in always.items():
        scales[table[b, pages]] = np.nan
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV
    kv = PagedKV(kv.k, kv.block_table, kv.ctx_len, codes=torch.zeros((n, 1, d), dtype=torch.int8).cuda(),
                 scales=torch.from_numpy(scales).cuda())
    dr = _drafter(shape, w, 3, 400)
    dr.set_path(path)
    tok, hid = _run(dr, dd, None, kv, 2, n_select=k, keep_first=1, keep_last=2)
    ref_L, ref_k = L.copy(), inp.k_full.copy()
    for b in range(3):
        m = -(-L[b] // P)
        picked = sorted({0, m - 1, m - 2} | set(always[b])) if m > k else list(range(m))
        rest = [p for p in range(m) if p not in picked]
        picked = sorted(picked + rest[:max(0, min(k, m) - len(picked))])
        rows = np.concatenate([inp.k_full[b, p * P:min(p * P + P, L[b])] for p in picked])
        ref_L[b] = len(rows)
        ref_k[b, :len(rows)] = rows
    ref = O.draft_block(O.Shape.of(shape), O.decode_weights(w), inp.hidden, inp.last_token, None, ref_k, ref_L, inp.pos, 2)
    compare_block(tok, hid, ref, dtype)
    # every page: the plain block
    full = O.draft_block(O.Shape.of(shape), O.decode_weights(w), inp.hidden, inp.last_token, None, inp.k_full, L,
                         inp.pos, 2)
    for n_select in (0, 25):
        tok, hid = _run(dr, dd, None, kv, 2, n_select=n_select)
        compare_block(tok, hid, full, dtype)
    dr.close()


@gpu
def test_paged_block_follows_its_buffers_and_refuses_other_shapes():
    shape = replace(C.TINY_F32, dtype="bf16", layer_types=("F",), n_head=4, n_kv_head=1, head_dim_swa=128,
                    head_dim_full=128)
    L = np.array([90, 40], np.int32)
    wl = C.Workload(batch=2, ctx=100, n_draft=1)
    w = G.make_weights(shape, 9)
    inp = G.make_step_inputs(shape, wl, 9, ctx_len=L)
    dd = inputs_to_device(inp, "bf16")
    dr = _drafter(shape, w, 2, 100)
    kv, _ = _paged(dd["k_full"], L, 16, 1)
    for lens in ([90, 40], [17, 33], [64, 1]):  # a cache whose lengths change between calls
        kv.ctx_len.copy_(torch.tensor(lens, dtype=torch.int32))
        ref = O.draft_block(O.Shape.of(shape), O.decode_weights(w), inp.hidden, inp.last_token, None, inp.k_full,
                            np.array(lens, np.int32), inp.pos, 1)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        tok, hid = dr.draft_block_paged(dd["hidden"], dd["last_token"], None, kv, dd["pos"], 1, stream=st.cuda_stream)
        st.synchronize()
        compare_block(tok.cpu().numpy(), hid.cpu().numpy(), ref, "bf16")
    other, _ = _paged(torch.zeros((2, 100, 1, 64), dtype=torch.bfloat16, device="cuda"), L, 16, 1)
    for bad in (dict(kv_full=other), dict(kv_full=None), dict(n_select=4), dict(n_draft=0)):
        a = dict(kv_full=kv, n_select=0, n_draft=1)
        a.update(bad)
        with pytest.raises(B.MtpError):
            dr.draft_block_paged(dd["hidden"], dd["last_token"], None, a["kv_full"], dd["pos"], a["n_draft"],
                                 n_select=a["n_select"])
    with pytest.raises(ValueError):
        dr.draft_block_paged(dd["hidden"][:1], dd["last_token"], None, kv, dd["pos"], 1)
    for path in (2, 7):
        dr.set_path(path)
        with pytest.raises(B.MtpError):
            dr.draft_block_paged(dd["hidden"], dd["last_token"], None, kv, dd["pos"], 1)
    dr.close()


def test_null_arguments_are_refused_without_a_device():
    build_mod.build()
    lib = B.load_library()
    n = ctypes.c_int64()
    assert lib.mtp_draft_block_paged(None, None, None, None, None, None, 1, 1, 0, 0, 1, None, None, None, 0,
                                     None) == B.MTP_ERR_INVALID_ARG
    assert lib.mtp_draft_block_paged_workspace(None, None, None, 1, 0, ctypes.byref(n)) == B.MTP_ERR_INVALID_ARG
    assert B.mtp_last_error()


@gpu
def test_one_sequence_of_a_batched_drafter():
    # B = 1 on a handle made for more takes the tensor-core phases
    shape = replace(C.TINY_F32, dtype="bf16", layer_types=("S", "F"), window=24, n_head=4, n_kv_head=1, head_dim_swa=128,
                    head_dim_full=256)
    L = np.array([77], np.int32)
    w = G.make_weights(shape, 21)
    inp = G.make_step_inputs(shape, C.Workload(batch=1, ctx=80, n_draft=3), 21, ctx_len=L)
    ref = O.draft_block(O.Shape.of(shape), O.decode_weights(w), inp.hidden, inp.last_token, inp.k_swa, inp.k_full, L,
                        inp.pos, 3)
    dr = _drafter(shape, w, 4, 80)
    dd = inputs_to_device(inp, "bf16")
    kv_s, _ = _paged(dd["k_swa"], L, 32, 1)
    kv_f, _ = _paged(dd["k_full"], L, 16, 2)
    for path in (0, 5, 1):
        dr.set_path(path)
        compare_block(*_run(dr, dd, kv_s, kv_f, 3), ref, "bf16")
    dr.close()


@gpu
def test_paged_block_checks_its_tensors():
    shape = replace(C.TINY_F32, dtype="bf16", layer_types=("F",), n_head=4, n_kv_head=1, head_dim_swa=128,
                    head_dim_full=128)
    L = np.array([90, 40], np.int32)
    w = G.make_weights(shape, 9)
    inp = G.make_step_inputs(shape, C.Workload(batch=2, ctx=100, n_draft=1), 9, ctx_len=L)
    dd = inputs_to_device(inp, "bf16")
    dr = _drafter(shape, w, 2, 100)
    kv, _ = _paged(dd["k_full"], L, 16, 1)
    good = dict(hidden=dd["hidden"], last_token=dd["last_token"], pos=dd["pos"], out_tokens=None, out_hidden=None)
    for bad in (dict(hidden=dd["hidden"].float()), dict(hidden=dd["hidden"].cpu()), dict(hidden=dd["hidden"][:, 8:]),
                dict(last_token=dd["last_token"].long()), dict(pos=dd["pos"][:1]), dict(pos=dd["pos"].cpu()),
                dict(out_tokens=torch.empty((2, 2), dtype=torch.int32, device="cuda")),
                dict(out_hidden=torch.empty((2, 1, shape.backbone), dtype=torch.bfloat16, device="cuda"))):
        a = {**good, **bad}
        with pytest.raises(ValueError):
            dr.draft_block_paged(a["hidden"], a["last_token"], None, kv, a["pos"], 1, out_tokens=a["out_tokens"],
                                 out_hidden=a["out_hidden"])
    dr.close()


@gpu
@pytest.mark.parametrize("cols,layers", [(16, "SF"), (1024, "SF"), (1024, "FS")])
def test_attention_timeout_is_reported_and_the_handle_recovers(cols, layers):
    # failure detection without a fault: the first layer's tensor-core attention looks up no page of
    # sequence 0, the waits for its keys give up after ~10 ms of cycles, the sequence's outputs are
    # NaN, the status word reads MTP_ERR_TIMEOUT, and the next call matches the oracle (path 1 has
    # no other waits). A full layer first and 1024 columns: keys dealt over the SMs; else a cluster
    # per sequence
    P, L = 16, np.array([200, 131, 77], np.int32)
    shape = replace(C.TINY_F32, dtype="bf16", layer_types=tuple(layers), window=24, n_head=4, n_kv_head=1,
                    head_dim_swa=128, head_dim_full=128)
    wl = C.Workload(batch=3, ctx=200, n_draft=2)
    w = G.make_weights(shape, 5)
    inp = G.make_step_inputs(shape, wl, 5, ctx_len=L)
    ref = O.draft_block(O.Shape.of(shape), O.decode_weights(w), inp.hidden, inp.last_token, inp.k_swa, inp.k_full,
                        inp.ctx_len, inp.pos, 2)
    dd = inputs_to_device(inp, "bf16")
    from mtp_speculative_decoding_gemma4_gb300 import PagedKV

    def wide(k, seed):
        kv, table = _paged(k, L, P, seed)
        t = np.full((3, cols), -1, np.int32)
        t[:, :min(cols, table.shape[1])] = table[:, :cols]
        return PagedKV(kv.k, torch.from_numpy(t).cuda(), kv.ctx_len)

    kv_s, kv_f = wide(dd["k_swa"], 1), wide(dd["k_full"], 2)
    dr = _drafter(shape, w, 3, 200)
    dr.set_path(1)
    dr.set_debug(skip_arrival_cta=0, spin_limit_cycles=20_000_000)
    tok, hid = dr.draft_block_paged(dd["hidden"], dd["last_token"], kv_s, kv_f, dd["pos"], 2)
    torch.cuda.synchronize()
    assert torch.isnan(hid[0, 0]).all()
    assert dr.status() == B.MTP_ERR_TIMEOUT
    assert dr.status() == B.MTP_OK
    dr.set_debug()
    tok, hid = _run(dr, dd, kv_s, kv_f, 2)
    compare_block(tok, hid, ref, "bf16")
    dr.close()


@gpu
@pytest.mark.parametrize("index,P,batch", [(2, 64, 0), (3, 32, 6), (4, 16, 9)])
def test_paged_block_of_the_benchmark_shapes_matches_the_oracle(index, P, batch):
    # tokens may differ only where the oracle's own margin is a near tie
    shape, wl, w, inp = config_data(index, batch)
    ref = oracle_block(index, n_draft=2, batch=batch)
    dr = _drafter(shape, w, wl.batch, wl.ctx)
    d = inputs_to_device(inp, shape.dtype)
    kv_s, _ = _paged(d["k_swa"], inp.ctx_len, P, 1)
    kv_f, _ = _paged(d["k_full"], inp.ctx_len, P, 2)
    tok, hid = _run(dr, d, kv_s, kv_f, 2)
    cmp = compare_block(tok, hid, ref, shape.dtype)
    assert len(cmp.tie_divergences) <= max(1, cmp.steps_compared // 50)
    dr.close()
