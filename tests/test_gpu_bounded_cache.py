"""The bounded paged cache as it is used: multi-axis positions, chunked prompts
and generated tokens under a window plus sinks, with pages granted, forked,
trimmed and compacted on the way; the whole step in a CUDA graph; calls on
several streams; offsets past 32 bits."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from hybrid_local_global_b200 import native, synth

from sinks_ref import attend64, attention_bound, axes64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def ok():
    assert native.gemma_attn_sync_status() == 0, native.gemma_last_error()


class Rows:
    """What the device should hold: every row's keys and values, from its first token on."""

    def __init__(self, n):
        self.k = [[] for _ in range(n)]
        self.v = [[] for _ in range(n)]

    def fork(self, parents):
        self.k = [list(self.k[p]) for p in parents]
        self.v = [list(self.v[p]) for p in parents]


@pytest.mark.parametrize("D,Hq,Hkv,window,sinks", [(512, 8, 1, 150, 6), (256, 4, 2, 128, 0), (256, 6, 2, 90, 140)])
def test_multimodal_beams_on_a_bounded_cache(D, Hq, Hkv, window, sinks):
    n, ps, pps, n_pages = 4, 128, 12, 40
    pairs, theta, scale = [D // 32, D // 16, D // 16], 1e6, D ** -0.5
    rng, gen = np.random.default_rng(D + window), synth.generator(D)
    book = native.PageBook(n, pps, n_pages, ps, DEV)
    pools = [torch.full((n_pages, Hkv, ps, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    lacking, n_live = i32([0]), i32([0])
    lens, rows = [0] * n, Rows(n)

    def positions(count):  # text and image coordinates, one triple per token
        return torch.tensor(rng.integers(0, 3000, (3, n, count)), dtype=torch.int32)

    def new_tokens(count):
        """count tokens for every row: grant pages, rotate, attend; checks the outputs."""
        native.gemma_kv_pages_reserve(book, pools, seq_lens=i32(lens), new_tokens=i32([count] * n), lacking=lacking)
        q, k, v = (synth.randn_bf16((n, count, h, D), gen) for h in (Hq, Hkv, Hkv))
        pos = positions(count)
        qd, kd = q.to(DEV), k.to(DEV)
        native.gemma_rope_axes(qd, kd, pos.to(DEV), axis_pairs=pairs, rope_theta=theta, q_out=qd, k_out=kd,
                               flags=native.GEMMA_ROPE_INTERLEAVED)
        out = torch.empty_like(qd)
        kw = dict(window=window, sinks=sinks, rope_frac=0.0, rope_theta=theta, scale=scale)
        if count == 1:
            native.gemma_attn_decode_sinks(qd[:, 0], kd[:, 0], v[:, 0].to(DEV), *pools, book.page_table, out=out[:, 0],
                                           seq_lens=i32([x + 1 for x in lens]), max_seq_len=pps * ps, **kw)
        else:
            native.gemma_attn_prefill_sinks(qd, kd, v.to(DEV), *pools, book.page_table, out=out,
                                            seq_lens_before=i32(lens), **kw)
        ok()
        assert lacking.item() == 0
        for b in range(n):
            at = pos[:, b]
            kr, qr = kd[b].cpu(), qd[b].cpu()
            for got, x in ((kr, k[b]), (qr, q[b])):
                want = axes64(x, at, pairs, theta, interleaved=True)
                # half a bf16 step, and 2^-20 of the pair for the 32-bit rotation
                assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * 8).all()
            rows.k[b] += list(kr)
            rows.v[b] += list(v[b])
            ref, _ = attend64(qr, torch.stack(rows.k[b]), torch.stack(rows.v[b]), list(range(lens[b], lens[b] + count)),
                              window, sinks, scale)
            got = out[b].double().cpu()
            assert torch.isfinite(got).all()
            assert (got - ref).abs().max() <= attention_bound(ref, float(v.abs().max()) + 3.0)
            lens[b] += count

    def trim_and_compact():
        native.gemma_kv_pages_trim(book, seq_lens=i32(lens), window=window, sinks=sinks)
        native.gemma_kv_pages_compact(book, pools, n_live=n_live)
        ok()
        held = book.page_table[book.page_table >= 0]
        assert n_live.item() == held.unique().numel() and int(held.max()) < n_live.item()
        per_row = math.ceil(sinks / ps) + math.ceil(window / ps) + 1
        assert (book.page_table >= 0).sum(1).max().item() <= per_row
        for p in pools:  # nothing may be read from the pages that were given back
            p[n_live.item():] = float("nan")

    for step, count in enumerate((200, 131, 1, 1, 67, 1, 140, 1, 1)):
        new_tokens(count)
        if step % 2 == 0:
            trim_and_compact()
        if step in (1, 2, 5, 7):
            parents = [int(x) for x in rng.integers(0, n, n)]
            native.gemma_kv_pages_fork(book, i32(parents))
            rows.fork(parents)
            lens = [lens[p] for p in parents]
    native.gemma_kv_pages_trim(book, seq_lens=i32([0] * n))
    ok()
    assert (book.page_table == -1).all() and (book.ref_count == 0).all()


def test_captured_generation_step():
    """Reserve, attend, advance and trim as one graph that follows the device's
    lengths; an idle slot; the same tokens without a graph give the same bits."""
    n, ps, pps, n_pages, Hq, Hkv, D, window, sinks = 3, 128, 8, 20, 8, 1, 512, 140, 5
    gen = synth.generator(3)
    steps = 150
    qs, ks, vs = (synth.randn_bf16((steps, n, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
    q, k, v = (torch.empty_like(t[0]) for t in (qs, ks, vs))
    out = torch.empty_like(q)
    kw = dict(window=window, sinks=sinks, rope_frac=0.25, rope_theta=1e6, scale=D ** -0.5, max_seq_len=pps * ps)

    def fresh():
        book = native.PageBook(n, pps, n_pages, ps, DEV)
        pools = [torch.zeros(n_pages, Hkv, ps, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        return book, pools, i32([0, 100, 0]), i32([1, 1, 0]), i32([0])  # row 1 starts inside a page, row 2 idles

    def step(book, pools, lens, new, lacking, ws):
        native.gemma_kv_pages_reserve(book, pools, seq_lens=lens, new_tokens=new, lacking=lacking, workspace=ws)
        lens += new
        native.gemma_attn_decode_sinks(q, k, v, *pools, book.page_table, seq_lens=lens, out=out, **kw)
        native.gemma_kv_pages_trim(book, seq_lens=lens, window=window, sinks=sinks)

    ws = torch.empty(native.gemma_kv_pages_workspace_size(n, pps, n_pages), dtype=torch.uint8, device=DEV)
    plain, state = [], fresh()
    for s in range(steps):
        q.copy_(qs[s]), k.copy_(ks[s]), v.copy_(vs[s])
        step(*state, ws)
        plain.append(out.clone())
    ok()
    state = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*state, ws)
    for s in range(steps):
        q.copy_(qs[s]), k.copy_(ks[s]), v.copy_(vs[s])
        graph.replay()
        assert torch.equal(out.view(torch.int16), plain[s].view(torch.int16)), s
    ok()
    assert (out[2] == 0).all() and state[2].tolist() == [steps, 100 + steps, 0]
    assert (state[0].page_table >= 0).sum().item() <= 2 * 4


FIRST_CALL = """
import torch
from hybrid_local_global_b200 import native
torch.zeros(1, device="cuda")
D, what = 256, %r
bf = dict(dtype=torch.bfloat16, device="cuda")
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
q, k = torch.ones(1, 1, 4, D, **bf), torch.ones(1, 1, 2, D, **bf)
out, pools = torch.zeros_like(q), [torch.zeros(4, 2, 128, D, **bf) for _ in range(2)]
book = native.PageBook(1, 4, 4, 128, "cuda")
book.page_table[0, 0], book.ref_count[0] = 0, 1
lens, one, lacking = i32([1]), i32([1]), i32([0])
POS = i32([[[0]]])
ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
kw = dict(window=8, sinks=1, rope_frac=1.0, rope_theta=1e4, scale=0.1, workspace=ws)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    if what == "decode":
        native.gemma_attn_decode_sinks(q[:, 0], k[:, 0], k[:, 0], *pools, book.page_table, seq_lens=one, max_seq_len=512,
                                       out=out[:, 0], **kw)
    elif what == "prefill":
        native.gemma_attn_prefill_sinks(q, k, k, *pools, book.page_table, out=out, **kw)
    elif what == "rope":
        native.gemma_rope_axes(q, k, POS, axis_pairs=[16], rope_theta=1e4, q_out=out, k_out=k)
    else:
        native.gemma_kv_pages_reserve(book, pools, seq_lens=lens, new_tokens=one, lacking=lacking, workspace=ws)
        native.gemma_kv_pages_compact(book, pools, n_live=lacking, workspace=ws)
        out.fill_(1)
g.replay()
assert native.gemma_attn_sync_status() == 0
assert (out == 1).all(), out
"""


@pytest.mark.parametrize("what", ["decode", "prefill", "rope", "pages"])
def test_first_call_of_a_process_may_be_captured(what):
    subprocess.run([sys.executable, "-c", FIRST_CALL % what], check=True, timeout=240,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_graphs_that_share_a_workspace_and_profiling():
    """Two prompts' graphs on one workspace, replayed in turn; the same calls
    with the library's launch events between the kernels."""
    gen = synth.generator(12)
    ws, jobs = torch.empty(64 << 20, dtype=torch.uint8, device=DEV), []
    for D, Hq, Hkv, S in ((256, 16, 8, 700), (512, 8, 1, 60), (512, 16, 8, 300)):
        pools = [torch.zeros(12, Hkv, 128, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        q, k, v = (synth.randn_bf16((1, S, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
        out, table = torch.empty_like(q), torch.randperm(12)[None, :8].int().to(DEV)

        def call(q=q, k=k, v=v, pools=pools, out=out, table=table, D=D):
            native.gemma_attn_prefill_sinks(q, k, v, *pools, table, out=out, window=140, sinks=6, rope_frac=0.25,
                                            rope_theta=1e6, scale=D ** -0.5, workspace=ws)

        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
            call()
        jobs.append((call, graph, out, out.clone()))
    for _ in range(3):
        for _, graph, out, _ in jobs:
            out.zero_()
            graph.replay()
    ok()
    for _, _, out, want in jobs:
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    native.gemma_attn_profile(True)
    try:
        for call, _, out, want in jobs:
            out.zero_()
            call()
            ok()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    finally:
        native.gemma_attn_profile(False)


def test_calls_on_several_streams_at_once():
    """Independent sequences decoded on four streams, many calls in flight."""
    gen = synth.generator(8)
    D, Hq, Hkv, ps, n = 256, 4, 2, 128, 4
    jobs = []
    for s in range(n):
        pools = [synth.randn_bf16((9, Hkv, ps, D), gen).to(DEV) for _ in range(2)]
        q, k, v = (synth.randn_bf16((2, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
        table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4) + s % 2
        jobs.append((q, k, v, *pools, table))
    kw = dict(max_seq_len=512, window=200, sinks=7, rope_frac=1.0, rope_theta=1e4, scale=0.06)
    lens = [i32([200 + 30 * s, 400 + s]) for s in range(n)]
    want = []
    for job, ln in zip(jobs, lens):
        o = torch.empty_like(job[0])
        native.gemma_attn_decode_sinks(*job, seq_lens=ln, out=o, **kw)
        want.append(o)
    ok()
    streams = [torch.cuda.Stream() for _ in range(n)]
    outs = [[torch.empty_like(j[0]) for _ in range(20)] for j in jobs]
    for i in range(20):
        for s, st in enumerate(streams):
            native.gemma_attn_decode_sinks(*jobs[s], seq_lens=lens[s], out=outs[s][i], stream=st, **kw)
    torch.cuda.synchronize()
    ok()
    for s in range(n):
        for o in outs[s]:
            assert torch.equal(o.view(torch.int16), want[s].view(torch.int16))


def test_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 of the pool: the same rows in low
    pages give the same bits."""
    D, Hkv, Hq, ps, n_pages = 512, 4, 8, 128, 8400  # 8400 pages of 2^18 elements
    gen = synth.generator(5)
    pools = [torch.zeros(n_pages, Hkv, ps, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    rows = [synth.randn_bf16((3, Hkv, ps, D), gen).to(DEV) for _ in range(2)]
    for p, r in zip(pools, rows):
        p[8395:8398] = r
    native.gemma_kv_pages_copy(pools, src=i32([8395, 8396, 8397]), dst=i32([2, 0, 8399]))
    ok()
    for p, r in zip(pools, rows):
        assert torch.equal(p[2], r[0]) and torch.equal(p[0], r[1]) and torch.equal(p[8399], r[2])
        p[1] = r[2]
    kw = dict(window=250, sinks=20, rope_frac=0.25, rope_theta=1e6, scale=D ** -0.5)
    q, k, v = (synth.randn_bf16((1, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
    outs = []
    for table in ([[8395, 8396, 8397]], [[2, 0, 1]]):
        o = torch.empty_like(q)
        native.gemma_attn_decode_sinks(q, k, v, *pools, i32(table), seq_lens=i32([333]), max_seq_len=384, out=o, **kw)
        outs.append(o)
    ok()
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16)) and outs[0].abs().sum() > 0
    for p in pools:
        assert torch.equal(p[8397, :, 76], p[1, :, 76])
    for S in (5, 45):
        q, k, v = (synth.randn_bf16((1, S, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
        outs = []
        for table in ([[8395, 8396, 8397]], [[2, 0, 1]]):
            o = torch.empty_like(q)
            native.gemma_attn_prefill_sinks(q, k, v, *pools, i32(table), seq_lens_before=i32([333]), out=o, **kw)
            outs.append(o)
        ok()
        assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16)) and outs[0].abs().sum() > 0
    book = native.PageBook(2, 3, n_pages, ps, DEV)
    book.page_table[0] = i32([8395, 8396, 8397])
    book.page_table[1] = i32([8395, 8396, 8397])
    book.ref_count[8395:8398] = 2
    book.ref_count[:1000] = 1  # in use elsewhere
    lacking = i32([0])
    native.gemma_kv_pages_reserve(book, pools, seq_lens=i32([300, 300]), new_tokens=i32([1, 1]), lacking=lacking)
    ok()
    assert book.page_table[0].tolist() == [8395, 8396, 1000]
    for p in pools:
        assert torch.equal(p[1000, :, :44], p[8397, :, :44])


def test_rotation_of_many_tokens():
    """More than 2^31 bytes of vectors, the last token checked."""
    tokens, H, D = 70001, 32, 512
    x = torch.zeros(tokens, H, D, dtype=torch.bfloat16, device=DEV)
    x[-1] = synth.randn_bf16((H, D), synth.generator(2)).to(DEV)
    pos = torch.arange(2 * tokens, dtype=torch.int32, device=DEV).view(2, tokens)
    last = x[-1].cpu().clone()
    native.gemma_rope_axes(x, None, pos, axis_pairs=[100, 28], rope_theta=1e6, q_out=x)
    ok()
    want = axes64(last[None], pos[:, -1:].cpu(), [100, 28], 1e6)[0]
    assert ((x[-1].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18).all()
    assert (x[:-1] == 0).all()
