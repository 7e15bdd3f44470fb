"""Window-plus-sinks attention on a paged cache (gemma_attn_prefill_sinks,
gemma_attn_decode_sinks) against its plain 64-bit form."""
import math

import numpy as np
import pytest
import torch

from hybrid_local_global_b200 import native, synth

from sinks_ref import attend64, attention_bound, kept_pages, rope64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bf16(x):
    return x.to(torch.bfloat16)


def make_cache(lens, held, Hkv, D, ps, pps, seed, keqv=False, poison=float("nan")):
    """Contiguous K and V [B][cap][Hkv][D] (already rotated keys) and the same
    rows in a pool whose other pages and rows hold `poison`. held[b]: page
    numbers that sequence b has."""
    rng = np.random.default_rng(seed)
    gen = synth.generator(seed)
    B, cap = len(lens), pps * ps
    K = synth.randn_bf16((B, cap, Hkv, D), gen)
    V = K.clone() if keqv else synth.randn_bf16((B, cap, Hkv, D), gen)
    n_pages = sum(len(h) for h in held) + 3
    ids = list(rng.permutation(n_pages))
    table = torch.full((B, pps), -1, dtype=torch.int32)
    kp = torch.full((n_pages, Hkv, ps, D), poison, dtype=torch.bfloat16)
    vp = kp.clone()
    for b in range(B):
        for i in held[b]:
            table[b, i] = int(ids.pop())
            n = min(ps, max(0, lens[b] - i * ps))
            kp[table[b, i], :, :n] = K[b, i * ps:i * ps + n].transpose(0, 1)
            vp[table[b, i], :, :n] = V[b, i * ps:i * ps + n].transpose(0, 1)
    return K, V, kp, vp, table


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


DECODE = [
    # lens (with the new token; 0 idle), window, sinks, Hq, Hkv, D, page size
    dict(lens=[1, 2, 0, 33, 600], window=64, sinks=4, Hq=8, Hkv=1, D=512, ps=128),
    dict(lens=[129, 700, 128], window=100, sinks=0, Hq=4, Hkv=2, D=256, ps=128),
    dict(lens=[1000], window=1, sinks=1, Hq=3, Hkv=1, D=512, ps=256),
    dict(lens=[1000, 517], window=1, sinks=0, Hq=7, Hkv=1, D=256, ps=128),
    dict(lens=[900, 301, 300], window=37, sinks=300, Hq=16, Hkv=2, D=256, ps=128),
    dict(lens=[2500], window=1024, sinks=16, Hq=32, Hkv=4, D=512, ps=128),
    dict(lens=[50, 1300, 4097, 0], window=1000, sinks=129, Hq=4, Hkv=4, D=256, ps=384),
    dict(lens=[300], window=1 << 30, sinks=5, Hq=2, Hkv=1, D=512, ps=128),
    dict(lens=[300, 20], window=40, sinks=1 << 30, Hq=2, Hkv=2, D=256, ps=128),
]


def run_decode(lens, window, sinks, Hq, Hkv, D, ps, seed=11, keqv=False, shared=False, frac=0.25, theta=1e6,
               poison_unseen=True, stream=None):
    B, pps = len(lens), max(lens) // ps + 2
    held = [sorted(kept_pages(n - 1, window, sinks, ps) | {(n - 1) // ps}) if n else [] for n in lens]
    cached = [n if shared else n - 1 for n in lens]
    K, V, kp, vp, table = make_cache(cached, held, Hkv, D, ps, pps, seed, keqv)
    gen = synth.generator(seed + 1)
    q = synth.randn_bf16((B, Hq, D), gen)
    kn, vn = synth.randn_bf16((B, Hkv, D), gen), synth.randn_bf16((B, Hkv, D), gen)
    if poison_unseen:  # rows of held pages that the token does not see
        for b, n in enumerate(lens):
            for i in held[b]:
                for r in range(ps):
                    j = i * ps + r
                    if j < n - 1 and not (j > n - 1 - window or j < sinks):
                        kp[table[b, i], :, r] = vp[table[b, i], :, r] = float("inf")
    kd, vd = kp.to(DEV), vp.to(DEV)
    out = torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    scale = D ** -0.5
    flags = (native.GEMMA_F_SHARED if shared else 0) | (native.GEMMA_F_KEQV if keqv else 0)
    native.gemma_attn_decode_sinks(
        q.to(DEV), None if shared else kn.to(DEV), None if shared or keqv else vn.to(DEV), kd, None if keqv else vd,
        table.to(DEV), seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), max_seq_len=max(max(lens), 1),
        window=window, sinks=sinks, rope_frac=frac, rope_theta=theta, scale=scale, out=out, flags=flags, stream=stream)
    assert native.gemma_attn_sync_status(stream) == 0, native.gemma_last_error()
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()
            continue
        if not shared:
            K[b, n - 1] = bf16(rope64(kn[b:b + 1], [n - 1], frac, theta)[0])
            V[b, n - 1] = K[b, n - 1] if keqv else vn[b]
            page, row = table[b, (n - 1) // ps], (n - 1) % ps
            got = kd[page, :, row].cpu()
            # one bf16 step of the exact rotation: a value next to a border may round either way
            assert (got.double() - K[b, n - 1].double()).abs().max() <= 2 * 2.0 ** -8 * K[b, n - 1].abs().max()
            K[b, n - 1] = got
            kp[page, :, row] = got
            if keqv:
                V[b, n - 1] = got
            else:
                assert same_bits(vd[page, :, row].cpu(), vn[b])
                vp[page, :, row] = vn[b]
        qr = bf16(rope64(q[b:b + 1], [n - 1], frac, theta))
        ref, _ = attend64(qr, K[b], V[b], [n - 1], window, sinks, scale)
        got = out[b].double().cpu()
        assert torch.isfinite(got).all(), (b, n)
        err = (got - ref[0]).abs().max()
        assert err <= attention_bound(ref, float(V[b, :n].abs().max())), (b, n, float(err))
    assert same_bits(kd.cpu(), kp)  # nothing else was written
    assert same_bits(vd.cpu(), vp)


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "%s-w%d-s%d-d%d" % (c["lens"], c["window"], c["sinks"], c["D"]))
def test_decode(case):
    run_decode(**case)


@pytest.mark.parametrize("keqv,shared", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("D", [256, 512])
def test_decode_keqv_and_shared(D, keqv, shared):
    run_decode(lens=[1, 47, 48, 49, 640], window=48, sinks=20, Hq=8, Hkv=2, D=D, ps=128, keqv=keqv, shared=shared,
               frac=1.0, theta=1e4)


@pytest.mark.parametrize("B,Hkv,window", [(1, 1, 4000), (2, 1, 700), (8, 4, 300), (40, 4, 200), (75, 4, 130)])
def test_decode_every_split_count(B, Hkv, window):
    """Batches small to large: clusters of 8 CTAs down to single ones."""
    lens = [window + 150 + 7 * b for b in range(B)]
    run_decode(lens=lens, window=window, sinks=40, Hq=2 * Hkv, Hkv=Hkv, D=512, ps=128)


@pytest.mark.parametrize("window", [14, 33, 60, 100, 127])
@pytest.mark.parametrize("sinks,D,Hkv,B", [(0, 512, 1, 1), (0, 256, 2, 2), (9, 256, 2, 3), (9, 256, 16, 24), (0, 512, 4, 80)])
def test_decode_small_window_across_a_tile_boundary(window, sinks, D, Hkv, B):
    """The window begins in one tile and ends in the next, less than 128
    positions on, in one CTA (many sequences) or two."""
    lens = [(134, 777, 129, 256 + window // 2, 391, 640 + window - 1)[b % 6] + 128 * (b // 6) for b in range(B)]
    run_decode(lens=lens, window=window, sinks=sinks, Hq=2 * Hkv, Hkv=Hkv, D=D, ps=128)


def test_decode_equals_global_paged_decode_when_everything_is_visible():
    lens, Hq, Hkv, D, ps = [700, 31], 8, 1, 512, 128
    held = [list(range(6)), [0]]
    K, V, kp, vp, table = make_cache([n - 1 for n in lens], held, Hkv, D, ps, 6, 5, poison=0.0)
    gen = synth.generator(6)
    q, kn, vn = (synth.randn_bf16((2, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
    kw = dict(seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), max_seq_len=700, rope_frac=0.25,
              rope_theta=1e6, scale=D ** -0.5)
    a, b = torch.empty_like(q), torch.empty_like(q)
    ka, va, kb, vb = kp.to(DEV), vp.to(DEV), kp.to(DEV), vp.to(DEV)
    t = table.clamp(min=0).to(DEV)
    native.gemma_attn_decode_sinks(q, kn, vn, ka, va, t, window=700, sinks=0, out=a, **kw)
    native.gemma_attn_decode_paged(q, kn, vn, kb, vb, t, out=b, **kw)
    assert native.gemma_attn_sync_status() == 0
    assert same_bits(ka, kb) and same_bits(va, vb)
    # both round their weights and outputs to bf16, the splits differ
    assert (a.double() - b.double()).abs().max() <= 2 * attention_bound(b.double(), float(va.abs().max()))


def test_decode_reports_bad_lengths_and_pages():
    lens, Hq, Hkv, D, ps = [200, 900, -3, 150], 2, 1, 256, 128
    held = [[0, 1], [0, 1, 2, 3], [0], [0, 1]]
    K, V, kp, vp, table = make_cache([199, 500, 1, 149], held, Hkv, D, ps, 8, 9, poison=0.0)
    table[3, 1] = kp.shape[0]  # the page of the new token and of visible keys lies outside the pool
    q = synth.randn_bf16((4, Hq, D), synth.generator(1)).to(DEV)
    kn = synth.randn_bf16((4, Hkv, D), synth.generator(2)).to(DEV)
    kd, vd, out = kp.to(DEV), vp.to(DEV), torch.full_like(q, float("nan"))
    native.gemma_attn_decode_sinks(q, kn, kn, kd, vd, table.to(DEV),
                                   seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), max_seq_len=300,
                                   window=50, sinks=3, rope_frac=1.0, rope_theta=1e4, scale=0.06, out=out)
    assert native.gemma_attn_sync_status() == native.GEMMA_ERR_DEVICE_RANGE
    assert (out[1] == 0).all() and (out[2] == 0).all() and torch.isfinite(out[0]).all()
    changed = (kd.cpu() != kp).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(table[0, 1])]  # only the good sequence's row was written


def test_decode_timeout_is_reported():
    """The first copy never comes: the waits run out, the call reports it and the next one works."""
    native.gemma_attn_set_wait_limit(2_000_000)
    native.gemma_attn_debug_drop_next_copy(True)
    try:
        with pytest.raises(AssertionError):
            run_decode(lens=[600], window=300, sinks=4, Hq=8, Hkv=1, D=512, ps=128)
        assert native.gemma_attn_sync_status() == 0
    finally:
        native.gemma_attn_set_wait_limit(0)
        native.gemma_attn_debug_timeout_info()
    run_decode(lens=[600], window=300, sinks=4, Hq=8, Hkv=1, D=512, ps=128)


def test_decode_on_another_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run_decode(lens=[300, 77], window=64, sinks=4, Hq=8, Hkv=1, D=512, ps=128, stream=s)


PREFILL = [
    # before (per sequence; None: no lengths given), new, window, sinks, Hq, Hkv, D, page size
    dict(before=None, S=1, window=1, sinks=0, Hq=2, Hkv=1, D=256, ps=128),
    dict(before=None, S=300, window=64, sinks=4, Hq=4, Hkv=2, D=256, ps=128),
    dict(before=[0, 130], S=257, window=100, sinks=130, Hq=2, Hkv=1, D=512, ps=128),
    dict(before=[1000], S=1, window=200, sinks=5, Hq=8, Hkv=1, D=512, ps=256),
    dict(before=[777, 64], S=130, window=333, sinks=16, Hq=3, Hkv=1, D=512, ps=128),
    dict(before=[900, 5], S=140, window=1, sinks=1, Hq=8, Hkv=1, D=512, ps=128),
    dict(before=[511], S=70, window=128, sinks=300, Hq=3, Hkv=3, D=256, ps=384),
    dict(before=[640], S=65, window=256, sinks=0, Hq=4, Hkv=1, D=512, ps=128),
    dict(before=[400], S=33, window=1 << 30, sinks=1 << 30, Hq=2, Hkv=1, D=256, ps=128),
]


def run_prefill(before, S, window, sinks, Hq, Hkv, D, ps, seed=21, keqv=False, shared=False, frac=0.25, theta=1e6,
                scale=None):
    lens = before or [0, 0]
    B, pps = len(lens), (max(lens) + S) // ps + 2
    held = [sorted(kept_pages(n, window, sinks, ps) | set(range(n // ps, (n + S - 1) // ps + 1))) for n in lens]
    cached = [n + S if shared else n for n in lens]
    K, V, kp, vp, table = make_cache(cached, held, Hkv, D, ps, pps, seed, keqv)
    gen = synth.generator(seed + 1)
    q = synth.randn_bf16((B, S, Hq, D), gen)
    kn, vn = synth.randn_bf16((B, S, Hkv, D), gen), synth.randn_bf16((B, S, Hkv, D), gen)
    kd, vd = kp.to(DEV), vp.to(DEV)
    out = torch.full((B, S, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(B, Hq, S, dtype=torch.float32, device=DEV)
    scale = D ** -0.5 if scale is None else scale
    flags = (native.GEMMA_F_SHARED if shared else 0) | (native.GEMMA_F_KEQV if keqv else 0)
    native.gemma_attn_prefill_sinks(
        q.to(DEV), None if shared else kn.to(DEV), None if shared or keqv else vn.to(DEV), kd, None if keqv else vd,
        table.to(DEV), window=window, sinks=sinks, rope_frac=frac, rope_theta=theta, scale=scale, out=out, lse=lse,
        seq_lens_before=None if before is None else torch.tensor(before, dtype=torch.int32, device=DEV), flags=flags)
    assert native.gemma_attn_sync_status() == 0, native.gemma_last_error()
    for b, n in enumerate(lens):
        pos = list(range(n, n + S))
        if not shared:
            exact = rope64(kn[b], pos, frac, theta)
            for i, j in enumerate(pos):
                page, row = table[b, j // ps], j % ps
                got = kd[page, :, row].cpu()
                assert (got.double() - exact[i]).abs().max() <= 2.0 ** -8 * 1.01 * exact[i].abs().max()
                K[b, j] = kp[page, :, row] = got
                V[b, j] = got if keqv else vn[b, i]
                if not keqv:
                    vp[page, :, row] = vn[b, i]
        # the queries are rounded once, as they are up to a power of two
        qr = bf16(rope64(q[b], pos, frac, theta))
        ref, ref_lse = attend64(qr, K[b], V[b], pos, window, sinks, scale)
        got = out[b].double().cpu()
        assert torch.isfinite(got).all()
        err = (got - ref).abs().max()
        assert err <= attention_bound(ref, float(V[b, :n + S].abs().max())), (b, float(err))
        # 32-bit sums of up to n + S terms and the logits' 32-bit accumulation
        assert (lse[b].double().cpu().T - ref_lse).abs().max() <= 1e-4 * (1 + float(ref_lse.abs().max()))
    assert same_bits(kd.cpu(), kp) and same_bits(vd.cpu(), vp)


# enough rows that the keys are not split over a cluster: the unsplit kernels
PREFILL += [
    dict(before=[300, 17], S=130, window=150, sinks=9, Hq=16, Hkv=8, D=512, ps=128),   # head pairs
    dict(before=[0, 260], S=129, window=70, sinks=140, Hq=8, Hkv=8, D=512, ps=128),    # one head per CTA
    dict(before=[513, 100], S=200, window=128, sinks=1, Hq=16, Hkv=16, D=256, ps=256),
    dict(before=[90, 600], S=190, window=300, sinks=0, Hq=48, Hkv=16, D=256, ps=128),
    # head_dim 256, several row tiles per CTA pair: pairs of heads, of row tiles (an odd number of
    # them), few and many key tiles each
    dict(before=[0, 130, 777], S=700, window=200, sinks=20, Hq=16, Hkv=8, D=256, ps=128),
    dict(before=None, S=1300, window=1, sinks=0, Hq=16, Hkv=8, D=256, ps=128),
    dict(before=[5, 300, 0, 128], S=600, window=130, sinks=140, Hq=9, Hkv=9, D=256, ps=256),
    dict(before=[40, 3], S=300, window=90, sinks=3, Hq=40, Hkv=8, D=256, ps=128),
    dict(before=[64, 700], S=300, window=256, sinks=33, Hq=16, Hkv=8, D=512, ps=128),
    dict(before=[11], S=300, window=100, sinks=2, Hq=15, Hkv=5, D=512, ps=128),
]


@pytest.mark.parametrize("case", PREFILL, ids=lambda c: "%s+%d-w%d-s%d-d%d" % (c["before"], c["S"], c["window"],
                                                                               c["sinks"], c["D"]))
def test_prefill(case):
    run_prefill(**case)


@pytest.mark.parametrize("keqv,shared", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("D", [256, 512])
def test_prefill_keqv_and_shared(D, keqv, shared):
    run_prefill([300, 0], 60, window=90, sinks=7, Hq=4, Hkv=1, D=D, ps=128, keqv=keqv, shared=shared, frac=1.0, theta=1e4)


@pytest.mark.parametrize("G", range(1, 9))
def test_prefill_every_group_size(G):
    """Short chunks pack 128 / G tokens x G heads into a tile."""
    run_prefill([200, 31], 150 // G + 3, window=80, sinks=5, Hq=2 * G, Hkv=2, D=256 if G % 2 else 512, ps=128)


@pytest.mark.parametrize("scale", [0.0, -0.03, 0.5, 2.0 ** -6, 1e-30])
@pytest.mark.parametrize("D", [256, 512])
def test_prefill_scales(D, scale):
    run_prefill([100], 40, window=60, sinks=3, Hq=4, Hkv=1, D=D, ps=128, scale=scale)
    run_prefill([100, 0], 130, window=60, sinks=3, Hq=16, Hkv=16, D=D, ps=128, scale=scale)


def test_prefill_of_no_tokens_does_nothing():
    q = torch.empty(2, 0, 4, 256, dtype=torch.bfloat16, device=DEV)
    kv = torch.empty(2, 0, 2, 256, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(1, 2, 128, 256, dtype=torch.bfloat16, device=DEV)
    table = torch.full((2, 1), -1, dtype=torch.int32, device=DEV)
    native.gemma_attn_prefill_sinks(q, kv, kv, pool, pool.clone(), table, window=4, sinks=1, rope_frac=1.0,
                                    rope_theta=1e4, scale=1.0, out=torch.empty_like(q))
    assert native.gemma_attn_sync_status() == 0


def test_prefill_reports_pages_outside_the_pool():
    q = synth.randn_bf16((1, 40, 2, 256), synth.generator(3)).to(DEV)
    pool = torch.zeros(2, 2, 128, 256, dtype=torch.bfloat16, device=DEV)
    for bad in (-1, 2):
        table = torch.tensor([[bad]], dtype=torch.int32, device=DEV)
        native.gemma_attn_prefill_sinks(q, q, q, pool, pool.clone(), table, window=16, sinks=4, rope_frac=1.0,
                                        rope_theta=1e4, scale=0.1, out=torch.empty_like(q))
        assert native.gemma_attn_sync_status() == native.GEMMA_ERR_DEVICE_RANGE
        assert (pool == 0).all()


@pytest.mark.parametrize("D,Hq,Hkv,S", [(256, 16, 8, 700), (256, 2, 1, 40), (512, 16, 8, 300), (512, 5, 5, 500),
                                        (256, 9, 9, 400)])
def test_prefill_leaves_out_sequences_without_room(D, Hq, Hkv, S):
    """Lengths that the table has no room for are reported; the others' rows
    are what they are alone, and the outputs of the bad ones stay as they were."""
    gen = synth.generator(41)
    pps = (S + 200) // 128 + 1
    q, k, v = (synth.randn_bf16((4, S, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
    kw = dict(window=150, sinks=5, rope_frac=0.25, rope_theta=1e6, scale=D ** -0.5)
    table = torch.arange(4 * pps, dtype=torch.int32, device=DEV).view(4, pps)

    def run(lens):
        pools = [torch.zeros(4 * pps, Hkv, 128, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        out = torch.full_like(q, 7.0)
        native.gemma_attn_prefill_sinks(q, k, v, *pools, table, out=out,
                                        seq_lens_before=torch.tensor(lens, dtype=torch.int32, device=DEV), **kw)
        return out, pools, native.gemma_attn_sync_status()

    good, pa, status = run([3, 0, 100, 1])
    assert status == 0
    some, pb, status = run([3, -1, 100, pps * 128 - S + 1])
    assert status == native.GEMMA_ERR_DEVICE_RANGE
    for b in (0, 2):
        assert same_bits(some[b], good[b])
    for b in (1, 3):
        assert (some[b] == 7).all() and all((p[b * pps:(b + 1) * pps] == 0).all() for p in pb)
    none, pc, status = run([-1, -5, 1 << 30, pps * 128])
    assert status == native.GEMMA_ERR_DEVICE_RANGE
    assert (none == 7).all() and all((p == 0).all() for p in pc)
    again, pd, status = run([3, 0, 100, 1])
    assert status == 0 and same_bits(again, good)


def test_chunks_and_steps_agree():
    """A prompt in one call, in chunks, and its last tokens one at a time give the same rows."""
    B, S, Hq, Hkv, D, ps, window, sinks = 1, 333, 8, 1, 512, 128, 96, 9
    gen = synth.generator(31)
    q, k, v = (synth.randn_bf16((B, S, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    kw = dict(window=window, sinks=sinks, rope_frac=0.25, rope_theta=1e6, scale=D ** -0.5)

    def pools():
        return [torch.zeros(3, Hkv, ps, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    whole, pa = torch.empty_like(q), pools()
    native.gemma_attn_prefill_sinks(q, k, v, *pa, table, out=whole, **kw)
    parts, pb, at = torch.empty_like(q), pools(), 0
    for n in (1, 127, 2, 130, 50):
        o = torch.empty(B, n, Hq, D, dtype=torch.bfloat16, device=DEV)
        native.gemma_attn_prefill_sinks(*(t[:, at:at + n].contiguous() for t in (q, k, v)), *pb, table, out=o,
                                        seq_lens_before=torch.tensor([at], dtype=torch.int32, device=DEV), **kw)
        parts[:, at:at + n] = o
        at += n
    for at in range(at, S):
        o = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV)
        native.gemma_attn_decode_sinks(*(t[:, at].contiguous() for t in (q, k, v)), *pb, table, out=o,
                                       seq_lens=torch.tensor([at + 1], dtype=torch.int32, device=DEV),
                                       max_seq_len=S, **kw)
        parts[:, at] = o
    assert native.gemma_attn_sync_status() == 0
    assert same_bits(pa[0], pb[0]) and same_bits(pa[1], pb[1])
    # chunked rows see the same tiles in another order; steps round q before the scale
    assert (whole.double() - parts.double()).abs().max() <= 2 * attention_bound(whole.double(), float(v.abs().max()))
