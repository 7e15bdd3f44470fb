"""NaN and infinities in what a query sees (window-plus-sinks attention): the
softmax of a logit that is no number is no number, so a head whose query or
visible keys hold one comes out as NaN, never as plausible zeros, and every
other head and token is, bit for bit, what it is without."""
import math

import pytest
import torch

from hybrid_local_global_b200 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
KW = dict(rope_frac=0.25, rope_theta=1e6)


def bits(t):
    return t.contiguous().view(torch.int16)


def cache(B, pps, Hkv, D, seed):
    gen = synth.generator(seed)
    pools = [synth.randn_bf16((B * pps, Hkv, 128, D), gen).to(DEV) for _ in range(2)]
    table = torch.randperm(B * pps, generator=torch.Generator().manual_seed(seed)).int().view(B, pps).to(DEV)
    return pools, table


def check(got, clean, hit, v_absmax=None):
    """hit: mask of the rows [..., heads] that must be NaN; the others as in
    `clean`, bit for bit, or (v_absmax given) as close as 32-bit sums taken
    against another running maximum come."""
    assert torch.isfinite(clean).all()
    assert torch.isnan(got[hit]).all(), torch.nonzero(~torch.isnan(got).all(-1) & hit)[:4].tolist()
    a, b = got[~hit], clean[~hit]
    if v_absmax is None:
        assert torch.equal(bits(a), bits(b))
    else:
        assert ((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + 2.0 ** -13 * v_absmax).all()


# sequences, q heads, KV heads, dim, window: clusters of several CTAs and single ones, groups of 1 to 8
DECODE = [(1, 8, 1, 512, 700), (1, 8, 1, 256, 300), (2, 7, 1, 512, 3000), (3, 4, 4, 256, 100), (64, 32, 4, 512, 300),
          (80, 8, 2, 256, 150)]


def decode_setup(B, Hq, Hkv, D, window):
    n = window + 260
    pools, table = cache(B, n // 128 + 1, Hkv, D, B + D)
    gen = synth.generator(window)
    q, k, v = (synth.randn_bf16((B, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
    lens = torch.tensor([n - 3 * (b % 40) for b in range(B)], dtype=torch.int32, device=DEV)

    def run(q, pools):
        out = torch.full_like(q, 7.0)
        native.gemma_attn_decode_sinks(q, k, v, *[p.clone() for p in pools], table, seq_lens=lens, max_seq_len=n,
                                       window=window, sinks=5, scale=D ** -0.5, out=out, **KW)
        assert native.gemma_attn_sync_status() == 0
        return out

    return q, pools, table, lens, run


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode_query(case, bad):
    B, Hq, Hkv, D, _ = case
    q, pools, _, _, run = decode_setup(*case)
    clean = run(q, pools)
    for heads in ([0], [Hq - 1], [h for h in range(Hq) if h % 4 == 0]):
        x, hit = q.clone(), torch.zeros(B, Hq, dtype=torch.bool, device=DEV)
        x[B // 2, heads, D - 1] = bad
        hit[B // 2, heads] = True
        # The new token's logit is then infinite, so the heads' running maxima move at that tile
        # where they would have stayed (by less than 2^8): the others' weights are formed against
        # another power of two. A weight is held as two bf16, off by 2^-8 of 2^-8 of itself: an
        # output differs by at most 2 * 2^-16 max|v| before its rounding (2^-13 covers the 32-bit
        # sums too), which may then fall to the next bf16, 2^-7 of it away.
        check(run(x, pools), clean, hit, None if math.isnan(bad) else float(pools[1].abs().max()))


@pytest.mark.parametrize("rows", ["one", "tile", "all"])
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode_keys(case, rows):
    """NaN in one visible key, in all of a 128-position tile, in every cached key of a KV head."""
    B, Hq, Hkv, D, window = case
    q, pools, table, lens, run = decode_setup(*case)
    clean = run(q, pools)
    b, g = B // 2, Hkv - 1
    n = int(lens[b])
    spots = {"one": [n - 2], "tile": range((n - 1) // 128 * 128 - 128, (n - 1) // 128 * 128), "all": range(n - 1)}[rows]
    if rows == "tile" and window < 256:
        spots = [j for j in spots if j >= n - window]
    k = pools[0].clone()
    for j in spots:
        k[table[b, j // 128], g, j % 128, 3] = math.nan
    hit = torch.zeros(B, Hq, dtype=torch.bool, device=DEV)
    hit[b, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)] = any(j >= n - window for j in spots)  # some key that is seen
    check(run(q, [k, pools[1]]), clean, hit)


# before, new tokens, window, q heads, KV heads, dim: a chunk split over a cluster, pairs that walk row
# tiles, head pairs, one head per CTA
PREFILL = [([300], 40, 700, 8, 1, 512), ([200, 31], 20, 90, 4, 1, 256), ([513, 100], 200, 128, 16, 16, 256),
           ([300, 17], 130, 150, 16, 8, 512), ([0, 260], 129, 70, 8, 8, 512)]


def prefill_setup(before, S, window, Hq, Hkv, D):
    B, pps = len(before), (max(before) + S) // 128 + 1
    pools, table = cache(B, pps, Hkv, D, S)
    gen = synth.generator(S + D)
    q, k, v = (synth.randn_bf16((B, S, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
    lens = torch.tensor(before, dtype=torch.int32, device=DEV)

    def run(q, k=k, pools=pools):
        out = torch.full_like(q, 7.0)
        lse = torch.full((B, Hq, S), 7.0, dtype=torch.float32, device=DEV)
        native.gemma_attn_prefill_sinks(q, k, v, *[p.clone() for p in pools], table, window=window, sinks=5,
                                        scale=D ** -0.5, out=out, lse=lse, seq_lens_before=lens, **KW)
        assert native.gemma_attn_sync_status() == 0
        return out, lse.transpose(1, 2)

    return q, k, pools, table, run


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_prefill_query(case, bad):
    before, S, _, Hq, _, D = case
    q, _, _, _, run = prefill_setup(*case)
    clean, clean_lse = run(q)
    x, hit = q.clone(), torch.zeros(len(before), S, Hq, dtype=torch.bool, device=DEV)
    for b, s, h in ((0, 0, 0), (0, 7, Hq - 1), (len(before) - 1, S - 1, Hq // 2)):
        x[b, s, h, D - 1] = bad
        hit[b, s, h] = True
    out, lse = run(x)
    check(out, clean, hit)
    assert torch.equal(lse[~hit], clean_lse[~hit])
    if math.isnan(bad):
        assert torch.isnan(lse[hit]).all(), lse[hit]


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_prefill_logits_all_minus_infinity(case):
    """0 / 0: the only key that the first token sees has a logit of -inf."""
    before, S, _, Hq, Hkv, D = case
    case = ([0] * len(before), S, 1, Hq, Hkv, D)
    q, k, _, _, run = prefill_setup(*case)
    k = k.clone()
    k[0, 0, :, D - 1] = 1.0
    clean, _ = run(q, k)
    x, hit = q.clone(), torch.zeros(len(before), S, Hq, dtype=torch.bool, device=DEV)
    x[0, 0, 1, D - 1] = -math.inf
    hit[0, 0, 1] = True
    out, lse = run(x, k)
    check(out, clean, hit)
    assert lse[0, 0, 1] == -math.inf


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_prefill_keys(case):
    """A cached key that is NaN reaches the tokens that see it, and no other."""
    before, S, window, Hq, Hkv, D = case
    q, _, pools, table, run = prefill_setup(*case)
    clean, clean_lse = run(q)
    b = max(range(len(before)), key=lambda i: before[i])
    j, g = before[b] - 3, Hkv - 1
    k = pools[0].clone()
    k[table[b, j // 128], g, j % 128, 9] = math.nan
    hit = torch.zeros(len(before), S, Hq, dtype=torch.bool, device=DEV)
    seen = [s for s in range(S) if j > before[b] + s - window]
    hit[b, seen, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)] = True
    out, lse = run(q, pools=[k, pools[1]])
    check(out, clean, hit)
    assert torch.isnan(lse[hit]).all() and torch.equal(lse[~hit], clean_lse[~hit])
