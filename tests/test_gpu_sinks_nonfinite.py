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
