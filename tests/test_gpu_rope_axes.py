"""Multi-axis rotary positions (gemma_rope_axes) against the 64-bit rotation."""
import itertools

import pytest
import torch

from hybrid_local_global_b200 import native, synth

from sinks_ref import axes64

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def flags_of(interleaved, ladders, inverse):
    return ((native.GEMMA_ROPE_INTERLEAVED if interleaved else 0) | (native.GEMMA_ROPE_AXIS_LADDERS if ladders else 0)
            | (native.GEMMA_ROPE_INVERSE if inverse else 0))


def check(got, x, want):
    """One bf16 rounding (half a step) of a 32-bit rotation. Its angle is
    reduced in 64 bits and then rounded to 32: off by at most 2^-24 half-turns
    of a value below 1, so 2^-24 pi < 2^-22; the sine and cosine are good to two
    32-bit steps, the two products and their sum to one each: 2^-21 (|a| + |b|) in all."""
    pair = x.double().abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(*x.shape[:-1], x.shape[-1] // 2, 2)
    tol = U * want.abs() + 2.0 ** -21 * pair.flatten(-2) * (1 + U) + 2.0 ** -133
    assert ((got.double().cpu() - want).abs() <= tol).all()


def positions(axes, tokens, far, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-far, far + 1, (axes, tokens), generator=g).to(torch.int32)


CASES = [
    # tokens, Hq, Hkv, D, pairs, theta, largest position
    (1, 1, 1, 8, [4], 1e4, 3),
    (5, 3, 1, 72, [10, 13, 13], 1e4, 5000),
    (9, 8, 1, 512, [16, 24, 24], 1e6, 262144),
    (130, 4, 2, 256, [32, 48, 48], 1e4, 100000),
    (33, 16, 16, 64, [16, 16], 1e4, 140),
    (7, 2, 1, 128, [0, 64], 1e6, 2 ** 31 - 1),
    (3, 2, 2, 80, [0, 0, 0], 1e4, 10),
    (2000, 2, 1, 96, [5, 1, 7, 9], 5e5, 2000000),
    (4, 33, 7, 512, [256], 1e4, 9),
]


@pytest.mark.parametrize("interleaved,ladders,inverse", list(itertools.product([False, True], repeat=3)))
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_64_bits(case, interleaved, ladders, inverse):
    tokens, Hq, Hkv, D, pairs, theta, far = case
    gen = synth.generator(tokens + D)
    q, k = synth.randn_bf16((tokens, Hq, D), gen), synth.randn_bf16((tokens, Hkv, D), gen)
    pos = positions(len(pairs), tokens, far, D)
    qo, ko = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
    native.gemma_rope_axes(q.to(DEV), k.to(DEV), pos.to(DEV), axis_pairs=pairs, rope_theta=theta, q_out=qo, k_out=ko,
                           flags=flags_of(interleaved, ladders, inverse))
    torch.cuda.synchronize()
    for x, got in ((q, qo), (k, ko)):
        check(got, x, axes64(x, pos, pairs, theta, interleaved, ladders, inverse))
        n = 2 * sum(pairs)
        assert torch.equal(got[..., n:].cpu(), x[..., n:])  # pairs of no axis are copied


@pytest.mark.parametrize("inplace", [False, True])
def test_slices_of_a_fused_projection(inplace):
    B, S, Hq, Hkv, D, pairs = 2, 19, 4, 2, 64, [8, 12, 12]
    qkv = synth.randn_bf16((B, S, Hq + 2 * Hkv, D), synth.generator(1))
    pos = positions(3, B * S, 900, 2)
    dev = qkv.to(DEV)
    q, k = dev[:, :, :Hq], dev[:, :, Hq:Hq + Hkv]
    qo, ko = (q, k) if inplace else (torch.empty(B, S, Hq, D, dtype=q.dtype, device=DEV),
                                     torch.zeros(B, S, 3 * Hkv, D, dtype=q.dtype, device=DEV)[:, :, Hkv:2 * Hkv])
    native.gemma_rope_axes(q, k, pos.view(3, B, S).to(DEV), axis_pairs=pairs, rope_theta=1e4, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    for got, lo, hi in ((qo, 0, Hq), (ko, Hq, Hq + Hkv)):
        x = qkv[:, :, lo:hi].reshape(B * S, hi - lo, D)
        check(got.reshape(B * S, hi - lo, D), x, axes64(x, pos, pairs, 1e4))
    assert torch.equal(dev[:, :, Hq + Hkv:].cpu(), qkv[:, :, Hq + Hkv:])  # v is as it was
    if not inplace:
        assert torch.equal(dev.cpu(), qkv)


def test_q_alone_and_no_tokens():
    x = synth.randn_bf16((6, 2, 64), synth.generator(4))
    pos = positions(2, 6, 50, 1)
    out = torch.empty_like(x, device=DEV)
    native.gemma_rope_axes(x.to(DEV), None, pos.to(DEV), axis_pairs=[10, 20], rope_theta=1e4, q_out=out)
    torch.cuda.synchronize()
    check(out, x, axes64(x, pos, [10, 20], 1e4))
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    native.gemma_rope_axes(e, e, torch.empty(2, 0, dtype=torch.int32, device=DEV), axis_pairs=[1, 1], rope_theta=1e4,
                           q_out=e, k_out=e)


def test_gradient_is_the_inverse():
    """d <w, rotate(x)> / dx = inverse(w), against differences in 64 bits."""
    D, pairs, n = 64, [8, 24], 3
    gen = synth.generator(7)
    x, w = synth.randn_bf16((n, 1, D), gen), synth.randn_bf16((n, 1, D), gen)
    pos = positions(2, n, 300, 3)
    grad = torch.empty_like(w, device=DEV)
    native.gemma_rope_axes(w.to(DEV), None, pos.to(DEV), axis_pairs=pairs, rope_theta=1e4, q_out=grad,
                           flags=native.GEMMA_ROPE_INVERSE)
    torch.cuda.synchronize()
    xd = x.double()
    for t in range(n):
        for d in range(D):
            up, dn = xd.clone(), xd.clone()
            up[t, 0, d] += 0.5
            dn[t, 0, d] -= 0.5
            diff = ((axes64(up, pos, pairs, 1e4) - axes64(dn, pos, pairs, 1e4)) * w.double()).sum()
            # the map is linear: the difference is the derivative
            tol = U * abs(float(diff)) + 2.0 ** -20 * float(w[t].abs().max()) * 2
            assert abs(float(grad[t, 0, d]) - float(diff)) <= tol


def test_equals_the_attention_calls_own_rotation():
    """All axes alike: the rotation that a decode call applies to a new key."""
    D, frac, theta, n = 512, 0.25, 1e6, 70001
    k = synth.randn_bf16((1, 2, D), synth.generator(9)).to(DEV)
    pos = torch.full((3, 1), n - 1, dtype=torch.int32, device=DEV)
    out = torch.empty_like(k)
    native.gemma_rope_axes(k, None, pos, axis_pairs=[16, 24, 24], rope_theta=theta, q_out=out)
    pps = n // 128 + 1
    pool = torch.zeros(1, 2, 128, D, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(1, pps, dtype=torch.int32, device=DEV)
    native.gemma_attn_decode_sinks(k, k, k, pool, pool.clone(), table, seq_lens=torch.tensor([n], dtype=torch.int32, device=DEV),
                                   max_seq_len=n, window=1, sinks=0, rope_frac=frac, rope_theta=theta, scale=0.1,
                                   out=torch.empty_like(k))
    assert native.gemma_attn_sync_status() == 0
    assert torch.equal(pool[0, :, (n - 1) % 128].view(torch.int16), out[0].view(torch.int16))
