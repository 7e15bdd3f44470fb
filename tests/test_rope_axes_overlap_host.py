"""Which outputs gemma_rope_axes takes: its own input, or memory that neither
input and no other output uses (refused on the host, before any launch)."""
import random

import pytest
import torch

from hybrid_local_global_b200 import native

from test_sinks_host import FAKE, raw_axes

BAD = native.GEMMA_ERR_INVALID_ARG
# q: 10 tokens of 8 heads of 64 at FAKE, k: 2 heads, 128 elements a token, at FAKE + 0x100000; outputs apart
KP = FAKE + 0x100000


@pytest.mark.parametrize("over", [
    dict(qo=KP, qos=512), dict(qo=KP + 1024),              # q_out over k (both ranges meet)
    dict(ko=FAKE), dict(ko=FAKE + 5 * 1024),               # k_out over q
    dict(ko=FAKE + 0x200000), dict(ko=FAKE + 0x200000 + 2048),  # k_out over q_out
    dict(k=FAKE, ks=128, ko=FAKE, kos=128, qo=FAKE),       # q and k alike, both in place
    dict(qs=1 << 60), dict(kos=1 << 62),                   # strides that no memory holds
], ids=str)
def test_refusals(over):
    assert raw_axes(**over) == BAD and native.gemma_last_error()


def test_other_slices_of_a_fused_buffer_are_refused_where_they_meet():
    # heads [q 8 | k 2 | free 8 | free 2] of 64, token stride 20 * 64
    fused = dict(qs=1280, ks=1280, qos=1280, kos=1280, q=FAKE, k=FAKE + 8 * 128)
    for q_out, k_out in ((1, 18), (9, 18), (11, 9), (10, 9), (10, 17), (13, 18), (10, 19), (3, 8)):
        # (13, ...): q_out's last head runs into the next token's q; (10, 19): k_out's into it
        assert raw_axes(qo=FAKE + q_out * 128, ko=FAKE + k_out * 128, **fused) == BAD, (q_out, k_out)


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would be launched on made-up addresses")
def test_against_a_count_of_shared_bytes():
    """Random slices with one stride: refused iff some byte is shared. (Without a
    device an accepted call fails at its launch, not as an argument.)"""
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        n, Hq, Hkv, D = rng.choice([1, 2, 5]), rng.randint(1, 3), rng.randint(1, 2), rng.choice([8, 16])
        heads = rng.randint(Hq, Hq + 9)
        at = {x: rng.randint(0, 3 * heads) for x in ("q", "k", "qo", "ko")}
        if rng.random() < 0.3:
            at["qo"] = at["q"]
        if rng.random() < 0.3:
            at["ko"] = at["k"]
        if heads < max(Hq, Hkv):
            continue

        def elements(x):
            h = Hq if x.startswith("q") else Hkv
            return {at[x] * D + t * heads * D + e for t in range(n) for e in range(h * D)}

        q, k, qo, ko = (elements(x) for x in ("q", "k", "qo", "ko"))
        bad = bool((at["qo"] != at["q"] and qo & q) or (at["ko"] != at["k"] and ko & k) or qo & k or ko & q or qo & ko)
        stride = heads * D
        rc = raw_axes(q=FAKE + at["q"] * D * 2, qs=stride, k=FAKE + at["k"] * D * 2, ks=stride, qo=FAKE + at["qo"] * D * 2,
                      qos=stride, ko=FAKE + at["ko"] * D * 2, kos=stride, n_axes=1, pairs=(D // 2,), tokens=n, Hq=Hq,
                      Hkv=Hkv, D=D)
        assert (rc == BAD) == bad and rc in (BAD, native.GEMMA_ERR_CUDA), (n, Hq, Hkv, D, heads, at)
        seen[bad] += 1
    assert min(seen.values()) > 300, seen
