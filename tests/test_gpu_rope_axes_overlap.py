"""gemma_rope_axes into other slices of a fused buffer, which lie between its
inputs' tokens without sharing bytes with them."""
import itertools

import pytest
import torch

from hybrid_local_global_b200 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("tokens", [1, 7, 2500])
@pytest.mark.parametrize("places", [p for p in itertools.permutations([0, 4, 6, 10]) if {p[0], p[2]} == {0, 6}], ids=str)
def test_outputs_between_the_inputs(tokens, places):
    """The four tensors at any places of [4 | 2 | 4 | 2] heads (q and q_out in the wide ones)."""
    D, pairs = 64, [8, 24]
    at = dict(zip(("q", "k", "qo", "ko"), places))
    buf = synth.randn_bf16((tokens, 12, D), synth.generator(tokens)).to(DEV)
    pos = torch.randint(-300, 300, (2, tokens), generator=synth.generator(1), dtype=torch.int32).to(DEV)
    q, qo = (buf[:, at[x]:at[x] + 4] for x in ("q", "qo"))
    k, ko = (buf[:, at[x]:at[x] + 2] for x in ("k", "ko"))
    before, kw = buf.clone(), dict(axis_pairs=pairs, rope_theta=1e4)
    qd, kd = q.contiguous(), k.contiguous()
    a, b = torch.empty_like(qd), torch.empty_like(kd)
    native.gemma_rope_axes(qd, kd, pos, q_out=a, k_out=b, **kw)
    native.gemma_rope_axes(q, k, pos, q_out=qo, k_out=ko, **kw)
    torch.cuda.synchronize()
    assert torch.equal(qo.contiguous().view(torch.int16), a.view(torch.int16))
    assert torch.equal(ko.contiguous().view(torch.int16), b.view(torch.int16))
    for x, n in (("q", 4), ("k", 2)):  # the inputs are as they were
        assert torch.equal(buf[:, at[x]:at[x] + n], before[:, at[x]:at[x] + n])


def test_meeting_outputs_are_refused():
    buf = torch.zeros(9, 12, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(1, 9, dtype=torch.int32, device=DEV)
    q, k = buf[:, :4], buf[:, 4:6]
    other = torch.empty(9, 2, 64, dtype=torch.bfloat16, device=DEV)
    for q_out, k_out in ((buf[:, 5:9], other), (buf[:, 6:10], buf[:, 9:11]), (q, buf[:, 3:5]), (buf[:, 1:5], other),
                         (buf[:, 6:10], q[:, 2:])):
        with pytest.raises(native.GemmaError) as e:
            native.gemma_rope_axes(q, k, pos, axis_pairs=[32], rope_theta=1e4, q_out=q_out, k_out=k_out)
        assert e.value.code == native.GEMMA_ERR_INVALID_ARG
    assert native.gemma_attn_sync_status() == 0 and (buf == 0).all()
