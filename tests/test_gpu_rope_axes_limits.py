"""A rotation of as many tokens as the argument holds."""
import pytest
import torch

from hybrid_local_global_b200 import native

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_most_tokens():
    """In place: the last tokens turn (43 GB in all)."""
    n, tail = 2 ** 31 - 1, 1000
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    x = torch.empty(n, 1, 8, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(1, n, dtype=torch.int32, device=DEV)
    x[-tail:] = torch.arange(8, device=DEV).to(torch.bfloat16)
    x[:tail] = 1.0
    pos[0, -tail:] = 1
    native.gemma_rope_axes(x, None, pos, axis_pairs=[1], rope_theta=1.0, q_out=x)
    assert native.gemma_attn_sync_status() == 0
    c, s = 0.5403023058681398, 0.8414709848078965  # of one radian
    got = x[-tail:, 0].double()
    # (0, 1) turned, rounded once; the 32-bit sine and cosine are off by far less than 2^-12 of that
    want = torch.tensor([-s, c], dtype=torch.float64, device=DEV)
    assert ((got[:, :2] - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -12) * want.abs()).all()
    assert (got[:, 2:] == torch.arange(2, 8, device=DEV)).all()
    assert (x[:tail] == 1).all()  # position 0
