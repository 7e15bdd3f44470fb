"""Numbers that a C int does not hold are refused: their low 32 bits would be
other arguments (sinks = 2^32 is no sinks at all)."""
import pytest
import torch

from hybrid_local_global_b200 import native

from test_scratch_stream_host import Tensor, i32, page_book

FAR = [1 << 31, 1 << 32, (1 << 32) + 64, 1 << 63, -(1 << 31) - 1]
ROPE = dict(rope_frac=0.25, rope_theta=1e6, scale=0.04)


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    def launch(*a):
        raise AssertionError("reached the library")
    for f in ("_prefill_sinks", "_decode_sinks", "_pages_trim", "_rope_axes"):
        monkeypatch.setattr(native, f, launch)
    monkeypatch.setattr(native, "_raw_stream", lambda index: 3)
    monkeypatch.setattr(native, "_current_device", lambda: 0)
    monkeypatch.setattr(native, "_scratch", lambda n, device, stream: Tensor(n, dtype=torch.uint8))


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("name", ["window", "sinks", "max_seq_len"])
def test_attention(name, far):
    pools, table = [Tensor(20, 1, 128, 512)] * 2, i32(2, 8)
    kw = dict(ROPE, window=64, sinks=4)
    step, one = Tensor(2, 8, 512), Tensor(2, 1, 512)
    with pytest.raises(ValueError, match=name):
        native.gemma_attn_decode_sinks(step, one, one, *pools, table, out=step, seq_lens=i32(2),
                                       **{**kw, "max_seq_len": 1000, name: far})
    if name != "max_seq_len":
        rows, new = Tensor(2, 16, 8, 512), Tensor(2, 16, 1, 512)
        with pytest.raises(ValueError, match=name):
            native.gemma_attn_prefill_sinks(rows, new, new, *pools, table, out=rows, **{**kw, name: far})
        with pytest.raises(ValueError, match=name):
            native.gemma_kv_pages_trim(page_book(), seq_lens=i32(2), **{"window": 64, "sinks": 4, name: far})


@pytest.mark.parametrize("tokens", [(1 << 31,), ((1 << 32) + 5,), (1 << 16, 1 << 16)])
def test_tokens_of_a_rotation(tokens):
    x = Tensor(*tokens, 1, 8)
    with pytest.raises(ValueError, match="tokens"):
        native.gemma_rope_axes(x, None, i32(1, *tokens), axis_pairs=[4], rope_theta=1e4, q_out=x)
