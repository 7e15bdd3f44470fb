"""Calls on a stream that is not the current one, with scratch of their own,
while the current stream allocates and overwrites blocks of the same sizes."""
import pytest
import torch

from hybrid_local_global_b200 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def beside(call, nbytes, rounds=20):
    """call(stream) on a side stream, `rounds` times, the current one busy with
    blocks of `nbytes` that it takes, fills and lets go of."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(rounds):
        call(side)
        for _ in range(3):
            torch.empty(nbytes, dtype=torch.uint8, device=DEV).fill_(0x7f)
    torch.cuda.synchronize()
    assert native.gemma_attn_sync_status() == 0


@pytest.mark.parametrize("D,Hq,Hkv,S", [(256, 16, 8, 700), (512, 8, 1, 60)])
def test_prefill(D, Hq, Hkv, S):
    gen = synth.generator(S)
    q, k, v = (synth.randn_bf16((1, S, h, D), gen).to(DEV) for h in (Hq, Hkv, Hkv))
    pools = [torch.zeros(8, Hkv, 128, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table, outs = torch.arange(8, dtype=torch.int32, device=DEV)[None], []

    def call(stream):
        outs.append(torch.full_like(q, 7.0))
        stream.wait_stream(torch.cuda.current_stream())
        native.gemma_attn_prefill_sinks(q, k, v, *pools, table, window=140, sinks=6, rope_frac=0.25, rope_theta=1e6,
                                        scale=D ** -0.5, out=outs[-1], stream=stream)

    beside(call, native.gemma_attn_prefill_workspace_size(1, S, Hq, Hkv, D, 0))
    want = torch.empty_like(q)
    native.gemma_attn_prefill_sinks(q, k, v, *pools, table, window=140, sinks=6, rope_frac=0.25, rope_theta=1e6,
                                    scale=D ** -0.5, out=want)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


def test_page_calls():
    """Ten beams split their last page over and over, and the pool is compacted."""
    n, pps, n_pages = 10, 6, 90
    book = native.PageBook(n, pps, n_pages, 128, DEV)
    pool = torch.zeros(n_pages, 2, 128, 256, dtype=torch.bfloat16, device=DEV)
    lens, one, first = i32([300] * n), i32([1] * n), i32([0] * n)
    lacking, n_live = i32([0]), i32([0])
    native.gemma_kv_pages_reserve(book, [pool], seq_lens=i32([0] * n), new_tokens=i32([300] + [0] * (n - 1)), lacking=lacking)
    native.gemma_kv_pages_fork(book, first)
    for i, page in enumerate(book.page_table[0, :3].tolist()):
        pool[page] = i + 1.0
    torch.cuda.synchronize()

    def call(stream):
        native.gemma_kv_pages_fork(book, first, stream=stream)
        native.gemma_kv_pages_reserve(book, [pool], seq_lens=lens, new_tokens=one, lacking=lacking, stream=stream)
        native.gemma_kv_pages_compact(book, [pool], n_live=n_live, stream=stream)

    beside(call, native.gemma_kv_pages_workspace_size(n, pps, n_pages))
    table = book.page_table.cpu()
    assert lacking.item() == 0 and n_live.item() == 2 + n
    assert (table[:, :2] == table[0, :2]).all() and len(set(table[:, 2].tolist())) == n and (table[:, 3:] == -1).all()
    assert sorted(set(table.flatten().tolist())) == [-1] + list(range(2 + n))
    for b in range(n):
        for i in range(3):
            rows = 128 if i < 2 else 300 - 256
            assert (pool[table[b, i], :, :rows] == i + 1.0).all()
