"""Page books at the sizes where a launch needs more shared memory than a
kernel gets unasked, and small ones beside them."""
import threading

import numpy as np
import pytest
import torch

from hybrid_local_global_b200 import native

pytestmark = pytest.mark.gpu
DEV = "cuda"


def one_page_each(n_seqs, n_pages):
    """A book whose row b holds the page n_pages - 1 - b alone."""
    book = native.PageBook(n_seqs, 1, n_pages, 128, DEV)
    book.page_table[:, 0] = torch.arange(n_pages - 1, n_pages - 1 - n_seqs, -1, dtype=torch.int32, device=DEV)
    book.ref_count[n_pages - n_seqs:] = 1
    return book


# one bit a page: 48 KB of shared memory hold 393216, those that the kernel declares taken off
@pytest.mark.parametrize("n_pages", [392192, 392193, 393216, 393217, 1 << 20])
def test_compact(n_pages):
    book = one_page_each(3, n_pages)
    n_live = torch.zeros(1, dtype=torch.int32, device=DEV)
    page_map = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    native.gemma_kv_pages_compact(book, [], n_live=n_live, page_map=page_map)
    assert native.gemma_attn_sync_status() == 0
    assert n_live.item() == 3 and book.page_table.flatten().tolist() == [2, 1, 0]
    assert book.ref_count[:3].tolist() == [1, 1, 1] and int(book.ref_count.sum()) == 3
    assert page_map[-3:].tolist() == [0, 1, 2] and int((page_map >= 0).sum()) == 3


@pytest.mark.parametrize("n_seqs", [1535, 1536, 1537, 4095, 4096])
def test_fork(n_seqs):
    book = one_page_each(n_seqs, 5000)
    rows = book.page_table.clone()
    parents = torch.from_numpy(np.random.default_rng(n_seqs).integers(-1, n_seqs, n_seqs).astype(np.int32)).to(DEV)
    native.gemma_kv_pages_fork(book, parents)
    assert native.gemma_attn_sync_status() == 0
    want = torch.where(parents[:, None] < 0, -1, rows[parents.clamp(min=0).long()])
    assert torch.equal(book.page_table, want)
    counts = torch.bincount(want[want >= 0].long(), minlength=5000).int()
    assert torch.equal(book.ref_count, counts)


def test_small_and_large_books_from_several_threads():
    """A thread with a small book beside one with a large: neither launch may
    depend on what the other asked for."""
    errors = []

    def work(n_seqs, n_pages, rounds):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                book = one_page_each(n_seqs, n_pages)
                n_live = torch.zeros(1, dtype=torch.int32, device=DEV)
                same = torch.arange(n_seqs, dtype=torch.int32, device=DEV)
                ws = torch.empty(native.gemma_kv_pages_workspace_size(n_seqs, 1, n_pages), dtype=torch.uint8, device=DEV)
                for _ in range(rounds):
                    native.gemma_kv_pages_compact(book, [], n_live=n_live, workspace=ws)
                    native.gemma_kv_pages_fork(book, same)
                stream.synchronize()
                assert n_live.item() == n_seqs
        except Exception as e:  # noqa: BLE001 -- handed to the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in ((4096, 1 << 20, 300), (1600, 400000, 300), (4, 50, 300))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert native.gemma_attn_sync_status() == 0
