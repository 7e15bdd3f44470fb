"""Page upkeep (gemma_kv_pages_*) against the same calls made one entry at a
time on lists; every result is exact."""
import numpy as np
import pytest
import torch

from hybrid_local_global_b200 import native, synth

from sinks_ref import Book, random_book

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def on_device(bk):
    dev = native.PageBook(len(bk.table), len(bk.table[0]), bk.n_pages, bk.ps, DEV)
    dev.page_table.copy_(torch.tensor(bk.table, dtype=torch.int32))
    dev.ref_count.copy_(torch.tensor(bk.refs, dtype=torch.int32))
    return dev


def check_book(dev, bk):
    assert dev.page_table.cpu().tolist() == bk.table
    assert dev.ref_count.cpu().tolist() == bk.refs


def ok():
    assert native.gemma_attn_sync_status() == 0, native.gemma_last_error()


def make_pools(n_pages, ps, seed, kinds=(("bf16", 1, 256), ("int8", 3, 256), ("bf16", 2, 512))):
    gen = synth.generator(seed, DEV)
    pools = []
    for kind, H, D in kinds:
        if kind == "int8":
            p = native.Int8KVCache(n_pages, H, ps, D, DEV)
            synth.fill_int8_cache_(p, gen)
        else:
            p = synth.randn_bf16((n_pages, H, ps, D), gen, DEV)
        pools.append(p)
    return pools


def parts(pool):
    """Tensors [n_pages, H, ps, ...] of a pool (int8: codes and params), as integers."""
    if isinstance(pool, native.Int8KVCache):
        return [pool.codes, pool.params.view(torch.int32)]
    return [pool.view(torch.int16)]


def snapshot(pools):
    return [[t.clone() for t in parts(p)] for p in pools]


def check_pools(pools, before, copies):
    """copies: (src, dst, rows) of distinct destinations, contents as before the call."""
    for p, old in zip(pools, before):
        for t, o in zip(parts(p), old):
            want = o.clone()
            for s, d, rows in copies:
                want[d, :, :rows] = o[s, :, :rows]
            assert torch.equal(t, want)


@pytest.mark.parametrize("n_seqs,pps,n_pages,fill", [(1, 1, 1, 1.0), (4, 9, 64, 0.6), (33, 70, 1500, 0.5), (1500, 3, 5000, 0.7),
                                                     (4096, 2, 9000, 0.4)])
def test_fork(n_seqs, pps, n_pages, fill):
    rng = np.random.default_rng(n_seqs)
    bk = random_book(rng, n_seqs, pps, n_pages, 128, fill)
    dev = on_device(bk)
    for step in range(3):
        parents = rng.integers(-1, n_seqs, n_seqs).tolist()
        if step == 1:
            parents = list(range(n_seqs))[::-1]  # a permutation
        if step == 2:
            parents = [0] * n_seqs
        native.gemma_kv_pages_fork(dev, i32(parents))
        bk.fork(parents)
        ok()
        check_book(dev, bk)


def test_fork_reports_bad_parents():
    bk = random_book(np.random.default_rng(1), 5, 4, 40, 128, 0.8)
    dev = on_device(bk)
    native.gemma_kv_pages_fork(dev, i32([1, 5, -2, 2 ** 31 - 1, 0]))
    assert native.gemma_attn_sync_status() == native.GEMMA_ERR_DEVICE_RANGE
    bk.fork([1, 1, 2, 3, 0])
    check_book(dev, bk)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (300, 0), (300, 5), (128, 128), (129, 129), (2 ** 31 - 1, 4),
                                          (5, 2 ** 31 - 1)])
def test_trim(window, sinks):
    rng = np.random.default_rng(window % 1000 + sinks % 1000)
    ps, pps = 128, 11
    bk = random_book(rng, 14, pps, 200, ps, 0.9)
    dev = on_device(bk)
    lens = [0, 1, 127, 128, 129, 300, 301, 427, 428, 429, 640, pps * ps, -1, 1000]
    for _ in range(2):  # the second call finds nothing to drop
        native.gemma_kv_pages_trim(dev, seq_lens=i32(lens), window=window, sinks=sinks)
        bk.trim(lens, window, sinks)
        ok()
        check_book(dev, bk)


def test_trim_reports_lengths_past_the_table():
    bk = random_book(np.random.default_rng(3), 2, 3, 20, 128, 1.0)
    dev = on_device(bk)
    native.gemma_kv_pages_trim(dev, seq_lens=i32([3 * 128 + 1, 128]))
    assert native.gemma_attn_sync_status() == native.GEMMA_ERR_DEVICE_RANGE
    bk.trim([-1, 128], 0, 0)
    check_book(dev, bk)


def reserve(dev, pools, lens, new):
    lacking = i32([77])
    native.gemma_kv_pages_reserve(dev, pools, seq_lens=i32(lens), new_tokens=i32(new), lacking=lacking)
    return lacking


# few bytes at most (one launch): int8 with an odd number of 8-byte rows, runs of several tiles of a
# CTA; many: a second launch copies
SMALL, LARGE = (("int8", 1, 48), ("bf16", 1, 16)), (("bf16", 1, 256), ("int8", 3, 256), ("bf16", 2, 512))


@pytest.mark.parametrize("kinds", [SMALL, (("bf16", 1, 320),), LARGE])
@pytest.mark.parametrize("ps", [128, 256])
@pytest.mark.parametrize("seed", range(4))
def test_reserve_random(seed, ps, kinds):
    rng = np.random.default_rng(100 + seed)
    n_seqs, pps, n_pages = 9, 8, 120
    bk = Book(n_seqs, pps, n_pages, ps)
    dev, pools = on_device(bk), make_pools(n_pages, ps, seed, kinds)
    lens = [0] * n_seqs
    for step in range(6):
        new = [int(x) for x in rng.integers(0, ps + 40, n_seqs)]
        new = [min(a, pps * ps - n) for a, n in zip(new, lens)]
        before = snapshot(pools)
        lacking = reserve(dev, pools, lens, new)
        want, copies = bk.reserve(lens, new)
        ok()
        assert lacking.item() == want == 0
        check_book(dev, bk)
        check_pools(pools, before, copies)
        lens = [n + a for n, a in zip(lens, new)]
        parents = [int(x) for x in rng.integers(0, n_seqs, n_seqs)]
        native.gemma_kv_pages_fork(dev, i32(parents))
        bk.fork(parents)
        lens = [lens[p] for p in parents]
        drop = [int(rng.integers(0, n + 1)) if rng.random() < 0.3 else n for n in lens]
        native.gemma_kv_pages_trim(dev, seq_lens=i32(drop))
        bk.trim(drop, 0, 0)
        lens = drop
        check_book(dev, bk)


def test_reserve_copy_on_write_rules():
    """Sharers outside the call force a copy for every writer; otherwise the
    last writer keeps the page; a page without rows of the sequence is
    replaced, not copied; a full last page is left shared."""
    ps = 128
    for lens, new in (([200] * 4, [1, 1, 0, 1]), ([200] * 4, [1, 1, 1, 1]), ([256] * 4, [1, 1, 1, 1]), ([100] * 4, [1, 0, 0, 5]),
                      ([200] * 4, [100, 1, 300, 0])):
        bk = Book(4, 4, 30, ps)
        bk.table = [[5, 9, -1, -1] for _ in range(4)]
        dev, pools = on_device(bk), make_pools(30, ps, 1)
        before = snapshot(pools)
        lacking = reserve(dev, pools, lens, new)
        want, copies = bk.reserve(lens, new)
        ok()
        assert lacking.item() == 0 == want
        check_book(dev, bk)
        check_pools(pools, before, copies)


def test_reserve_without_enough_pages_changes_nothing():
    bk = Book(3, 4, 5, 128)
    bk.table = [[0, 1, -1, -1], [0, 1, -1, -1], [-1] * 4]
    dev, pools = on_device(bk), make_pools(5, 128, 2)
    before = snapshot(pools)
    lacking = reserve(dev, pools, [200, 200, 0], [1, 100, 400])  # 1 split + 1 fresh + 4 fresh, 3 free
    assert native.gemma_attn_sync_status() == native.GEMMA_ERR_DEVICE_RANGE
    assert lacking.item() == 3 == bk.reserve([200, 200, 0], [1, 100, 400])[0]
    check_book(dev, bk)
    check_pools(pools, before, [])
    lacking = reserve(dev, pools, [200, 200, 0], [0, 0, 384])  # exactly the three that are free
    ok()
    bk.reserve([200, 200, 0], [0, 0, 384])
    assert lacking.item() == 0
    check_book(dev, bk)


def test_reserve_leaves_bad_rows_out():
    ps, pps = 128, 3
    bk = Book(6, pps, 30, ps)
    dev, pools = on_device(bk), make_pools(30, ps, 2)
    lens, new = [0, -1, 0, pps * ps, 2 ** 31 - 1, 383], [1, 5, -5, 1, 2 ** 31 - 1, 1]
    lacking = reserve(dev, pools, lens, new)
    assert native.gemma_attn_sync_status() == native.GEMMA_ERR_DEVICE_RANGE
    bk.reserve([0, 0, 0, 0, 0, 383], [1, 0, 0, 0, 0, 1])
    assert lacking.item() == 0
    check_book(dev, bk)


def test_reserve_large_prompts():
    """More slots and pages than one pass of the plan takes."""
    ps, pps, n_seqs, n_pages = 128, 700, 5, 9000
    bk = random_book(np.random.default_rng(4), n_seqs, pps, n_pages, ps, 0.1)
    dev = on_device(bk)
    lens, new = [0, 5, 128, 70000, 89599], [pps * ps, 80000, 1, 19600, 1]
    lacking = reserve(dev, [], lens, new)
    assert bk.reserve(lens, new)[0] == 0
    ok()
    assert lacking.item() == 0
    check_book(dev, bk)


@pytest.mark.parametrize("n_seqs,pps,n_pages,fill", [(1, 1, 1, 0.0), (1, 1, 1, 1.0), (3, 5, 33, 0.5), (9, 40, 700, 0.6),
                                                     (7, 300, 40000, 0.3)])
def test_compact(n_seqs, pps, n_pages, fill):
    rng = np.random.default_rng(n_pages)
    bk = random_book(rng, n_seqs, pps, n_pages, 128, fill)
    dev = on_device(bk)
    pools = make_pools(n_pages, 128, 7) if n_pages < 1000 else []
    before = snapshot(pools)
    n_live, page_map = i32([-1]), torch.full((n_pages,), -9, dtype=torch.int32, device=DEV)
    native.gemma_kv_pages_compact(dev, pools, n_live=n_live, page_map=page_map)
    want, names = bk.compact()
    ok()
    assert n_live.item() == want and page_map.cpu().tolist() == names
    check_book(dev, bk)
    check_pools(pools, before, [(p, t, 128) for p, t in enumerate(names) if t >= 0 and t != p])
    native.gemma_kv_pages_compact(dev, pools, n_live=n_live)  # again: nothing moves
    ok()
    check_book(dev, bk)
    check_pools(pools, before, [(p, t, 128) for p, t in enumerate(names) if t >= 0 and t != p])


def test_compact_reports_entries_that_name_no_live_page():
    bk = Book(2, 3, 10, 128)
    bk.table = [[7, -1, -1], [8, 7, -1]]
    dev = on_device(bk)
    dev.page_table[0, 2] = 9   # count 0
    dev.page_table[1, 2] = 10  # outside
    n_live = i32([0])
    native.gemma_kv_pages_compact(dev, [], n_live=n_live)
    assert native.gemma_attn_sync_status() == native.GEMMA_ERR_DEVICE_RANGE
    assert n_live.item() == 2 and dev.page_table.cpu().tolist() == [[0, -1, 9], [1, 0, 10]]


@pytest.mark.parametrize("kinds", [(("bf16", 1, 256),), (("int8", 3, 512), ("bf16", 5, 512)), (("bf16", 1, 16),) * 70])
def test_copy(kinds):
    n_pages = 41
    pools = make_pools(n_pages, 128, 9, kinds)
    for n in (0, 1, 20):
        ids = np.random.default_rng(n).permutation(n_pages)
        src, dst = ids[:n].tolist(), ids[n:2 * n].tolist()
        if n == 20:
            src[3] = src[4] = src[0]  # one source, several destinations
        before = snapshot(pools)
        native.gemma_kv_pages_copy(pools, src=i32(src), dst=i32(dst))
        ok()
        check_pools(pools, before, [(s, d, 128) for s, d in zip(src, dst)])


def test_copy_skips_conflicts():
    pools = make_pools(12, 128, 9)
    before = snapshot(pools)
    #      good    chain: 2 reads what 1 writes   same dst twice   swap              self   outside      self read by another
    src = [0, 1, 2, 4, 5, 7, 8, 9, 12, 0, 9]
    dst = [10, 2, 3, 6, 6, 8, 7, 9, 0, -1, 11]
    native.gemma_kv_pages_copy(pools, src=i32(src), dst=i32(dst))
    assert native.gemma_attn_sync_status() == native.GEMMA_ERR_DEVICE_RANGE
    # pair 0 reads page 0, which the bad pair (12 -> 0) names as its destination: skipped as well
    check_pools(pools, before, [(1, 2, 128), (9, 11, 128)])


def test_captured_upkeep_follows_the_device_state():
    """fork, reserve, trim and compact in one graph, replayed on changing rows."""
    ps, n_seqs, pps, n_pages = 128, 4, 6, 60
    rng = np.random.default_rng(8)
    bk = Book(n_seqs, pps, n_pages, ps)
    dev, pools = on_device(bk), make_pools(n_pages, ps, 3)
    lens = [130, 5, 260, 0]
    reserve(dev, pools, [0] * n_seqs, lens)
    bk.reserve([0] * n_seqs, lens)
    parents, dl, dn, lacking, n_live = i32([0] * 4), i32(lens), i32([0] * 4), i32([0]), i32([0])
    ws = torch.empty(native.gemma_kv_pages_workspace_size(n_seqs, pps, n_pages), dtype=torch.uint8, device=DEV)
    after = torch.empty_like(dl)

    def step():
        native.gemma_kv_pages_fork(dev, parents)
        native.gemma_kv_pages_reserve(dev, pools, seq_lens=dl, new_tokens=dn, lacking=lacking, workspace=ws)
        torch.add(dl, dn, out=after)
        native.gemma_kv_pages_trim(dev, seq_lens=after, window=200, sinks=3)
        native.gemma_kv_pages_compact(dev, pools, n_live=n_live, workspace=ws)

    ok()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    saved, pools_saved = dev.state.clone(), snapshot(pools)
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    dev.state.copy_(saved)
    for p, old in zip(pools, pools_saved):
        for t, o in zip(parts(p), old):
            t.copy_(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        par = [int(x) for x in rng.integers(0, n_seqs, n_seqs)]
        lens = [lens[p] for p in par]
        new = [int(x) for x in rng.integers(1, 60, n_seqs)]
        before = snapshot(pools)
        parents.copy_(i32(par)), dl.copy_(i32(lens)), dn.copy_(i32(new))
        graph.replay()
        ok()
        bk.fork(par)
        short, copies = bk.reserve(lens, new)
        lens = [a + b for a, b in zip(lens, new)]
        bk.trim(lens, 200, 3)
        want, names = bk.compact()
        assert lacking.item() == short == 0 and n_live.item() == want
        check_book(dev, bk)
        for p, old in zip(pools, before):
            for t, o in zip(parts(p), old):
                w = o.clone()
                for a, b, rows in copies:
                    w[b, :, :rows] = o[a, :, :rows]
                w2 = w.clone()
                for a, b in enumerate(names):
                    if b >= 0 and b != a:
                        w2[b] = w[a]
                assert torch.equal(t, w2)
