"""Refusals of the window-plus-sinks, page and multi-axis rotation calls, which
happen before any device work (no GPU needed), and the block walk that the
decode kernel takes over a sequence's visible keys."""
import ctypes
import os
import re

import pytest
import torch

from hybrid_local_global_b200 import native

from sinks_ref import Book, attend64, kept_pages, sees

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "gemma_attn.h")
FAKE = 0x10000  # never dereferenced
E = native


def raw_prefill(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, table=FAKE, ps=128, pps=8, n_pages=20, before=FAKE, B=2, S=16, W=64,
             sinks=4, Hq=8, Hkv=1, D=512, frac=0.25, theta=1e6, scale=0.04, out=FAKE, lse=None, ws=FAKE, wsb=1 << 30,
             flags=0)
    a.update(over)
    return native._prefill_sinks(a["q"], a["k"], a["v"], a["kp"], a["vp"], a["table"], a["ps"], a["pps"], a["n_pages"],
                                 a["before"], a["B"], a["S"], a["W"], a["sinks"], a["Hq"], a["Hkv"], a["D"], a["frac"],
                                 a["theta"], a["scale"], a["out"], a["lse"], a["ws"], a["wsb"], a["flags"], None)


def raw_decode(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, table=FAKE, ps=128, pps=8, n_pages=20, lens=FAKE, top=1000, B=2, W=64,
             sinks=4, Hq=8, Hkv=1, D=512, frac=0.25, theta=1e6, scale=0.04, out=FAKE, ws=FAKE, wsb=1 << 30, flags=0)
    a.update(over)
    return native._decode_sinks(a["q"], a["k"], a["v"], a["kp"], a["vp"], a["table"], a["ps"], a["pps"], a["n_pages"],
                                a["lens"], a["top"], a["B"], a["W"], a["sinks"], a["Hq"], a["Hkv"], a["D"], a["frac"],
                                a["theta"], a["scale"], a["out"], a["ws"], a["wsb"], a["flags"], None)


BAD = [
    (dict(q=None), E.GEMMA_ERR_INVALID_ARG), (dict(out=None), E.GEMMA_ERR_INVALID_ARG),
    (dict(k=None), E.GEMMA_ERR_INVALID_ARG), (dict(v=None), E.GEMMA_ERR_INVALID_ARG),
    (dict(kp=None), E.GEMMA_ERR_INVALID_ARG), (dict(vp=None), E.GEMMA_ERR_INVALID_ARG),
    (dict(table=None), E.GEMMA_ERR_INVALID_ARG), (dict(q=FAKE + 8), E.GEMMA_ERR_INVALID_ARG),
    (dict(kp=FAKE + 2), E.GEMMA_ERR_INVALID_ARG), (dict(v=FAKE + 4), E.GEMMA_ERR_INVALID_ARG),
    (dict(ps=64), E.GEMMA_ERR_INVALID_ARG), (dict(ps=0), E.GEMMA_ERR_INVALID_ARG),
    (dict(ps=1 << 24, pps=1 << 10), E.GEMMA_ERR_INVALID_ARG), (dict(n_pages=0), E.GEMMA_ERR_INVALID_ARG),
    (dict(pps=0), E.GEMMA_ERR_INVALID_ARG), (dict(B=0), E.GEMMA_ERR_INVALID_ARG), (dict(B=70000), E.GEMMA_ERR_INVALID_ARG),
    (dict(W=0), E.GEMMA_ERR_INVALID_ARG), (dict(W=-5), E.GEMMA_ERR_INVALID_ARG), (dict(sinks=-1), E.GEMMA_ERR_INVALID_ARG),
    (dict(Hq=9, Hkv=2), E.GEMMA_ERR_INVALID_ARG), (dict(Hq=9, Hkv=1), E.GEMMA_ERR_UNSUPPORTED),
    (dict(D=128), E.GEMMA_ERR_UNSUPPORTED), (dict(frac=1.5), E.GEMMA_ERR_INVALID_ARG),
    (dict(theta=0.0), E.GEMMA_ERR_INVALID_ARG), (dict(scale=float("nan")), E.GEMMA_ERR_INVALID_ARG),
    (dict(flags=E.GEMMA_F_KV_INT8), E.GEMMA_ERR_UNSUPPORTED), (dict(flags=64), E.GEMMA_ERR_INVALID_ARG),
    (dict(flags=E.GEMMA_F_SOURCE_WINDOW), E.GEMMA_ERR_INVALID_ARG),
    (dict(flags=E.GEMMA_F_SHARED), E.GEMMA_ERR_INVALID_ARG),  # with k_new
    (dict(flags=E.GEMMA_F_KEQV), E.GEMMA_ERR_INVALID_ARG),    # with v_new
    (dict(flags=E.GEMMA_F_KEQV, v=None, vp=FAKE + 64), E.GEMMA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("over,code", BAD + [
    (dict(S=-1), E.GEMMA_ERR_INVALID_ARG), (dict(S=1025), E.GEMMA_ERR_CAPACITY), (dict(wsb=64), E.GEMMA_ERR_CAPACITY),
    (dict(ws=None), E.GEMMA_ERR_CAPACITY), (dict(ws=FAKE + 8), E.GEMMA_ERR_INVALID_ARG)])
def test_prefill_refusals(over, code):
    assert raw_prefill(**over) == code and native.gemma_last_error()


@pytest.mark.parametrize("over,code", BAD + [
    (dict(lens=None), E.GEMMA_ERR_INVALID_ARG), (dict(top=0), E.GEMMA_ERR_INVALID_ARG),
    (dict(top=1025), E.GEMMA_ERR_CAPACITY)])
def test_decode_refusals(over, code):
    assert raw_decode(**over) == code and native.gemma_last_error()


def book(**over):
    a = dict(page_table=FAKE, ref_count=FAKE, n_seqs=4, pages_per_seq=8, n_pages=40, page_size=128)
    a.update(over)
    return native.gemma_page_book(*a.values())


def pools(n=1, **over):
    a = dict(pool=FAKE, n_kv_heads=2, head_dim=256, flags=0)
    a.update(over)
    return (native.gemma_page_pool * max(n, 1))(*[native.gemma_page_pool(*a.values()) for _ in range(n)])


def page_calls(bk, pl, n=1, ints=FAKE, ws=FAKE, wsb=1 << 30):
    """Every call that takes a book."""
    b = ctypes.byref(bk)
    yield native._pages_fork(b, ints, None)
    yield native._pages_trim(b, ints, 0, 0, None)
    yield native._pages_reserve(b, pl, n, ints, ints, ints, ws, wsb, None)
    yield native._pages_compact(b, pl, n, ints, None, ws, wsb, None)


@pytest.mark.parametrize("over,code", [
    (dict(page_table=None), E.GEMMA_ERR_INVALID_ARG), (dict(ref_count=None), E.GEMMA_ERR_INVALID_ARG),
    (dict(ref_count=FAKE + 2), E.GEMMA_ERR_INVALID_ARG), (dict(n_seqs=0), E.GEMMA_ERR_INVALID_ARG),
    (dict(pages_per_seq=-1), E.GEMMA_ERR_INVALID_ARG), (dict(n_pages=0), E.GEMMA_ERR_INVALID_ARG),
    (dict(page_size=100), E.GEMMA_ERR_INVALID_ARG), (dict(pages_per_seq=1 << 24), E.GEMMA_ERR_INVALID_ARG),
    (dict(n_seqs=4097), E.GEMMA_ERR_UNSUPPORTED), (dict(n_pages=(1 << 20) + 1), E.GEMMA_ERR_UNSUPPORTED),
    (dict(n_seqs=4096, pages_per_seq=(1 << 18) + 1), E.GEMMA_ERR_UNSUPPORTED)])
def test_book_refusals(over, code):
    for rc in page_calls(book(**over), pools()):
        assert rc == code


def test_page_call_refusals():
    b = ctypes.byref(book())
    assert native._pages_fork(None, FAKE, None) == E.GEMMA_ERR_INVALID_ARG
    for rc in page_calls(book(), pools(), ints=None):
        assert rc == E.GEMMA_ERR_INVALID_ARG
    for rc in page_calls(book(), pools(), ints=FAKE + 1):
        assert rc == E.GEMMA_ERR_INVALID_ARG
    assert native._pages_trim(b, FAKE, -1, 0, None) == E.GEMMA_ERR_INVALID_ARG
    assert native._pages_trim(b, FAKE, 0, -1, None) == E.GEMMA_ERR_INVALID_ARG
    need = native.gemma_kv_pages_workspace_size(4, 8, 40)
    assert need > 0 and native.gemma_kv_pages_workspace_size(0, 8, 40) == 0
    for kw in (dict(ws=None), dict(wsb=need - 1)):
        assert list(page_calls(book(), pools(), **kw))[2:] == [E.GEMMA_ERR_CAPACITY] * 2
    assert list(page_calls(book(), pools(), ws=FAKE + 4))[2:] == [E.GEMMA_ERR_INVALID_ARG] * 2
    assert native._pages_compact(b, pools(), 1, FAKE, FAKE + 3, FAKE, 1 << 30, None) == E.GEMMA_ERR_INVALID_ARG


@pytest.mark.parametrize("over,code", [
    (dict(pool=None), E.GEMMA_ERR_INVALID_ARG), (dict(pool=FAKE + 8), E.GEMMA_ERR_INVALID_ARG),
    (dict(n_kv_heads=0), E.GEMMA_ERR_INVALID_ARG), (dict(head_dim=24), E.GEMMA_ERR_INVALID_ARG),
    (dict(flags=1), E.GEMMA_ERR_INVALID_ARG), (dict(n_kv_heads=1 << 15), E.GEMMA_ERR_UNSUPPORTED)])
def test_pool_refusals(over, code):
    assert list(page_calls(book(), pools(**over)))[2:] == [code] * 2
    assert native._pages_copy(pools(**over), 1, 40, 128, FAKE, FAKE, 3, None) == code


def test_copy_refusals():
    p = pools()
    for args in ((p, 1, 40, 100, FAKE, FAKE, 3), (p, 1, 0, 128, FAKE, FAKE, 3), (p, 1, 40, 128, FAKE, FAKE, -1),
                 (p, 1, 40, 128, None, FAKE, 3), (p, 1, 40, 128, FAKE, FAKE + 2, 3), (p, 1, 40, 128, FAKE, FAKE, 41),
                 (None, 1, 40, 128, FAKE, FAKE, 3), (p, -1, 40, 128, FAKE, FAKE, 3)):
        assert native._pages_copy(*args, None) == E.GEMMA_ERR_INVALID_ARG
    assert native._pages_copy(p, 1, 40, 128, None, None, 0, None) == 0  # nothing to copy
    assert native._pages_copy(None, 0, 40, 128, FAKE, FAKE, 3, None) == 0


def raw_axes(**over):
    a = dict(q=FAKE, qs=512, k=FAKE + 0x100000, ks=128, pos=FAKE, n_axes=3, pairs=(8, 12, 12), tokens=10, Hq=8, Hkv=2, D=64,
             theta=1e4, qo=FAKE + 0x200000, qos=512, ko=FAKE + 0x300000, kos=128, flags=0)
    a.update(over)
    pairs = None if a["pairs"] is None else (ctypes.c_int * max(len(a["pairs"]), 1))(*a["pairs"])
    return native._rope_axes(a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["n_axes"], pairs, a["tokens"], a["Hq"], a["Hkv"],
                             a["D"], a["theta"], a["qo"], a["qos"], a["ko"], a["kos"], a["flags"], None)


@pytest.mark.parametrize("over,code", [
    (dict(flags=8), E.GEMMA_ERR_INVALID_ARG), (dict(tokens=-1), E.GEMMA_ERR_INVALID_ARG),
    (dict(Hq=0), E.GEMMA_ERR_INVALID_ARG), (dict(Hkv=-1), E.GEMMA_ERR_INVALID_ARG), (dict(D=60), E.GEMMA_ERR_UNSUPPORTED),
    (dict(D=520), E.GEMMA_ERR_UNSUPPORTED), (dict(n_axes=0), E.GEMMA_ERR_INVALID_ARG),
    (dict(n_axes=5), E.GEMMA_ERR_INVALID_ARG), (dict(pairs=None), E.GEMMA_ERR_INVALID_ARG),
    (dict(pairs=(8, -1, 1)), E.GEMMA_ERR_INVALID_ARG), (dict(pairs=(8, 12, 13)), E.GEMMA_ERR_INVALID_ARG),
    (dict(theta=-1.0), E.GEMMA_ERR_INVALID_ARG), (dict(theta=float("inf")), E.GEMMA_ERR_INVALID_ARG),
    (dict(q=None), E.GEMMA_ERR_INVALID_ARG), (dict(ko=None), E.GEMMA_ERR_INVALID_ARG),
    (dict(pos=None), E.GEMMA_ERR_INVALID_ARG), (dict(pos=FAKE + 1), E.GEMMA_ERR_INVALID_ARG),
    (dict(q=FAKE + 8), E.GEMMA_ERR_INVALID_ARG), (dict(qs=516), E.GEMMA_ERR_INVALID_ARG),
    (dict(qs=504), E.GEMMA_ERR_INVALID_ARG), (dict(kos=64), E.GEMMA_ERR_INVALID_ARG),
    (dict(qo=FAKE + 1024), E.GEMMA_ERR_INVALID_ARG), (dict(qo=FAKE, qos=1024), E.GEMMA_ERR_INVALID_ARG)])
def test_axes_refusals(over, code):
    assert raw_axes(**over) == code and native.gemma_last_error()


def test_axes_of_no_tokens():
    assert raw_axes(tokens=0, q=None, k=None, qo=None, ko=None, pos=None) == 0


def test_binding_checks():
    z = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):  # not on a GPU
        native.gemma_rope_axes(z, None, torch.zeros(1, 2, dtype=torch.int32), axis_pairs=[4], rope_theta=1e4, q_out=z)
    bk = native.PageBook(2, 3, 7, 128, "cpu")
    assert (bk.n_seqs, bk.pages_per_seq, bk.n_pages) == (2, 3, 7)
    assert (bk.page_table == -1).all() and (bk.ref_count == 0).all() and bk.state.numel() == 13
    with pytest.raises(TypeError):
        native.gemma_kv_pages_fork(bk, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        native.gemma_kv_pages_fork(bk, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        native.gemma_kv_pages_trim(bk, seq_lens=torch.zeros(2, dtype=torch.int64))


@pytest.mark.parametrize("name", ["gemma_page_book", "gemma_page_pool"])
def test_struct_fields_match_the_header(name):
    text = open(HEADER).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", " ", body, flags=re.S)
    fields = [d.replace("*", " * ").split() for d in body.split(";") if d.split()]
    got = getattr(native, name)._fields_
    assert [f[-1] for f in fields] == [n for n, _ in got]
    for f, (_, t) in zip(fields, got):
        want = ctypes.c_void_p if "*" in f else {"int": ctypes.c_int, "unsigned": ctypes.c_uint}[f[0]]
        assert t is want


# ------------------------------------------------------------ the decode kernel's walk
def walk(length, window, sinks):
    """sink_span and block0 of csrc/common.cuh, restated: [(first position, 32-position blocks)] of every tile."""
    lo = max(0, length - window)
    first, start = 0, lo // 128 * 128
    if sinks > 0:
        end = min(sinks, lo)
        if -(-end // 128) * 128 < start:
            first = -(-end // 128)
        else:
            start = 0
    out = []
    for i in range(first + -(-(length - start) // 128)):
        p = i * 128 if i < first else start + (i - first) * 128
        begin, to = p, min(p + 128, length)
        if lo > begin and sinks <= begin:
            begin = lo // 32 * 32
        if lo >= p + 128 and sinks < to:
            to = sinks
        out.append((begin, -(-(to - begin) // 32)))
    return out


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 128, 129, 300, 1 << 30])
@pytest.mark.parametrize("sinks", [0, 1, 31, 32, 33, 70, 128, 129, 300, 1 << 30])
def test_walk_covers_every_visible_key_once(window, sinks):
    for length in [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 200, 256, 333, 400, 513, 700]:
        lo = max(0, length - window)
        tiles = walk(length, window, sinks)
        read = []
        for begin, blocks in tiles:
            rows = list(range(begin, begin + 32 * blocks))
            # in one aligned 128-position tile, whole blocks, the first and the last with a visible key
            assert begin % 32 == 0 and 1 <= blocks <= 4 and begin // 128 == rows[-1] // 128
            for block in (rows[:32], rows[-32:]):
                assert any(p < length and (p >= lo or p < sinks) for p in block), (length, begin, blocks)
            read += rows
        assert len(set(read)) == len(read) and length - 1 in range(tiles[-1][0], tiles[-1][0] + 32 * tiles[-1][1])
        seen = [p for p in read if p < length and (p >= lo or p < sinks)]
        assert seen == [j for j in range(length) if sees(j, length - 1, window, sinks)]


def test_reference_book_and_attention_are_what_they_say():
    assert kept_pages(300, 0, 0, 128) == {0, 1, 2} and kept_pages(300, 1, 0, 128) == set()
    assert kept_pages(300, 2, 1, 128) == {0, 2} and kept_pages(0, 5, 5, 128) == set()
    bk = Book(3, 3, 6, 128)
    assert bk.reserve([0, 0, 0], [200, 0, 0]) == (0, []) and bk.table[0] == [0, 1, -1]
    bk.fork([0, 0, -1])
    assert bk.refs == [2, 2, 0, 0, 0, 0]
    assert bk.reserve([200, 200, 0], [1, 1, 0]) == (0, [(1, 2, 72)])
    assert bk.table[:2] == [[0, 2, -1], [0, 1, -1]]
    bk.trim([0, 200, 0], 0, 0)
    assert bk.compact() == (2, [0, 1, -1, -1, -1, -1])
    K = torch.zeros(3, 1, 2)
    V = torch.tensor([[[1.0, 0]], [[float("nan"), 0]], [[3.0, 0]]])
    out, lse = attend64(torch.zeros(1, 1, 2), K, V, [2], 1, 1, 1.0)
    assert out[0, 0, 0] == 2.0 and abs(float(lse) - 0.6931471805599453) < 1e-15
