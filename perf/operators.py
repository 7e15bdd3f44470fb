"""Cases of the serving operators around a bounded paged cache: rotary
positions on several axes, attention to a sliding window plus a few first
tokens (prompts and single tokens), and the upkeep of the cache's pages
(forking, copy-on-write growth, trimming, compacting, copying).

``run`` computes a case either with the library's entry points (``own``) or in
plain torch, from what ``prepare`` made; ``exact`` gives the same results in 64
bits, written from the definitions.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE = 128


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One generation step of eight requests of a multimodal model on its
        # global layers: a quarter of the 256 pairs turns, by (time, height,
        # width). Nothing but latency.
        dict(name="axes_step_b8", op="axes", tokens=8, hq=8, hkv=1, dim=512, pairs="16 24 24",
             interleaved=False, ladders=False, inverse=False, theta=1e6, fused=False, far=200000),
        # A long prompt of text and images on a 31B-shaped local layer, q and k
        # being slices of one fused projection, axes interleaved over the pairs.
        dict(name="axes_prompt_31b", op="axes", tokens=8192, hq=32, hkv=16, dim=256, pairs="32 48 48",
             interleaved=True, ladders=False, inverse=False, theta=1e4, fused=True, far=60000),
        # The gradient of a vision tower's two-axis rotation (height, width,
        # each with frequencies of its own): images of odd sizes.
        dict(name="axes_vision_grad", op="axes", tokens=19881, hq=16, hkv=16, dim=64, pairs="16 16",
             interleaved=False, ladders=True, inverse=True, theta=1e4, fused=False, far=141),
        # A short user turn after a long conversation: E2B-shaped global layer
        # bounded to 512 recent tokens and 4 first ones.
        dict(name="sinks_turn_e2b", op="prefill", batch=1, new=64, lo=8011, hi=8011, hq=8, hkv=1, dim=512,
             window=512, sinks=4, frac=0.25, theta=1e6),
        # A whole prompt on a 31B-shaped local layer, one token short of 8192.
        dict(name="sinks_prompt_local", op="prefill", batch=1, new=8191, lo=0, hi=0, hq=32, hkv=16, dim=256,
             window=1024, sinks=16, frac=1.0, theta=1e4),
        # Chunks of two long documents (ragged lengths) on a 31B-shaped global
        # layer bounded to 4096 recent tokens and 64 first ones.
        dict(name="sinks_chunk_31b", op="prefill", batch=2, new=4096, lo=30000, hi=100000, hq=32, hkv=4, dim=512,
             window=4096, sinks=64, frac=0.25, theta=1e6),
        # One request generating: E2B-shaped bounded global layer. Latency.
        dict(name="sinks_step_b1", op="decode", batch=1, idle=0, lo=8200, hi=8200, hq=8, hkv=1, dim=512,
             window=512, sinks=4, frac=0.25, theta=1e6),
        # A local layer of a mid-sized batch, a window that no tile divides.
        dict(name="sinks_step_local_b16", op="decode", batch=16, idle=1, lo=3, hi=9000, hq=32, hkv=16, dim=256,
             window=1000, sinks=3, frac=1.0, theta=1e4),
        # A full serving batch on a 31B-shaped global layer, lengths U[4096,
        # 131072], two slots of the batch idle.
        dict(name="sinks_step_b64", op="decode", batch=64, idle=2, lo=4096, hi=131072, hq=32, hkv=4, dim=512,
             window=4096, sinks=64, frac=0.25, theta=1e6),
        # A beam step of 4 requests x 4 beams: the beams are reordered and every
        # row gets room for its next token, the shared last page copied on write.
        dict(name="pages_beam_step", op="beam", groups=4, width=4, prompt=900, grown=173, new=1, pools=2, hkv=1,
             dim=512, spare=24),
        # Sequences trimmed to window and sinks, then the pool compacted so that
        # its tail can be given back.
        dict(name="pages_trim_compact", op="compact", batch=48, lo=300, hi=6000, window=1024, sinks=16, pools=2,
             hkv=4, dim=256, spare=100),
        # Cached prompts copied into fresh pages: 8 layers' K and V at once.
        dict(name="pages_copy_prefix", op="copy", copies=61, pages=160, pools=16, hkv=1, dim=512),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["axes", "prefill", "decode", "beam", "compact", "copy"])
    if op == "axes":
        dim = rng.choice([64, 72, 80, 96, 128, 256, 512])
        axes = rng.choice([1, 2, 3])
        left, pairs = dim // 2, []
        for _ in range(axes):
            pairs.append(rng.randint(0, left))
            left -= pairs[-1]
        if not sum(pairs):
            pairs[0] = dim // 2
        hkv = rng.choice([1, 2, 4, 5])
        return dict(op=op, tokens=_spread(rng, 1, 9000), hq=hkv * rng.choice([1, 2, 3, 8]), hkv=hkv, dim=dim,
                    pairs=" ".join(map(str, pairs)), interleaved=rng.random() < 0.5, ladders=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, theta=rng.choice([1e4, 1e6]), fused=rng.random() < 0.5,
                    far=_spread(rng, 10, 1000000))
    if op in ("prefill", "decode"):
        dim = rng.choice([256, 512])
        hkv = rng.choice([1, 2, 3, 4])
        case = dict(op=op, hq=hkv * rng.choice([1, 2, 3, 4, 7, 8]), hkv=hkv, dim=dim, window=_spread(rng, 1, 4096),
                    sinks=rng.choice([0, 1, 4, rng.randint(5, 300)]), frac=rng.choice([0.25, 1.0]),
                    theta=rng.choice([1e4, 1e6]))
        if op == "prefill":
            first = rng.random() < 0.3
            hi = 0 if first else _spread(rng, 1, 20000)
            case.update(batch=rng.randint(1, 2), new=_spread(rng, 1, 3000), lo=hi // 3, hi=hi)
        else:
            batch, hi = _spread(rng, 1, 48), _spread(rng, 1, 40000)
            case.update(batch=batch, idle=rng.randint(0, batch // 4), lo=max(1, hi // 5), hi=hi)
        return case
    if op == "beam":
        return dict(op=op, groups=_spread(rng, 1, 16), width=rng.randint(1, 8), prompt=_spread(rng, 1, 4000),
                    grown=_spread(rng, 1, 500), new=_spread(rng, 1, 200), pools=rng.randint(1, 4),
                    hkv=rng.choice([1, 2]), dim=rng.choice([256, 512]), spare=rng.randint(0, 60))
    if op == "compact":
        hi = _spread(rng, 10, 6000)
        return dict(op=op, batch=_spread(rng, 1, 40), lo=hi // 8, hi=hi, window=rng.choice([0, _spread(rng, 1, 2000)]),
                    sinks=rng.choice([0, 4, 200]), pools=rng.randint(1, 2), hkv=rng.choice([1, 2]),
                    dim=rng.choice([256, 512]), spare=rng.randint(0, 200))
    pages = _spread(rng, 4, 300)
    return dict(op=op, copies=rng.randint(1, max(1, pages // 2 - 1)), pages=pages, pools=rng.randint(1, 6),
                hkv=rng.choice([1, 2]), dim=rng.choice([256, 512]))


# ------------------------------------------- what a case's scheduler knows
def _pairs(case):
    """Turning pairs of each axis."""
    return [int(n) for n in case["pairs"].split()]


def _lens(case):
    """Tokens that each sequence holds (decode: with the new one; 0 = idle slot)."""
    rng = random.Random(case["lo"] * 7919 + case["hi"] * 31 + case["batch"])
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    for i in range(case.get("idle", 0)):
        lens[(3 * i + 1) % case["batch"]] = 0
    return lens


def _kept(length, window, sinks):
    """Page numbers of a sequence that hold a position still to be seen."""
    first = max(0, length - window + 1) if window else 0
    pages = {p // PAGE for p in range(0, min(sinks, length), PAGE)} | {(min(sinks, length) - 1) // PAGE}
    pages |= set(range(first // PAGE, -(-length // PAGE))) if first < length else set()
    return sorted(p for p in pages if p >= 0)


def _deal(rows, n_pages, per_seq, rng):
    """A page table whose listed (row, page number) entries get the pages of
    a shuffled pool in turn, as a pool looks after some time in use."""
    pool = list(range(n_pages))
    rng.shuffle(pool)
    table = np.full((len(rows), per_seq), -1, dtype=np.int32)
    for b, numbers in enumerate(rows):
        for i in numbers:
            table[b, i] = pool.pop()
    return table


def _attn_pages(case):
    """Page numbers that each sequence holds when the call is made."""
    rows = []
    for n in _lens(case):
        old, new = (n, case["new"]) if case["op"] == "prefill" else (max(n - 1, 0), min(n, 1))
        held = set(_kept(old, case["window"], case["sinks"])) | set(range(old // PAGE, -(-(old + new) // PAGE)))
        rows.append(sorted(held))
    return rows


def _beam_plan(case):
    """Tables before the step: a group's beams share the prompt's full pages
    and hold the rest of their pages alone; every second beam is dropped."""
    g, w = case["groups"], case["width"]
    length = case["prompt"] + case["grown"]
    shared, total = case["prompt"] // PAGE, -(-length // PAGE)
    per_seq = -(-(length + case["new"]) // PAGE)
    grow = per_seq - total + 1
    n_pages = g * (shared + w * (total - shared)) + g * w * grow + case["spare"]
    pool = list(range(n_pages))
    random.Random(length).shuffle(pool)
    table = np.full((g * w, per_seq), -1, dtype=np.int32)
    for r in range(g):
        for i in range(shared):
            table[r * w:(r + 1) * w, i] = pool.pop()
        for b in range(w):
            for i in range(shared, total):
                table[r * w + b, i] = pool.pop()
    parents = [r * w + b // 2 for r in range(g) for b in range(w)]
    return table, n_pages, length, parents


def _compact_plan(case):
    lens = _lens(case)
    rows = [list(range(-(-n // PAGE))) for n in lens]
    n_pages = sum(len(r) for r in rows) + case["spare"]
    per_seq = max(1, max(len(r) for r in rows))
    return _deal(rows, n_pages, per_seq, random.Random(n_pages)), n_pages, lens


def _copy_plan(case):
    pool = list(range(case["pages"]))
    random.Random(case["copies"]).shuffle(pool)
    n = case["copies"]
    return pool[:n], pool[n:2 * n]


# ------------------------------------------------------------------ prepare
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _pool(gen, n_pages, hkv, dim):
    pool = torch.empty(n_pages, hkv, PAGE, dim, device=DEV, dtype=torch.bfloat16)
    step = max(1, (64 << 20) // (hkv * PAGE * dim))
    for i in range(0, n_pages, step):
        pool[i:i + step] = _normal(gen, *pool[i:i + step].shape)
    return pool


def _ints(values):
    return torch.as_tensor(np.asarray(values), dtype=torch.int32, device=DEV)


def _positions(case, gen):
    """Runs of text (all axes alike) with images between them (time stands,
    height and width run over the picture), far into a conversation."""
    n, axes = case["tokens"], len(_pairs(case))
    i = torch.arange(n, device=DEV)
    side = 23
    start = torch.randint(0, case["far"], (1,), generator=gen, device=DEV)
    block, inside = i // (side * side), i % (side * side)
    image = block % 2 == 1
    t = torch.where(image, start + block * side, start + block * side + inside)
    rows = [t, torch.where(image, t + inside // side, t), torch.where(image, t + inside % side, t)]
    if case["ladders"]:  # a vision tower's patches: small coordinates
        rows = [torch.randint(0, case["far"] + 1, (n,), generator=gen, device=DEV) for _ in rows]
    return torch.stack(rows[-axes:]).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = _gen(seed)
    st = dict(case=case)
    if case["op"] == "axes":
        n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["dim"]
        if case["fused"]:  # q | k | v of one projection: q and k are strided slices of it
            qkv = _normal(gen, n, hq + 2 * hkv, d)
            st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv])
        else:
            st.update(q=_normal(gen, n, hq, d), k=_normal(gen, n, hkv, d))
        st.update(positions=_positions(case, gen), q_out=torch.empty(n, hq, d, device=DEV, dtype=torch.bfloat16),
                  k_out=torch.empty(n, hkv, d, device=DEV, dtype=torch.bfloat16))
    elif case["op"] in ("prefill", "decode"):
        b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["dim"]
        lens, rows = _lens(case), _attn_pages(case)
        s = (case["new"],) if case["op"] == "prefill" else ()
        n_pages = max(1, sum(len(r) for r in rows))
        top = max(lens) + (case["new"] if s else 0)
        per_seq = max(1, -(-top // PAGE))
        st.update(q=_normal(gen, b, *s, hq, d), k=_normal(gen, b, *s, hkv, d), v=_normal(gen, b, *s, hkv, d),
                  k_pool=_pool(gen, n_pages, hkv, d), v_pool=_pool(gen, n_pages, hkv, d),
                  table=_ints(_deal(rows, n_pages, per_seq, random.Random(seed))), lens=lens, seq_lens=_ints(lens),
                  top=max(1, top), busy=torch.tensor([i for i, n in enumerate(lens) if n], device=DEV),
                  out=torch.empty(b, *s, hq, d, device=DEV, dtype=torch.bfloat16))
        if own:
            from hybrid_local_global_b200 import native
            size = (native.gemma_attn_prefill_workspace_size(b, *s, hq, hkv, d, 0) if s else
                    native.gemma_attn_decode_sinks_workspace_size(b, hq, hkv, d, case["window"], case["sinks"], st["top"]))
            st["workspace"] = torch.empty(max(size, 1), device=DEV, dtype=torch.uint8)
    elif case["op"] == "copy":
        src, dst = _copy_plan(case)
        st.update(pools=[_pool(gen, case["pages"], case["hkv"], case["dim"]) for _ in range(case["pools"])],
                  src=_ints(src), dst=_ints(dst))
    else:
        if case["op"] == "beam":
            table, n_pages, length, parents = _beam_plan(case)
            st.update(parents=_ints(parents), seq_lens=_ints([length] * len(table)),
                      new_tokens=_ints([case["new"]] * len(table)))
        else:
            table, n_pages, lens = _compact_plan(case)
            st.update(seq_lens=_ints(lens))
        refs = np.bincount(table[table >= 0], minlength=n_pages)
        start = _ints(np.concatenate([table.ravel(), refs]))
        st.update(pools=[_pool(gen, n_pages, case["hkv"], case["dim"]) for _ in range(case["pools"])],
                  start=start, n_seqs=table.shape[0], per_seq=table.shape[1], n_pages=n_pages,
                  count=torch.zeros(1, dtype=torch.int32, device=DEV))
        if own:
            from hybrid_local_global_b200 import native
            st["book"] = native.PageBook(table.shape[0], table.shape[1], n_pages, PAGE, DEV)
            size = native.gemma_kv_pages_workspace_size(table.shape[0], table.shape[1], n_pages)
            st["workspace"] = torch.empty(max(size, 1), device=DEV, dtype=torch.uint8)
    return st


# ---------------------------------------------------------------------- run
def run(st):
    case = st["case"]
    if own:
        return _OWN[case["op"]](st, case)
    return _PLAIN[case["op"]](st, case)


# ------------------------------------------------ the library's entry points
def _own_axes(st, case):
    from hybrid_local_global_b200 import native
    flags = ((native.GEMMA_ROPE_INTERLEAVED if case["interleaved"] else 0)
             | (native.GEMMA_ROPE_AXIS_LADDERS if case["ladders"] else 0)
             | (native.GEMMA_ROPE_INVERSE if case["inverse"] else 0))
    native.gemma_rope_axes(st["q"], st["k"], st["positions"], axis_pairs=_pairs(case), rope_theta=case["theta"],
                           q_out=st["q_out"], k_out=st["k_out"], flags=flags)
    return st["q_out"], st["k_out"]


def _own_prefill(st, case):
    from hybrid_local_global_b200 import native
    native.gemma_attn_prefill_sinks(
        st["q"], st["k"], st["v"], st["k_pool"], st["v_pool"], st["table"], window=case["window"], sinks=case["sinks"],
        rope_frac=case["frac"], rope_theta=case["theta"], scale=case["dim"] ** -0.5, out=st["out"],
        seq_lens_before=st["seq_lens"], workspace=st["workspace"])
    return st["out"], st["k_pool"], st["v_pool"]


def _own_decode(st, case):
    from hybrid_local_global_b200 import native
    native.gemma_attn_decode_sinks(
        st["q"], st["k"], st["v"], st["k_pool"], st["v_pool"], st["table"], seq_lens=st["seq_lens"],
        max_seq_len=st["top"], window=case["window"], sinks=case["sinks"], rope_frac=case["frac"],
        rope_theta=case["theta"], scale=case["dim"] ** -0.5, out=st["out"], workspace=st["workspace"])
    return st["out"], st["k_pool"], st["v_pool"]


def _own_beam(st, case):
    from hybrid_local_global_b200 import native
    book = st["book"]
    book.state.copy_(st["start"])
    native.gemma_kv_pages_fork(book, st["parents"])
    native.gemma_kv_pages_reserve(book, st["pools"], seq_lens=st["seq_lens"], new_tokens=st["new_tokens"],
                                  lacking=st["count"], workspace=st["workspace"])
    return [book.page_table, book.ref_count, st["count"], *st["pools"]]


def _own_compact(st, case):
    from hybrid_local_global_b200 import native
    book = st["book"]
    book.state.copy_(st["start"])
    native.gemma_kv_pages_trim(book, seq_lens=st["seq_lens"], window=case["window"], sinks=case["sinks"])
    native.gemma_kv_pages_compact(book, st["pools"], n_live=st["count"], workspace=st["workspace"])
    return [book.page_table, book.ref_count, st["count"], *st["pools"]]


def _own_copy(st, case):
    from hybrid_local_global_b200 import native
    native.gemma_kv_pages_copy(st["pools"], src=st["src"], dst=st["dst"])
    return list(st["pools"])


_OWN = dict(axes=_own_axes, prefill=_own_prefill, decode=_own_decode, beam=_own_beam, compact=_own_compact,
            copy=_own_copy)


# ------------------------------------------------------------- plain forms
def _axis_of_pairs(pairs, interleaved):
    """(axis, rank within the axis) of every turning pair, first pair first."""
    listed_ = [(a, r) for a, n in enumerate(pairs) for r in range(n)]
    return sorted(listed_, key=lambda ar: (ar[1], ar[0])) if interleaved else listed_


def _turn(x, cos, sin):
    """Pairs (2i, 2i + 1) of x [tokens, heads, dim] turned; cos and sin [tokens, turning pairs]."""
    y = x.float()
    n = cos.shape[1]
    a, b = y[..., 0:2 * n:2], y[..., 1:2 * n:2]
    c, s = cos[:, None, :], sin[:, None, :]
    y = y.clone()
    y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * c - b * s, a * s + b * c
    return y


def _plain_axes(st, case):
    order = _axis_of_pairs(_pairs(case), case["interleaved"])
    i = torch.arange(len(order), device=DEV, dtype=torch.float64)
    expo = i / (case["dim"] / 2)
    if case["ladders"]:
        expo = torch.tensor([r / _pairs(case)[a] for a, r in order], device=DEV, dtype=torch.float64)
    freq = torch.exp(-expo * math.log(case["theta"]))
    axis = torch.tensor([a for a, _ in order], device=DEV)
    angle = st["positions"].double()[axis].T * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if case["inverse"]:
        sin = -sin
    st["q_out"].copy_(_turn(st["q"], cos, sin))
    st["k_out"].copy_(_turn(st["k"], cos, sin))
    return st["q_out"], st["k_out"]


def _rope(x, pos, case):
    """x [n, heads, dim] turned at positions pos [n] by one axis, in 32 bits."""
    d = case["dim"]
    n = int(case["frac"] * (d // 2))
    freq = torch.exp(torch.arange(n, device=DEV, dtype=torch.float64) * (-2.0 / d * math.log(case["theta"])))
    angle = pos.double()[:, None] * freq
    return _turn(x, torch.cos(angle).float(), torch.sin(angle).float())


def _rows(st, b, pos):
    """(page, row) of positions of sequence b."""
    return st["table"][b].long()[pos // PAGE], pos % PAGE


def _attend(q, k, v, seen):
    """q [n, hq, d], k and v [m, hkv, d], seen [n, m] -> [n, hq, d], in the type of q."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    qg = q.view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    s = (qg @ k.permute(1, 2, 0)).view(hkv, hq // hkv, n, -1) * d ** -0.5
    s = s.masked_fill(~seen, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p.view(hkv, -1, p.shape[-1]) @ v.permute(1, 0, 2)
    return o.view(hkv, hq // hkv, n, d).permute(2, 0, 1, 3).reshape(n, hq, d)


def _plain_prefill(st, case):
    window, sinks, new = case["window"], case["sinks"], case["new"]
    block = 512
    for b, before in enumerate(st["lens"]):
        pos = torch.arange(before, before + new, device=DEV)
        page, row = _rows(st, b, pos)
        st["k_pool"][page, :, row] = _rope(st["k"][b], pos, case).to(torch.bfloat16)
        st["v_pool"][page, :, row] = st["v"][b]
        q = _rope(st["q"][b], pos, case)
        for i in range(0, new, block):
            p = pos[i:i + block]
            lo, hi = max(before + i - window + 1, 0), before + min(i + block, new)
            keys = torch.cat([torch.arange(min(sinks, lo), device=DEV), torch.arange(lo, hi, device=DEV)])
            page, row = _rows(st, b, keys)
            seen = (keys <= p[:, None]) & ((keys < sinks) | (keys > p[:, None] - window))
            st["out"][b, i:i + block] = _attend(q[i:i + block], st["k_pool"][page, :, row].float(),
                                                st["v_pool"][page, :, row].float(), seen).to(torch.bfloat16)
    return st["out"], st["k_pool"], st["v_pool"]


def _plain_decode(st, case):
    window, sinks = case["window"], case["sinks"]
    lens = st["seq_lens"].long()
    live = lens > 0
    pos = (lens - 1).clamp(min=0)
    b = torch.arange(len(lens), device=DEV)
    page, row = st["table"].long()[b, pos // PAGE].clamp(min=0), pos % PAGE
    q, k = _rope(st["q"], pos, case), _rope(st["k"], pos, case).to(torch.bfloat16)
    keep = live[:, None, None]
    sel = st["busy"]
    st["k_pool"][page[sel], :, row[sel]] = k[sel]
    st["v_pool"][page[sel], :, row[sel]] = st["v"][sel]
    span = min(window, st["top"])
    first = torch.arange(min(sinks, st["top"]), device=DEV)
    for i in range(0, len(lens), 4):
        p = pos[i:i + 4, None]
        recent = p - span + 1 + torch.arange(span, device=DEV)
        keys = torch.cat([first.expand(len(p), -1), recent], 1)
        seen = torch.cat([first <= p - window, recent >= 0], 1)  # a first token inside the window counts once
        at = keys.clamp(min=0)
        page = torch.gather(st["table"][i:i + 4].long(), 1, at // PAGE).clamp(min=0)
        kk, vv = st["k_pool"][page, :, at % PAGE].float(), st["v_pool"][page, :, at % PAGE].float()
        n, m, hkv, d = kk.shape
        s = torch.einsum("bhgd,bmhd->bhgm", q[i:i + 4].view(n, hkv, -1, d), kk) * d ** -0.5
        s = s.masked_fill(~seen[:, None, None], -math.inf)
        w = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.einsum("bhgm,bmhd->bhgd", w / w.sum(-1, keepdim=True), vv).reshape(n, -1, d)
        st["out"][i:i + 4] = torch.where(keep[i:i + 4], o, torch.zeros_like(o)).to(torch.bfloat16)
    return st["out"], st["k_pool"], st["v_pool"]


def _open_book(st):
    state = st["start"].clone()
    n = st["n_seqs"] * st["per_seq"]
    return state[:n].view(st["n_seqs"], st["per_seq"]), state[n:]


def _count_refs(table, n_pages):
    flat = table.flatten().long()
    refs = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    refs.scatter_add_(0, torch.where(flat >= 0, flat, n_pages), torch.ones_like(flat, dtype=torch.int32))
    return refs[:n_pages]


def _plain_beam(st, case):
    table, _ = _open_book(st)
    n_pages, per_seq = st["n_pages"], st["per_seq"]
    table = table[st["parents"].long()]
    refs = _count_refs(table, n_pages)
    # entries that the new tokens will write
    lens, new = st["seq_lens"].long(), st["new_tokens"].long()
    number = torch.arange(per_seq, device=DEV)
    first, last = lens // PAGE, (lens + new - 1) // PAGE
    write = (number >= first[:, None]) & (number <= last[:, None]) & (new > 0)[:, None]
    old = table.long()
    held = old.clamp(min=0)
    shared = write & (old >= 0) & (refs[held] > 1)
    # of a page that only rows of this call hold, the last one keeps it
    place = torch.arange(table.numel(), device=DEV).view_as(old)
    spot = torch.where(shared, held, n_pages).flatten()
    writers = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    writers.scatter_add_(0, spot, torch.ones_like(spot, dtype=torch.int32))
    latest = torch.full((n_pages + 1,), -1, dtype=torch.int64, device=DEV)
    latest.scatter_reduce_(0, spot, place.flatten(), "amax")
    split = shared & ~((writers[held] == refs[held]) & (latest[held] == place))
    fresh = (write & (old < 0)) | split
    pages = torch.arange(n_pages, device=DEV)
    free = torch.sort(torch.where(refs == 0, pages, n_pages + pages)).values
    n_free, n_fresh = (refs == 0).sum(), fresh.sum()
    st["count"].copy_((n_fresh - n_free).clamp(min=0))
    enough = n_fresh <= n_free
    turn = (torch.cumsum(fresh.flatten().long(), 0) - 1).view_as(old).clamp(0, n_pages - 1)
    out = torch.where(fresh & enough, free[turn], old)
    refs_out = _count_refs(out, n_pages)
    # the rows that a split page already holds go along
    at = first[:, None].clamp(max=per_seq - 1)
    src, dst = old.gather(1, at)[:, 0], out.gather(1, at)[:, 0]
    moved = split.gather(1, at)[:, 0] & enough
    src, dst = torch.where(moved, src, dst).clamp(min=0), dst.clamp(min=0)
    rows = (torch.arange(PAGE, device=DEV) < (lens % PAGE)[:, None]) & moved[:, None]
    for pool in st["pools"]:
        pool[dst] = torch.where(rows[:, None, :, None], pool[src], pool[dst])
    return [out.to(torch.int32), refs_out, st["count"], *st["pools"]]


def _plain_compact(st, case):
    table, _ = _open_book(st)
    n_pages = st["n_pages"]
    lens, window, sinks = st["seq_lens"].long()[:, None], case["window"], case["sinks"]
    begin = torch.arange(st["per_seq"], device=DEV) * PAGE
    end = torch.minimum(begin + PAGE, lens)
    recent = end > (lens - window + 1 if window else lens * 0)
    keep = (begin < lens) & (recent | (begin < sinks))
    table = torch.where(keep, table, -1)
    refs = _count_refs(table, n_pages)
    # the k-th live page past the live count moves into the k-th hole before it
    live = refs > 0
    n_live = live.sum()
    st["count"].copy_(n_live)
    pages = torch.arange(n_pages, device=DEV)
    hole = ~live & (pages < n_live)
    mover = live & (pages >= n_live)
    moves = mover.sum()
    most = n_pages // 2
    to = torch.sort(torch.where(hole, pages, n_pages + pages)).values[:most]
    src = torch.sort(torch.where(mover, pages, torch.where(hole, 2 * n_pages, n_pages) + pages)).values[:most] % n_pages
    real = torch.arange(most, device=DEV) < moves
    dst = torch.where(real, to % n_pages, src)
    new_name = pages.clone()
    new_name[src] = dst
    flat = table.long()
    out = torch.where(flat >= 0, new_name[flat.clamp(min=0)], -1).to(torch.int32)
    for pool in st["pools"]:
        pool[dst] = pool[src]
    return [out, _count_refs(out, n_pages), st["count"], *st["pools"]]


def _plain_copy(st, case):
    src, dst = st["src"].long(), st["dst"].long()
    for pool in st["pools"]:
        pool[dst] = pool[src]
    return list(st["pools"])


_PLAIN = dict(axes=_plain_axes, prefill=_plain_prefill, decode=_plain_decode, beam=_plain_beam, compact=_plain_compact,
              copy=_plain_copy)


# ------------------------------------------------------------------- work
def _seen_pairs(first, new, window, sinks):
    """(query, key) pairs of queries at first .. first + new - 1."""
    total = 0
    for p in range(first, first + new):
        total += min(p + 1, window) + min(sinks, max(0, p + 1 - window))
    return total


def work(case):
    if case["op"] == "axes":
        vec = case["tokens"] * (case["hq"] + case["hkv"])
        return dict(bytes=2 * vec * case["dim"] * 2 + case["tokens"] * len(_pairs(case)) * 4,
                    flops=vec * sum(_pairs(case)) * 6)
    if case["op"] == "prefill":
        n, hq, hkv, d, w, s = (case[x] for x in ("new", "hq", "hkv", "dim", "window", "sinks"))
        flops = keys = 0
        for before in _lens(case):
            flops += 4 * hq * d * _seen_pairs(before, n, w, s)
            lo = max(0, before - w + 1)
            keys += (before - lo) + min(s, lo)
        rows = case["batch"] * n
        return dict(bytes=2 * (rows * (2 * hq + 4 * hkv) * d + 2 * keys * hkv * d), flops=flops)
    if case["op"] == "decode":
        hq, hkv, d = case["hq"], case["hkv"], case["dim"]
        lens = [n for n in _lens(case) if n]
        pairs = sum(_seen_pairs(n - 1, 1, case["window"], case["sinks"]) for n in lens)
        return dict(bytes=2 * (2 * (pairs - len(lens)) * hkv * d + len(lens) * (2 * hq + 4 * hkv) * d),
                    flops=4 * hq * d * pairs)
    page = case["hkv"] * PAGE * case["dim"] * 2
    if case["op"] == "copy":
        return dict(bytes=2 * case["copies"] * case["pools"] * page + 8 * case["copies"], flops=0)
    if case["op"] == "beam":
        table, n_pages, length, parents = _beam_plan(case)
        tails = {}
        if length % PAGE:
            for p in parents:
                tails[p] = tails.get(p, 0) + 1
        copies = sum(n - 1 for n in tails.values())
        held = copies * (length % PAGE) * page // PAGE
        return dict(bytes=2 * held * case["pools"] + 8 * table.size + 8 * n_pages, flops=0)
    table, n_pages, lens = _compact_plan(case)
    kept = [set(_kept(n, case["window"], case["sinks"])) for n in lens]
    live = {int(table[b, i]) for b, numbers in enumerate(kept) for i in numbers}
    moves = sum(1 for p in live if p >= len(live))
    return dict(bytes=2 * moves * page * case["pools"] + 8 * table.size + 8 * n_pages, flops=0)


# ------------------------------------------------------------------ exact
def _exact_turn(x, pos_of_pair, freq, sign):
    """x [n, heads, dim] in 64 bits; pair i of row t turned by sign * pos_of_pair[i][t] * freq[i]."""
    y = x.double().clone()
    for i, f in enumerate(freq):
        angle = pos_of_pair[i].double() * (sign * f)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        z = turn * torch.complex(x[..., 2 * i].double(), x[..., 2 * i + 1].double())
        y[..., 2 * i], y[..., 2 * i + 1] = z.real, z.imag
    return y


def _exact_rope(x, pos, case):
    d = case["dim"]
    n = int(math.floor(case["frac"] * d / 2))
    freq = [case["theta"] ** (-2.0 * i / d) for i in range(n)]
    return _exact_turn(x, [pos] * n, freq, 1.0)


def _exact_attention(st, case, b, q, pos):
    """Queries q [n, hq, d] at positions pos of sequence b over the pool as it stands, head by head."""
    n, hq, d = q.shape
    group = hq // case["hkv"]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=DEV)
    p = pos[:, None]
    first, last = int(pos[0]), int(pos[-1])
    keys = [j for j in range(last + 1) if j < case["sinks"] or j > first - case["window"]]
    j = torch.tensor(keys, device=DEV)
    where = st["table"][b].long()
    hidden = (j > p) | ((j >= case["sinks"]) & (j <= p - case["window"]))
    for g in range(case["hkv"]):
        k = st["k_pool"][where[j // PAGE], g, j % PAGE].double()
        v = st["v_pool"][where[j // PAGE], g, j % PAGE].double()
        for h in range(g * group, (g + 1) * group):
            s = q[:, h] @ k.T / math.sqrt(d)
            out[:, h] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v
    return out


def _exact_pages(case, st):
    """The page calls one entry at a time, on lists."""
    n = st["n_seqs"] * st["per_seq"]
    state = st["start"].tolist()
    table = [state[i:i + st["per_seq"]] for i in range(0, n, st["per_seq"])]
    n_pages = st["n_pages"]

    def references():
        refs = [0] * n_pages
        for r in table:
            for e in r:
                if e >= 0:
                    refs[e] += 1
        return refs

    if case["op"] == "beam":
        table = [list(table[p]) for p in st["parents"].tolist()]
        refs = references()
        free = [p for p in range(n_pages) if not refs[p]]
        length, grants, left = case["prompt"] + case["grown"], [], refs[:]
        for b in range(len(table)):
            for i in range(length // PAGE, (length + case["new"] - 1) // PAGE + 1):
                e = table[b][i]
                if e < 0 or left[e] > 1:
                    grants.append((b, i, e))
                    if e >= 0:
                        left[e] -= 1
        count = max(0, len(grants) - len(free))
        if not count:
            for (b, i, e), f in zip(grants, free):
                if e >= 0 and i == length // PAGE:
                    for pool in st["pools"]:
                        pool[f, :, :length % PAGE] = pool[e, :, :length % PAGE].clone()
                table[b][i] = f
    else:
        for b, length in enumerate(_lens(case)):
            kept = set(_kept(length, case["window"], case["sinks"]))
            table[b] = [e if i in kept else -1 for i, e in enumerate(table[b])]
        refs = references()
        count = sum(1 for r in refs if r)
        holes = [p for p in range(count) if not refs[p]]
        named = {}
        for p in range(count, n_pages):
            if refs[p]:
                named[p] = holes[len(named)]
        for p, to in named.items():
            for pool in st["pools"]:
                pool[to] = pool[p].clone()
        table = [[named.get(e, e) for e in r] for r in table]
    return [_ints(table), _ints(references()), _ints([count]), *st["pools"]]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "axes":
        order = _axis_of_pairs(_pairs(case), case["interleaved"])
        if case["ladders"]:
            freq = [case["theta"] ** (-float(r) / _pairs(case)[a]) for a, r in order]
        else:
            freq = [case["theta"] ** (-2.0 * i / case["dim"]) for i in range(len(order))]
        at = [st["positions"][a] for a, _ in order]
        sign = -1.0 if case["inverse"] else 1.0
        return _exact_turn(st["q"], at, freq, sign), _exact_turn(st["k"], at, freq, sign)
    if case["op"] == "copy":
        src, dst = _copy_plan(case)
        for pool in st["pools"]:
            for a, b in zip(src, dst):
                pool[b] = pool[a].clone()
        return list(st["pools"])
    if case["op"] in ("beam", "compact"):
        return _exact_pages(case, st)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["lens"]):
        if case["op"] == "prefill":
            pos, q, k, v = torch.arange(n, n + case["new"], device=DEV), st["q"][b], st["k"][b], st["v"][b]
        elif n:
            pos, q, k, v = torch.tensor([n - 1], device=DEV), st["q"][b:b + 1], st["k"][b:b + 1], st["v"][b:b + 1]
        else:
            continue
        page = st["table"][b].long()[pos // PAGE]
        st["k_pool"][page, :, pos % PAGE] = _exact_rope(k, pos, case).to(torch.bfloat16)
        st["v_pool"][page, :, pos % PAGE] = v
        q = _exact_rope(q, pos, case)
        o = torch.cat([_exact_attention(st, case, b, q[i:i + 1024], pos[i:i + 1024]) for i in range(0, len(pos), 1024)])
        if case["op"] == "prefill":
            out[b] = o
        else:
            out[b] = o[0]
    return out, st["k_pool"], st["v_pool"]
