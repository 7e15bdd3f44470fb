"""Window-plus-sinks attention at random sizes against its definition in 64
bits (on the GPU): groups, windows from one position to everything, sinks,
page sizes, lengths, K = V and shared layers, poison in every row and page that
the call must not read, and every pool row that it must not write."""
import math
import random

import pytest
import torch

from hybrid_local_global_b200 import native

from sinks_ref import attention_bound

pytestmark = pytest.mark.gpu
DEV = "cuda"


def log_uniform(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def randn(*shape):
    return torch.randn(*shape, device=DEV).bfloat16()


class Case:
    """lens[b] positions per sequence, the last `new` of them this call's."""

    def __init__(self, rng, new):
        self.new, self.D, self.Hkv = new, rng.choice([256, 512]), log_uniform(rng, 1, 16)
        self.G = rng.choice([1, 2, 2, 3, 4, 5, 6, 7, 8])
        self.B = min(log_uniform(rng, 1, 60 if new == 1 else 3), max(1, 400 // self.Hkv))
        self.window = rng.choice([1, log_uniform(rng, 1, 200), log_uniform(rng, 32, 1500), 1 << 30])
        self.sinks = rng.choice([0, 0, 1, 4, 128, log_uniform(rng, 1, 400), 1 << 30 if rng.random() < 0.2 else 7])
        self.ps, self.scale = rng.choice([128, 256, 384]), rng.choice([self.D ** -0.5, -0.02, 0.15])
        top = rng.choice([log_uniform(rng, 1, 300), log_uniform(rng, 100, 1500)])
        self.lens = [rng.randint(0, top) + new for _ in range(self.B)]
        if new == 1 and rng.random() < 0.3:
            self.lens[rng.randrange(self.B)] = 0  # an idle slot
        self.keqv, self.shared = rng.random() < 0.25, rng.random() < 0.25
        self.flags = (native.GEMMA_F_KEQV if self.keqv else 0) | (native.GEMMA_F_SHARED if self.shared else 0)
        B, ps = self.B, self.ps
        self.pps = (max(max(self.lens), 1) + ps - 1) // ps
        n_pages = B * self.pps + 2
        self.k, self.v = randn(B, new, self.Hkv, self.D), randn(B, new, self.Hkv, self.D)
        self.q = randn(B, new, self.Hkv * self.G, self.D)
        if self.keqv:
            self.v = self.k
        self.K = randn(n_pages, self.Hkv, ps, self.D)
        self.V = self.K if self.keqv else randn(n_pages, self.Hkv, ps, self.D)
        page = torch.randperm(n_pages, device=DEV)[:B * self.pps].view(B, self.pps)
        L = torch.tensor(self.lens, device=DEV)
        pos = torch.arange(self.pps * ps, device=DEV)
        at = (L - new)[:, None] + torch.arange(new, device=DEV)  # [B, new]
        self.see = ((pos <= at[..., None]) & ((pos > at[..., None] - self.window) | (pos < self.sinks))
                    & (L > 0)[:, None, None])
        mine = (pos >= (L - new)[:, None]) & (pos < L[:, None]) & (not self.shared)
        read = self.see.any(1) & ~mine
        # poison all else; entries of pages that are neither read nor written name no page
        bad = torch.ones(n_pages, ps, dtype=torch.bool, device=DEV)
        bad[page.view(-1)] = ~read.view(-1, ps)
        poison = rng.choice([float("nan"), float("inf")])
        self.K.masked_fill_(bad[:, None, :, None], poison)
        self.V.masked_fill_(bad[:, None, :, None], poison)
        used = (read | mine).view(B, self.pps, ps).any(-1)
        self.table = torch.where(used, page, rng.choice([-1, n_pages, 1 << 30])).int()
        # the pools afterwards
        self.K2, self.V2 = self.K.clone(), self.V.clone()
        if not self.shared:
            for b in range(B):
                for i in range(new if self.lens[b] else 0):
                    j = self.lens[b] - new + i
                    self.K2[page[b, j // ps], :, j % ps] = self.k[b, i]
                    self.V2[page[b, j // ps], :, j % ps] = self.v[b, i]
        self.page = page

    def expected(self, b):
        """(out [new, Hq, D], lse [new, Hq], largest |v|) in 64 bits."""
        rows = self.see[b].any(0).nonzero().flatten()
        at = self.page[b, rows // self.ps], slice(None), rows % self.ps
        k, v = self.K2[at].double(), self.V2[at].double()  # [rows, Hkv, D]
        q = self.q[b].double().view(self.new, self.Hkv, self.G, self.D)
        s = torch.einsum("ihgd,khd->ihgk", q, k) * self.scale
        s = s.masked_fill(~self.see[b][:, rows][:, None, None], -math.inf)
        out = torch.einsum("ihgk,khd->ihgd", torch.softmax(s, -1), v)
        return out.reshape(self.new, -1, self.D), torch.logsumexp(s, -1).reshape(self.new, -1), float(v.abs().max())

    def check_pools(self, K, V):
        assert same_bits(K, self.K2) and same_bits(V, self.V2), vars(self)

    def __str__(self):
        return str({k: v for k, v in vars(self).items() if not isinstance(v, torch.Tensor)})


@pytest.mark.parametrize("seed", range(12))
def test_decode_random(seed):
    rng = random.Random(seed)
    torch.manual_seed(seed)
    for _ in range(12):
        c = Case(rng, 1)
        K, V, out = c.K.clone(), c.V.clone(), torch.full_like(c.q[:, 0], float("nan"))
        native.gemma_attn_decode_sinks(
            c.q[:, 0].contiguous(), None if c.shared else c.k[:, 0].contiguous(),
            None if c.shared or c.keqv else c.v[:, 0].contiguous(), K, None if c.keqv else V, c.table,
            seq_lens=torch.tensor(c.lens, dtype=torch.int32, device=DEV), max_seq_len=max(max(c.lens), 1),
            window=c.window, sinks=c.sinks, rope_frac=0.0, rope_theta=1e4, scale=c.scale, out=out, flags=c.flags)
        assert native.gemma_attn_sync_status() == 0, str(c)
        c.check_pools(K, K if c.keqv else V)
        for b, n in enumerate(c.lens):
            if n == 0:
                assert (out[b] == 0).all()
                continue
            want, _, vmax = c.expected(b)
            # the output's rounding; queries and weights keep 16 bits and the sums 32 (logits up to about 16)
            err = (out[b].double() - want[0]).abs() - (2.0 ** -8 * want[0].abs() + 2.0 ** -11 * vmax)
            assert err.max() <= 0, (b, float(err.max()), str(c))


@pytest.mark.parametrize("seed", range(12))
def test_prefill_random(seed):
    rng = random.Random(100 + seed)
    torch.manual_seed(seed)
    for _ in range(5):
        c = Case(rng, rng.choice([2, log_uniform(rng, 2, 200), log_uniform(rng, 100, 900)]))
        K, V, out = c.K.clone(), c.V.clone(), torch.full_like(c.q, float("nan"))
        lse = torch.full((c.B, c.Hkv * c.G, c.new), float("nan"), device=DEV)
        native.gemma_attn_prefill_sinks(
            c.q, None if c.shared else c.k, None if c.shared or c.keqv else c.v, K, None if c.keqv else V, c.table,
            seq_lens_before=torch.tensor([n - c.new for n in c.lens], dtype=torch.int32, device=DEV), window=c.window,
            sinks=c.sinks, rope_frac=0.0, rope_theta=1e4, scale=c.scale, out=out, lse=lse, flags=c.flags)
        assert native.gemma_attn_sync_status() == 0, str(c)
        c.check_pools(K, K if c.keqv else V)
        for b in range(c.B):
            want, want_lse, vmax = c.expected(b)
            err = (out[b].double() - want).abs().max()
            assert err <= attention_bound(want, vmax), (b, float(err), str(c))
            # 32-bit sums of up to 2400 terms and the logits' 32-bit accumulation
            assert (lse[b].double().T - want_lse).abs().max() <= 1e-4 * (1 + float(want_lse.abs().max())), str(c)
