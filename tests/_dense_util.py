"""Caches of chosen bytes and the 64-bit definition of dense attention, with
the bounds its kernels are held to."""
from __future__ import annotations

import math

import torch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


class DenseCase:
    """A paged cache of random codes and scales on the GPU, and its dequantised
    rows in 64 bits on the CPU.  Slots that hold no entry (behind a sequence's
    last, pages of no sequence) hold NaN scales."""

    def __init__(self, csa2, lens, page=64, seed=0, spare=2, extra_cols=1, scale_lo=0.1):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page = list(lens), page
        need = [-(-n // page) for n in lens]
        P = sum(need) + spare
        perm = torch.randperm(P, generator=g).int()
        table = torch.full((len(lens), max(need + [0]) + extra_cols), -1, dtype=torch.int32)
        o = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[o:o + n]
            o += n
        codes = torch.randint(0, 256, (P * page, 128), generator=g, dtype=torch.uint8)
        s = (torch.rand((P * page, 16), generator=g) * 0.5 + scale_lo).to(torch.float8_e4m3fn)
        scales = torch.full((P * page, 16), 0x7F, dtype=torch.uint8)
        self.table = table
        for b, n in enumerate(lens):
            sl = self.slots(b, n)
            scales[sl] = s.view(torch.uint8)[sl]
        self.codes, self.scales = codes, scales
        self.csa2 = csa2
        self.upload()

    def upload(self):
        self.cache = self.csa2.KVCache.from_tensors(self.codes.cuda(), self.scales.cuda(), self.table.cuda(), self.page)
        self.max_len = self.table.shape[1] * self.page
        return self

    def slots(self, b, n):
        pos = torch.arange(n)
        return self.table[b].long()[pos // self.page] * self.page + pos % self.page

    def rows(self, b):
        """[n, 256] fp64: K | V of the sequence's entries."""
        sl = self.slots(b, self.lens[b])
        c = self.codes[sl].int()
        x = torch.stack([E2M1[c & 15], E2M1[c >> 4]], 2).view(-1, 256)
        return x * self.scales[sl].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


def queries(n, seed=1, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, 16, 128), generator=g) * gain).to(torch.bfloat16)


def reference(q, rows, seen, hidden=None):
    """The definition for q [n, 16, 128] over rows [L, 256]; seen [n] leading
    entries each; hidden: indices nobody sees.  Returns out, lse and their
    bounds (before the output's own rounding), all fp64.

    Bounds.  A score is 128 products, each exact in fp32 or wider, summed in
    fp32: its error is at most 128 * 2^-24 of sum |q k|, and the scaling by
    log2(e) / sqrt(128) adds 2^-22 of |s|; call the largest over an entry row ds.
    exp moves by ds relative, its own error is below 2^-20, the sum of n weights
    n * 2^-24; numerator and denominator each, so
      out: 2 (ds + 2^-20 + n 2^-24) sum w |v|   lse: ds + 2^-20 + n 2^-24 + 2^-23 |lse|
    and the weights' rounding (the caller's) comes on top.  Weights are held as
    fp16 times 2^7 over a maximum that is at most the largest score, so the
    smallest fp16 step, 2^-24, rounds a weight far below the largest by up to
    2^-25 / 2^7 = 2^-32 (of a sum that is at least 1): 2^-32 sum |v| more."""
    n, L = q.shape[0], rows.shape[0]
    out = torch.zeros((n, 16, 128), dtype=torch.float64)
    lse = torch.full((n, 16), -math.inf, dtype=torch.float64)
    spread, b_out, b_lse = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(lse)
    qd = q.double()
    for i in range(n):
        m = int(seen[i])
        keep = torch.ones(m, dtype=torch.bool)
        if hidden is not None:
            keep[[h for h in hidden if h < m]] = False
        k, v = rows[:m][keep, :128], rows[:m][keep, 128:]
        if not k.shape[0]:
            continue
        s = qd[i] @ k.T / math.sqrt(128)
        mag = qd[i].abs() @ k.abs().T / math.sqrt(128)
        lse[i] = torch.logsumexp(s, 1)
        w = torch.exp(s - lse[i][:, None])
        out[i] = w @ v
        spread[i] = w @ v.abs()
        ds = (mag * 128 * 2.0 ** -24 + s.abs() * 2.0 ** -22).amax(1)
        e = ds + 2.0 ** -20 + k.shape[0] * 2.0 ** -24
        b_out[i] = 2 * e[:, None] * spread[i] + v.abs().sum(0) * 2.0 ** -32
        b_lse[i] = e + lse[i].abs() * 2.0 ** -23
    return out, lse, spread, b_out, b_lse


def check(out, lse, ref, what=""):
    """Weights rounded to fp16 (half a step: 2^-11) for a bf16 result, carried in
    two fp16 terms (2^-22) for an fp32 one; the result's own rounding is 2^-8 or
    2^-24 of it."""
    r_out, r_lse, spread, b_out, b_lse = ref
    bf = out.dtype == torch.bfloat16
    got, gl = out.double().cpu(), lse.double().cpu()
    tol = b_out + spread * (2.0 ** -11 if bf else 2.0 ** -22) + r_out.abs() * (2.0 ** -8 if bf else 2.0 ** -24)
    assert torch.equal(torch.isnan(got), torch.isnan(r_out)), f"{what}: NaN where none belongs, or the other way"
    fine = ~torch.isnan(r_out)
    worst = ((got - r_out).abs() - tol)[fine]
    assert not fine.any() or worst.max() <= 0, f"{what}: out off by {worst.max():.3g} beyond its bound"
    empty = r_lse == -math.inf
    assert torch.equal(gl == -math.inf, empty), f"{what}: empty rows"
    ok = ~empty & ~torch.isnan(r_lse)
    d = ((gl - r_lse).abs() - b_lse)[ok]
    assert not ok.any() or d.max() <= 0, f"{what}: lse off by {d.max():.3g} beyond its bound"
