"""Shared helpers for the tests over a paged latent cache: inputs, the plain
definitions in 64 bits on the CPU, and the tolerances.

Tolerances (derived from the arithmetic, not from a run):
* a score is an fp32 sum of 576 exact bf16 products: each of at most 576
  additions is off by at most 2^-23 of the sum of magnitudes, so a score is off
  by at most d = 576 * 2^-23 * scale * sum |q||x|, plus 2^-22 of its own size
  for the scaling and the subtraction of the reference;
* a weight exp(score - lse) is then off by a factor of at most exp(2 d) and one
  rounding to bf16 (2^-8) before the product with the values; the weights are
  normalised by the sum of the rounded ones, which adds another 2^-8;
* the output is rounded once to bf16: 2^-8 of its value;
* lse: d, plus the rounding of a sum of n positive fp32 numbers (at most
  n * 2^-24, and 2^-22 for the exponentials), plus 2^-22 of the lse itself.
"""
import numpy as np
import torch

D, DV = 576, 512
SCALE = D ** -0.5


def seen(n, window, sinks):
    """Boolean [n]: the entries of a sequence of n that its newest token sees."""
    s = np.arange(n)
    return np.ones(n, bool) if window == 0 else (s >= n - window) | (s < sinks)


class Cache:
    """A pool of pages on the CPU, a shuffled block table and queries.  Rows
    that no sequence's length covers hold NaN; pages of another layer lie
    between the pool's when layers > 1."""

    def __init__(self, lens, page=16, H=16, seed=0, layers=1, spare=0, q_mul=2.0, extra_pages=0,
                 table_pad=0, poison=True):
        g = torch.Generator().manual_seed(seed)
        self.lens_list, self.page, self.H, self.B = list(lens), page, H, len(lens)
        need = [-(-n // page) for n in lens]
        total = sum(need) + extra_pages
        self.n_pages = max(total, 1) + spare
        x = torch.randn((self.n_pages, layers, page, D), generator=g).to(torch.bfloat16)
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        cols = max(max(need, default=0), 1) + table_pad
        table = torch.full((self.B, cols), -1, dtype=torch.int32)
        at = 0
        covered = torch.zeros((self.n_pages, page), dtype=torch.bool)
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m]
            at += m
            for j in range(m):
                rows = min(page, lens[b] - j * page)
                covered[table[b, j].long(), :rows] = True
        self.free_pages = order[at:]
        if poison:
            x[:, 0][~covered] = float("nan")
        self.full = x
        self.pool = x[:, 0]                     # strided when layers > 1
        self.table, self.lens = table, torch.tensor(lens, dtype=torch.int32).reshape(-1)
        self.max_len = max(lens, default=0)
        self.q = (torch.randn((self.B, H, D), generator=g) * q_mul).to(torch.bfloat16)

    def rows(self, b):
        """The latents of sequence b, [n, 576] bf16."""
        n = self.lens_list[b]
        pages = self.table[b, :-(-n // self.page)].long()
        return self.pool[pages].reshape(-1, D)[:n]

    def to_gpu(self):
        full = self.full.cuda()
        return full[:, 0], self.table.cuda(), self.lens.cuda(), self.q.cuda()


def attention64(q, x, vis, scale=SCALE):
    """One query row set q [H, 576] over latents x [n, 576], entries vis [n]:
    (out, lse, tolerance of out, tolerance of lse) in 64 bits."""
    H = q.shape[0]
    q, x = q.double(), x[torch.from_numpy(vis)].double()
    if x.shape[0] == 0:
        z = torch.zeros((H, DV), dtype=torch.float64)
        return z, torch.full((H,), -np.inf, dtype=torch.float64), z, torch.zeros(H).double()
    s = scale * (q @ x.T)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    out = p @ x[:, :DV]
    d = (576 * 2.0 ** -23 * scale * (q.abs() @ x.abs().T)).amax(1) + 2.0 ** -21 * s.abs().amax(1)
    spread = p @ x[:, :DV].abs()
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -7 * 1.02 + 2.1 * d[:, None]) * spread + 1e-30
    tol_lse = d + x.shape[0] * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -21 * lse.abs()
    return out, lse, tol, tol_lse


def check_rows(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.double().cpu(), tol.double().cpu()
    assert torch.equal(torch.isneginf(got), torch.isneginf(want)), what
    fin = torch.isfinite(want)
    assert torch.isfinite(got[fin]).all(), f"{what}: not finite"
    over = ((got - want).abs() - tol)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{what}: {int((over > 0).sum())} outside, by up to {float(over.max()):.3e}"


class SharedPages:
    """Sequences longer than a pool: block tables that name the pool's pages again and again.
    row(b): the pool row of each entry of sequence b."""

    def __init__(self, lens, page, n_pages, H, seed):
        g = torch.Generator().manual_seed(seed)
        self.lens_list, self.page, self.B, self.H = list(lens), page, len(lens), H
        self.pool = torch.randn((n_pages, page, D), generator=g).to(torch.bfloat16)
        cols = -(-max(lens) // page)
        self.table = torch.randint(0, n_pages, (self.B, cols), generator=g).to(torch.int32)
        self.q = (torch.randn((self.B, H, D), generator=g) * 2).to(torch.bfloat16)

    def row(self, b):
        s = torch.arange(self.lens_list[b])
        return self.table[b].long()[s // self.page] * self.page + s % self.page
