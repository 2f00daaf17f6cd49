"""The paged-cache operators together, as a serving step uses them: a prompt
through the windowed MHA form, its latents in a paged cache, decode steps that
append a latent, attend and add up the weights, then a cut of the cache and
further steps on what is left.

The two forms of MLA meet here: with per-head projections that pick (signed)
latent dims, the prompt's last row in the MHA form equals the decode call's
output of that token, projected."""
import numpy as np
import pytest
import torch

import sparse_attention_08_b200 as dsa
from tests import paged_cases as C
from tests.dsa_cases import assert_no_device_error

pytestmark = pytest.mark.gpu

H, PAGE, WINDOW, SINKS = 16, 16, 150, 4


class Model:
    """Signed-selection projections between a 576-d latent and the MHA form."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        pick = lambda: torch.stack([torch.randperm(512, generator=g)[:128] for _ in range(H)])  # noqa: E731
        sign = lambda: (torch.randint(0, 2, (H, 128), generator=g) * 2 - 1).float()  # noqa: E731
        self.ik, self.sk, self.iv, self.sv = pick(), sign(), pick(), sign()

    def kv(self, lat):
        lat = lat.float()
        k = lat[:, self.ik] * self.sk                                   # [n, H, 128]
        rope = lat[:, None, 512:].expand(-1, H, -1)
        return torch.cat([k, rope], 2).to(torch.bfloat16), (lat[:, self.iv] * self.sv).to(torch.bfloat16)

    def absorbed(self, q):
        """Queries [n, H, 192] of the MHA form as latent queries [n, H, 576]."""
        out = torch.zeros((q.shape[0], H, 576))
        at = self.ik.expand(q.shape[0], -1, -1)
        out.scatter_(2, at, q[..., :128].float() * self.sk)
        out[..., 512:] = q[..., 128:].float()
        return out.to(torch.bfloat16)

    def project(self, out):
        return out.gather(2, self.iv.expand(out.shape[0], -1, -1)) * self.sv


def test_serving_steps():
    g = torch.Generator().manual_seed(90)
    model = Model(91)
    lens = [200, 77]
    B, steps, budget, recent = len(lens), 5, 64, 16
    scale = 192 ** -0.5
    lat = [torch.randn((n + 2 * steps, 576), generator=g).to(torch.bfloat16) for n in lens]
    q = [(torch.randn((n + 2 * steps, H, 192), generator=g) * 1.5).to(torch.bfloat16) for n in lens]

    # the prompt
    kv = [model.kv(x[:n]) for x, n in zip(lat, lens)]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
    T = sum(lens)
    out = torch.empty((T, H, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, H), device="cuda")
    dsa.dsa_window_mha_fwd(torch.cat([x[:n] for x, n in zip(q, lens)]).cuda(),
                           torch.cat([k for k, _ in kv]).cuda(), torch.cat([v for _, v in kv]).cuda(),
                           cu, cu, B, max(lens), max(lens), WINDOW, SINKS, scale, out, lse)
    assert_no_device_error()

    # its latents in pages
    pages = 16
    order = torch.randperm(B * pages + B * 8, generator=g).to(torch.int32)
    table = order[:B * pages].reshape(B, pages)
    free = order[B * pages:].reshape(B, 8)
    pool = torch.full((order.numel(), PAGE, 576), float("nan"), dtype=torch.bfloat16)
    for b, n in enumerate(lens):
        for s in range(n):
            pool[table[b, s // PAGE].long(), s % PAGE] = lat[b][s]
    pool, table, free = pool.cuda(), table.cuda(), free.cuda()
    n_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    most = max(lens) + 2 * steps
    mass = torch.zeros((B, most), device="cuda")
    o = torch.empty((B, H, 512), dtype=torch.bfloat16, device="cuda")
    ls = torch.empty((B, H), device="cuda")

    def decode(tokens, tab, m):
        ql = model.absorbed(torch.stack([q[b][t] for b, t in enumerate(tokens)]))
        dsa.dsa_paged_mla_decode(ql.cuda(), pool, tab, n_d, most, scale, o, ls, window=WINDOW,
                                 sinks=SINKS)
        dsa.dsa_paged_attn_mass(ql.cuda(), pool, tab, n_d, ls, most, scale, m, mass_in=m,
                                window=WINDOW, sinks=SINKS)
        return ql

    # the prompt's last token again, through the cache
    decode([n - 1 for n in lens], table, mass)
    assert_no_device_error()
    got = model.project(o.cpu().float())
    for b in range(B):
        last = int(cu[b + 1]) - 1
        want = out[last].cpu().float()
        # both forms round the weights (2^-8 of them) and the result (2^-8)
        tol = 4 * 2.0 ** -8 * (want.abs() + 4.0 * float(lat[b][:lens[b]].float().std()))
        assert ((got[b] - want).abs() <= tol).all()
        assert float((ls[b] - lse[last]).abs().max()) < 1e-3
    mass.zero_()

    def append(b, row, n, tab):
        pool[tab[b, n // PAGE].long(), n % PAGE] = row.cuda()

    held = [x[:n].clone() for x, n in zip(lat, lens)]
    total = [torch.zeros(most, dtype=torch.float64) for _ in lens]

    def check(ql):
        for b in range(B):
            vis = C.seen(held[b].shape[0], WINDOW, SINKS)
            w, wl, tol, tol_l = C.attention64(ql[b], held[b], vis, scale)
            C.check_rows(o[b], w, tol, f"out of sequence {b}")
            C.check_rows(ls[b], wl, tol_l, f"lse of sequence {b}")
            v = torch.from_numpy(vis).nonzero().flatten()
            z = scale * (held[b][v].double() @ ql[b].double().T)
            total[b][v] += torch.exp(z - wl).sum(1)

    def run_steps(first, tab, m):
        for i in range(steps):
            for b in range(B):
                append(b, lat[b][lens[b] + first + i], held[b].shape[0], tab)
                held[b] = torch.cat([held[b], lat[b][lens[b] + first + i][None]])
            n_d.add_(1)
            ql = decode([n + first + i for n in lens], tab, m)
            assert_no_device_error()
            check(ql)

    run_steps(0, table, mass)
    for b in range(B):
        n = held[b].shape[0]
        assert float((mass[b, :n].cpu().double() - total[b][:n]).abs().max()) < 1e-4 * steps * H

    # the cut, by the totals the calls added up
    new_lens = torch.empty_like(n_d)
    idx = torch.empty((B, budget), dtype=torch.int32, device="cuda")
    new_mass = torch.zeros((B, most), device="cuda")
    dsa.dsa_cache_evict(pool, table, n_d, mass, most, budget, SINKS, recent, free, new_lens, idx,
                        new_mass)
    assert_no_device_error()
    for b in range(B):
        n = held[b].shape[0]
        row = mass[b].cpu()
        mid = sorted(range(SINKS, n - recent), key=lambda i: (-float(row[i]), i))
        keep = sorted(list(range(SINKS)) + mid[:budget - SINKS - recent] + list(range(n - recent, n)))
        assert idx[b].tolist() == keep
        held[b] = held[b][keep]
        total[b] = torch.zeros(most, dtype=torch.float64)
        total[b][:budget] = row[keep].double()
    n_d.copy_(new_lens)
    run_steps(steps, free, new_mass)
    for b in range(B):
        n = held[b].shape[0]
        assert n == budget + steps
        assert float((new_mass[b, :n].cpu().double() - total[b][:n]).abs().max()) < 1e-4 * 2 * steps * H


def test_empty_batches():
    """No sequences, or sequences without room for an entry: the addresses of empty tensors are
    null, and nothing is to be read or written through them."""
    dev, bf16, i32 = "cuda", torch.bfloat16, torch.int32
    pool = torch.full((3, PAGE, 576), float("nan"), dtype=bf16, device=dev)
    for B, most in ((0, 40), (0, 0), (2, 0)):
        q = torch.ones((B, H, 576), dtype=bf16, device=dev)
        table = torch.full((B, 3), -1, dtype=i32, device=dev)
        n = torch.zeros(B, dtype=i32, device=dev)
        out = torch.full((B, H, 512), 7.0, dtype=bf16, device=dev)
        lse = torch.full((B, H), 7.0, device=dev)
        mass = torch.empty((B, most), device=dev)
        new_mass = torch.full((B, 20), 7.0, device=dev)
        new_n, idx = torch.full_like(n, 7), torch.full((B, 20), 7, dtype=i32, device=dev)
        dsa.dsa_paged_mla_decode(q, pool, table, n, most, 0.04, out, lse)
        dsa.dsa_paged_attn_mass(q, pool, table, n, lse, most, 0.04, mass, mass_in=mass)
        dsa.dsa_cache_evict(pool, table, n, mass, most, 20, 2, 4, table + 1, new_n, idx, new_mass)
        assert_no_device_error()
        assert (out == 0).all() and torch.isneginf(lse).all()
        assert (new_n == 0).all() and (idx == -1).all() and (new_mass == 0).all()
    assert torch.isnan(pool.float()).all()


def test_pages_far_apart():
    """Offsets that pass 32 bits: pages 2^27 elements apart (a page of many layers), the last ones
    5 GB behind the first."""
    budget, window, sinks = 64, 100, 3
    c = C.Cache([300, 170], page=16, H=H, seed=92, extra_pages=8)
    far = torch.empty((c.n_pages, 1 << 27), dtype=torch.bfloat16, device="cuda")
    pool = far[:, :16 * 576].view(c.n_pages, 16, 576)
    pool.copy_(c.pool)
    table, n, q = c.table.cuda(), c.lens.cuda(), c.q.cuda()
    o, ls = torch.empty((2, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((2, H), device="cuda")
    mass = torch.zeros((2, 300), device="cuda")
    dsa.dsa_paged_mla_decode(q, pool, table, n, 300, C.SCALE, o, ls, window=window, sinks=sinks)
    dsa.dsa_paged_attn_mass(q, pool, table, n, ls, 300, C.SCALE, mass, mass_in=mass, window=window, sinks=sinks)
    free = c.free_pages[:8].reshape(2, 4)
    idx, new_n = torch.empty((2, budget), dtype=torch.int32, device="cuda"), torch.empty_like(n)
    dsa.dsa_cache_evict(pool, table, n, mass, 300, budget, 4, 16, free.cuda(), new_n, idx)
    assert_no_device_error()
    for b, k in enumerate(c.lens_list):
        want, wl, tol, tol_l = C.attention64(c.q[b], c.rows(b), C.seen(k, window, sinks))
        C.check_rows(o[b], want, tol, f"out of sequence {b}")
        C.check_rows(ls[b], wl, tol_l, f"lse of sequence {b}")
        got = pool[free[b].long().cuda()].reshape(-1, 576)[:budget].cpu()
        kept = idx[b].cpu().long()
        assert kept.tolist()[:4] == [0, 1, 2, 3] and kept.tolist()[-16:] == list(range(k - 16, k))
        assert torch.equal(got.view(torch.int16), c.rows(b)[kept].view(torch.int16))
