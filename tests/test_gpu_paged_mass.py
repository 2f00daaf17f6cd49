"""dsa_paged_attn_mass against the plain definition in 64 bits.

Tolerance: a score and its lse enter an exponential, so with d the bound on a
score's error (tests/paged_cases.py) a weight is off by a factor of at most
exp(d) plus 2^-22 of it; the sum over H heads and the addition to the total round
H + 2 times, each by at most 2^-24 of the result."""
import numpy as np
import pytest
import torch

import sparse_attention_08_b200 as dsa
from tests import paged_cases as C
from tests.dsa_cases import assert_no_device_error

pytestmark = pytest.mark.gpu


def want(c, lse, mass_in, window, sinks):
    out, tol = [], []
    for b, n in enumerate(c.lens_list):
        vis = torch.from_numpy(C.seen(n, window, sinks))
        m = mass_in[b, :n].double()
        t = 2.0 ** -23 * m.abs()
        if n:
            x = c.rows(b)[vis].double()
            q = c.q[b].double()
            s = C.SCALE * (x @ q.T)
            d = 576 * 2.0 ** -23 * C.SCALE * (x.abs() @ q.abs().T) + 2.0 ** -21 * (s.abs() + lse[b].double().abs())
            e = torch.exp(s - lse[b].double())
            w = e.sum(1)
            m[vis] += w
            t[vis] += (e * (torch.exp(d) - 1 + 2.0 ** -21)).sum(1) + (c.H + 2) * 2.0 ** -24 * m[vis].abs()
        out.append(m)
        tol.append(t + 1e-30)
    return out, tol


def run(c, window=0, sinks=0, lse=None, in_place=False, no_in=False, pad=3):
    g = torch.Generator().manual_seed(5)
    width = c.max_len + pad
    mass_in = torch.rand((c.B, width), generator=g) * 3
    if lse is None:
        lse = torch.stack([C.attention64(c.q[b], c.rows(b), C.seen(n, window, sinks))[1].float()
                           for b, n in enumerate(c.lens_list)])
    pool, table, lens, q = c.to_gpu()
    m_in = mass_in.cuda()
    out = m_in if in_place else torch.full((c.B, width), -7.0, device="cuda")
    dsa.dsa_paged_attn_mass(q, pool, table, lens, lse.cuda(), c.max_len, C.SCALE, out,
                            mass_in=None if no_in else m_in, window=window, sinks=sinks)
    assert_no_device_error()
    base = torch.zeros_like(mass_in) if no_in else mass_in
    rows, tol = want(c, lse, base, window, sinks)
    got = out.cpu()
    for b, n in enumerate(c.lens_list):
        C.check_rows(got[b, :n], rows[b], tol[b], f"sequence {b}")
        rest = mass_in[b, n:] if in_place else torch.full((width - n,), -7.0)
        assert torch.equal(got[b, n:], rest), "entries past the length"
    return out


@pytest.mark.parametrize("lens,H,page", [
    ([1], 16, 16), ([5, 0, 128, 129], 16, 16), ([127, 300, 1], 32, 48), ([700, 64, 257], 64, 64),
    ([513, 1000], 128, 32), ([260, 5], 192, 256), ([130, 33], 256, 128),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_small(lens, H, page, in_place):
    run(C.Cache(lens, page=page, H=H, seed=40 + H), in_place=in_place)


@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 0), (128, 4), (300, 130), (640, 1), (9999, 3)])
@pytest.mark.parametrize("in_place,no_in", [(False, False), (True, False), (False, True)])
def test_window(window, sinks, in_place, no_in):
    c = C.Cache([1, 77, 640, 1029, 0, 2000], page=16, H=16, seed=41)
    for b, n in enumerate(c.lens_list):
        vis = torch.from_numpy(C.seen(n, window, sinks))
        for s in (~vis).nonzero().flatten().tolist():
            c.pool[c.table[b, s // 16].long(), s % 16] = float("nan")
    run(c, window, sinks, in_place=in_place, no_in=no_in)


def test_long_many_and_strided():
    run(C.Cache([20111], page=64, H=16, seed=42))
    run(C.Cache([(37 * i) % 211 for i in range(700)], page=16, H=16, seed=43))
    run(C.Cache([300, 290, 40], page=32, H=32, seed=44, layers=3, table_pad=5, spare=2))


def test_with_the_decode_call_and_in_a_graph():
    """The weights of one token add up to H, whatever the window."""
    c = C.Cache([3000, 17, 129], page=64, H=128, seed=45)
    pool, table, lens, q = c.to_gpu()
    out = torch.empty((3, 128, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 128), device="cuda")
    mass = torch.zeros((3, 3000), device="cuda")

    def step():
        dsa.dsa_paged_mla_decode(q, pool, table, lens, 3000, C.SCALE, out, lse, window=500, sinks=4)
        dsa.dsa_paged_attn_mass(q, pool, table, lens, lse, 3000, C.SCALE, mass, mass_in=mass,
                                window=500, sinks=4)

    step()
    assert_no_device_error()
    # weights of a softmax whose lse has relative error d: sums within H * (d + roundings)
    assert float((mass.double().sum(1) - 128).abs().max()) < 128 * 1e-4
    first = mass.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    graph.replay()
    assert_no_device_error()
    assert torch.allclose(mass, 3 * first, rtol=1e-6)


def test_infinite_total_and_nan_entry():
    c = C.Cache([200, 130], page=16, H=16, seed=46)
    lse = torch.stack([C.attention64(c.q[b], c.rows(b), np.ones(n, bool))[1].float()
                       for b, n in enumerate(c.lens_list)])
    c.pool[c.table[0, 3].long(), 2] = float("nan")
    pool, table, lens, q = c.to_gpu()
    m = torch.zeros((2, 200), device="cuda")
    m[1, 5] = float("inf")
    dsa.dsa_paged_attn_mass(q, pool, table, lens, lse.cuda(), 200, C.SCALE, m, mass_in=m)
    assert_no_device_error()
    assert torch.isnan(m[0, 50]) and int(torch.isnan(m).sum()) == 1
    assert torch.isinf(m[1, 5]) and int(torch.isinf(m).sum()) == 1


@pytest.mark.parametrize("B", [3, 41, 300, 700])
def test_totals_between_the_first_tokens_and_the_window(B):
    """Gaps from none to several thousand entries, in more and in fewer sequences than there are
    warps to copy them."""
    top = 20000 if B < 10 else 900
    lens = [(1 + 7919 * i) % top for i in range(B)]
    lens[-1] = top
    for window, sinks, no_in in ((60, 1, False), (300, 130, False), (60, 5, True), (0, 0, False)):
        run(C.Cache(lens, page=16, H=16, seed=47), window, sinks, no_in=no_in)


def test_weights_of_far_scores_are_as_exact_as_near_ones():
    """Scores that are exact (whole numbers times 1/16) around a large lse, one head at a time (the
    others' weights are 0), so that only the exponential rounds: t = score - lse once (2^-24 of
    t), the change to base 2 by its constant and its product (2^-24 each of t), exp2 by 2^-22
    of the weight."""
    n, H, scale = 61, 16, 1.0 / 16
    c = C.Cache([n], page=16, H=H, seed=48)
    d = torch.arange(n).float()
    for s in range(n):
        c.pool[c.table[0, s // 16].long(), s % 16] = 8.0
        c.pool[c.table[0, s // 16].long(), s % 16, 0] = 8.0 + d[s]
    c.q[:] = 1.0
    pool, table, lens, q = c.to_gpu()
    at = torch.tensor([288.37, 290.3, 291.77] * 6)[:H]
    for h in range(H):
        lse = torch.full((1, H), 1e30)
        lse[0, h] = at[h]
        out = torch.zeros((1, n), device="cuda")
        dsa.dsa_paged_attn_mass(q, pool, table, lens, lse.cuda(), n, scale, out)
        assert_no_device_error()
        t = (4608 + d.double()) * scale - lse[0, h].double()
        off = (out[0].cpu().double() / torch.exp(t) - 1).abs()
        assert (off <= 3 * 2.0 ** -24 * t.abs() + 2.0 ** -22 + 1e-9).all(), float(off.max())


@pytest.mark.parametrize("window,sinks", [(0, 0), ((1 << 23) + 5, 1000)])
def test_longest_sequences_entry_by_entry(window, sinks):
    """One head without a query and with lse = 0 (the others' weights are 0): every entry that is
    seen gets exactly 1."""
    lens = [1 << 24, (1 << 24) - 37]
    c = C.SharedPages(lens, 64, 400, 16, seed=49)
    c.q[:, 5] = 0
    lse = torch.full((2, 16), 1e30)
    lse[:, 5] = 0
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    m = torch.full((2, 1 << 24), 2.0, device="cuda")
    out = torch.full((2, 1 << 24), -7.0, device="cuda")
    dsa.dsa_paged_attn_mass(c.q.cuda(), c.pool.cuda(), c.table.cuda(), n, lse.cuda(), 1 << 24, C.SCALE, out,
                            mass_in=m, window=window, sinks=sinks)
    assert_no_device_error()
    for b, k in enumerate(lens):
        want = torch.full((1 << 24,), -7.0)
        want[:k] = 2.0 + torch.from_numpy(C.seen(k, window, sinks)).float()
        assert torch.equal(out[b].cpu(), want)
