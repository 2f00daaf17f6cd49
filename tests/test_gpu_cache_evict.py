"""dsa_cache_evict against sorting on the CPU: positions, totals and latents are
copies, so everything is compared exactly."""
import pytest
import torch

import sparse_attention_08_b200 as dsa
from tests import paged_cases as C
from tests.dsa_cases import assert_no_device_error

pytestmark = pytest.mark.gpu

DSA_ERR_BOUNDS = 7


def keep_of(row, n, budget, sinks, recent):
    if n <= budget:
        return list(range(n))
    mid = list(range(sinks, n - recent))
    key = row.double()
    key = torch.where(torch.isnan(key), torch.full_like(key, float("inf")), key).tolist()
    nan = torch.isnan(row).tolist()
    mid.sort(key=lambda i: (not nan[i], -key[i], i))
    return sorted(list(range(sinks)) + mid[:budget - sinks - recent] + list(range(n - recent, n)))


def run(c, mass, budget, sinks, recent, with_mass=True, max_len=None):
    kept = [min(n, budget) for n in c.lens_list]
    need = [-(-k // c.page) for k in kept]
    most = max_len or c.max_len
    cols = max(-(-min(budget, most) // c.page), 1)
    new_table = torch.full((c.B, cols + 2), -5, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        new_table[b, :m] = c.free_pages[at:at + m]
        at += m
    full = c.full.cuda()
    pool = full[:, 0]
    table, lens, m = c.table.cuda(), c.lens.cuda(), mass.cuda()
    idx = torch.full((c.B, budget), -9, dtype=torch.int32, device="cuda")
    new_lens = torch.full((c.B,), -9, dtype=torch.int32, device="cuda")
    new_mass = torch.full((c.B, budget + 3), -9.0, device="cuda") if with_mass else None
    dsa.dsa_cache_evict(pool, table, lens, m, most, budget, sinks, recent, new_table.cuda(),
                        new_lens, idx, new_mass)
    assert_no_device_error()
    want_pool = c.full.clone()
    for b, n in enumerate(c.lens_list):
        keep = keep_of(mass[b], n, budget, sinks, recent)
        assert int(new_lens[b]) == len(keep)
        got = idx[b].cpu().tolist()
        assert got == keep + [-1] * (budget - len(keep)), f"positions of sequence {b}"
        if with_mass:
            w = torch.cat([mass[b, keep], torch.zeros(budget - len(keep)), torch.full((3,), -9.0)])
            assert torch.equal(new_mass[b].cpu().view(torch.int32), w.view(torch.int32))
        rows = c.rows(b)[keep]
        for j in range(len(keep)):
            want_pool[new_table[b, j // c.page].long(), 0, j % c.page] = rows[j]
    # the old pages, other layers and the rows behind the kept ones are untouched
    assert torch.equal(full.cpu().view(torch.int16), want_pool.view(torch.int16))


def pages_for(lens, budget, page):
    return sum(-(-min(n, budget) // page) for n in lens)


def cache(lens, page, budget, seed, **kw):
    return C.Cache(lens, page=page, H=16, seed=seed, extra_pages=pages_for(lens, budget, page), **kw)


def totals(c, seed, kind="heavy"):
    g = torch.Generator().manual_seed(seed)
    m = torch.exp(2 * torch.randn((c.B, c.max_len + 1), generator=g))
    if kind == "zeros":
        m[torch.rand(m.shape, generator=g) < 0.7] = 0.0
        m[torch.rand(m.shape, generator=g) < 0.1] = -0.0
    elif kind == "equal":
        m.fill_(1.25)
    elif kind == "few":
        m = torch.randint(0, 3, m.shape, generator=g).float() - 1
    elif kind == "rising":
        m = torch.arange(m.shape[1]).float().repeat(c.B, 1)
    elif kind == "odd":
        m[torch.rand(m.shape, generator=g) < 0.02] = float("nan")
        m[torch.rand(m.shape, generator=g) < 0.02] = float("inf")
        m[torch.rand(m.shape, generator=g) < 0.02] = float("-inf")
        m[torch.rand(m.shape, generator=g) < 0.2] *= -1
        m[torch.rand(m.shape, generator=g) < 0.1] = 1e-42
    return m


@pytest.mark.parametrize("kind", ["heavy", "zeros", "equal", "few", "rising", "odd"])
@pytest.mark.parametrize("lens,page,budget,sinks,recent", [
    ([1, 0, 100, 101, 700], 16, 100, 4, 32),
    ([333, 64, 65], 48, 64, 0, 0),
    ([500, 3], 32, 1, 0, 1),                  # a budget of the newest entry alone
    ([500, 40], 16, 37, 37, 0),               # of the first entries alone
    ([9000, 8193, 20], 64, 2000, 4, 100),     # a cluster per sequence
])
def test_kept_entries(kind, lens, page, budget, sinks, recent):
    c = cache(lens, page, budget, seed=60)
    run(c, totals(c, 61, kind), budget, sinks, recent)


def test_long_rows_and_one_cta_limit():
    c = cache([40000, 8192, 33000], 128, 5000, seed=62)
    run(c, totals(c, 63, "heavy"), 5000, 16, 512)
    c = cache([8192, 8191], 16, 8191, seed=64)
    run(c, totals(c, 65, "zeros"), 8191, 1, 1, max_len=8192)


def test_strided_pool_without_totals_out():
    c = cache([300, 90], 16, 128, seed=66, layers=3, table_pad=4)
    run(c, totals(c, 67), 128, 2, 10, with_mass=False)


def test_bad_pages_are_reported_and_skipped():
    c = cache([100, 100], 16, 32, seed=68)
    m = totals(c, 69).cuda()
    pool, table, lens, _ = c.to_gpu()
    before = pool.clone()
    new_table = torch.tensor([[10 ** 6, 0], [-1, -1]], dtype=torch.int32, device="cuda")
    new_table[0, 1] = c.free_pages[0]
    idx = torch.empty((2, 32), dtype=torch.int32, device="cuda")
    nl = torch.empty(2, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_evict(pool, table, lens, m, 100, 32, 1, 1, new_table, nl, idx)
    assert dsa.dsa_get_device_error() == DSA_ERR_BOUNDS
    same = (pool.view(torch.int16) == before.view(torch.int16)).flatten(1).all(1)
    same[c.free_pages[0].long()] = True
    assert same.all()
    assert nl.tolist() == [32, 32]


def test_replayed_in_a_graph_follows_the_lengths():
    c = cache([300, 200], 16, 64, seed=70)
    m = totals(c, 71)
    pool, table, lens, _ = c.to_gpu()
    nt = c.free_pages[:8].reshape(2, 4).cuda()
    idx = torch.empty((2, 64), dtype=torch.int32, device="cuda")
    nl = torch.empty(2, dtype=torch.int32, device="cuda")
    md = m.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_cache_evict(pool, table, lens, md, 300, 64, 4, 8, nt, nl, idx)
    for ns in ([300, 200], [10, 65], [0, 64]):
        lens.copy_(torch.tensor(ns, dtype=torch.int32))
        graph.replay()
        assert_no_device_error()
        for b, n in enumerate(ns):
            keep = keep_of(m[b], n, 64, 4, 8)
            assert idx[b].cpu().tolist() == keep + [-1] * (64 - len(keep))
            assert int(nl[b]) == len(keep)


@pytest.mark.parametrize("graph", [False, True])
def test_cuts_of_cuts_without_a_pause(graph):
    """Each cut reads the lengths, totals, table and latents that the one before it on the
    stream has only just written (or is still writing when it starts)."""
    lens, page, budgets = [30000, 9000, 2500, 31000], 64, [9000, 4000, 900]
    c = C.Cache(lens, page=page, H=16, seed=72, extra_pages=sum(pages_for(lens, k, page) for k in budgets))
    m = totals(c, 73, "zeros")
    tables, at = [], 0
    for k in budgets:
        t = torch.full((4, -(-k // page)), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            need = -(-min(n, k) // page)
            t[b, :need] = c.free_pages[at:at + need]
            at += need
        tables.append(t)
    pool, table, n_d, _ = c.to_gpu()
    first = pool.clone()
    dev = [t.cuda() for t in tables]
    idx = [torch.empty((4, k), dtype=torch.int32, device="cuda") for k in budgets]
    n_new = [torch.empty_like(n_d) for _ in budgets]
    m_new = [torch.empty((4, k), device="cuda") for k in budgets]
    m_d = m.cuda()

    def cuts():
        tab, n, mass, most = table, n_d, m_d, c.max_len
        for i, k in enumerate(budgets):
            dsa.dsa_cache_evict(pool, tab, n, mass, most, k, 4, 100, dev[i], n_new[i], idx[i], m_new[i])
            tab, n, mass, most = dev[i], n_new[i], m_new[i], k

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cuts()
        g.replay()
        g.replay()
    else:
        cuts()
    assert_no_device_error()
    assert torch.equal(table, c.table.cuda())
    for b, n in enumerate(lens):
        row, rows, held = m[b], c.rows(b), n
        for i, k in enumerate(budgets):
            keep = keep_of(row, held, k, 4, 100)
            held = len(keep)
            assert int(n_new[i][b]) == held
            assert idx[i][b].cpu().tolist() == keep + [-1] * (k - held)
            row, rows = torch.cat([row[keep], torch.zeros(k - held)]), rows[keep]
            assert torch.equal(m_new[i][b].cpu().view(torch.int32), row.view(torch.int32))
            got = pool[tables[i][b, :-(-held // page)].long().cuda()].reshape(-1, 576)[:held].cpu()
            assert torch.equal(got.view(torch.int16), rows.view(torch.int16))
    used = torch.cat([t[t >= 0] for t in tables]).long()
    rest = torch.ones(c.n_pages, dtype=torch.bool)
    rest[used] = False
    assert torch.equal(pool[rest.cuda()].view(torch.int16), first[rest.cuda()].view(torch.int16))


@pytest.mark.parametrize("lens,budget,kind", [
    ([262144, 262143, 150000], 8192, "heavy"), ([262144], 262143, "zeros"), ([262144, 262000], 2048, "few"),
])
def test_longest_rows(lens, budget, kind):
    """Rows of the largest size that is allowed, over a pool whose pages they name many times."""
    page, shared, B = 128, 200, len(lens)
    per = -(-budget // page)
    c = C.SharedPages(lens, page, shared + B * per, 16, seed=74)
    c.table %= shared
    new_table = shared + torch.randperm(B * per, generator=torch.Generator().manual_seed(75)).reshape(B, per).to(torch.int32)
    c.max_len = 262144
    m = totals(c, 76, kind)
    pool = c.pool.cuda()
    idx = torch.empty((B, budget), dtype=torch.int32, device="cuda")
    new_n = torch.empty(B, dtype=torch.int32, device="cuda")
    new_m = torch.empty((B, budget), device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_evict(pool, c.table.cuda(), n, m.cuda(), 262144, budget, 4, 1000, new_table.cuda(), new_n, idx, new_m)
    assert_no_device_error()
    assert new_n.tolist() == [min(k, budget) for k in lens]
    want = c.pool.reshape(-1, 576).clone()
    for b, k in enumerate(lens):
        keep = torch.tensor(keep_of(m[b], k, budget, 4, 1000))
        assert torch.equal(idx[b].cpu().long(), keep)
        assert torch.equal(new_m[b].cpu().view(torch.int32), m[b, keep].view(torch.int32))
        j = torch.arange(keep.numel())
        want[new_table[b].long()[j // page] * page + j % page] = c.pool.reshape(-1, 576)[c.row(b)[keep]]
    assert torch.equal(pool.cpu().view(torch.int16), want.reshape(pool.shape).view(torch.int16))
