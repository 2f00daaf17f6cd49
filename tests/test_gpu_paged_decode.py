"""dsa_paged_mla_decode against the plain definition in 64 bits."""
import pytest
import torch

import sparse_attention_08_b200 as dsa
from tests import paged_cases as C
from tests.dsa_cases import assert_no_device_error

pytestmark = pytest.mark.gpu

DSA_ERR_BOUNDS = 7


def run(c, window=0, sinks=0, lse=True, **kw):
    pool, table, lens, q = c.to_gpu()
    out = torch.full((c.B, c.H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((c.B, c.H), float("nan"), device="cuda") if lse else None
    dsa.dsa_paged_mla_decode(q, pool, table, lens, c.max_len, C.SCALE, out, ls, window=window,
                             sinks=sinks, **kw)
    assert_no_device_error()
    return out, ls


def check(c, out, lse, window=0, sinks=0):
    for b in range(c.B):
        vis = C.seen(c.lens_list[b], window, sinks)
        o, l, tol, tol_l = C.attention64(c.q[b], c.rows(b), vis)
        C.check_rows(out[b], o, tol, f"out of sequence {b}")
        if lse is not None:
            C.check_rows(lse[b], l, tol_l, f"lse of sequence {b}")


@pytest.mark.parametrize("lens,H,page", [
    ([1], 16, 16),                              # one entry
    ([5, 0, 128, 129], 16, 16),                 # an empty sequence, a full tile, one over
    ([127, 300, 1], 32, 48),                    # pages of 48 rows: tiles and pages end apart
    ([700, 64, 257], 64, 64),
    ([513, 1000], 128, 32),                     # two head groups
    ([260], 192, 256),                          # three head groups, a page beyond the tile
    ([130, 33], 256, 128),
])
def test_small(lens, H, page):
    c = C.Cache(lens, page=page, H=H, seed=len(lens) + H)
    check(c, *run(c))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (100, 0), (128, 4), (300, 130), (5000, 7),
                                          (640, 1)])
def test_window_and_sinks(window, sinks):
    c = C.Cache([1, 77, 640, 1029, 0], page=16, H=16, seed=7)
    # what a windowed layer's cache holds outside the window is not looked at
    for b, n in enumerate(c.lens_list):
        vis = torch.from_numpy(C.seen(n, window, sinks))
        for s in (~vis).nonzero().flatten().tolist():
            c.pool[c.table[b, s // 16].long(), s % 16] = float("nan") if s % 2 else float("inf")
    check(c, *run(c, window, sinks), window, sinks)


def test_split_over_the_gpu():
    # 158 tiles on 148 pieces, and a batch whose sequences end inside pieces
    c = C.Cache([20111], page=64, H=16, seed=21)
    check(c, *run(c))
    c = C.Cache([9000, 3, 12345, 0, 4097], page=128, H=64, seed=22)
    check(c, *run(c))


@pytest.mark.parametrize("tiles", [
    [9] * 20,                               # (the join in four groups of threads)
    [21] * 41,                              # four whole pieces of five or six tiles each
    [1 + b % 5 for b in range(120)],        # whole pieces once they may hold a tile more
    [1 + b % 8 for b in range(128)],        # no whole pieces: cut where the line falls
    [1 + b % 8 for b in range(129)],        # more sequences than one round takes
    [40, 0, 90, 3],
])
def test_pieces_of_whole_sequences(tiles):
    lens = [max(0, 64 * n - 7 * b % 60) for b, n in enumerate(tiles)]
    c = C.Cache(lens, page=32, H=16, seed=len(tiles))
    check(c, *run(c))


def test_many_short_sequences():
    lens = [(37 * i) % 211 for i in range(700)]
    c = C.Cache(lens, page=16, H=16, seed=23)
    check(c, *run(c))


def test_rescale_and_far_references():
    # keys along the query with a factor that grows: the running reference is
    # left behind by far more than its slack, tile after tile; and shrinks, so
    # that later tiles have no weight at all
    c = C.Cache([1500, 1500], page=16, H=16, seed=24)
    for b, ramp in ((0, torch.linspace(0, 40, 1500)), (1, torch.linspace(40, 0, 1500))):
        x = (c.q[b, 0].float() / 24)[None, :] * ramp[:, None] + c.rows(b).float() * 0.2
        for s in range(1500):
            c.pool[c.table[b, s // 16].long(), s % 16] = x[s].to(torch.bfloat16)
    check(c, *run(c))


def test_very_negative_scores():
    c = C.Cache([300], page=16, H=16, seed=25)
    for s in range(300):
        c.pool[c.table[0, s // 16].long(), s % 16] = (-c.q[0, 0].float() * (5 + s % 3)).to(torch.bfloat16)
    c.q[0, :] = c.q[0, :1]
    check(c, *run(c))


def test_a_single_entry_gives_its_value():
    """Weights that add up to one exactly: a token that sees one entry gets its value's bits."""
    c = C.Cache([1, 77, 300], page=16, H=16, seed=32)
    out, _ = run(c, window=1)
    for b, n in enumerate(c.lens_list):
        assert torch.equal(out[b].cpu(), c.rows(b)[n - 1, :512].expand(16, -1))


def test_nan_entry_stays_in_its_sequence():
    c = C.Cache([200, 200], page=16, H=16, seed=26)
    c.pool[c.table[0, 3].long(), 2] = float("nan")
    out, lse = run(c)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    o, l, tol, tol_l = C.attention64(c.q[1], c.rows(1), C.seen(200, 0, 0))
    C.check_rows(out[1], o, tol, "out")
    C.check_rows(lse[1], l, tol_l, "lse")


def test_nan_head_stays_in_its_head():
    """A head with a NaN query beside heads whose references have to move."""
    c = C.Cache([700], page=16, H=16, seed=31)
    ramp = torch.linspace(0, 60, 700)
    x = (c.q[0, 3].float() / 24)[None, :] * ramp[:, None] + c.rows(0).float() * 0.2
    for s in range(700):
        c.pool[c.table[0, s // 16].long(), s % 16] = x[s].to(torch.bfloat16)
    c.q[0, 2, 5] = float("nan")
    out, lse = run(c)
    assert torch.isnan(out[0, 2]).all() and torch.isnan(lse[0, 2])
    o, l, tol, tol_l = C.attention64(c.q[0], c.rows(0), C.seen(700, 0, 0))
    rest = [h for h in range(16) if h != 2]
    C.check_rows(out[0, rest], o[rest], tol[rest], "out")
    C.check_rows(lse[0, rest], l[rest], tol_l[rest], "lse")


def test_strided_pages_shared_pages_and_table_slices():
    c = C.Cache([300, 290, 40], page=32, H=32, seed=27, layers=3, table_pad=5, spare=2)
    c.table[1, :9] = c.table[0, :9]             # a shared prefix of 288 entries
    c.pool[c.table[1, 9].long(), :2] = 1.0
    pool, table, lens, q = c.to_gpu()
    wide = torch.full((3, 40), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 7:7 + table.shape[1]] = table
    out = torch.empty((3, 32, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 32), device="cuda")
    dsa.dsa_paged_mla_decode(q, pool, wide[:, 7:7 + table.shape[1]], lens, 4000, C.SCALE, out, lse)
    assert_no_device_error()
    check(c, out, lse)


def test_no_lse_and_small_scale():
    c = C.Cache([500, 2], page=16, H=64, seed=28)
    out, _ = run(c, lse=False)
    check(c, out, None)


def test_same_bits_again_and_in_a_graph_on_another_stream():
    c = C.Cache([7000, 10, 3001], page=64, H=128, seed=29)
    out, lse = run(c)
    out2, lse2 = run(c)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    pool, table, lens, q = c.to_gpu()
    o = torch.zeros_like(out)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    dsa.dsa_paged_mla_decode(q, pool, table, lens, c.max_len, C.SCALE, o, stream=st)
    st.synchronize()
    assert torch.equal(o, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_paged_mla_decode(q, pool, table, lens, c.max_len, C.SCALE, o)
    # lengths are read on the device: a replay follows them
    lens.copy_(torch.tensor([6000, 0, 2500], dtype=torch.int32))
    graph.replay()
    assert_no_device_error()
    for b, n in enumerate([6000, 0, 2500]):
        want, _, tol, _ = C.attention64(c.q[b], c.rows(b)[:n], C.seen(n, 0, 0))
        C.check_rows(o[b], want, tol, f"replayed sequence {b}")


def test_out_of_range_lengths_and_pages_are_reported():
    c = C.Cache([100, 60], page=16, H=16, seed=30, spare=1)
    pool, table, lens, q = c.to_gpu()
    out = torch.zeros((2, 16, 512), dtype=torch.bfloat16, device="cuda")
    args = dict(max_len_k=100, sm_scale=C.SCALE, out=out)
    dsa.dsa_paged_mla_decode(q, pool, table, torch.tensor([100, -3], dtype=torch.int32, device="cuda"),
                             **args)
    assert dsa.dsa_get_device_error() == DSA_ERR_BOUNDS
    assert (out[1] == 0).all()
    dsa.dsa_paged_mla_decode(q, pool, table, torch.tensor([100, 200], dtype=torch.int32, device="cuda"),
                             **args)
    assert dsa.dsa_get_device_error() == DSA_ERR_BOUNDS
    bad = table.clone()
    bad[0, 2] = c.n_pages
    dsa.dsa_paged_mla_decode(q, pool, bad, lens, **args)
    assert dsa.dsa_get_device_error() == DSA_ERR_BOUNDS
    want, _, tol, _ = C.attention64(c.q[1], c.rows(1), C.seen(60, 0, 0))
    C.check_rows(out[1], want, tol, "the sequence beside it")
    assert dsa.dsa_get_device_error() == 0


@pytest.mark.parametrize("lens,H,window,sinks", [
    ([131072], 128, 0, 0),                          # one full context
    ([1 << 24, (1 << 24) - 37], 16, 0, 0),          # the longest that are allowed
    ([(1 << 24) - 1], 64, (1 << 23) + 5, 1000),
])
def test_longest_sequences(lens, H, window, sinks):
    """Against 64 bits with each pool row weighted by how often it is seen.  Beside the
    tolerances of the short cases: O adds up 4 products of 16 keys for each of a CTA's tiles, each off
    by at most 2^-22 of the sum of magnitudes; a thread adds its weights of every other tile
    (2^-24 each), and the parts (at most 148) are added up once more.  Head 0 has no query: its
    weights are all 1, so that its lse counts the entries (to 4 units in its last place)."""
    c = C.SharedPages(lens, 64, 400, H, seed=35)
    c.q[:, 0] = 0
    out = torch.empty((c.B, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((c.B, H), device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dsa.dsa_paged_mla_decode(c.q.cuda(), c.pool.cuda(), c.table.cuda(), n, max(lens), C.SCALE, out, lse,
                             window=window, sinks=sinks)
    assert_no_device_error()
    tiles = sum(lens) // 64 // (148 // -(-H // 64)) + 8
    for b in range(c.B):
        row = c.row(b)[torch.from_numpy(C.seen(lens[b], window, sinks))]
        often = torch.bincount(row, minlength=400 * 64).double()
        q, x = c.q[b].double(), c.pool.reshape(-1, 576).double()
        s = C.SCALE * (q @ x.T)
        want_l = torch.logsumexp(s + often.log(), 1)
        p = torch.exp(s - want_l[:, None]) * often
        o, spread = p @ x[:, :512], p @ x[:, :512].abs()
        d = (576 * 2.0 ** -23 * C.SCALE * (q.abs() @ x.abs().T)).amax(1) + 2.0 ** -21 * s.abs().amax(1)
        sums = (tiles / 2 + 200) * 2.0 ** -24
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -7 * 1.02 + 2.1 * d[:, None] + 4 * tiles * 2.0 ** -22 + sums) * spread
        C.check_rows(out[b], o, tol, f"out of sequence {b}")
        C.check_rows(lse[b], want_l, d + sums + 2.0 ** -21 + 2.0 ** -21 * want_l.abs(), f"lse of sequence {b}")
        count = float(torch.tensor(float(row.numel())).double().log())
        assert abs(float(lse[b, 0]) - count) <= 4 * 2.0 ** -19, "entries seen"


def test_large_values_under_a_reference_left_behind():
    """The stated range: values up to 2^70, with weights that grow to 2^31 over a sequence's first."""
    c = C.Cache([1500], page=16, H=16, seed=36)
    c.q[..., :512] = 0
    c.q[..., 512:] = c.q[:, :1, 512:]
    rope = c.q[0, 0, 512:].float()
    up = torch.linspace(0, 31 * 0.6931, 1500)[:, None] * rope / (C.SCALE * float(rope @ rope))
    for s in range(1500):
        c.pool[c.table[0, s // 16].long(), s % 16, :512] *= 2.0 ** 68
        c.pool[c.table[0, s // 16].long(), s % 16, 512:] = up[s].to(torch.bfloat16)
    assert float(c.rows(0)[:, :512].abs().max()) <= 2.0 ** 70 + 2.0 ** 69
    check(c, *run(c))
