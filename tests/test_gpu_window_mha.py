"""dsa_window_mha_fwd against the plain definition in 64 bits.

Tolerances: those of tests/paged_cases.py with 192 dims in a score: a score is off
by at most d = 192 * 2^-23 * scale * sum |q||k| (and 2^-21 of its size), a weight
by exp(2 d) and its rounding to bf16 (2^-8, and 2^-8 again in the normalising sum,
which is of the rounded weights), the output by its own rounding (2^-8)."""
import numpy as np
import pytest
import torch

import sparse_attention_08_b200 as dsa
from tests import paged_cases as C
from tests.dsa_cases import assert_no_device_error

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
DSA_ERR_BOUNDS = 7


def make(lens, lens_q, H, seed, q_mul=2.0):
    g = torch.Generator().manual_seed(seed)
    lens_q = lens if lens_q is None else lens_q
    T_q, T_k = sum(lens_q), sum(lens)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q = (r(T_q, H, 192) * q_mul).to(torch.bfloat16)
    k, v = r(T_k, H, 192).to(torch.bfloat16), r(T_k, H, 128).to(torch.bfloat16)
    cu = lambda n: torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)  # noqa: E731
    return q, k, v, cu(lens_q), cu(lens), lens_q


def call(q, k, v, cu_q, cu_k, lens_q, lens, window, sinks, lse=True, stream=None):
    out = torch.full((q.shape[0], q.shape[1], 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
    dsa.dsa_window_mha_fwd(q.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), cu_k.cuda(), len(lens),
                           max(lens_q), max(lens), window, sinks, SCALE, out, ls, stream=stream)
    return out, ls


def check(q, k, v, cu_q, cu_k, out, lse, window, sinks, seqs=None):
    out = out.cpu()
    lse = None if lse is None else lse.cpu()
    for b in range(cu_q.shape[0] - 1) if seqs is None else seqs:
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        if q0 == q1:
            continue
        p = torch.arange(k1 - k0 - (q1 - q0), k1 - k0)[:, None]
        s = torch.arange(k1 - k0)[None]
        see = s <= p
        if window:
            see &= (s > p - window) | (s < sinks)
        for h in range(q.shape[1]):
            Q, K, V = q[q0:q1, h].double(), k[k0:k1, h].double(), v[k0:k1, h].double()
            z = SCALE * (Q @ K.T)
            d = 192 * 2.0 ** -23 * SCALE * (Q.abs() @ K.abs().T) + 2.0 ** -21 * z.abs()
            d = d.masked_fill(~see, 0).amax(1)
            z = z.masked_fill(~see, -np.inf)
            ls = torch.logsumexp(z, 1)
            w = torch.exp(z - ls[:, None])
            o = w @ V
            tol = 2.0 ** -8 * o.abs() + (2.0 ** -7 * 1.02 + 2.1 * d[:, None]) * (w @ V.abs()) + 1e-30
            C.check_rows(out[q0:q1, h], o, tol, f"out of sequence {b}, head {h}")
            if lse is not None:
                t = d + (k1 - k0) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -21 * ls.abs()
                C.check_rows(lse[q0:q1, h], ls, t, f"lse of sequence {b}, head {h}")


CASES = [
    ([1], None, 1, 4, 1),
    ([300], None, 2, 64, 4),                      # a second pair of query tiles with one tile
    ([129, 1, 400], [129, 1, 7], 3, 128, 1),      # chunks: queries late in the sequence
    ([700, 256, 257], None, 2, 1, 0),             # only oneself
    ([513], None, 2, 0, 0),                       # no limit
    ([900], None, 1, 200, 300),                   # first tokens over several tiles
    ([1500], [40], 2, 37, 130),                   # a gap of many tiles in between
    ([1030], None, 7, 5000, 3),                   # a window beyond the sequence
    ([260, 0, 390], [260, 0, 390], 2, 129, 128),  # an empty sequence
    ([2300], None, 1, 1000, 16),                  # value tiles around the ring's end
]


@pytest.mark.parametrize("lens,lens_q,H,window,sinks", CASES)
def test_small(lens, lens_q, H, window, sinks):
    q, k, v, cu_q, cu_k, lens_q = make(lens, lens_q, H, seed=80)
    out, lse = call(q, k, v, cu_q, cu_k, lens_q, lens, window, sinks)
    assert_no_device_error()
    check(q, k, v, cu_q, cu_k, out, lse, window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (128, 0), (129, 3), (200, 0), (256, 16), (300, 140)])
@pytest.mark.parametrize("off", [0, 77, 301])
def test_ends_of_the_window_of_two_query_tiles(window, sinks, off):
    """A pair of query tiles shares all key tiles but the window's first and last."""
    lens_q = [513, 256, 384]
    lens = [n + off for n in lens_q]
    q, k, v, cu_q, cu_k, lens_q = make(lens, lens_q, 2, 77 + window + off)
    out, lse = call(q, k, v, cu_q, cu_k, lens_q, lens, window, sinks)
    check(q, k, v, cu_q, cu_k, out, lse, window, sinks)
    assert_no_device_error()


@pytest.mark.parametrize("ramp", [(0, 30), (30, 0)])
def test_references_left_behind(ramp):
    q, k, v, cu_q, cu_k, lens_q = make([640], None, 2, seed=81)
    grow = torch.linspace(*ramp, 640)[:, None, None]
    k = (k.float() * 0.2 + grow * q[300:301].float() / 20).to(torch.bfloat16)
    for window, sinks in ((0, 0), (200, 4)):
        out, lse = call(q, k, v, cu_q, cu_k, lens_q, [640], window, sinks)
        assert_no_device_error()
        check(q, k, v, cu_q, cu_k, out, lse, window, sinks)


@pytest.mark.parametrize("shift", [-300.0, -60.0, 60.0, 300.0])
def test_scores_far_from_zero(shift):
    """All of a row's scores far below or above zero, some rows changing sides."""
    q, k, v, cu_q, cu_k, lens_q = make([400], None, 2, seed=87, q_mul=1.0)
    q[:, :, 0] = 32.0
    k[:, :, 0] = shift / (32.0 * SCALE)
    k[200:260, :, 0] *= -1
    for window, sinks in ((0, 0), (70, 2)):
        out, lse = call(q, k, v, cu_q, cu_k, lens_q, [400], window, sinks)
        assert_no_device_error()
        check(q, k, v, cu_q, cu_k, out, lse, window, sinks)


def test_a_single_key_gives_its_value():
    """Weights that add up to one exactly: a row that sees one key gets its value's bits."""
    q, k, v, cu_q, cu_k, lens_q = make([300], None, 3, seed=88, q_mul=3.0)
    out, _ = call(q, k, v, cu_q, cu_k, lens_q, [300], 1, 0)
    assert_no_device_error()
    assert torch.equal(out.cpu(), v)


def test_another_sequences_nan_stays_there():
    lens = [200, 130, 77]
    q, k, v, cu_q, cu_k, lens_q = make(lens, None, 2, seed=82)
    for t in (q, k, v):
        t[200:330] = float("nan")
    out, lse = call(q, k, v, cu_q, cu_k, lens_q, lens, 64, 4)
    assert_no_device_error()
    check(q, k, v, cu_q, cu_k, out, lse, 64, 4, seqs=[0, 2])
    assert torch.isnan(out[200:330]).all()


def test_rows_behind_the_last_sequence_are_left_alone():
    q, k, v, cu_q, cu_k, lens_q = make([150], None, 2, seed=83)
    out = torch.full((200, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((200, 2), 7.0, device="cuda")
    q2 = torch.cat([q, torch.full((50, 2, 192), float("nan"), dtype=torch.bfloat16)])
    dsa.dsa_window_mha_fwd(q2.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), cu_k.cuda(), 1, 200, 200, 64,
                           1, SCALE, out, lse)
    assert_no_device_error()
    check(q, k, v, cu_q, cu_k, out[:150], lse[:150], 64, 1)
    assert (out[150:] == 7).all() and (lse[150:] == 7).all()


def test_many_items_graph_and_stream():
    lens = [333, 64, 1000, 129, 5]
    q, k, v, cu_q, cu_k, lens_q = make(lens, None, 64, seed=84)
    out, lse = call(q, k, v, cu_q, cu_k, lens_q, lens, 150, 4)
    assert_no_device_error()
    check(q, k, v, cu_q, cu_k, out, lse, 150, 4, seqs=[1, 3, 4])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        out2, lse2 = call(q, k, v, cu_q, cu_k, lens_q, lens, 150, 4)
    st.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    dq, dk, dv, a, b = q.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), cu_k.cuda()
    o = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_window_mha_fwd(dq, dk, dv, a, b, 5, 1000, 1000, 150, 4, SCALE, o)
    graph.replay()
    assert_no_device_error()
    assert torch.equal(o, out)


def test_all_keys_equals_the_masked_mode():
    """window = 0 is the masked MHA mode with every causal key selected."""
    lens = [300]
    q, k, v, cu_q, cu_k, lens_q = make(lens, None, 4, seed=85)
    out, lse = call(q, k, v, cu_q, cu_k, lens_q, lens, 0, 0)
    idx = torch.arange(300, dtype=torch.int32).repeat(300, 1).cuda()
    o2 = torch.empty_like(out)
    l2 = torch.empty_like(lse)
    dsa.dsa_masked_mha_fwd(q.cuda(), k.cuda(), v.cuda(), idx, cu_q.cuda(), cu_k.cuda(), 1, 300, 300,
                           300, SCALE, o2, l2)
    assert_no_device_error()
    # both round each weight to bf16 and the result once
    assert float((out.float() - o2.float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.abs().max())
    assert float((lse - l2).abs().max()) < 1e-4


def test_more_queries_than_keys_is_reported():
    q, k, v, _, _, _ = make([60], None, 1, seed=86)
    cu_q = torch.tensor([0, 40, 60], dtype=torch.int32)
    cu_k = torch.tensor([0, 30, 60], dtype=torch.int32)
    out = torch.full((60, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_window_mha_fwd(q.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), cu_k.cuda(), 2, 40, 40, 8, 1,
                           SCALE, out)
    assert dsa.dsa_get_device_error() == DSA_ERR_BOUNDS
    assert (out[:40] == 7).all()
    check(q, k, v, cu_q, cu_k, out, None, 8, 1, seqs=[1])


@pytest.mark.parametrize("lens,most", [([250, 100], 200), ([600, 10], 305)])
def test_more_queries_than_the_bound_is_reported(lens, most):
    """Rows past max_len_q get no output, and the call says so."""
    q, k, v, cu_q, cu_k, _ = make(lens, None, 2, seed=89)
    out = torch.full((sum(lens), 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((sum(lens), 2), 7.0, device="cuda")
    dsa.dsa_window_mha_fwd(q.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), cu_k.cuda(), 2, most,
                           max(lens), 64, 2, SCALE, out, lse)
    assert dsa.dsa_get_device_error() == DSA_ERR_BOUNDS
    assert (out[most:lens[0]] == 7).all() and (lse[most:lens[0]] == 7).all()
    # the other rows are those of a call that allows the length
    full, full_lse = call(q, k, v, cu_q, cu_k, lens, lens, 64, 2)
    assert_no_device_error()
    out[most:lens[0]], lse[most:lens[0]] = full[most:lens[0]], full_lse[most:lens[0]]
    for o, l in ((full, full_lse), (out, lse)):
        check(q, k, v, cu_q, cu_k, o, l, 64, 2)


def test_no_queries():
    """Nothing to do, with the null addresses that empty tensors have."""
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    e = lambda d: torch.empty((0, 2, d), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dsa.dsa_window_mha_fwd(e(192), e(192), e(128), cu, cu, 2, 8, 8, 4, 1, SCALE, e(128),
                           torch.empty((0, 2), device="cuda"))
    dsa.dsa_window_mha_fwd(e(192), e(192), e(128), cu[:1], cu[:1], 0, 0, 0, 4, 1, SCALE, e(128))
    assert_no_device_error()


def test_rows_behind_two_billion_elements():
    """A short sequence behind a long one: its rows' offsets pass 32 bits."""
    lens, H = [88000, 300], 128
    T = sum(lens)
    t = [torch.zeros((T, H, d), dtype=torch.bfloat16, device="cuda") for d in (192, 192, 128)]
    q, k, v, _, _, _ = make([300], None, H, seed=90)
    for a, b in zip(t, (q, k, v)):
        a[88000:] = b.cuda()
    cu = torch.tensor([0, 88000, T], dtype=torch.int32, device="cuda")
    out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    dsa.dsa_window_mha_fwd(*t, cu, cu, 2, 88000, 88000, 40, 2, SCALE, out, lse)
    assert_no_device_error()
    one = torch.tensor([0, 300], dtype=torch.int32)
    check(q, k, v, one, one, out[88000:], lse[88000:], 40, 2)
    # zeros before it: the values' zeros, and the log of how many keys a row sees
    assert (out[:88000] == 0).all()
    seen = torch.arange(1, 88001, device="cuda").clamp_max(42).double().log()
    assert float((lse[:88000].double() - seen[:, None]).abs().max()) <= 2.0 ** -20 * 4


@pytest.mark.parametrize("v_mul,ramp", [(2.0 ** 68, (0.0, 31.0)), (2.0 ** -90, (-31.0, -28.0))])
def test_large_and_small_values_under_a_reference_left_behind(v_mul, ramp):
    """The stated range: values from 2^-90 to 2^70, with a row's weights from 2^-31 to 2^31."""
    q, k, v, cu_q, cu_k, lens_q = make([500], None, 2, seed=91)
    q[:] = q[:1]
    up = torch.linspace(*ramp, 500)[:, None] * 0.6931
    for h in range(2):
        x = q[0, h].float()
        k[:, h] = (up * x / (SCALE * float(x @ x))).to(torch.bfloat16)
    v *= v_mul
    for window, sinks in ((0, 0), (200, 4)):
        out, lse = call(q, k, v, cu_q, cu_k, lens_q, [500], window, sinks)
        assert_no_device_error()
        check(q, k, v, cu_q, cu_k, out, lse, window, sinks)
