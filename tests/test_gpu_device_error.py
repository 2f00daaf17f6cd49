"""What a report in the device error word does to other launches: nothing.

A captured launch keeps its number in every replay, so a later launch's report must
not make its waits give up.  That is made visible with the library's test hook: a
captured indexer launch leaves out its first key-tile load, and has to say so itself
(DSA_ERR_TIMEOUT) after its own wait limit of 20 ms, whatever was reported before."""
import time

import pytest
import torch

import sparse_attention_08_b200 as dsa
from sparse_attention_08_b200 import workloads as W
from tests import dsa_cases as C
from tests import paged_cases as P

pytestmark = pytest.mark.gpu

DSA_ERR_TIMEOUT, DSA_ERR_BOUNDS = 6, 7


def bad_length():
    """A call with an input error that is cut to range and reported."""
    c = P.Cache([100, 60], page=16, H=16, seed=30)
    pool, table, _, q = c.to_gpu()
    lens = torch.tensor([100, -3], dtype=torch.int32, device="cuda")
    out = torch.zeros((2, 16, 512), dtype=torch.bfloat16, device="cuda")
    dsa.dsa_paged_mla_decode(q, pool, table, lens, 100, P.SCALE, out)
    assert dsa.dsa_get_device_error() == DSA_ERR_BOUNDS


def lost_load(gpu):
    """A call whose wait runs out."""
    dsa.dsa_debug_fault_injection(20_000_000, True)
    try:
        C.gpu_indexer(gpu)
        assert dsa.dsa_get_device_error() == DSA_ERR_TIMEOUT
    finally:
        dsa.dsa_debug_fault_injection(0, False)


@pytest.mark.parametrize("kind", ["bounds", "timeout"])
def test_a_report_does_not_end_the_waits_of_an_older_graph(kind):
    gpu = W.make_small(H_I=4, d_I=64, H=16, L=1500, k=64, integer=True, seed=131).to("cuda")
    C.assert_no_device_error()
    graph = torch.cuda.CUDAGraph()
    dsa.dsa_debug_fault_injection(20_000_000, True)
    try:
        with torch.cuda.graph(graph):
            C.gpu_indexer(gpu)
    finally:
        dsa.dsa_debug_fault_injection(0, False)
    if kind == "bounds":
        bad_length()
    else:
        lost_load(gpu)
    assert dsa.dsa_get_device_error() == 0
    graph.replay()
    assert dsa.dsa_get_device_error() == DSA_ERR_TIMEOUT
    # and its own report is cleared with the word: the next replay finds out for itself
    graph.replay()
    assert dsa.dsa_get_device_error() == DSA_ERR_TIMEOUT
    assert dsa.dsa_get_device_error() == 0


def test_a_bad_page_reads_as_zeros_and_the_rest_is_computed():
    """One bad id among many long sequences: the bits of a page of zeros in its place."""
    lens = [4000 + 211 * i for i in range(24)]
    c = P.Cache(lens, page=64, H=16, seed=33, spare=1)
    zero = int(c.free_pages[0])
    c.pool[zero] = 0
    pool, table, n, q = c.to_gpu()
    o = torch.empty((2, c.B, 16, 512), dtype=torch.bfloat16, device="cuda")
    l = torch.empty((2, c.B, 16), device="cuda")
    m = torch.zeros((2, c.B, c.max_len), device="cuda")
    for i, page in enumerate((zero, c.n_pages + 7)):
        t = table.clone()
        t[11, 40] = page
        dsa.dsa_paged_mla_decode(q, pool, t, n, c.max_len, P.SCALE, o[i], l[i])
        assert dsa.dsa_get_device_error() == (DSA_ERR_BOUNDS if i else 0)
        dsa.dsa_paged_attn_mass(q, pool, t, n, l[i], c.max_len, P.SCALE, m[i])
        assert dsa.dsa_get_device_error() == (DSA_ERR_BOUNDS if i else 0)
    for x in (o, l, m):
        assert torch.isfinite(x.float()).all() and torch.equal(x[0], x[1])


def calls():
    """The kernels with roles that wait for one another: name, call and outputs."""
    c = P.Cache([5000, 70, 3000, 64, 1], page=64, H=64, seed=34)
    pool, table, n, q = c.to_gpu()
    ws = torch.zeros(dsa.dsa_paged_mla_decode_workspace_size(c.B, 64, c.max_len), dtype=torch.uint8,
                     device="cuda")
    o, l = torch.empty((c.B, 64, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((c.B, 64), device="cuda")
    m = torch.zeros((c.B, c.max_len), device="cuda")
    g = torch.Generator().manual_seed(35)
    cu = torch.tensor([0, 600, 610, 1010], dtype=torch.int32, device="cuda")
    x = [torch.randn((1010, 16, d), generator=g).to(torch.bfloat16).cuda() for d in (192, 192, 128)]
    wo, wl = torch.empty_like(x[2]), torch.empty((1010, 16), device="cuda")
    return [
        ("decode", lambda: dsa.dsa_paged_mla_decode(q, pool, table, n, c.max_len, P.SCALE, o, l, workspace=ws),
         [o, l]),
        ("mass", lambda: dsa.dsa_paged_attn_mass(q, pool, table, n, l, c.max_len, P.SCALE, m), [m]),
        ("window", lambda: dsa.dsa_window_mha_fwd(*x, cu, cu, 3, 600, 600, 200, 4, 0.07, wo, wl), [wo, wl]),
    ]


@pytest.mark.parametrize("which", [0, 1, 2], ids=["decode", "mass", "window"])
def test_a_timed_out_wait_is_reported_and_the_next_call_has_the_same_bits(which):
    todo = calls()
    todo[0][1]()
    name, call, outs = todo[which]
    call()
    C.assert_no_device_error()
    want = [t.clone() for t in outs]
    dsa.dsa_debug_fault_injection(20_000_000, True)
    try:
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        assert dsa.dsa_get_device_error() == DSA_ERR_TIMEOUT, name
    finally:
        dsa.dsa_debug_fault_injection(0, False)
    # a dozen limits of 20 ms one after the other, not the default 2 s
    assert took < 1.5, took
    if which:
        todo[0][1]()
    call()
    C.assert_no_device_error()
    for a, b in zip(outs, want):
        assert torch.equal(a, b), name
