"""What the calls over a paged cache refuse, on the host, before any launch."""
import ctypes

import pytest
import torch

import sparse_attention_08_b200 as dsa

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE, CUDA = 0, 1, 2, 3, 4, 5
P = ctypes.c_void_p(0x10000)


def off(n):
    return ctypes.c_void_p(0x10000 + n)


CACHE = dict(kv=P, n_pages=100, page=64, stride=64 * 576, table=P, ld=10, pages=10, lens=P, B=4,
             max_len=640)


def cache_args(a):
    return [a[k] for k in ("kv", "n_pages", "page", "stride", "table", "ld", "pages", "lens", "B",
                           "max_len")]


BAD_CACHE = [
    (dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(B=-1), INVALID), (dict(max_len=-1), INVALID), (dict(n_pages=0), INVALID),
    (dict(page=0), INVALID), (dict(pages=0), INVALID), (dict(ld=9), INVALID),
    (dict(stride=64 * 576 - 8), INVALID),
    (dict(page=8), UNSUPPORTED), (dict(page=63), UNSUPPORTED), (dict(page=1), UNSUPPORTED),
    (dict(max_len=(1 << 24) + 1), UNSUPPORTED), (dict(n_pages=1 << 31), UNSUPPORTED),
    (dict(kv=off(8)), ALIGN), (dict(stride=64 * 576 + 4), ALIGN),
]


def decode(**kw):
    a = dict(CACHE, q=P, H=128, d_qk=576, d_v=512, window=0, sinks=0, scale=0.04, out=P, lse=P,
             ws=P, nbytes=1 << 40)
    a.update(kw)
    return dsa.load().dsa_paged_mla_decode(a["q"], *cache_args(a), a["H"], a["d_qk"], a["d_v"],
                                           a["window"], a["sinks"], a["scale"], a["out"], a["lse"],
                                           a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(H=8), UNSUPPORTED), (dict(H=320), UNSUPPORTED), (dict(d_qk=512), UNSUPPORTED),
    (dict(d_v=576), UNSUPPORTED), (dict(q=off(2)), ALIGN), (dict(out=off(8)), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(nbytes=100), WORKSPACE), (dict(ws=off(4)), ALIGN),
    (dict(B=0), OK),
])
def test_decode_refuses(kw, status):
    assert decode(**kw) == status


def test_decode_workspace_size():
    size = dsa.dsa_paged_mla_decode_workspace_size
    assert size(1, 128, 131072) >= 2 * 148 * 64 * (512 * 4 + 16)
    assert size(1, 128, 100) < size(1, 128, 131072)
    assert size(-1, 128, 100) == 0 and size(1, 100, 100) == 0 and size(1, 128, -1) == 0


def test_wrappers_check_tensors():
    t = torch.zeros
    with pytest.raises(ValueError):         # CPU tensors
        dsa.dsa_paged_mla_decode(t((1, 16, 576), dtype=torch.bfloat16),
                                 t((2, 16, 576), dtype=torch.bfloat16),
                                 t((1, 2), dtype=torch.int32), t(1, dtype=torch.int32), 32, 0.04,
                                 t((1, 16, 512), dtype=torch.bfloat16))


def mass(**kw):
    a = dict(CACHE, q=P, H=128, d_qk=576, window=0, sinks=0, scale=0.04, lse=P, m_in=P, m_out=P,
             ld_m=640)
    a.update(kw)
    return dsa.load().dsa_paged_attn_mass(a["q"], *cache_args(a), a["H"], a["d_qk"], a["window"],
                                          a["sinks"], a["scale"], a["lse"], a["m_in"], a["m_out"],
                                          a["ld_m"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(m_out=None), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=-1.0), INVALID),
    (dict(ld_m=639), INVALID), (dict(H=100), UNSUPPORTED), (dict(d_qk=512), UNSUPPORTED),
    (dict(q=off(2)), ALIGN), (dict(B=0), OK), (dict(max_len=0), OK),
])
def test_mass_refuses(kw, status):
    assert mass(**kw) == status


def evict(**kw):
    a = dict(CACHE, mass=P, ld_m=640, budget=128, sinks=4, recent=16, nt=off(16), nt_ld=2, nt_pages=2,
             nl=off(32), idx=P, nm=off(48), ld_nm=128)
    a.update(kw)
    return dsa.load().dsa_cache_evict(*cache_args(a), a["mass"], a["ld_m"], a["budget"],
                                      a["sinks"], a["recent"], a["nt"], a["nt_ld"], a["nt_pages"],
                                      a["nl"], a["idx"], a["nm"], a["ld_nm"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(mass=None), INVALID), (dict(nt=None), INVALID), (dict(nl=None), INVALID),
    (dict(idx=None), INVALID), (dict(budget=0), INVALID), (dict(sinks=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(sinks=120, recent=9), INVALID), (dict(ld_m=639), INVALID),
    (dict(ld_nm=127), INVALID), (dict(nt_pages=1, nt_ld=1), INVALID), (dict(nt_ld=1), INVALID),
    (dict(nl=P), INVALID),                     # the lengths themselves
    (dict(nm=P), INVALID),                     # the totals themselves
    (dict(max_len=262145, ld_m=262145), UNSUPPORTED), (dict(B=0), OK),
])
def test_evict_refuses(kw, status):
    assert evict(**kw) == status


def window_mha(**kw):
    a = dict(q=P, k=P, v=P, cq=P, ck=P, B=1, mlq=64, mlk=64, tq=64, tk=64, H=128, d_qk=192, d_v=128,
             window=32, sinks=4, scale=0.07, out=P, lse=P)
    a.update(kw)
    return dsa.load().dsa_window_mha_fwd(*[a[n] for n in (
        "q", "k", "v", "cq", "ck", "B", "mlq", "mlk", "tq", "tk", "H", "d_qk", "d_v", "window",
        "sinks", "scale", "out", "lse")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(cq=None), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(scale=0.0), INVALID), (dict(mlq=65), INVALID),
    (dict(tq=65), INVALID), (dict(tk=0), INVALID), (dict(H=0), UNSUPPORTED),
    (dict(d_qk=128), UNSUPPORTED), (dict(d_v=192), UNSUPPORTED),
    (dict(mlk=(1 << 24) + 1), UNSUPPORTED), (dict(q=off(4)), ALIGN), (dict(out=off(8)), ALIGN),
    (dict(tq=0), OK), (dict(B=0, tq=0, tk=0), OK),
])
def test_window_mha_refuses(kw, status):
    assert window_mha(**kw) == status


def test_stream_of_another_device_is_refused():
    class Stream:
        cuda_stream, device = 0, torch.device("cuda", 1)

    with pytest.raises(ValueError, match="cuda:1"):
        dsa._On(0, Stream())


def test_null_addresses_of_empty_tensors():
    """Nothing to read or write: no address is needed for it."""
    none = dict(B=0, table=None, lens=None, q=None, out=None, lse=None, m_in=None, m_out=None,
                mass=None, nt=None, nl=None, idx=None, nm=None)
    for n in (640, 0):
        assert decode(**none, max_len=n) == OK
        assert mass(**none, max_len=n) == OK
        assert evict(**none, max_len=n) == OK
    assert mass(max_len=0, m_in=None, m_out=None) == OK
    # (a sequence without a cache still has an output)
    assert decode(max_len=0, out=None) == INVALID
    assert evict(max_len=0, idx=None) == INVALID and evict(max_len=0, nl=None) == INVALID
    assert mass(**dict(none, B=4)) == INVALID and mass(m_out=None) == INVALID
    assert window_mha(tq=0, q=None, out=None) == OK
    assert window_mha(tq=0, tk=0, mlq=0, mlk=0, B=0, q=None, k=None, v=None, out=None) == OK
    # what is no tensor's address is still looked at
    assert decode(**none, window=-1) == INVALID and decode(**none, H=8) == UNSUPPORTED
    assert evict(**none, budget=0) == INVALID and window_mha(tq=0, q=None, H=0) == UNSUPPORTED


@pytest.mark.parametrize("B,tiles,status", [(65535, 32768, UNSUPPORTED), (1 << 20, 2048, UNSUPPORTED),
                                            (65535, 32767, WORKSPACE)])
def test_more_tiles_than_32_bits_count_are_refused(B, tiles, status):
    """The tiles of all sequences stand in one line whose positions are 32-bit numbers, those
    of the last pieces' ends too."""
    page = 65536
    big = dict(B=B, max_len=64 * (tiles - 1), page=page, stride=page * 576, pages=40, ld=40, H=16)
    assert decode(**big, nbytes=16) == status
    if status == UNSUPPORTED:
        assert mass(**big, ld_m=64 * tiles) == status
