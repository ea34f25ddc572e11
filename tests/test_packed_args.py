"""Refusals of the packed, paged and rotary entry points before anything touches the device, and workspace sizes."""

import ctypes

import pytest
import torch

from exact_io_aware_56_b200 import fa

INV, UNS, OK = fa.FA_ERR_INVALID_ARGUMENT, fa.FA_ERR_UNSUPPORTED, fa.FA_OK
P = 1 << 20  # aligned, never dereferenced: rejected before use
BIG = 1 << 40


def rows(ts=512, hs=64, data=P):
    return fa.Rows(data, ts, hs)


def pages(ps=4096, hs=1024, ss=64, data=P):
    return fa.Pages(data, ps, hs, ss)


def packed_fwd(q=rows(), k=rows(), v=rows(), o=rows(), r=None, lse=P, cu=P, S=2, T=64, Hq=4, Hkv=2, d=64, causal=1,
               scale=0.125, ws=P, n=BIG):
    return fa.lib().fa_packed_fwd(q, k, v, o, r, lse, cu, S, T, Hq, Hkv, d, causal, scale, ws, n, None)


def packed_bwd(q=rows(), dout=rows(), dk=rows(), lse=P, cu=P, S=2, T=64, Hq=4, Hkv=2, d=64, causal=1, scale=0.125,
               ws=P, n=BIG):
    return fa.lib().fa_packed_bwd(q, rows(), rows(), rows(), None, dout, lse, rows(), dk, rows(), cu, S, T, Hq, Hkv, d,
                                  causal, scale, ws, n, None)


def paged(q=rows(), kp=pages(), vp=pages(), o=rows(), lse=P, n_pages=9, page=16, bt=P, bts=8, mp=8, ln=P, cu=P, S=2, T=4,
          max_q=3, Hq=4, Hkv=2, d=64, causal=1, scale=0.125, ws=P, n=BIG):
    return fa.lib().fa_paged_fwd(q, kp, vp, o, lse, n_pages, page, bt, bts, mp, ln, cu, S, T, max_q, Hq, Hkv, d, causal,
                                 scale, ws, n, None)


def rope(q=rows(), k=rows(), qo=rows(), ko=rows(), pos=P, f=P, sec=(32,), T=4, Hq=4, Hkv=2, d=64, inter=0, inv=0):
    c = (ctypes.c_int * len(sec))(*sec) if sec is not None else None
    return fa.lib().fa_rope(q, k, qo, ko, pos, f, c, 0 if sec is None else len(sec), T, Hq, Hkv, d, inter, inv, None)


def append(q=rows(), k=rows(), v=rows(), qo=rows(), kp=pages(), vp=pages(), n_pages=9, page=16, bt=P, bts=8, mp=8, ln=P,
           cu=P, S=2, T=4, pos=P, f=P, sec=(32,), Hq=4, Hkv=2, d=64, inter=0):
    c = (ctypes.c_int * len(sec))(*sec) if sec else None
    return fa.lib().fa_paged_append(q, k, v, qo, kp, vp, n_pages, page, bt, bts, mp, ln, cu, S, T, pos, f, c, len(sec),
                                    Hq, Hkv, d, inter, None)


@pytest.mark.parametrize("call", [packed_fwd, packed_bwd, paged])
def test_shapes(call):
    assert call(S=-1) == INV and call(T=-1) == INV and call(Hkv=0) == INV and call(causal=2) == INV
    assert call(scale=0.0) == INV and call(scale=float("nan")) == INV and call(scale=float("inf")) == INV
    assert call(d=96) == UNS and call(Hq=3) == UNS and call(Hq=258, Hkv=2) == UNS and call(T=(1 << 30) + 1) == UNS
    assert call(S=0) == OK and call(T=0) == OK
    assert call(ws=None) == INV and call(ws=P + 8) == INV and call(n=16) == INV
    assert call(lse=None) == INV and call(lse=P + 2) == INV


@pytest.mark.parametrize("call", [packed_fwd, packed_bwd])
def test_packed_pointers(call):
    assert call(cu=None) == INV and call(cu=P + 1) == INV
    assert call(q=None) == INV


def test_strides():
    for bad in (rows(ts=0), rows(hs=0), rows(ts=-512), rows(ts=511), rows(hs=4), rows(data=P + 8), rows(data=None),
                rows(ts=1 << 40)):
        assert packed_fwd(q=bad) == INV and packed_fwd(o=bad) == INV and packed_fwd(r=bad) == INV
        assert packed_bwd(dout=bad) == INV and packed_bwd(dk=bad) == INV
        assert paged(q=bad) == INV and paged(o=bad) == INV
        assert rope(q=bad) == INV and rope(ko=bad) == INV
        assert append(k=bad) == INV and append(qo=bad) == INV
    for bad in (pages(ps=0), pages(hs=3), pages(ss=-64), pages(data=P + 2), pages(data=None)):
        assert paged(kp=bad) == INV and paged(vp=bad) == INV and append(kp=bad) == INV and append(vp=bad) == INV


def test_cache():
    for call in (paged, append):
        assert call(page=0) == INV and call(page=12) == UNS and call(n_pages=-1) == INV and call(n_pages=0) == INV
        assert call(mp=0) == INV and call(mp=1 << 27) == UNS and call(bt=None) == INV and call(bts=7) == INV
        assert call(ln=None) == INV and call(cu=None) == INV  # no offsets: one token each, S = T
    assert paged(max_q=0) == INV and paged(max_q=-1) == INV
    assert append(S=0) == OK and append(T=0) == OK


def test_rotation():
    for call in (rope, append):
        assert call(sec=(33,)) == INV and call(sec=(0, 32)) == INV and call(sec=(-8, 40)) == INV and call(sec=(12,)) == UNS
        assert call(sec=(8, 8, 8, 4, 4)) == UNS and call(f=None) == INV and call(f=P + 4) == INV and call(inter=2) == INV
        assert call(d=32) == UNS and call(sec=(16, 16), pos=None) == INV
    assert rope(pos=None) == INV and rope(sec=None) == INV and rope(inv=2) == INV and rope(Hq=0, Hkv=0) == INV
    assert rope(T=0) == OK and rope(q=None) == INV and append(Hkv=0) == INV


def test_workspaces():
    L = fa.lib()
    assert L.fa_packed_fwd_workspace_bytes(2, 64, 4, 3, 64) == 0 and L.fa_packed_fwd_workspace_bytes(2, 64, 4, 2, 96) == 0
    assert L.fa_packed_bwd_workspace_bytes(-1, 64, 4, 2, 64) == 0
    assert L.fa_paged_fwd_workspace_bytes(2, 64, 8, 4, 2, 64, 12, 8) == 0
    # The backward holds an fp32 D and dQ per query row; the forward a list of its units, and partial results only
    # where the units can be few.
    n = L.fa_packed_bwd_workspace_bytes(3, 1000, 4, 2, 128)
    assert 4 * 4 * 1000 * 129 <= n < 4 * 4 * 1000 * 129 + (1 << 22)
    assert 0 < L.fa_packed_fwd_workspace_bytes(3, 1000, 4, 2, 128) < 1 << 24
    assert 0 < L.fa_packed_fwd_workspace_bytes(8, 1 << 17, 32, 8, 128) < 1 << 18
    # Paged: partial results; more rows per sequence need more.
    one = L.fa_paged_fwd_workspace_bytes(32, 32, 1, 32, 8, 128, 16, 512)
    four = L.fa_paged_fwd_workspace_bytes(32, 128, 4, 32, 8, 128, 16, 512)
    assert 0 < one < four


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 4, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        fa.attention_packed_forward(x, x, x, torch.tensor([0, 4], dtype=torch.int32), True)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        fa.attention_packed_backward(x, x, x, x, x, x, torch.tensor([0, 4], dtype=torch.int32), True)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        fa.attention_paged(x, x[None], x[None], i, i)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        fa.paged_append(x, x, x[None], x[None], i, i)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        fa.rope(x, x, i, f)
    with pytest.raises(ValueError, match="required"):
        fa.rope(None, None, i, f)
    with pytest.raises(TypeError):
        fa.rope("q", x, i, f)
