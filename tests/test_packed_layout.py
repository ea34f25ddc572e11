"""Host logic of the packed forward's launch (CPU, no GPU): what it lays out in the workspace, read through the
fa_test_packed_layout hook, fits what the size queries ask for on a device of any number of multiprocessors, and the
CTAs that find their units without a list have at most two each."""

import ctypes

import numpy as np
import pytest

from exact_io_aware_56_b200 import fa


def layout(S, T, Hq, Hkv, d, page, max_pages, sms):
    L = fa.lib()
    L.fa_test_packed_layout.argtypes = [ctypes.c_int] * 8 + [ctypes.POINTER(ctypes.c_longlong)]
    L.fa_test_packed_layout.restype = ctypes.c_int
    out = (ctypes.c_longlong * 5)()
    assert L.fa_test_packed_layout(S, T, Hq, Hkv, d, page, max_pages, sms, out) == fa.FA_OK
    return dict(zip(["bytes", "runs", "direct", "units", "grid"], list(out)))


def shapes():
    rng = np.random.default_rng(11)
    for _ in range(400):
        hkv = int(rng.choice([1, 2, 4, 8]))
        r = int(rng.choice([1, 2, 3, 4, 8]))
        S = int(rng.integers(1, 40))
        T = int(np.exp(rng.uniform(np.log(S), np.log(20000))))
        d = int(rng.choice([64, 128]))
        page = int(rng.choice([0, 16, 64, 256]))
        max_pages = -(-int(np.exp(rng.uniform(0, np.log(40000)))) // page) if page else 0
        yield S, max(S, T), hkv * r, hkv, d, page, max_pages


@pytest.mark.parametrize("kind", ["packed", "paged"])
def test_launch_fits_the_workspace(kind):
    runs = direct = 0
    for S, T, Hq, Hkv, d, page, max_pages in shapes():
        if (page > 0) != (kind == "paged") or (page and Hq // Hkv * T <= 128):
            continue
        room = fa.fa_paged_fwd_workspace_bytes(S, T, T, Hq, Hkv, d, page, max_pages) if page else \
            fa.fa_packed_fwd_workspace_bytes(S, T, Hq, Hkv, d)
        for sms in (1, 2, 7, 20, 33, 64, 74, 100, 130, 132, 147, 148, 160):
            x = layout(S, T, Hq, Hkv, d, page, max_pages, sms)
            assert x["bytes"] <= room, (S, T, Hq, Hkv, d, page, max_pages, sms)
            assert 1 <= x["grid"] <= min(sms, 148) * (1 if d == 128 else 2)
            assert not x["direct"] or (not x["runs"] and x["units"] <= 2 * x["grid"])
            runs += x["runs"]
            direct += x["direct"]
    assert runs > 100 and (direct > 100) == (kind == "packed")


def test_backward_holds_key_gradients_only_where_units_may_be_cut():
    # fp32 dK and dV (8 bytes per element) are zeroed and kept for fewer than 208 tiles of 128 keys times KV heads. (The
    # list of units takes the 4 MB at most.)
    for T, Hq, Hkv, d in ((1536, 32, 16, 128), (6528, 16, 4, 128), (13184, 8, 2, 64), (200 * 128, 1, 1, 64)):
        rest = 4 * T * Hq * (d + 1)
        assert fa.fa_packed_bwd_workspace_bytes(1, T, Hq, Hkv, d) >= rest + 8 * T * Hkv * d
    for T, Hq, Hkv, d in ((1664, 32, 16, 128), (6656, 16, 4, 128), (13312, 8, 2, 64), (31000, 1, 1, 64)):
        rest = 4 * T * Hq * (d + 1)
        assert fa.fa_packed_bwd_workspace_bytes(1, T, Hq, Hkv, d) < rest + (4 << 20)
