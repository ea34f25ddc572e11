"""Shared helpers of the tests of packed sequences, the paged cache and rotary positions: inputs, bounds."""

import numpy as np
import torch

from exact_io_aware_56_b200 import fa, to_f64

# Error bounds, from the arithmetic. A bf16 rounding is off by at most half a step, 2^-8 of the value.
#  * Softmax weights are rounded to bf16 before P V (2^-8 each). Beyond that a weight is off by the error of its
#    exponent: S in fp32 over d = 128 products, at most 128 * 2^-24 * scale * sum_c |q_c k_c| (7 to 14 for these
#    inputs, so 1.1e-4), and the exponential's own (2^-22). In the backward P comes from S and L, twice that. Together
#    below 2^-11.
#    So |O - exact| <= W sum_j P_ij |v_j| + 2^-8 |exact|, W = 2^-8 + 2^-11 (and 1e-6 for exact zeros).
#  * L: the error of S, 1.1e-4, and fp32 of |m| < 100 (6e-6): below 1.5e-4.
#  * Gradients: dS is rounded to bf16 as the weights are; oracle.packed_bwd_ref carries W through.
HALF = 2.0 ** -8
W = 2.0 ** -8 + 2.0 ** -11
TOL_L = 1.5e-4


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def normal(seed, *shape):
    """bf16 standard normals on the CPU."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def assert_within(name, got, ref, bound):
    got = to_f64(got) if isinstance(got, torch.Tensor) else got
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), f"{name}: finite values differ"
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin]), name
    over = np.abs(got - np.where(fin, ref, 0.0)) - np.broadcast_to(bound, ref.shape)
    over = over[fin]
    assert not over.size or over.max() <= 0, f"{name}: over its bound by {over.max():.3e}"


def assert_forward(o, lse, O, L, A):
    """o and lse against the oracle in the rows that belong to a sequence (NaN elsewhere in the oracle's)."""
    rows = ~np.isnan(O).any(axis=(1, 2))
    assert_within("O", to_f64(o)[rows], O[rows], W * A[rows] + HALF * np.abs(O[rows]) + 1e-6)
    assert_within("L", to_f64(lse)[:, rows], L[:, rows], TOL_L)


def done():
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK


class Cache:
    """A paged cache with scattered pages, its unused slots poisoned with NaN; on the CPU, with its device copies."""

    def __init__(self, seed, lens, page, hkv, d, spare=3, token_major=False):
        rng = np.random.default_rng(seed)
        used = [-(-n // page) for n in lens]
        pool = sum(used) + spare
        self.n_pages, self.page, self.lens = pool, page, np.array(lens, dtype=np.int32)
        self.table = np.full((len(lens), max(used + [1])), 2 ** 30, dtype=np.int32)  # never to be read
        order = rng.permutation(pool)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.k = torch.full((pool, hkv, page, d), float("nan"), dtype=torch.bfloat16)
        self.v = self.k.clone()
        for b, n in enumerate(lens):
            kb, vb = normal(seed * 1000 + 2 * b, n, hkv, d), normal(seed * 1000 + 2 * b + 1, n, hkv, d)
            for i in range(used[b]):
                m = min(page, n - i * page)
                self.k[self.table[b, i], :, :m] = kb[i * page:i * page + m].transpose(0, 1)
                self.v[self.table[b, i], :, :m] = vb[i * page:i * page + m].transpose(0, 1)
        self.token_major = token_major

    def cuda(self):
        def up(x):
            if self.token_major:  # stored [pages, page, heads, d]
                return x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
            return x.cuda()

        return (up(self.k), up(self.v), torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda())
