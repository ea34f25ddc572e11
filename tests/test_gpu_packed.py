"""GPU parity of attention over packed sequences (fa_packed_fwd, fa_packed_bwd) against the fp64 oracle: lengths from
none to several tiles, grouped heads whose group does not divide a tile, both head dims, causal and not; NaN in other
sequences and behind the last; strided views; graphs; finite differences."""

import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_56_b200 import fa, to_f64

from .packed import HALF, TOL_L, W, assert_forward, assert_within, done, normal, offsets

pytestmark = pytest.mark.gpu

# (lengths, Hq, Hkv)
SHAPES = [
    ([1], 1, 1),
    ([128], 2, 2),
    ([129, 1, 127], 4, 2),
    ([300, 0, 17, 256, 64], 4, 1),
    ([5, 63, 65, 200, 33], 6, 2),       # groups of three
    ([400], 5, 1),                      # a group of five
    ([1] * 30 + [2, 3], 8, 8),
    ([513, 255], 3, 3),
    ([70, 90], 16, 1),
]


def inputs(lens, hq, hkv, d, seed, pad=0):
    T = int(sum(lens)) + pad
    return [normal(seed + i, T, h, d) for i, h in enumerate((hq, hkv, hkv, hq))]


def backward_check(q, k, v, dout, grads, cu, causal, scale):
    ref = oracle.packed_bwd_ref(*(to_f64(x) for x in (q, k, v, dout)), cu, causal, scale, W)
    for name, got, want, err in zip(("dQ", "dK", "dV"), grads, ref[:3], ref[3:]):
        rows = ~np.isnan(want).any(axis=(1, 2))
        assert_within(name, to_f64(got)[rows], want[rows], err[rows] + HALF * np.abs(want[rows]) + 1e-5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, d, causal):
    lens, hq, hkv = shape
    q, k, v, _ = inputs(lens, hq, hkv, d, seed=sum(lens) + d)
    cu = offsets(lens)
    o, lse = fa.attention_packed_forward(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(cu).cuda(), causal, 0.125)
    done()
    assert_forward(o, lse, *oracle.packed_fwd_ref(to_f64(q), to_f64(k), to_f64(v), cu, causal, 0.125))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, d, causal):
    lens, hq, hkv = shape
    host = inputs(lens, hq, hkv, d, seed=2 * sum(lens) + d)
    q, k, v, dout = (x.cuda() for x in host)
    cu = offsets(lens)
    cud = torch.from_numpy(cu).cuda()
    o, lse, resid = fa.attention_packed_forward(q, k, v, cud, causal, 0.125, residual=True)
    ref = oracle.packed_fwd_ref(*(to_f64(x) for x in host[:3]), cu, causal, 0.125)
    assert_forward(o, lse, *ref)
    # o + o_resid carries O to 16 bits: what is left is the weights' rounding.
    assert_within("O + residual", to_f64(o) + to_f64(resid), ref[0], W * ref[2] + 2.0 ** -15 * np.abs(ref[0]) + 1e-6)
    grads = fa.attention_packed_backward(q, k, v, o, dout, lse, cud, causal, 0.125, o_resid=resid)
    done()
    backward_check(*host, grads, cu, causal, 0.125)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_nan_and_infinity_stay_in_their_sequence(d, causal):
    # The second of three sequences and the rows around all of them hold NaN and infinities.
    lens, hq, hkv = [100, 60, 150], 4, 2
    cu = offsets(lens) + 2
    host = inputs(lens, hq, hkv, d, 77, pad=9)
    for i, x in enumerate(host):
        x[102:162] = (float("nan"), float("inf"), float("-inf"), float("nan"))[i]
        x[:2] = x[-7:] = float("nan")
    q, k, v, dout = (x.cuda() for x in host)
    cud = torch.from_numpy(cu).cuda()
    T = q.shape[0]
    o, resid = (torch.full_like(q, 7.0) for _ in range(2))
    lse = torch.full((hq, T), 7.0, device="cuda")
    ws = torch.empty(fa.fa_packed_fwd_workspace_bytes(3, T, hq, hkv, d), dtype=torch.uint8, device="cuda")
    fa.fa_packed_fwd(q, k, v, o, lse, cud, causal, 0.125, ws, o_resid=resid)
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    ws = torch.empty(fa.fa_packed_bwd_workspace_bytes(3, T, hq, hkv, d), dtype=torch.uint8, device="cuda")
    fa.fa_packed_bwd(q, k, v, o, dout, lse, dq, dk, dv, cud, causal, 0.125, ws, o_resid=resid)
    done()
    for x in (o, resid, dq, dk, dv, lse.t()):
        assert (x[:2] == 7).all() and (x[-7:] == 7).all()
    for lo, hi in ((2, 102), (162, 312)):
        part = [x[lo:hi] for x in host]
        c = np.array([0, hi - lo], dtype=np.int32)
        assert_forward(o[lo:hi], lse[:, lo:hi], *oracle.packed_fwd_ref(*(to_f64(x) for x in part[:3]), c, causal, 0.125))
        backward_check(*part, [x[lo:hi] for x in (dq, dk, dv)], c, causal, 0.125)


@pytest.mark.parametrize("d", [64, 128])
def test_strided_views(d):
    # q, k, v are slices of one fused projection, their gradients slices of one buffer; o and dout head-major.
    lens, hq, hkv = [130, 50, 128], 4, 2
    cu = offsets(lens)
    T = int(cu[-1])
    fused = normal(5, T, hq + 2 * hkv, d).cuda()
    q, k, v = fused.split((hq, hkv, hkv), 1)
    dfused = torch.full_like(fused, 7.0)
    o = torch.empty(hq, T, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    dout = normal(6, hq, T, d).cuda().transpose(0, 1)
    lse = torch.empty(hq, T, device="cuda")
    cud = torch.from_numpy(cu).cuda()
    ws = torch.empty(fa.fa_packed_fwd_workspace_bytes(3, T, hq, hkv, d), dtype=torch.uint8, device="cuda")
    fa.fa_packed_fwd(q, k, v, o, lse, cud, True, 0.125, ws)
    ws = torch.empty(fa.fa_packed_bwd_workspace_bytes(3, T, hq, hkv, d), dtype=torch.uint8, device="cuda")
    dq, dk, dv = dfused.split((hq, hkv, hkv), 1)
    fa.fa_packed_bwd(q, k, v, o, dout, lse, dq, dk, dv, cud, True, 0.125, ws)
    done()
    host = [x.cpu().contiguous() for x in (q, k, v, dout)]
    assert_forward(o, lse, *oracle.packed_fwd_ref(*(to_f64(x) for x in host[:3]), cu, True, 0.125))
    # Without the residual D carries o's rounding too: 2^-8 |O| <= 2^-8 sum P|v|, once more W.
    ref = oracle.packed_bwd_ref(*(to_f64(x) for x in host), cu, True, 0.125, 2 * W)
    for got, want, err in zip((dq, dk, dv), ref[:3], ref[3:]):
        assert_within("gradient", to_f64(got), want, err + HALF * np.abs(want) + 1e-5)


@pytest.mark.parametrize("d", [64, 128])
def test_agrees_with_the_equal_length_kernels(d):
    # Two sequences of 256 tokens, as a batch and as a pack.
    q, k, v, dout = (x.cuda() for x in inputs([512], 4, 2, d, 91))
    cu = torch.tensor([0, 256, 512], dtype=torch.int32, device="cuda")

    def batch(x):
        return x.unflatten(0, (2, 256)).transpose(1, 2).contiguous()

    ob, lb, rb = fa.attention_forward(batch(q), batch(k), batch(v), True, residual=True)
    gb = fa.attention_backward(batch(q), batch(k), batch(v), ob, batch(dout), lb, True, o_resid=rb)
    o, lse, r = fa.attention_packed_forward(q, k, v, cu, True, residual=True)
    g = fa.attention_packed_backward(q, k, v, o, dout, lse, cu, True, o_resid=r)
    done()
    # Each is within W sum P|v| + 2^-8 |O| of the same exact value, and sum P|v| <= max |v|.
    assert (batch(o).float() - ob.float()).abs().max() <= 2 * (W + HALF) * v.float().abs().max()
    # (The equal-length kernel evaluates some exponentials by a polynomial of relative error 1.2e-4.)
    assert (lse.unflatten(1, (2, 256)).transpose(0, 1) - lb).abs().max() <= 2 * TOL_L + 1.2e-4
    backward_check(*(x.cpu() for x in (q, k, v, dout)), g, np.array([0, 256, 512]), True, d ** -0.5)
    backward_check(*(x.cpu() for x in (q, k, v, dout)), [x.transpose(1, 2).flatten(0, 1) for x in gb],
                   np.array([0, 256, 512]), True, d ** -0.5)


def test_gradients_against_differences():
    # d/dt sum(dout * O(x + t u)) by central differences of the fp64 oracle along random directions.
    lens, hq, hkv, d = [37, 150], 2, 1, 64
    host = inputs(lens, hq, hkv, d, 101)
    cu = offsets(lens)
    q, k, v, dout = (x.cuda() for x in host)
    cud = torch.from_numpy(cu).cuda()
    o, lse, r = fa.attention_packed_forward(q, k, v, cud, True, 0.125, residual=True)
    grads = fa.attention_packed_backward(q, k, v, o, dout, lse, cud, True, 0.125, o_resid=r)
    done()
    ref = oracle.packed_bwd_ref(*(to_f64(x) for x in host), cu, True, 0.125, W)
    x = [to_f64(t) for t in host]
    rng = np.random.default_rng(3)
    for i in range(3):
        u = rng.choice([-1.0, 1.0], size=x[i].shape)
        at = []
        for t in (1e-4, -1e-4):
            y = list(x[:3])
            y[i] = y[i] + t * u
            at.append((x[3] * oracle.packed_fwd_ref(*y, cu, True, 0.125)[0]).sum())
        slope = (at[0] - at[1]) / 2e-4
        bound = (ref[3 + i] + HALF * np.abs(ref[i])).sum()  # the elements' bounds, |u| = 1
        assert abs((to_f64(grads[i]) * u).sum() - slope) <= bound + 1e-3


def test_out_of_range_offsets_are_reported_and_nothing_is_written():
    q, k, v, dout = (x.cuda() for x in inputs([64, 200], 2, 2, 64, 111))
    for cu in ([0, 300, 264], [-1, 64, 264], [0, 64, 265], [0, 264, 64]):
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, dq, dk, dv = (torch.full_like(q, 7.0) for _ in range(4))
        lse = torch.full((2, 264), 7.0, device="cuda")
        ws = torch.empty(fa.fa_packed_fwd_workspace_bytes(2, 264, 2, 2, 64), dtype=torch.uint8, device="cuda")
        fa.fa_packed_fwd(q, k, v, o, lse, cud, True, 0.125, ws)
        assert fa.fa_check_device_error() == fa.FA_ERR_DATA
        ws = torch.empty(fa.fa_packed_bwd_workspace_bytes(2, 264, 2, 2, 64), dtype=torch.uint8, device="cuda")
        fa.fa_packed_bwd(q, k, v, o, dout, lse, dq, dk, dv, cud, True, 0.125, ws)
        assert fa.fa_check_device_error() == fa.FA_ERR_DATA
        for x in (o, dq, dk, dv, lse):
            assert (x == 7).all()


def test_captured_training_step_replays_on_other_lengths():
    T, hq, hkv, d = 400, 4, 2, 64
    host = inputs([T], hq, hkv, d, 121)
    q, k, v, dout = (x.cuda() for x in host)
    cu = torch.tensor([0, 100, 250, 400], dtype=torch.int32, device="cuda")

    def step():
        o, lse, r = fa.attention_packed_forward(q, k, v, cu, True, 0.125, residual=True)
        return (o, lse) + fa.attention_packed_backward(q, k, v, o, dout, lse, cu, True, 0.125, o_resid=r)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for lens in ([100, 150, 150], [1, 0, 399], [400, 0, 0]):
        c = offsets(lens)
        cu.copy_(torch.from_numpy(c))
        g.replay()
        done()
        assert_forward(out[0], out[1], *oracle.packed_fwd_ref(*(to_f64(x) for x in host[:3]), c, True, 0.125))
        backward_check(*host, out[2:], c, True, 0.125)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,heads", [(64, 18), (128, 12)])
def test_two_units_for_some_ctas(d, heads, causal):
    # More units than CTAs, fewer than twice as many: first units taken by length, second ones in turn. Replayed on
    # lengths of one unit per CTA and of a single sequence.
    lens = [300, 1, 77, 128, 129, 255, 64, 33, 2, 190, 256, 17, 0, 100]
    q, k, v, _ = inputs(lens, heads, heads, d, 141)
    cu = torch.from_numpy(offsets(lens)).cuda()
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    fa.attention_packed_forward(qd, kd, vd, cu, causal, 0.125)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fa.attention_packed_forward(qd, kd, vd, cu, causal, 0.125)
    for c in (lens, [128, 256, 384, 700] + [0] * 10, [0] * 13 + [sum(lens)]):
        c = offsets(c)
        assert c[-1] <= q.shape[0]
        cu.copy_(torch.from_numpy(c))
        g.replay()
        done()
        ref = oracle.packed_fwd_ref(to_f64(q), to_f64(k), to_f64(v), c, causal, 0.125)
        rows = slice(0, c[-1])
        assert_forward(o[rows], lse[:, rows], *(x[:, rows] if i == 1 else x[rows] for i, x in enumerate(ref)))


def test_many_sequences():
    # More sequences than the list's one-block kernel has threads, most of them empty or short.
    rng = np.random.default_rng(7)
    lens = rng.choice([0, 0, 1, 2, 5], size=2500)
    lens[1234] = 300
    cu = offsets(lens)
    q, k, v, dout = inputs(lens, 2, 1, 64, 131)
    cud = torch.from_numpy(cu).cuda()
    o, lse, r = fa.attention_packed_forward(q.cuda(), k.cuda(), v.cuda(), cud, True, 0.125, residual=True)
    g = fa.attention_packed_backward(q.cuda(), k.cuda(), v.cuda(), o, dout.cuda(), lse, cud, True, 0.125, o_resid=r)
    done()
    assert_forward(o, lse, *oracle.packed_fwd_ref(to_f64(q), to_f64(k), to_f64(v), cu, True, 0.125))
    backward_check(q, k, v, dout, g, cu, True, 0.125)


def weight_error(q, k, scale):
    """Relative error of a weight for scores of any size: half a bf16 step, plus the error of its exponent: S in fp32
    over d products (d 2^-24 of the sum of their magnitudes), L's own error of that size, and 1.2e-4 each for the
    exponentials and for fp32 of large exponents."""
    d = q.shape[-1]
    most = scale * float(np.abs(to_f64(q)).max(0).max(0) @ np.abs(to_f64(k)).max(0).max(0))
    return HALF + 2 * (d * 2.0 ** -24 * most + 1.2e-4)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_large_and_rising_scores(d, causal):
    # Peaky rows: q, k three times as large, and keys that rise along the sequence, so that a row's max keeps growing
    # by less and by more than the forward's rescale threshold.
    lens, hq, hkv = [700, 300], 4, 2
    q, k, v, dout = inputs(lens, hq, hkv, d, 141)
    u = normal(142, 1, 1, d).float()
    u = u / u.norm()
    rise = torch.cat([torch.linspace(0, 60, n) for n in lens])[:, None, None]
    q = (2 * q.float() + 4 * u).to(torch.bfloat16)
    k = (2 * k.float() + rise * u).to(torch.bfloat16)
    cu = offsets(lens)
    cud = torch.from_numpy(cu).cuda()
    scale = d ** -0.5
    w = weight_error(q, k, scale)
    O, L, A = oracle.packed_fwd_ref(to_f64(q), to_f64(k), to_f64(v), cu, causal, scale)
    for residual in (False, True):
        got = fa.attention_packed_forward(q.cuda(), k.cuda(), v.cuda(), cud, causal, scale, residual=residual)
        done()
        assert_within("O", got[0], O, w * A + HALF * np.abs(O) + 1e-6)
        assert_within("L", got[1], L, (w - HALF) + 2.0 ** -22 * np.abs(L))
    grads = fa.attention_packed_backward(q.cuda(), k.cuda(), v.cuda(), got[0], dout.cuda(), got[1], cud, causal, scale,
                                         o_resid=got[2])
    done()
    ref = oracle.packed_bwd_ref(*(to_f64(x) for x in (q, k, v, dout)), cu, causal, scale, w)
    for got_, want, err in zip(grads, ref[:3], ref[3:]):
        assert_within("gradient", got_, want, err + HALF * np.abs(want) + 1e-4)


def test_saturated_rows_are_exact():
    # One key carries all of a row's weight: O = v of that key, bit for bit, and dQ = dK = 0.
    lens, hq, hkv, d = [200, 129, 1], 4, 2, 64
    T = sum(lens)
    g = torch.Generator().manual_seed(5)
    k = (torch.randint(0, 2, (T, hkv, d), generator=g) * 2 - 1).to(torch.bfloat16)
    v, dout = normal(6, T, hkv, d), normal(7, T, hq, d)
    cu = offsets(lens)
    rng = np.random.default_rng(5)
    pick = np.zeros((T, hq), dtype=np.int64)
    for b in range(3):
        for t in range(cu[b], cu[b + 1]):
            pick[t] = rng.integers(cu[b], t + 1, size=hq)
    heads = np.arange(hq) // 2
    q = 64 * k[torch.from_numpy(pick), torch.from_numpy(heads)[None]]
    kf = to_f64(k)
    for b in range(3):  # every other visible key is far below
        for t in range(cu[b], cu[b + 1]):
            for h in range(hq):
                dots = kf[cu[b]:t + 1, heads[h]] @ kf[pick[t, h], heads[h]]
                dots[pick[t, h] - cu[b]] = -1e9
                assert 64 * 0.125 * np.log2(np.e) * (d - dots.max()) > 160
    cud = torch.from_numpy(cu).cuda()
    o, lse, r = fa.attention_packed_forward(q.cuda(), k.cuda(), v.cuda(), cud, True, 0.125, residual=True)
    dq, dk, dv = fa.attention_packed_backward(q.cuda(), k.cuda(), v.cuda(), o, dout.cuda(), lse, cud, True, 0.125,
                                              o_resid=r)
    done()
    assert torch.equal(o.cpu(), v[torch.from_numpy(pick), torch.from_numpy(heads)[None]])
    assert (lse.cpu().t() / (0.125 * 64 * d) - 1).abs().max() < 2e-6
    assert (r == 0).all()


@pytest.mark.parametrize("r", [3, 5, 7])
@pytest.mark.parametrize("d", [64, 128])
def test_groups_that_leave_rows_of_a_tile_free_repeat(d, r):
    # 128 % r rows of a query tile belong to no token. Whatever another call left in shared memory there (zeros, or
    # queries with scores of hundreds), the results are the same bits.
    lens, hkv = [700, 300, 129], 4
    q, k, v, _ = (x.cuda() for x in inputs(lens, r * hkv, hkv, d, 500 + r))
    cu = torch.from_numpy(offsets(lens)).cuda()
    other = normal(510, 8192, 16, d).cuda()
    whole = torch.tensor([0, 4096, 8192], dtype=torch.int32, device="cuda")
    pages = [x.view(-1, 16, hkv, d).transpose(1, 2).contiguous() for x in (k[:1024], v[:1024])]
    table, ln = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32), torch.tensor([500, 400], dtype=torch.int32, device="cuda")
    new = torch.from_numpy(offsets([200, 130])).cuda()
    got = []
    for gain in (0.0, 100.0, 0.0, -100.0):
        fa.attention_packed_forward(other * gain, other, other, whole, False, 0.125)
        got.append(fa.attention_packed_forward(q, k, v, cu, True, 0.125))
        fa.attention_packed_forward(other * gain, other, other, whole, False, 0.125)
        got[-1] += fa.attention_paged(q[:330], *pages, table, ln, new, 200, True, 0.125)
    done()
    for x in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, got[0]))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 4), (64, 8, 2), (128, 4, 4), (128, 8, 2)])
def test_a_neighbours_queries_change_no_bit(d, hq, hkv, causal):
    # The first sequence's last query tile also holds the second one's first queries, of large scores or none.
    lens = [300, 300]
    q, k, v, _ = (x.cuda() for x in inputs(lens, hq, hkv, d, 520))
    cu = torch.from_numpy(offsets(lens)).cuda()
    got = []
    for gain in (0.0, 100.0, 1.0):
        x = q.clone()
        x[300:] *= gain
        got.append(fa.attention_packed_forward(x, k, v, cu, causal, 0.125))
    done()
    for o, lse in got[1:]:
        assert torch.equal(o[:300], got[0][0][:300]) and torch.equal(lse[:, :300], got[0][1][:, :300])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_key_gradients_repeat_with_208_units(d, causal):
    # 52 tiles of 128 keys times 4 KV heads: every tile's dk and dv come from one CTA. With fewer, parts are added up by
    # several, in any order: bounds hold, the last bits may differ.
    scale = 0.125
    for lens, repeats in (([2900, 127, 1, 2300, 1100], True), ([700], False)):
        tiles = sum(-(-n // 128) for n in lens)
        assert (tiles * 4 >= 208) == repeats
        host = inputs(lens, 8, 4, d, 530)
        q, k, v, dout = (x.cuda() for x in host)
        cu = offsets(lens)
        cud = torch.from_numpy(cu).cuda()
        o, lse, resid = fa.attention_packed_forward(q, k, v, cud, causal, scale, residual=True)
        first = None
        for _ in range(10):
            grads = fa.attention_packed_backward(q, k, v, o, dout, lse, cud, causal, scale, o_resid=resid)
            first = first or grads
            assert not repeats or (torch.equal(grads[1], first[1]) and torch.equal(grads[2], first[2]))
        done()
        if not repeats:
            backward_check(*host, grads, cu, causal, scale)
