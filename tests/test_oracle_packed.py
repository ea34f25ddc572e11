"""Pins of the packed, paged and rotary oracle functions: against the equal-length definitions, one another, and the
rotation's identities."""

import numpy as np

import oracle


def draw(*shapes, seed=0):
    rng = np.random.default_rng(seed)
    return [rng.normal(size=s) for s in shapes]


def test_packed_is_the_definition_per_sequence():
    q, k, v, g = draw((11, 4, 8), (11, 2, 8), (11, 2, 8), (11, 4, 8))
    cu = np.array([1, 5, 5, 11])
    for causal in (True, False):
        O, L, A = oracle.packed_fwd_ref(q, k, v, cu, causal, 0.3)
        grads = oracle.packed_bwd_ref(q, k, v, g, cu, causal, 0.3, 0.01)
        assert np.isnan(O[0]).all() and np.isnan(L[:, 0]).all() and np.isnan(grads[1][0]).all()
        for lo, hi in ((1, 5), (5, 11)):
            b = [x[lo:hi].transpose(1, 0, 2)[None] for x in (q, k, v, g)]
            Ob, Lb = oracle.attn_fwd_ref(*b[:3], causal, 0.3)
            np.testing.assert_allclose(O[lo:hi], Ob[0].transpose(1, 0, 2), atol=1e-13)
            np.testing.assert_allclose(L[:, lo:hi], Lb[0], atol=1e-13)
            for x, y in zip(grads[:3], oracle.attn_bwd_ref(*b, causal, 0.3)):
                np.testing.assert_allclose(x[lo:hi], y[0].transpose(1, 0, 2), atol=1e-12)
        assert (A[1:] >= np.abs(O[1:]) - 1e-13).all() and all((e >= 0).all() for e in grads[3:])


def test_paged_is_packed_with_a_table():
    lens, new, page = [7, 5], [3, 5], 4
    q, k, v = draw((8, 2, 8), (12, 1, 8), (12, 1, 8), seed=1)
    table = np.array([[2, 0], [3, 1]])
    kp, vp = np.full((4, 1, page, 8), np.nan), np.full((4, 1, page, 8), np.nan)
    cu = np.array([0, 3, 8])
    # The caches are filled by the append, old tokens first.
    full = np.array([0, 7, 12])
    kp, vp = (oracle.append_ref(p, x, table, np.array(lens), full) for p, x in ((kp, k), (vp, v)))
    O, L, _ = oracle.paged_ref(q, kp, vp, table, lens, cu, True, 0.3)
    qq = np.zeros((12, 2, 8))
    qq[4:7], qq[7:] = q[:3], q[3:]
    Op, Lp, _ = oracle.packed_fwd_ref(qq, k, v, full, True, 0.3)
    np.testing.assert_allclose(O, np.concatenate([Op[4:7], Op[7:]]), atol=1e-13)
    np.testing.assert_allclose(L, np.concatenate([Lp[:, 4:7], Lp[:, 7:]], 1), atol=1e-13)
    # Rows without keys.
    O, L, _ = oracle.paged_ref(q, kp, vp, table, [1, 0], cu, True, 0.3)
    assert (O[:2] == 0).all() and np.isneginf(L[:, :2]).all() and np.isfinite(L[:, 2]).all() and (O[3:] == 0).all()
    assert oracle.places([1, 0], cu, 8)[:3] == [(0, -2), (0, -1), (0, 0)]


def test_rotation_identities():
    x, y = draw((6, 3, 16), (6, 3, 16), seed=2)
    f = 100.0 ** (-np.arange(6) / 6)
    pos = np.random.default_rng(3).integers(0, 50, size=(2, 6))
    for interleaved in (False, True):
        a = oracle.rope_ref(x, pos, f, [2, 4], interleaved, False)
        np.testing.assert_allclose(oracle.rope_ref(a, pos, f, [2, 4], interleaved, True), x, atol=1e-13)
        assert np.array_equal(a[..., 12:], x[..., 12:])
        np.testing.assert_allclose((a ** 2).sum(-1), (x ** 2).sum(-1), atol=1e-12)
        # Scores go by differences of positions alone.
        s = (oracle.rope_ref(x, pos, f, [2, 4], interleaved, False) * oracle.rope_ref(y, pos + 7, f, [2, 4], interleaved, False)).sum(-1)
        t = (oracle.rope_ref(x, pos * 0, f, [2, 4], interleaved, False) * oracle.rope_ref(y, pos * 0 + 7, f, [2, 4], interleaved, False)).sum(-1)
        np.testing.assert_allclose(s, t, atol=1e-12)
    # The pairs are those named: half apart, or neighbours.
    e = np.zeros((1, 1, 4))
    e[0, 0, 0] = 1.0
    one = np.array([[1]])
    np.testing.assert_allclose(oracle.rope_ref(e, one, np.array([0.5, 9.0]), [2], False, False)[0, 0], [np.cos(0.5), 0, np.sin(0.5), 0])
    np.testing.assert_allclose(oracle.rope_ref(e, one, np.array([0.5, 9.0]), [2], True, False)[0, 0], [np.cos(0.5), np.sin(0.5), 0, 0])
