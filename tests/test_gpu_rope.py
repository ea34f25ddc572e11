"""GPU parity of rotary positions (fa_rope) and the append to a paged cache (fa_paged_append) against the fp64 oracle,
their refusals of bad pages, and the two paths they belong to: prompt -> cache -> attention, and a training step."""

import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_56_b200 import fa, to_f64

from .packed import HALF, Cache, W, assert_forward, assert_within, done, normal, offsets

pytestmark = pytest.mark.gpu

# The rotation is in fp32 of exact bf16 inputs. For positions below 2^24 the float64 angle is off by less than 2^-28;
# its fp32 fraction of a turn (2^-25 pi) and the function (two units of 2^-24) leave cos and sin off by 2^-22, the fp32
# products and their sum by another 2^-23: an element by less than 2^-21 (|x| + |y|) before its rounding to bf16.
FINE = 2.0 ** -21


def freqs(pairs, base=10000.0):
    return base ** (-np.arange(pairs) / pairs)


def check_turned(name, got, x, positions, f, sections, interleaved, inverse):
    ref = oracle.rope_ref(to_f64(x), positions, f, sections, interleaved, inverse)
    size = np.abs(to_f64(x)).max()
    assert_within(name, got, ref, HALF * np.abs(ref) + FINE * 2 * size)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,sections", [(1, 1, 1, 64, [32]), (77, 5, 1, 128, [64]), (700, 4, 2, 128, [16, 24, 24]),
                                                 (33, 3, 3, 64, [4, 3, 1]), (50, 2, 1, 128, [8, 8, 8, 8])])
def test_rope(T, hq, hkv, d, sections, interleaved, inverse):
    q, k = normal(1, T, hq, d), normal(2, T, hkv, d)
    rng = np.random.default_rng(T)
    pos = rng.integers(-5, 1 << 24, size=(len(sections), T)).astype(np.int32)
    pos[:, ::3] = rng.integers(0, 4096, size=pos[:, ::3].shape)
    f = freqs(sum(sections))
    args = (torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), sections, interleaved, inverse)
    qd, kd = q.cuda(), k.cuda()
    qo, ko = fa.rope(qd, kd, *args)
    done()
    check_turned("q", qo, q, pos, f, sections, interleaved, inverse)
    check_turned("k", ko, k, pos, f, sections, interleaved, inverse)
    assert torch.equal(qd.cpu(), q) and torch.equal(kd.cpu(), k)
    # One of the two alone, and in place.
    assert torch.equal(fa.rope(None, kd, *args)[1], ko)
    assert torch.equal(fa.rope(qd, None, *args)[0], qo)
    fa.fa_rope(qd, kd, qd, kd, *args)
    done()
    assert torch.equal(qd, qo) and torch.equal(kd, ko)


def test_rope_of_strided_views():
    fused = normal(3, 40, 8, 64).cuda()
    q, k, _ = fused.split((4, 2, 2), 1)
    pos, f = np.arange(40, dtype=np.int32)[None], freqs(16)
    want_q, want_k = q.cpu(), k.cpu()
    rest = fused[:, 6:].clone()
    fa.fa_rope(q, k, q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda())
    done()
    check_turned("q", q, want_q, pos, f, [16], False, False)
    check_turned("k", k, want_k, pos, f, [16], False, False)
    assert torch.equal(fused[:, 6:], rest)


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("new,lens,page,hq,hkv,d,sections", [
    ([1], [1], 16, 2, 1, 64, [32]),
    ([1, 1, 1], [500, 17, 16], 16, 4, 2, 128, None),
    ([40, 0, 3, 200], [40, 7, 100, 333], 48, 3, 3, 64, [8, 4, 4]),
    ([5, 2], [3, 0], 8, 2, 2, 64, [32]),   # places below 0 are left out
    ([1] * 70, list(range(1, 71)), 32, 4, 1, 128, [64]),
])
def test_append(new, lens, page, hq, hkv, d, sections, token_major):
    cache = Cache(5, lens, page, hkv, d, token_major=token_major)
    kp, vp, table, ln = cache.cuda()
    cu = offsets(new) + 2
    T = int(cu[-1]) + 3
    q, k, v = normal(6, T, hq, d), normal(7, T, hkv, d), normal(8, T, hkv, d)
    f = None if sections is None else freqs(sum(sections))
    multi = sections is not None and len(sections) > 1
    pos = np.random.default_rng(1).integers(0, 100000, size=(len(sections), T)).astype(np.int32) if multi else None
    q_out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_paged_append(q.cuda(), k.cuda(), v.cuda(), q_out, kp, vp, table, ln, torch.from_numpy(cu).cuda(),
                       None if pos is None else torch.from_numpy(pos).cuda(),
                       None if f is None else torch.from_numpy(f).cuda(), sections)
    done()
    where = oracle.places(lens, cu, T)
    if pos is None:
        pos = np.array([[max(at, -10 ** 6) for _, at in where]], dtype=np.int32)
    rk = oracle.rope_ref(to_f64(k), pos, f, sections, False, False) if f is not None else to_f64(k)
    rq = oracle.rope_ref(to_f64(q), pos, f, sections, False, False) if f is not None else to_f64(q)
    kref, vref = to_f64(cache.k), to_f64(cache.v)
    kref, vref = (oracle.append_ref(x, y, cache.table, cache.lens, cu) for x, y in ((kref, rk), (vref, to_f64(v))))
    assert np.array_equal(to_f64(vp), vref, equal_nan=True)
    touched = np.zeros(kref.shape, dtype=bool)
    for b, at in where:
        if b >= 0 and at >= 0:
            touched[cache.table[b, at // page], :, at % page] = True
    got = to_f64(kp)
    assert np.array_equal(got[~touched], kref[~touched], equal_nan=True)
    assert_within("k", got[touched], kref[touched], HALF * np.abs(kref[touched]) + FINE * 10)
    assert_within("q", q_out[2:-3], rq[2:-3], HALF * np.abs(rq[2:-3]) + FINE * 10)
    assert (q_out[:2] == 7).all() and (q_out[-3:] == 7).all()


def test_append_leaves_bad_pages_and_sequences_out():
    cache = Cache(15, [40, 40], 16, 1, 64)
    for what in ("page", "len"):
        kp, vp, table, ln = cache.cuda()
        before = kp.clone()
        if what == "page":
            table[0, 2] = cache.n_pages
        else:
            ln[0] = table.shape[1] * 16 + 1
        k, v = normal(16, 10, 1, 64).cuda(), normal(17, 10, 1, 64).cuda()
        fa.paged_append(k, v, kp, vp, table, ln, torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda"))
        assert fa.fa_check_device_error() == fa.FA_ERR_DATA
        got, page = kp.cpu(), cache.table[1, 2]
        assert torch.equal(got[page, 0, 3:8], k[5:, 0].cpu())
        got[page, 0, 3:8] = before.cpu()[page, 0, 3:8]
        assert torch.equal(got.nan_to_num(7.0), before.cpu().nan_to_num(7.0))


@pytest.mark.parametrize("d", [64, 128])
def test_serving_path(d):
    # Prompts appended and attended to in chunks, then token by token, equal the packed prompt's rows.
    hq, hkv, page = 4, 2, 16
    lens = [70, 200]
    cu = offsets(lens)
    T = int(cu[-1])
    q, k, v = (normal(s, T, h, d).cuda() for s, h in ((1, hq), (2, hkv), (3, hkv)))
    f = torch.from_numpy(freqs(d // 2)).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens])[None]
    qr, kr = fa.rope(q, k, pos, f)
    want_o, want_l = fa.attention_packed_forward(qr, kr, v, torch.from_numpy(cu).cuda(), True)
    pages = 2 * -(-max(lens) // page)
    kp = torch.full((pages, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    table = torch.randperm(pages).to(torch.int32).view(2, -1).cuda()
    at = [0, 0]
    for chunk in ([40, 130], [29, 0], [0, 68], [1, 1], [0, 1]):
        rows = torch.cat([torch.arange(cu[b] + at[b], cu[b] + at[b] + chunk[b]) for b in range(2)]).cuda()
        at = [a + c for a, c in zip(at, chunk)]
        ln = torch.tensor(at, dtype=torch.int32, device="cuda")
        cc = torch.from_numpy(offsets(chunk)).cuda()
        qq = fa.paged_append(k[rows], v[rows], kp, vp, table, ln, cc, q=q[rows], inv_freq=f)
        assert torch.equal(qq, qr[rows])
        o, lse = fa.attention_paged(qq, kp, vp, table, ln, cc, max(chunk))
        done()
        # Two results of the same exact value, each off by its weights' and its own rounding (|O| and the weighted
        # |v| are below 4 here).
        assert (o.float() - want_o[rows].float()).abs().max() <= 2 * 4 * (W + HALF)
        assert (lse - want_l[:, rows]).abs().max() <= 6e-4
    assert at == lens


def test_training_path_gradients():
    # rope -> packed attention -> backward -> inverse rope: the gradients of the unturned q and k.
    lens, hq, hkv, d = [60, 131], 4, 2, 64
    cu = offsets(lens)
    T = int(cu[-1])
    host = [normal(s, T, h, d) for s, h in ((1, hq), (2, hkv), (3, hkv), (4, hq))]
    q, k, v, dout = (x.cuda() for x in host)
    f, sec = freqs(32), [8, 12, 12]
    pos = np.random.default_rng(0).integers(0, 1000, size=(3, T)).astype(np.int32)
    rope = (torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), sec)
    cud = torch.from_numpy(cu).cuda()
    qr, kr = fa.rope(q, k, *rope)
    o, lse, r = fa.attention_packed_forward(qr, kr, v, cud, True, 0.125, residual=True)
    gq, gk, gv = fa.attention_packed_backward(qr, kr, v, o, dout, lse, cud, True, 0.125, o_resid=r)
    dq, dk = fa.rope(gq, gk, *rope, inverse=True)
    done()
    # From the turned bf16 q and k on, exactly; the inverse turns the bounds like the values.
    ref = oracle.packed_bwd_ref(to_f64(qr), to_f64(kr), to_f64(host[2]), to_f64(host[3]), cu, True, 0.125, W)
    for got, want, err in ((dq, ref[0], ref[3]), (dk, ref[1], ref[4])):
        exact = oracle.rope_ref(want, pos, f, sec, False, True)
        e = err + HALF * np.abs(want) + 1e-5  # before the turn: of a pair, at most the sum of both bounds
        pair = np.concatenate([e[..., :32] + e[..., 32:]] * 2, -1)
        assert_within("turned gradient", got, exact, pair * (1 + HALF) + HALF * np.abs(exact) + 1e-5)
    assert_within("dV", gv, ref[2], ref[5] + HALF * np.abs(ref[2]) + 1e-5)
