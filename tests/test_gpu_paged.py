"""GPU parity of attention over a paged cache (fa_paged_fwd) against the fp64 oracle: single tokens, drafted tokens,
chunks and mixtures; page sizes that end inside a key tile; empty caches and rows without keys; NaN in unused slots;
strided views; out-of-range pages, lengths and offsets; graphs, streams and guard rows."""

import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_56_b200 import fa, to_f64

from .packed import Cache, assert_forward, done, normal, offsets

pytestmark = pytest.mark.gpu


def run(new, lens, page, hq, hkv, d, causal=True, seed=1, max_q=None, token_major=False, cu=None):
    cache = Cache(seed, lens, page, hkv, d, token_major=token_major)
    cu = offsets(new) if cu is None else np.array(cu, dtype=np.int32)
    q = normal(seed + 7, int(cu[-1]), hq, d)
    kp, vp, table, ln = cache.cuda()
    o, lse = fa.attention_paged(q.cuda(), kp, vp, table, ln, torch.from_numpy(cu).cuda(),
                                max(new) if max_q is None else max_q, causal, 0.125)
    done()
    ref = oracle.paged_ref(to_f64(q), to_f64(cache.k), to_f64(cache.v), cache.table, cache.lens, cu, causal, 0.125)
    assert_forward(o, lse, *ref)
    return o, lse


# (new tokens, cached tokens, page, Hq, Hkv)
FEW = [
    ([1], [1], 16, 1, 1),
    ([1], [129], 16, 16, 16),
    ([1, 1, 1], [1000, 1, 257], 64, 8, 2),
    ([4, 1, 3], [300, 64, 3], 32, 8, 1),        # 32 rows: four copies
    ([8, 2], [500, 700], 48, 6, 1),             # 48 rows: two copies, pages that do not divide a tile
    ([16, 0, 9], [200, 50, 130], 128, 8, 1),    # 128 rows, an empty sequence between
    ([7, 25], [40, 2000], 256, 5, 1),           # 125 rows, group of five
    ([1] * 40, [17 + 31 * i for i in range(40)], 8, 4, 4),
    ([128], [128], 16, 1, 1),
    ([1, 0, 1], [5, 700, 260], 24, 128, 1),     # a group of 128: one token fills the tile
    ([2, 9], [100, 40], 16, 14, 2),             # groups of seven, 63 rows
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", FEW)
def test_few_rows(case, d):
    new, lens, page, hq, hkv = case
    run(new, lens, page, hq, hkv, d, seed=sum(lens) + d)


CHUNKS = [
    ([129], [129], 16, 1, 1),
    ([300], [300], 64, 4, 2),
    ([200, 1, 0, 33], [1000, 77, 10, 33], 16, 8, 2),
    ([64, 64], [64, 3000], 48, 12, 4),          # groups of three
    ([257, 1, 1], [400, 2500, 1], 128, 4, 1),
    ([40], [5000], 256, 10, 2),                 # groups of five, few units: cut along the keys
    ([140, 3], [141, 4000], 8, 2, 2),
    ([2, 3], [400, 1000], 16, 128, 1),          # a group of 128
    ([70, 1, 9, 2], [1500, 300, 9, 2000], 40, 7, 1),
    ([130] * 6, [130, 1130, 2130, 700, 300, 1999], 64, 2, 1),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CHUNKS)
def test_chunks(case, d):
    new, lens, page, hq, hkv = case
    run(new, lens, page, hq, hkv, d, seed=sum(lens) + d)


@pytest.mark.parametrize("new", [[3, 5], [130, 70]])
@pytest.mark.parametrize("d", [64, 128])
def test_not_causal(new, d):
    run(new, [333, 700], 32, 4, 2, d, causal=False, seed=5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [([4, 2], [2, 0]), ([150, 140, 1], [20, 0, 0]), ([3, 1], [0, 5])])
def test_rows_without_keys(new, lens, d):
    # New tokens at places below 0 (a cache shorter than its new tokens) and empty caches: O = 0, L = -inf.
    o, lse = run(new, lens, 16, 4, 2, d, seed=9)
    n, m = new[0], lens[0]
    assert (o[:n - m] == 0).all() and torch.isneginf(lse[:, :n - m]).all()
    run(new, lens, 16, 4, 2, d, causal=False, seed=9)


@pytest.mark.parametrize("new", [[1, 1], [100, 60]])
def test_a_loose_bound_on_new_tokens(new):
    # max_q above the longest sequence may take the other kernel; the result is the same to rounding.
    run(new, [300, 400], 16, 4, 2, 128, seed=11, max_q=200)


@pytest.mark.parametrize("new", [[2, 3], [150, 20]])
@pytest.mark.parametrize("d", [64, 128])
def test_strided_views(new, d):
    lens, hq, hkv = [200, 333], 4, 2
    cache = Cache(3, lens, 16, hkv, d, token_major=True)
    kp, vp, table, ln = cache.cuda()
    cu = offsets(new)
    T = int(cu[-1])
    fused = normal(4, T, hq + 2 * hkv, d).cuda()   # q is a slice of a fused projection
    wide = torch.full((2, table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    out = torch.full((hq, T + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")  # head-major output
    lse = torch.empty(hq, T, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(2, T, max(new), hq, hkv, d, 16, table.shape[1]),
                     dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(fused[:, :hq], kp, vp, out.transpose(0, 1)[:T], lse, wide[:, :table.shape[1]], ln,
                    torch.from_numpy(cu).cuda(), max(new), True, 0.125, ws)
    done()
    ref = oracle.paged_ref(to_f64(fused[:, :hq]), to_f64(cache.k), to_f64(cache.v), cache.table, cache.lens, cu, True,
                           0.125)
    assert_forward(out.transpose(0, 1)[:T], lse, *ref)
    assert (out[:, T:] == 7.0).all()


@pytest.mark.parametrize("lens,max_q", [([100, 200], 4), ([300, 150], 140)])
def test_rows_outside_the_sequences_stay(lens, max_q):
    # Offsets that start behind row 0 and end before the last: those rows are left as they were.
    new = [min(4, max_q), max_q]
    cache = Cache(21, lens, 16, 2, 64)
    kp, vp, table, ln = cache.cuda()
    cu = offsets(new) + 3
    T = int(cu[-1]) + 5
    q = normal(22, T, 4, 64)
    q[:3] = q[-5:] = float("nan")
    o = torch.full((T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, T), 7.0, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(2, T, max_q, 4, 2, 64, 16, table.shape[1]), dtype=torch.uint8,
                     device="cuda")
    fa.fa_paged_fwd(q.cuda(), kp, vp, o, lse, table, ln, torch.from_numpy(cu).cuda(), max_q, True, 0.125, ws)
    done()
    assert_forward(o, lse, *oracle.paged_ref(to_f64(q), to_f64(cache.k), to_f64(cache.v), cache.table, cache.lens, cu,
                                             True, 0.125))
    assert (o[:3] == 7).all() and (o[-5:] == 7).all() and (lse[:, :3] == 7).all() and (lse[:, -5:] == 7).all()


def test_single_tokens_without_offsets_and_shared_pages():
    # No offsets: one token each. Both sequences read the same pages.
    cache = Cache(31, [500], 16, 2, 128)
    kp, vp, table, _ = cache.cuda()
    table2 = table.repeat(3, 1)
    lens = np.array([500, 123, 500], dtype=np.int32)
    q = normal(32, 3, 8, 128)
    o, lse = fa.attention_paged(q.cuda(), kp, vp, table2, torch.from_numpy(lens).cuda(), scale=0.125)
    done()
    ref = oracle.paged_ref(to_f64(q), to_f64(cache.k), to_f64(cache.v), np.repeat(cache.table, 3, 0), lens,
                           offsets([1, 1, 1]), True, 0.125)
    assert_forward(o, lse, *ref)


@pytest.mark.parametrize("rows", [[2, 3], [140, 150]])
@pytest.mark.parametrize("break_", ["len", "negative_len", "order", "end", "max_q"])
def test_out_of_range_lengths_are_reported_and_nothing_is_written(rows, break_):
    cache = Cache(41, [200, 300], 16, 2, 64)
    kp, vp, table, ln = cache.cuda()
    cu = offsets(rows)
    T, max_q = int(cu[-1]), max(rows)
    if break_ == "len":
        ln[1] = table.shape[1] * 16 + 1
    elif break_ == "negative_len":
        ln[0] = -1
    elif break_ == "order":
        cu[1] = T + 1
    elif break_ == "end":
        cu[2] = T + 1
    else:
        max_q -= 1
    q = normal(42, T, 4, 64).cuda()
    o = torch.full((T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, T), 7.0, device="cuda")
    ws = torch.empty(fa.fa_paged_fwd_workspace_bytes(2, T, max_q, 4, 2, 64, 16, table.shape[1]), dtype=torch.uint8,
                     device="cuda")
    fa.fa_paged_fwd(q, kp, vp, o, lse, table, ln, torch.from_numpy(cu).cuda(), max_q, True, 0.125, ws)
    assert fa.fa_check_device_error() == fa.FA_ERR_DATA
    assert fa.fa_check_device_error() == fa.FA_OK
    assert (o == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("new", [1, 150])
@pytest.mark.parametrize("bad", [-1, 2 ** 30])
def test_a_page_outside_the_pool_is_read_as_zeros_and_reported(new, bad):
    cache = Cache(51, [300], 16, 2, 64)
    kp, vp, table, ln = cache.cuda()
    table[0, 3] = bad
    q = normal(52, new, 4, 64)
    o, lse = fa.attention_paged(q.cuda(), kp, vp, table, ln, torch.from_numpy(offsets([new])).cuda(), new, True, 0.125)
    assert fa.fa_check_device_error() == fa.FA_ERR_DATA
    page = cache.table[0, 3]
    cache.k[page] = cache.v[page] = 0
    assert_forward(o, lse, *oracle.paged_ref(to_f64(q), to_f64(cache.k), to_f64(cache.v), cache.table, cache.lens,
                                             offsets([new]), True, 0.125))


@pytest.mark.parametrize("new", [[1, 1], [90, 100]])
def test_captured_call_replays_on_grown_sequences(new):
    page, hq, hkv, d = 16, 4, 2, 64
    cache = Cache(61, [700, 900], page, hkv, d)
    kp, vp, table, ln = cache.cuda()
    q = normal(62, sum(new), hq, d).cuda()
    cu = torch.from_numpy(offsets(new)).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fa.attention_paged(q, kp, vp, table, ln, cu, max(new), True, 0.125)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fa.attention_paged(q, kp, vp, table, ln, cu, max(new), True, 0.125)
    for lens in ([700, 900], [150, 899], [101, 333]):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        done()
        want = fa.attention_paged(q, kp, vp, table, ln, cu, max(new), True, 0.125)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        ref = oracle.paged_ref(to_f64(q), to_f64(cache.k), to_f64(cache.v), cache.table, np.array(lens), offsets(new),
                               True, 0.125)
        assert_forward(o, lse, *ref)


def test_on_another_stream():
    cache = Cache(71, [700, 900], 16, 2, 128)
    kp, vp, table, ln = cache.cuda()
    q = normal(72, 2, 8, 128).cuda()
    want = fa.attention_paged(q, kp, vp, table, ln, scale=0.125)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = fa.attention_paged(q, kp, vp, table, ln, scale=0.125, stream=stream)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits():
    # A pool of more than 2^32 bytes per tensor and 2^31 elements: pages at its end.
    page, hkv, d = 256, 8, 128
    n_pages = (1 << 31) // (page * hkv * d) + 9
    k = torch.zeros(n_pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = Cache(81, [1000], page, hkv, d, spare=0)
    table = small.table + (n_pages - small.n_pages)
    k[n_pages - small.n_pages:] = small.k.cuda()
    v[n_pages - small.n_pages:] = small.v.cuda()
    for new in (1, 140):
        q = normal(82, new, 16, d)
        o, lse = fa.attention_paged(q.cuda(), k, v, torch.from_numpy(table).cuda(),
                                    torch.from_numpy(small.lens).cuda(), torch.from_numpy(offsets([new])).cuda(), new,
                                    True, 0.125)
        done()
        assert_forward(o, lse, *oracle.paged_ref(to_f64(q), to_f64(small.k), to_f64(small.v), small.table, small.lens,
                                                 offsets([new]), True, 0.125))


@pytest.mark.parametrize("d", [64, 128])
def test_results_repeat(d):
    # Chunks beside single tokens, some units cut along the keys, some whole: every run gives the same bits.
    new, lens = [200, 130, 1, 33], [700, 2048, 3000, 33]
    cache = Cache(91, lens, 16, 4, d)
    kp, vp, table, ln = cache.cuda()
    q = normal(92, sum(new), 16, d).cuda()
    cu = torch.from_numpy(offsets(new)).cuda()
    first = None
    for _ in range(40):
        got = fa.attention_paged(q, kp, vp, table, ln, cu, max(new), True, 0.125)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    done()


def test_binding_refusals():
    cache = Cache(95, [40], 16, 2, 64)
    kp, vp, table, ln = cache.cuda()
    q = normal(96, 1, 4, 64).cuda()
    ok = dict(k_pages=kp, v_pages=vp, block_table=table, seq_lens=ln)

    def call(q=q, **kw):
        a = dict(ok, **kw)
        return fa.attention_paged(q, a.pop("k_pages"), a.pop("v_pages"), a.pop("block_table"), a.pop("seq_lens"), **a)

    call()
    for kw, err in ((dict(q=q.float()), TypeError), (dict(q=q[..., ::2]), ValueError), (dict(q=q[0]), ValueError),
                    (dict(k_pages=kp[0]), ValueError), (dict(v_pages=vp[:, :1]), ValueError),
                    (dict(block_table=table.long()), TypeError), (dict(block_table=table[0]), ValueError),
                    (dict(seq_lens=ln.repeat(2)), ValueError), (dict(seq_lens=ln.cpu()), RuntimeError),
                    (dict(cu_seqlens=torch.tensor([0, 1], device="cuda")), TypeError),
                    (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), fa.FaError),
                    (dict(scale=float("nan")), fa.FaError), (dict(max_q=-1), fa.FaError),
                    (dict(q=normal(1, 1, 3, 64).cuda()), fa.FaError),
                    (dict(k_pages=kp[:, :, :12], v_pages=vp[:, :, :12]), fa.FaError)):
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(fa.FaError) as e:
        call(max_q=0)
    assert e.value.status == fa.FA_ERR_INVALID_ARGUMENT and "fa_paged_fwd" in str(e.value)
    done()


@pytest.mark.parametrize("new,lens", [([1, 1, 1], [300, 5, 1000]), ([150, 3, 40], [700, 3, 1000])])
@pytest.mark.parametrize("d", [64, 128])
def test_workspace_contents_do_not_matter(new, lens, d):
    cache = Cache(97, lens, 16, 2, d)
    kp, vp, table, ln = cache.cuda()
    q = normal(98, sum(new), 4, d).cuda()
    cu = torch.from_numpy(offsets(new)).cuda()
    n = fa.fa_paged_fwd_workspace_bytes(3, sum(new), max(new), 4, 2, d, 16, table.shape[1])
    ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
    got = []
    for fill, at in ((0, 0), (0xFF, 0), (0x7F, 16)):  # NaN and huge patterns, another alignment
        ws.fill_(fill)
        got.append(fa.attention_paged(q, kp, vp, table, ln, cu, max(new), True, 0.125, workspace=ws[at:at + n]))
        done()
        assert torch.equal(got[-1][0], got[0][0]) and torch.equal(got[-1][1], got[0][1])


def test_no_tokens_and_no_sequences():
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    o, lse = fa.attention_paged(q, kp, kp, torch.zeros(0, 3, **i32), torch.zeros(0, **i32))
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    o, lse = fa.attention_paged(q, kp, kp, torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(3, **i32), 5)
    assert o.shape == (0, 4, 64)
    k = q[:, :2]
    assert fa.paged_append(k, k, kp, kp, torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(3, **i32), q=q).shape == q.shape
    fa.attention_packed_forward(q, k, k, torch.zeros(4, **i32), True)
    done()


def test_thousands_of_sequences():
    # More sequences than a warp sums in one step, some without new tokens or without keys.
    rng = np.random.default_rng(5)
    S = 2100
    new = rng.choice([0, 1, 1, 1, 2], size=S)
    lens = new + rng.choice([0, 1, 15, 40], size=S)
    lens[77], lens[1999] = 900, 2300
    new[77] = new[1999] = 1
    run([int(x) for x in new], [int(x) for x in lens], 16, 2, 1, 64, seed=3)
    # ... and through the prompt kernel.
    new[5] = 140
    lens[5] = 170
    run([int(x) for x in new], [int(x) for x in lens], 16, 2, 1, 64, seed=4)


def test_two_calls_at_once():
    # Chunks and single tokens on two streams, each with its own outputs and workspace, beside a packed prompt.
    a, b = Cache(101, [900, 2000], 16, 2, 64), Cache(102, [3000, 400], 32, 2, 128)
    da, db = a.cuda(), b.cuda()
    qa, qb, qp = normal(103, 280, 4, 64).cuda(), normal(104, 2, 8, 128).cuda(), normal(105, 700, 4, 64).cuda()
    cua, cup = torch.from_numpy(offsets([150, 130])).cuda(), torch.from_numpy(offsets([300, 400])).cuda()

    def calls(streams):
        return [fa.attention_paged(qa, *da, cua, 150, True, 0.125, stream=streams[0]),
                fa.attention_paged(qb, *db, scale=0.125, stream=streams[1]),
                fa.attention_packed_forward(qp, qp[:, :2], qp[:, 2:], cup, True, 0.125, stream=streams[2])]

    want = calls([None] * 3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        got = calls(streams)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    done()


@pytest.mark.parametrize("new", [[1, 3], [200, 9]])
@pytest.mark.parametrize("d", [64, 128])
def test_large_and_rising_scores(new, d):
    from .packed import HALF, assert_within
    from .test_gpu_packed import weight_error

    lens, hq, hkv, page = [900, 2000], 8, 2, 16
    cache = Cache(111, lens, page, hkv, d)
    u = normal(112, 1, 1, 1, d).float()
    u = u / u.norm()
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            p = cache.table[b, j]
            cache.k[p] = (2 * cache.k[p].float() + 60.0 * j * page / n * u[0]).to(torch.bfloat16)
    q = (2 * normal(113, sum(new), hq, d).float() + 4 * u[0]).to(torch.bfloat16)
    kp, vp, table, ln = cache.cuda()
    cu = offsets(new)
    scale = d ** -0.5
    o, lse = fa.attention_paged(q.cuda(), kp, vp, table, ln, torch.from_numpy(cu).cuda(), max(new), True, scale)
    done()
    O, L, A = oracle.paged_ref(to_f64(q), to_f64(cache.k), to_f64(cache.v), cache.table, cache.lens, cu, True, scale)
    w = weight_error(q, cache.k.nan_to_num(0.0).flatten(0, 1).flatten(0, 1)[:, None], scale)
    assert_within("O", o, O, w * A + HALF * np.abs(O) + 1e-6)
    assert_within("L", lse, L, (w - HALF) + 2.0 ** -22 * np.abs(L))


@pytest.mark.parametrize("new", [1, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_repeat_where_warps_differ(new, d):
    # Four, two and one copies of 4, 64 and 128 rows, about 14 key tiles in a row per CTA. Scores of some warps' rows
    # rise from tile to tile by 4 in all, those of the others fall, so that some warps rescale O at most tiles and the
    # others, which run ahead of them, at none.
    S, n, page, hkv, r = 16, 4096, 64, 4, 4 if new == 1 else 8
    k, v = normal(101, n, hkv, d).float() / 2, normal(102, n, hkv, d)
    j = torch.arange(n)
    rise = 32.0 * (j // 128) / (n // 128 - 1)
    k[:, :, 0] = (rise if new == 16 else torch.where(j % 128 < 64, rise, -rise))[:, None]
    q = normal(103, S, new, hkv, r, d)
    row = torch.arange(new * r).view(new, r)
    q[..., 0] = torch.where(row // 32 % 2 == 0, 1.0, -1.0)[:, None].to(torch.bfloat16)
    q = q.view(S * new, hkv * r, d)
    # All sequences share the pages of one, and end at different keys.
    order = torch.from_numpy(np.random.default_rng(104).permutation(n // page).astype(np.int32))
    kp, vp = (torch.empty(n // page, hkv, page, d, dtype=torch.bfloat16) for _ in range(2))
    for pages, x in ((kp, k.to(torch.bfloat16)), (vp, v)):
        pages[order.long()] = x.view(n // page, page, hkv, d).transpose(1, 2)
    table = order[None].repeat(S, 1)
    lens = np.array([n - 37 * b for b in range(S)], dtype=np.int32)
    cu = offsets([new] * S)
    args = [x.cuda() for x in (q, kp, vp, table, torch.from_numpy(lens), torch.from_numpy(cu))]
    first = None
    for _ in range(100):
        got = fa.attention_paged(*args, new, True, 0.125)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    done()
    assert_forward(*first, *oracle.paged_ref(to_f64(q), to_f64(kp), to_f64(vp), table.numpy(), lens, cu, True, 0.125))
