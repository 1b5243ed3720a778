"""attn_decode_paged on the GPU against the float64 paged oracle, with the
error bounds that the oracle derives from the kernel's roundings, and a run of
the cache's calls together."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_44_b200 as A
import oracle

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, FP: 2.0 ** -11}          # half a step of the weights' and the output's type
STEP = {BF: 0.0, FP: 2.0 ** -25}             # fp16: half the step below the normal range


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


def build(lens, H, Hk, N_q, d, page, dt, seed=0, cols=None, extra=3, shared=0, std=1.0):
    """Random pages for the lengths (garbage, NaN and infinities included, in every
    row that holds no position), the table in random order with -1 behind."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    cols = cols or max(1, max(-(-n // page) for n in lens))
    own = [max(0, -(-n // page) - shared // page) for n in lens]
    n_pages = sum(own) + shared // page + extra
    ids = rng.permutation(n_pages)
    k = rng.standard_normal((n_pages, Hk, page, d)).astype(np.float32) * std
    v = rng.standard_normal((n_pages, Hk, page, d)).astype(np.float32)
    real = np.zeros((n_pages, page), bool)
    prefix, at = ids[:shared // page], shared // page
    real[prefix] = True
    table = np.full((B, cols), -1)
    for b, n in enumerate(lens):
        mine = np.concatenate([prefix, ids[at:at + own[b]]])[:-(-n // page)]
        at += own[b]
        table[b, :len(mine)] = mine
        for j in range(0, n, page):
            real[mine[j // page], :min(page, n - j)] = True
    junk = np.array([np.nan, np.inf, -np.inf, 3e38], np.float32)
    for x in (k, v):
        bad = np.broadcast_to(~real[:, None, :, None], x.shape)
        x[bad] = rng.choice(junk, int(bad.sum()))
    k, v = (torch.from_numpy(x).to(dt) for x in (k, v))
    q = torch.from_numpy(rng.standard_normal((B, H, N_q, d)).astype(np.float32)).to(dt)
    cache = A.PagedCache(k.cuda(), v.cuda(), i32(table), i32(lens))
    return q, cache, prefix


def check(q, cache, causal=True, window=0, n_sink=0, scale=None, out_f32=False, status=0, got=None, **kw):
    d, dt = q.shape[3], q.dtype
    scale = A.default_scale(d) if scale is None else scale
    if got is None:
        A.get_status()
        got = A.decode_paged(q.cuda(), cache, causal=causal, window=window, n_sink=n_sink, scale=scale,
                             out_f32=out_f32, **kw)
        torch.cuda.synchronize()
        assert A.get_status() == status
    o, l = got
    assert o.dtype == (torch.float32 if out_f32 else dt)
    O, L, tO, tL = oracle.decode_paged(f64(q), f64(cache.k), f64(cache.v), cache.table.cpu().numpy(),
                                       cache.lens.cpu().numpy(), scale, causal, window, n_sink, u=U[dt],
                                       u_out=0.0 if out_f32 else U[dt], step=STEP[dt])
    o, l = f64(o), f64(l)
    empty = np.isneginf(L)
    assert (np.isneginf(l) == empty).all() and (o[empty] == 0).all()
    assert np.isfinite(o).all() and np.isfinite(l[~empty]).all()
    over = np.abs(o - O) - tO
    assert over.max() <= 0, (over.max(), np.abs(o - O).max())
    assert (np.abs(l[~empty] - L[~empty]) <= tL[~empty]).all(), np.abs(l[~empty] - L[~empty]).max()
    return got


# lens, H, H_kv, N_q, d, page, dtype, causal, window, n_sink
SWEEP = [
    ([1], 1, 1, 1, 64, 16, BF, 1, 0, 0),
    ([1, 0, 17], 4, 2, 1, 128, 16, FP, 1, 0, 0),
    ([15, 16, 17, 127, 128, 129], 4, 4, 1, 64, 16, BF, 1, 0, 0),
    ([300, 1, 0, 900, 33], 8, 2, 1, 128, 32, BF, 1, 0, 0),
    ([5000], 32, 8, 1, 128, 64, BF, 1, 0, 0),
    ([2500, 700], 8, 1, 2, 64, 128, FP, 1, 0, 0),
    ([640, 3, 1, 0], 6, 2, 4, 128, 256, BF, 1, 0, 0),      # rows before position 0
    ([640, 3, 1, 0], 6, 2, 4, 64, 16, FP, 0, 0, 0),
    ([999, 250], 16, 1, 1, 128, 16, BF, 0, 0, 0),          # 16 rows a group
    ([999, 250], 17, 1, 1, 64, 16, BF, 1, 0, 0),           # 17: a second row tile
    ([777, 130], 32, 1, 4, 128, 32, FP, 1, 0, 0),          # 128 rows
    ([400], 5, 1, 30, 64, 16, BF, 1, 0, 0),                # 150 rows
    ([3000, 900, 20], 8, 4, 3, 64, 16, BF, 1, 100, 5),
    ([3000, 900, 20], 8, 4, 3, 128, 64, FP, 1, 1, 0),
    ([3000, 900, 0], 4, 1, 2, 128, 16, BF, 1, 128, 200),   # more sinks than a tile
    ([700, 64], 2, 1, 1, 64, 32, FP, 1, 5000, 3),          # a window longer than the sequences
    # more rows a K/V head: tcgen05, groups of 128 rows and of 256
    ([700, 0, 1, 129, 128], 34, 2, 1, 128, 16, BF, 1, 0, 0),      # 17 rows
    ([2100, 40], 33, 1, 1, 64, 128, FP, 1, 0, 0),                 # 33 rows
    ([900, 0, 33, 2], 40, 2, 5, 128, 64, FP, 1, 0, 0),            # 100 rows, some before position 0
    ([900, 0, 33, 2], 40, 2, 5, 64, 256, BF, 0, 0, 0),
    ([3000, 900, 20, 0], 24, 1, 2, 128, 16, BF, 1, 100, 5),       # 48 rows under a window
    ([3000, 900, 20], 96, 2, 1, 64, 32, FP, 1, 1, 0),             # the diagonal alone
    ([2000, 700], 260, 2, 1, 128, 128, BF, 1, 0, 0),              # 130 rows: 256 a group
    ([1300, 0, 131], 160, 1, 2, 64, 16, BF, 1, 300, 200),         # 320 rows in two groups, window and sinks
    ([270, 1], 70, 2, 8, 128, 32, FP, 0, 0, 0),                   # 280 rows
    ([300, 190], 2, 2, 200, 64, 16, BF, 1, 0, 0),                 # 200 new rows of one head
    ([300, 190], 2, 2, 200, 128, 32, FP, 1, 50, 7),
    ([140] * 30 + [0], 68, 2, 1, 64, 16, FP, 1, 0, 0),            # more groups than ranges of a CTA's own
]


def _id(c):
    l, H, Hk, Nq, d, pg, dt, ca, w, s = c
    return f"n{max(l)}B{len(l)}H{H}k{Hk}q{Nq}d{d}p{pg}{'bf' if dt == BF else 'fp'}{'c' if ca else 'n'}w{w}s{s}"


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case", SWEEP, ids=[_id(c) for c in SWEEP])
def test_sweep(case, f32):
    lens, H, Hk, N_q, d, page, dt, causal, window, n_sink = case
    q, cache, _ = build(lens, H, Hk, N_q, d, page, dt, seed=sum(lens) + H)
    check(q, cache, bool(causal), window, n_sink, out_f32=f32)


@pytest.mark.parametrize("seed", range(24))
def test_random_cases(seed):
    rng = np.random.default_rng(500 + seed)
    B = int(rng.integers(1, 20))
    top = int(np.exp(rng.uniform(0, np.log(1500))))
    lens = [int(x) for x in rng.integers(0, top + 1, B)]
    Hk = int(rng.integers(1, 4))
    G = int(rng.choice([1, 2, 3, 4, 8, 20]))
    N_q = int(rng.choice([1, 1, 2, 3, 5]))
    window = int(rng.integers(1, 600)) if seed % 3 == 0 else 0
    q, cache, _ = build(lens, G * Hk, Hk, N_q, int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128, 256])),
                        [BF, FP][seed % 2], seed=seed)
    check(q, cache, bool(window) or seed % 4 != 1, window, int(rng.integers(0, 300)) if window else 0,
          out_f32=seed % 5 == 0)


# lens, H, H_kv, N_q, d, page, dtype, causal, shared
SHARED = [
    ([130, 128, 200], 2, 1, 1, 64, 16, BF, 1, 128),
    ([1500, 1100, 1024, 0, 1025], 4, 2, 1, 128, 64, BF, 1, 1024),
    ([700] * 9 + [0, 641], 8, 2, 2, 64, 16, FP, 1, 640),
    ([530, 513, 512, 900], 8, 8, 3, 128, 256, BF, 0, 512),
    ([514, 513, 512, 900], 8, 8, 3, 128, 256, FP, 1, 512),  # rows inside the prefix
    ([300, 160], 32, 1, 3, 64, 32, BF, 1, 160),             # part of a tile beyond whole ones
    ([400] * 40, 16, 2, 1, 128, 16, BF, 1, 384),            # several row tiles of the prefix
    ([300] * 5, 160, 20, 1, 64, 32, FP, 1, 256),            # 40 rows of each of 20 K/V heads
    ([300, 0, 290] * 3, 180, 60, 2, 64, 128, BF, 1, 256),   # 60 K/V heads
    ([300, 280], 340, 170, 12, 64, 16, FP, 1, 128),         # more groups than ranges
    ([350, 310, 0], 60, 2, 4, 128, 16, BF, 1, 256),         # 120 rows a sequence, 360 of the prefix
    ([150] * 600 + [0], 1, 1, 1, 64, 16, BF, 1, 128),       # more sequences than lengths kept on chip
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case", SHARED, ids=[f"B{len(c[0])}H{c[1]}q{c[3]}d{c[4]}s{c[8]}c{c[7]}" for c in SHARED])
def test_shared_prefix(case, f32):
    lens, H, Hk, N_q, d, page, dt, causal, shared = case
    q, cache, prefix = build(lens, H, Hk, N_q, d, page, dt, seed=shared + H, shared=shared)
    o, l = check(q, cache, bool(causal), out_f32=f32, shared_len=shared, shared_table=i32(prefix))
    check(q, cache, bool(causal), out_f32=f32)
    # a window: every sequence reads its own pages, the same bits
    a = A.decode_paged(q.cuda(), cache, window=77, shared_len=shared, shared_table=i32(prefix))
    b = A.decode_paged(q.cuda(), cache, window=77)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("H", [8, 64])
def test_a_window_that_masks_nothing_is_no_window(H):
    """At max_pages * page_size and beyond the bits are those of window 0, shared prefix or
    not; one position less is a window, under which nothing is shared."""
    q, cache, prefix = build([700] * 6 + [0, 321], H, 2, 2, 64, 16, FP, seed=25, shared=320, cols=44)
    q, cap = q.cuda(), 44 * 16
    shared = dict(shared_len=320, shared_table=i32(prefix))
    for kw in ({}, shared):
        want = A.decode_paged(q, cache, **kw)
        for window, n_sink in ((cap, 0), (cap + 1, 5), (2 ** 31 - 1, 2 ** 31 - 1)):
            got = A.decode_paged(q, cache, window=window, n_sink=n_sink, **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(q.cpu(), cache, True, cap, 5, **shared)
    a = A.decode_paged(q, cache, window=cap - 1, **shared)
    b = A.decode_paged(q, cache, window=cap - 1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_sequences_shorter_than_the_shared_prefix():
    """The prefix's pages are listed for the longest; short sequences use their part of it."""
    q, cache, prefix = build([900, 700, 650], 4, 2, 2, 64, 16, BF, seed=4, shared=640)
    cache.lens.copy_(i32([900, 300, 1]))
    check(q, cache, True, shared_len=640, shared_table=i32(prefix))
    cache.lens.copy_(i32([0, 0, 0]))
    check(q, cache, True, shared_len=640, shared_table=i32(prefix))


# query heads over 2 K/V heads: 2, 16, 40 and 150 rows take different kernels
HEADS = [4, 32, 80, 300]


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale, H):
    q, cache, _ = build([333, 40], H, 2, 1, 64, 16, BF, seed=8)
    check(q, cache, scale=scale, out_f32=True)


@pytest.mark.parametrize("H", HEADS)
def test_scale_zero_with_large_products(H):
    """Products of 1e30 times a scale of 0 are 0: every kept row weighs the same, and
    LSE is the logarithm of their number."""
    q, cache, prefix = build([333, 200], H, 2, 1, 64, 16, BF, seed=24, std=1e18, shared=128)
    q = q * 1e12
    check(q, cache, scale=0.0, out_f32=True)
    check(q, cache, scale=0.0, out_f32=True, shared_len=128, shared_table=i32(prefix))


@pytest.mark.parametrize("H", HEADS)
def test_large_logits_move_the_maximum(H):
    q, cache, _ = build([2000], H, 2, 1, 128, 16, BF, seed=9, std=8.0)
    check(q, cache, out_f32=True)


@pytest.mark.parametrize("H", HEADS)
def test_values_that_propagate(H):
    """A kept NaN row reaches the sequence that keeps it and no other."""
    q, cache, _ = build([300, 300, 300], H, 2, 1, 64, 16, BF, seed=10)
    o0, l0 = A.decode_paged(q.cuda(), cache)
    cache.k[cache.table[1, 3], 0, 5] = float("nan")
    o, l = A.decode_paged(q.cuda(), cache)
    assert o[1, :H // 2].isnan().all() and l[1, :H // 2].isnan().all()
    keep = torch.ones_like(l, dtype=torch.bool)
    keep[1, :H // 2] = False
    assert torch.equal(o[keep], o0[keep]) and torch.equal(l[keep], l0[keep])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shared", [0, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H", HEADS)
def test_rows_that_keep_nothing_are_zero_beside_values_that_are_not_finite(H, bad, shared, d):
    """An empty slot, and a row before position 0 whose neighbour keeps the bad V row,
    are 0 and minus infinity exactly; with a shared prefix the bad row is every sequence's."""
    q, cache, prefix = build([300, 200, 300], H, 2, 2, d, 16, BF, seed=23, shared=shared)
    cache.lens.copy_(i32([300, 0, 1]))
    kw = dict(shared_len=shared, shared_table=i32(prefix)) if shared else {}
    cache.v[cache.table[2, 0], :, 0] = bad
    for f32 in (False, True):
        o, l = A.decode_paged(q.cuda(), cache, out_f32=f32, **kw)
        torch.cuda.synchronize()
        assert A.get_status() == 0
        assert (o[1] == 0).all() and l[1].isneginf().all()
        assert (o[2, :, 0] == 0).all() and l[2, :, 0].isneginf().all()
        assert not o[2, :, 1].isfinite().any() and l[2, :, 1].isfinite().all()
        assert o[0].isfinite().all() == (shared == 0) and l[0].isfinite().all()


@pytest.mark.parametrize("H", HEADS)
def test_pages_that_do_not_exist_are_not_read(H):
    """Bad entries read as rows of zeros and are reported; the others are right."""
    q, cache, _ = build([300, 300, 40], H, 2, 1, 64, 16, BF, seed=11)
    o0, l0 = A.decode_paged(q.cuda(), cache)
    for bad in (-1, -2 ** 31, 2 ** 31 - 1, cache.k.shape[0]):
        cache.table[1, 2] = bad
        o, l = A.decode_paged(q.cuda(), cache)
        torch.cuda.synchronize()
        assert A.get_status() == A.ATTN_ERR_INVALID_ARG
        assert torch.equal(o[0], o0[0]) and torch.equal(o[2], o0[2]) and o[1].isfinite().all()


def test_lengths_that_do_not_fit_are_clamped():
    q, cache, _ = build([64, 64, 64], 4, 2, 1, 64, 16, BF, seed=12)
    o0, l0 = A.decode_paged(q.cuda(), cache)
    cache.lens.copy_(i32([2 ** 31 - 1, -5, 64]))
    o, l = A.decode_paged(q.cuda(), cache)
    torch.cuda.synchronize()
    assert A.get_status() == A.ATTN_ERR_INVALID_ARG
    assert torch.equal(o[0], o0[0]) and torch.equal(o[2], o0[2])
    assert (o[1] == 0).all() and l[1].isneginf().all()


@pytest.mark.parametrize("H", HEADS)
def test_rows_of_the_table_behind_a_window_are_not_read(H):
    """What lies left of every row's window and behind the sinks may be gone: the rows
    hold NaN, the pages are no longer in the table."""
    q, cache, _ = build([900, 700], H, 2, 2, 64, 16, BF, seed=13)
    a = A.decode_paged(q.cuda(), cache, window=200, n_sink=3)
    for b, n in enumerate([900, 700]):
        first = n - 2 - 200 + 1
        for j in range(3, first):
            cache.k[cache.table[b, j // 16], :, j % 16] = float("nan")
            cache.v[cache.table[b, j // 16], :, j % 16] = float("nan")
        cache.table[b, 1:first // 16] = -1
    cache.table[:, 60:] = 2 ** 30
    o, l = A.decode_paged(q.cuda(), cache, window=200, n_sink=3)
    torch.cuda.synchronize()
    assert A.get_status() == 0
    assert torch.equal(o, a[0]) and torch.equal(l, a[1])


def wide(cache, cols, n_pages):
    """The same sequences in a wide table and a large pool, whose further pages hold NaN."""
    big = [torch.full((n_pages, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda") for x in (cache.k, cache.v)]
    for x, y in zip(big, (cache.k, cache.v)):
        x[:y.shape[0]] = y
    table = torch.full((cache.lens.shape[0], cols), -1, dtype=torch.int32, device="cuda")
    table[:, :cache.table.shape[1]] = cache.table
    return A.PagedCache(*big, table, cache.lens)


# lens, H, H_kv, N_q, page, dtype, causal, window, n_sink, shared
WIDE = [
    ([3000, 0, 129, 1], 40, 2, 1, 16, BF, 1, 0, 0, 0),              # 20 rows
    ([3000, 0, 129, 3], 16, 4, 8, 64, FP, 1, 0, 0, 0),              # 32 rows, some before position 0
    ([2000, 300] * 3, 17, 1, 1, 256, BF, 0, 0, 0, 0),
    ([2000, 0, 300], 64, 2, 1, 16, FP, 1, 100000, 5, 0),            # a window that would see enough
    ([2000, 0, 300], 64, 2, 1, 16, FP, 1, 200, 5, 0),               # and one that does not
    ([900, 640, 0, 700], 64, 2, 1, 16, BF, 1, 0, 0, 640),
    ([5, 8], 32, 1, 1, 32, BF, 1, 0, 0, 0),
]


@pytest.mark.parametrize("cols", [16384, 64])
@pytest.mark.parametrize("case", WIDE, ids=[f"n{max(c[0])}H{c[1]}k{c[2]}q{c[3]}p{c[4]}w{c[7]}s{c[9]}" for c in WIDE])
def test_17_to_32_rows_in_wide_tables(case, cols):
    """At d = 64 these take one kernel or the other, by what the table and the pages may
    hold; a workspace of the bytes asked for, filled before, serves both."""
    lens, H, Hk, N_q, page, dt, causal, window, n_sink, shared = case
    q, cache, prefix = build(lens, H, Hk, N_q, 64, page, dt, seed=26 + H, shared=shared)
    kw = dict(shared_len=shared, shared_table=i32(prefix)) if shared else {}
    big = wide(cache, max(cols * 16 // page, cache.table.shape[1]), (140 << 20) // (4 * 64 * Hk * page))
    need = A.decode_paged_workspace_bytes(len(lens), H, Hk, N_q, 64, shared)
    got = []
    for _ in range(2):
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        A.get_status()
        got.append(A.decode_paged(q.cuda(), big, causal=bool(causal), window=window, n_sink=n_sink, workspace=ws, **kw))
        torch.cuda.synchronize()
        assert A.get_status() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    check(q, cache, bool(causal), window, n_sink, got=got[0])


@pytest.mark.parametrize("shared", [65520, 65536, 65700])
def test_prefix_of_17_to_32_rows_beyond_l2(shared):
    """A prefix of 128 MB (the pages it lists repeat, so few hold it) goes to one kernel,
    a shorter one to the other.  Against float64 sums on the GPU; the bounds are the
    oracle's, with |v_j - O| taken as |v_j| + |O| and the largest logit error for all."""
    B, H, Hk, d, page = 2, 80, 8, 64, 16                          # 10 rows a sequence
    rng = np.random.default_rng(27)
    k, v = (torch.from_numpy(rng.standard_normal((40, Hk, page, d)).astype(np.float32)).to(BF).cuda() for _ in range(2))
    pages = -(-shared // page)
    lens = [shared + 5, shared]
    table = i32(np.stack([rng.permutation(np.resize(np.arange(40), pages + 1)) for _ in range(2)]))
    table[1, :pages] = table[0, :pages]
    cache = A.PagedCache(k, v, table, i32(lens))
    q = torch.from_numpy(rng.standard_normal((B, H, 1, d)).astype(np.float32)).to(BF).cuda()
    A.get_status()
    o, l = A.decode_paged(q, cache, shared_len=shared, shared_table=table[0, :pages].contiguous(), out_f32=True)
    torch.cuda.synchronize()
    assert A.get_status() == 0
    scale, f, u = A.default_scale(d), 2.0 ** -24, U[BF]
    for b, n in enumerate(lens):
        for g in range(Hk):
            kk, vv = (x[table[b].long(), g].reshape(-1, d)[:n].double() for x in (k, v))
            x = q[b, 10 * g:10 * g + 10, 0].double()
            s = scale * (x @ kk.T)
            L = torch.logsumexp(s, 1, keepdim=True)
            w = torch.exp(s - L)
            O, mass = w @ vv, w @ vv.abs()
            e = (d + 4) * f * scale * float((x.abs() @ kk.abs().T).max()) + 4 * f * float(s.abs().max()) + 4 * f
            sums = (n + 16) * f
            rel = (u + e) / (1 - u - e) + sums
            assert ((o[b, 10 * g:10 * g + 10, 0] - O).abs() <= rel * (mass + O.abs())).all()
            bound = e + sums + 4 * f * (float(s.abs().max()) + float(L.abs().max()) + 1)
            assert ((l[b, 10 * g:10 * g + 10] - L).abs() <= bound).all()


def test_many_sequences():
    """More sequences than the kernel has threads in a CTA, most of them empty or short."""
    rng = np.random.default_rng(14)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    lens[650] = 600
    q, cache, _ = build(lens, 2, 1, 1, 64, 16, BF, seed=14)
    check(q, cache)


def test_equal_inputs_give_equal_bits_and_buffers_are_used():
    q, cache, _ = build([3000, 100, 0], 8, 2, 2, 128, 16, BF, seed=15)
    need = A.decode_paged_workspace_bytes(3, 8, 2, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q, device="cuda")
    lse = torch.empty(3, 8, 2, device="cuda")
    a = A.decode_paged(q.cuda(), cache, out=out, lse=lse, workspace=ws)
    assert a[0] is out and a[1] is lse
    b = A.decode_paged(q.cuda(), cache)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = A.decode_paged(q.cuda(), cache, return_lse=False)
    assert c[1] is None and torch.equal(c[0], b[0])


@pytest.mark.parametrize("H", HEADS)
def test_withheld_loads_end_in_a_status(H):
    q, cache, _ = build([3000, 100, 0], H, 2, 1, 128, 16, BF, seed=16)
    want = A.decode_paged(q.cuda(), cache)
    before = A.set_watchdog_ns(50_000_000)
    try:
        A.test_withhold_loads(1)
        A.decode_paged(q.cuda(), cache)
        torch.cuda.synchronize()
        assert A.get_status() == A.ATTN_ERR_DEVICE_TIMEOUT
    finally:
        A.test_withhold_loads(0)
        A.set_watchdog_ns(before)
    got = A.decode_paged(q.cuda(), cache)
    torch.cuda.synchronize()
    assert A.get_status() == 0 and torch.equal(got[0], want[0])


def test_withheld_loads_of_a_shared_prefix():
    """Both launches side by side give up, one after the other, and the next call works."""
    q, cache, prefix = build([900] * 9, 16, 2, 1, 64, 16, BF, seed=21, shared=640)
    kw = dict(shared_len=640, shared_table=i32(prefix))
    want = A.decode_paged(q.cuda(), cache, **kw)
    before = A.set_watchdog_ns(50_000_000)
    try:
        A.test_withhold_loads(1)
        A.decode_paged(q.cuda(), cache, **kw)
        torch.cuda.synchronize()
        assert A.get_status() == A.ATTN_ERR_DEVICE_TIMEOUT
    finally:
        A.test_withhold_loads(0)
        A.set_watchdog_ns(before)
    got = A.decode_paged(q.cuda(), cache, **kw)
    torch.cuda.synchronize()
    assert A.get_status() == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_shared_prefix_calls_back_to_back():
    """Steps whose launches overlap (append, prefix, own positions, merge) for many steps
    in one captured graph equal the same steps one at a time."""
    rng = np.random.default_rng(22)
    B, H, Hk, d = 12, 32, 2, 64

    def rows(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(BF).cuda()

    cache = A.paged_cache(B, 30, 500, Hk, 16, d, BF)
    A.pages_append(cache, rows(B, Hk, 300, d), rows(B, Hk, 300, d), i32([300] + [0] * (B - 1)))
    A.pages_fork(cache, i32([0] * (B - 1)), i32(range(1, B)))
    table = cache.table[0, :16].clone()
    steps = [(rows(B, Hk, 1, d), rows(B, Hk, 1, d), rows(B, H, 1, d)) for _ in range(20)]
    lens0, table0, refs0 = cache.lens.clone(), cache.table.clone(), cache.refs.clone()
    pages0 = cache.k.clone(), cache.v.clone()

    def run(sync):
        outs = []
        for kn, vn, q in steps:
            A.pages_append(cache, kn, vn)
            outs.append(A.decode_paged(q, cache, shared_len=256, shared_table=table))
            if sync:
                torch.cuda.synchronize()
        return outs

    def reset():
        for x, y in ((cache.lens, lens0), (cache.table, table0), (cache.refs, refs0), (cache.k, pages0[0]),
                     (cache.v, pages0[1])):
            x.copy_(y)
        torch.cuda.synchronize()

    A.get_status()
    want = [(o.clone(), l.clone()) for o, l in run(True)]
    reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(False)
    for _ in range(3):
        reset()
        g.replay()
        torch.cuda.synchronize()
        assert A.get_status() == 0
        for (o, l), (o1, l1) in zip(want, got):
            assert torch.equal(o, o1) and torch.equal(l, l1)


def test_two_streams_with_their_own_workspaces():
    q, cache, _ = build([3000, 2000], 8, 2, 1, 128, 16, BF, seed=17)
    q = q.cuda()
    want = A.decode_paged(q, cache)
    torch.cuda.synchronize()
    need = A.decode_paged_workspace_bytes(2, 8, 2, 1, 128)
    lanes = []
    for _ in range(2):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        lanes.append((torch.cuda.Stream(), torch.empty_like(q), torch.empty(2, 8, 1, device="cuda"), ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, l, ws in lanes:
            with torch.cuda.stream(s):
                A.decode_paged(q, cache, out=o, lse=l, workspace=ws)
    torch.cuda.synchronize()
    for _, o, l, _ in lanes:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_serving_run():
    """Prompts appended, a beam forked, steps with the shared prefix, beams dropped,
    the cache compacted: every step's attention is the oracle's over what was appended."""
    rng = np.random.default_rng(18)
    B, H, Hk, d, page = 6, 8, 2, 64, 16
    cache = A.paged_cache(B, 30, 90, Hk, page, d, BF)
    A.get_status()

    def rows(n):
        return torch.from_numpy(rng.standard_normal((B, Hk, n, d)).astype(np.float32)).to(BF)

    def step(counts, **kw):
        kn, vn = rows(1), rows(1)
        A.pages_append(cache, kn.cuda(), vn.cuda(), i32(counts))
        q = torch.from_numpy(rng.standard_normal((B, H, 1, d)).astype(np.float32)).to(BF)
        return q, check(q, cache, **kw)

    A.pages_append(cache, rows(333).cuda(), rows(333).cuda(), i32([333, 40, 0, 0, 0, 0]))
    step([1, 1, 0, 0, 0, 0])
    A.pages_fork(cache, i32([0, 0, 0]), i32([2, 3, 4]))
    step([1, 0, 1, 1, 1, 0])
    A.pages_trim(cache, None, i32([1]))
    shared = dict(shared_len=320, shared_table=cache.table[0, :20].clone())
    for _ in range(20):
        step([1, 0, 1, 1, 1, 0], **shared)
    A.pages_trim(cache, i32([0, 340]), i32([3, 0]))
    A.pages_fork(cache, i32([2]), i32([5]))
    q, before = step([0, 0, 1, 0, 1, 1])
    live = A.pages_compact(cache)
    torch.cuda.synchronize()
    assert int(live) == int((cache.refs > 0).sum()) and int(cache.table.max()) < int(live)
    after = A.decode_paged(q.cuda(), cache)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    A.pages_trim(cache)
    torch.cuda.synchronize()
    assert A.get_status() == 0 and int(cache.refs.abs().sum()) == 0 and int(cache.lens.sum()) == 0


def test_captured_decoding_loop():
    """Append and decode captured once; the lengths grow on the device at each replay."""
    rng = np.random.default_rng(19)
    B, H, Hk, d = 3, 4, 2, 128

    def rows(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(BF).cuda()

    cache = A.paged_cache(B, 20, 70, Hk, 16, d, BF)
    A.pages_append(cache, rows(B, Hk, 140, d), rows(B, Hk, 140, d), i32([140, 1, 0]))
    kn, vn, q = rows(B, Hk, 1, d), rows(B, Hk, 1, d), rows(B, H, 1, d)
    out, lse = torch.empty_like(q), torch.empty(B, H, 1, device="cuda")
    ws = torch.empty(A.decode_paged_workspace_bytes(B, H, Hk, 1, d), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(4096, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        A.decode_paged(q, cache, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.pages_append(cache, kn, vn, workspace=ws2)
        A.decode_paged(q, cache, out=out, lse=lse, workspace=ws)
    A.get_status()
    for n in range(3):
        for x in (kn, vn, q):
            x.copy_(rows(*x.shape))
        g.replay()
        torch.cuda.synchronize()
        assert A.get_status() == 0 and cache.lens.tolist() == [141 + n, 2 + n, 1 + n]
        check(q.cpu(), cache, got=(out, lse))


@pytest.mark.parametrize("H", [80, 300])
def test_more_sequences_than_threads_in_the_kernel_of_many_rows(H):
    """40 and 150 rows of each of 2 K/V heads over 1000 sequences: runs begin in every
    384 of them, behind empty ones, and long sequences lie in the last."""
    rng = np.random.default_rng(28)
    lens = [int(x) for x in rng.integers(0, 20, 1000)]
    for b in (0, 383, 384, 767, 768, 999):
        lens[b] = int(rng.integers(200, 600))
    lens[390:700] = [0] * 310
    q, cache, _ = build(lens, H, 2, 1, 64, 16, BF, seed=28)
    o, l = A.decode_paged(q.cuda(), cache)
    few = [0, 1, 383, 384, 385, 389, 390, 699, 700, 766, 767, 768, 769, 998, 999]
    part = A.PagedCache(cache.k, cache.v, cache.table[few].contiguous(), cache.lens[few].contiguous())
    torch.cuda.synchronize()
    assert A.get_status() == 0
    check(q[few], part, got=(o[few], l[few]))
    # the others against calls of at most 250 sequences: each side is off by at most
    # 2^-8 (sum w |v - O| + |O|), where |v| <= 6 and so |v - O| <= 12, and an LSE by 1.3e-4
    # (|q| |k| <= 144, 620 positions); 2.1 is both sides with what is of second order
    for b in range(0, 1000, 250):
        part = A.PagedCache(cache.k, cache.v, cache.table[b:b + 250].contiguous(), cache.lens[b:b + 250].contiguous())
        O, L = A.decode_paged(q[b:b + 250].cuda(), part)
        empty = part.lens == 0
        assert (o[b:b + 250][empty] == 0).all() and l[b:b + 250][empty].isneginf().all()
        away = (o[b:b + 250].float() - O.float()).abs()
        assert (away <= 2.1 * 2.0 ** -8 * (12 + O.float().abs())).all()
        assert ((l[b:b + 250][~empty] - L[~empty]).abs() <= 2.1 * 1.3e-4).all()
