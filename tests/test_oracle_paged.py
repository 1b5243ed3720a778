"""The paged oracle and the model of the page management, on the CPU: against
the dense decode oracle, and against hand-made cases and random runs."""
import numpy as np
import pytest

import oracle


def paged_of(K, V, page, extra, rng):
    """Dense K, V [B, H_kv, N, d] cut into pages in random places; table, pages."""
    B, Hk, N, d = K.shape
    cols = -(-N // page)
    ids = rng.permutation(B * cols + extra)
    kp = np.full((len(ids), Hk, page, d), np.nan)
    vp = kp.copy()
    table = ids[:B * cols].reshape(B, cols)
    for b in range(B):
        for j in range(N):
            kp[table[b, j // page], :, j % page] = K[b, :, j]
            vp[table[b, j // page], :, j % page] = V[b, :, j]
    return kp, vp, table


@pytest.mark.parametrize("causal,window,n_sink", [(True, 0, 0), (False, 0, 0), (True, 9, 3), (True, 1, 0)])
def test_decode_paged_matches_the_dense_oracle(causal, window, n_sink):
    rng = np.random.default_rng(1)
    B, H, Hk, n_q, N, d = 2, 4, 2, 3, 37, 8
    Q, K, V = (rng.standard_normal(s) for s in ((B, H, n_q, d), (B, Hk, N, d), (B, Hk, N, d)))
    kp, vp, table = paged_of(K, V, 16, 2, rng)
    O, L, tO, tL = oracle.decode_paged(Q, kp, vp, table, [N] * B, 0.3, causal, window, n_sink)
    O2, L2 = oracle.decode(Q, K, V, 0.3, causal, window, n_sink)
    assert np.allclose(O, O2, rtol=0, atol=1e-13) and np.allclose(L, L2, rtol=0, atol=1e-13)
    assert (tO > 0).all() and tO.max() < 1e-4


def test_rows_that_keep_nothing():
    rng = np.random.default_rng(2)
    Q = rng.standard_normal((2, 1, 3, 4))
    kp = rng.standard_normal((1, 1, 16, 4))
    O, L, _, _ = oracle.decode_paged(Q, kp, kp, np.array([[0], [-1]]), [2, 0], 1.0)
    assert (O[1] == 0).all() and np.isneginf(L[1]).all()          # an empty sequence
    assert (O[0, 0, 0] == 0).all() and np.isneginf(L[0, 0, 0])    # a row before position 0
    assert np.allclose(O[0, 0, 1], kp[0, 0, 0])                   # the row at position 0 keeps itself


def test_book_by_hand():
    b = oracle.PageBook(np.zeros((6, 1, 4, 1)), np.zeros((6, 1, 4, 1)), -np.ones((3, 3), int),
                        np.zeros(3, int), np.zeros(6, int))
    rows = np.arange(1, 1 + 3 * 6).reshape(3, 1, 6, 1).astype(float)
    assert b.append(rows, -rows, [6, 0, 3]) == 0
    assert b.table.tolist() == [[0, 1, -1], [-1, -1, -1], [2, -1, -1]]
    assert b.fork([0], [1]) == 0 and b.refs.tolist() == [2, 2, 1, 0, 0, 0]
    assert b.append(rows, rows, [0, 1, 0]) == 0                   # copy on write
    assert b.table[1].tolist() == [0, 3, -1] and b.refs.tolist() == [2, 1, 1, 1, 0, 0]
    assert b.k[3, 0, :, 0].tolist() == [5, 6, 7, 0]
    assert b.trim(rows=[0]) == 0 and b.refs.tolist() == [1, 0, 1, 1, 0, 0]
    assert b.compact() == 3
    assert b.table.tolist() == [[-1, -1, -1], [0, 1, -1], [2, -1, -1]]
    assert b.append(rows, rows, [6, 6, 6]) == -1                  # 7 + 6 > 12
    b.check()
    assert b.fork([1, 1], [2, 2]) == -1                           # row 2 is not empty
    assert b.lens.tolist() == [6, 7, 3] and b.refs.tolist() == [1, 1, 1, 1, 1, 0]
    assert b.append(rows, rows, [0, 0, 6]) == -6                  # two pages needed, one free
    assert b.lens.tolist() == [6, 7, 3] and b.append(rows, rows, [0, 0, 5]) == 0
    b.check()


def test_book_random_runs_keep_their_counts():
    rng = np.random.default_rng(3)
    for _ in range(20):
        B, page, cols, n = 6, 4, 5, 17
        b = oracle.PageBook(np.zeros((n, 2, page, 3)), np.zeros((n, 2, page, 3)), -np.ones((B, cols), int),
                            np.zeros(B, int), np.zeros(n, int))
        for _ in range(12):
            what = rng.integers(4)
            if what == 0:
                x = rng.standard_normal((B, 2, 7, 3))
                b.append(x, x, rng.integers(0, 8, B))
            elif what == 1:
                b.trim(rng.integers(0, 20, 2), rng.integers(0, B, 2))
            elif what == 2:
                b.fork(rng.integers(0, B, 2), rng.integers(0, B, 2))
            else:
                b.compact()
            b.check()
            assert (b.refs >= 0).all()


def test_book_trim_leaves_lengths_that_cannot_be_right():
    b = oracle.PageBook(np.zeros((6, 1, 4, 1)), np.zeros((6, 1, 4, 1)), -np.ones((2, 3), int),
                        np.zeros(2, int), np.zeros(6, int))
    rows = np.ones((2, 1, 12, 1))
    assert b.append(rows, rows, [12, 5]) == 0
    table, refs = b.table.copy(), b.refs.copy()
    for bad in (13, 2 ** 31 - 1, -1):
        b.lens[0] = bad
        assert b.trim([0, 4], [0, 0]) == -1 and b.lens[0] == bad
        assert (b.table == table).all() and (b.refs == refs).all()
