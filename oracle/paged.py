"""Float64 oracle of a decoding step over a K/V cache of pages, and a
sequential model of the page management.

TEST INFRASTRUCTURE ONLY (see ``oracle/definition.py``).

* "USAAIO Lesson 91", slide 31 ("MHA KV cache is the inference bottleneck"):
  every decoding step re-reads the whole cache; slide 32: with MQA / GQA the
  query heads share K/V heads.

Readings taken (the pages know no paged cache):

* position j of sequence b is row j % page_size of page table[b][j // page_size];
* the N_q new query rows of sequence b sit at positions lens[b] - N_q + i and keep key
  j iff j < lens[b] and the forward's mask rule holds; a row that keeps nothing
  has O = 0 and LSE = -inf;
* a shared prefix changes what is read and not what is computed, so it has
  no oracle of its own.
"""
from __future__ import annotations

import numpy as np

from .definition import kv_head_of


def gather(pages, row, n):
    """The first n rows [n, H_kv, d] of the sequence whose table row is `row`."""
    page = pages.shape[2]
    out = np.empty((n, pages.shape[1], pages.shape[3]), pages.dtype)
    for j in range(n):
        out[j] = pages[row[j // page], :, j % page]
    return out


def kept(n, n_q, i, causal, window, n_sink):
    """Positions 0..n-1 that query row i of n_q keeps, as a boolean array."""
    j = np.arange(n)
    pos = n - n_q + i
    keep = np.ones(n, bool)
    if causal:
        keep &= j <= pos
    if window > 0:
        keep &= (pos - j < window) | (j < n_sink)
    return keep


def decode_paged(Q, K, V, table, lens, scale, causal=True, window=0, n_sink=0, u=0.0, u_out=0.0,
                 step=0.0):
    """O [B, H, N_q, d], LSE [B, H, N_q] and bounds of both errors for a kernel
    that rounds its weights by a relative `u` (or, below the normal range, by an absolute
    `step` of the largest), its output by `u_out`, and sums in float32:

    * a logit is off by e = (d + 4) 2^-24 scale sum_k |q_k k_k| (d rounded
      products and sums, and the scaling), the exponent's argument by 2 units in
      its last place, the exponential by 2^-22;
    * weights off by (1 + x_j) move O by at most sum_j w_j |x_j| |v_j - O| / (1 - max x);
    * the sums of n weights and products are off by at most (n + 16) 2^-24 of
      the sum of the absolute terms (16: the merging of partial results).
    """
    B, H, n_q, d = Q.shape
    O = np.zeros((B, H, n_q, d))
    L = np.full((B, H, n_q), -np.inf)
    tO = np.zeros((B, H, n_q, d))
    tL = np.zeros((B, H, n_q))
    f = 2.0 ** -24
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        k, v = gather(K, table[b], n), gather(V, table[b], n)
        for h in range(H):
            g = kv_head_of(h, H, K.shape[1])
            for i in range(n_q):
                on = kept(n, n_q, i, causal, window, n_sink)
                if not on.any():
                    continue
                kk, vv, q = k[on, g], v[on, g], Q[b, h, i]
                s = scale * (kk @ q)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                w = p / l
                o = w @ vv
                O[b, h, i] = o
                L[b, h, i] = m + np.log(l)
                e = (d + 4) * f * abs(scale) * (np.abs(kk) @ np.abs(q)) + 4 * f * np.abs(s).max() + 4 * f
                e = np.expm1(np.minimum(e, 1.0))
                sums = (on.sum() + 16) * f
                away = np.abs(vv - o)
                x = u + e
                tO[b, h, i] = ((w * x) @ away + step / l * away.sum(0)) / (1 - min(0.5, x.max())) \
                    + sums * (w @ np.abs(vv) + np.abs(o))
                tO[b, h, i] += u_out * (np.abs(o) + tO[b, h, i]) + 1e-30
                tL[b, h, i] = (w @ e) + sums + 4 * f * (abs(m) + abs(L[b, h, i]) + 1)
    return O, L, tO, tL


class PageBook:
    """The page management, one sequence and one page at a time, on numpy arrays:
    k, v [n_pages, H_kv, page_size, d], table [B, max_pages], lens [B], refs
    [n_pages].  Each method returns the status it would leave (0, -1: something in the
    device arrays was out of range, -6: too few free pages)."""

    def __init__(self, k, v, table, lens, refs):
        self.k, self.v, self.table, self.lens, self.refs = (np.array(x) for x in (k, v, table, lens, refs))
        self.page = self.k.shape[2]

    def pages_of(self, n):
        return -(-n // self.page)

    def append(self, k_new, v_new, counts=None):
        B, n_new = k_new.shape[0], k_new.shape[2]
        refs0, status, out_of_pages = self.refs.copy(), 0, False
        free = [int(p) for p in np.flatnonzero(refs0 <= 0)]
        cap = self.table.shape[1] * self.page
        for b in range(B):
            c = n_new if counts is None else int(counts[b])
            start = int(self.lens[b])
            if c < 0 or c > n_new or start < 0 or start + c > cap:
                status = -1
                continue
            if c == 0:
                continue
            part, col = start % self.page, start // self.page
            old = int(self.table[b, col]) if part else -1
            if part and (not 0 <= old < len(self.refs) or refs0[old] < 1):
                status = -1
                continue
            copy = part > 0 and refs0[old] > 1
            need = self.pages_of(start + c) - self.pages_of(start) + int(copy)
            if need and (out_of_pages or need > len(free)):
                out_of_pages = True
                status = status or -6
                continue
            got, free = free[:need], free[need:]
            for p in got:
                self.refs[p] = 1
            if copy:
                new = got.pop(0)
                self.k[new, :, :part] = self.k[old, :, :part]
                self.v[new, :, :part] = self.v[old, :, :part]
                self.refs[old] -= 1
                self.table[b, col] = new
            for i, p in enumerate(got):
                self.table[b, self.pages_of(start) + i] = p
            for i in range(c):
                p, r = self.table[b, (start + i) // self.page], (start + i) % self.page
                self.k[p, :, r] = k_new[b, :, i]
                self.v[p, :, r] = v_new[b, :, i]
            self.lens[b] = start + c
        return status

    def trim(self, new_lens=None, rows=None):
        if rows is None:
            rows = range(len(self.lens) if new_lens is None else len(new_lens))
        status = 0
        for i, b in enumerate(rows):
            n = 0 if new_lens is None else int(new_lens[i])
            if not 0 <= b < len(self.lens) or n < 0:
                status = -1
                continue
            old = int(self.lens[b])
            if not 0 <= old <= self.table.shape[1] * self.page:
                status = -1
                continue
            if n >= old:
                continue
            for c in range(self.pages_of(n), self.pages_of(old)):
                p = int(self.table[b, c])
                self.table[b, c] = -1
                if 0 <= p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1
                else:
                    status = -1
            self.lens[b] = n
        return status

    def fork(self, parents, children):
        status, seen = 0, set()
        lens0 = self.lens.copy()
        for p, c in zip(parents, children):
            p, c = int(p), int(c)
            first = c not in seen
            seen.add(c)
            inside = 0 <= p < len(self.lens) and 0 <= c < len(self.lens)
            if not inside or not first or p in [int(x) for x in children] or lens0[c] != 0:
                status = -1
                continue
            n = self.pages_of(int(self.lens[p]))
            self.table[c] = -1
            self.table[c, :n] = self.table[p, :n]
            for page in self.table[p, :n]:
                self.refs[page] += 1
            self.lens[c] = self.lens[p]
        return status

    def compact(self):
        """Moves the live pages in place; returns their number."""
        n = int((self.refs > 0).sum())
        holes = [p for p in range(n) if self.refs[p] == 0]
        for p in range(n, len(self.refs)):
            if self.refs[p] > 0:
                to = holes.pop(0)
                self.k[to], self.v[to] = self.k[p], self.v[p]
                self.refs[to], self.refs[p] = self.refs[p], 0
                self.table[self.table == p] = to
        return n

    def check(self):
        """The counts are what the table holds."""
        held = np.zeros(len(self.refs), int)
        for b, n in enumerate(self.lens):
            for p in self.table[b, :self.pages_of(int(n))]:
                held[p] += 1
        assert (held == self.refs).all()
