"""Refusals of the paged cache's entry points, before any device work: the
binding's checks on CPU tensors, and the C ABI's on addresses that are never
dereferenced."""
import ctypes

import pytest
import torch

import exact_tiled_attention_44_b200 as A

BF = torch.bfloat16
INV, UNS, MIS = A.ATTN_ERR_INVALID_ARG, A.ATTN_ERR_UNSUPPORTED, A.ATTN_ERR_MISALIGNED


def cpu_cache(B=3, cols=4, n=8, Hk=2, page=16, d=64, dt=BF, refs=True):
    c = A.paged_cache(B, cols, n, Hk, page, d, dt, "cpu")
    return c if refs else A.PagedCache(c.k, c.v, c.table, c.lens)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_cache_tensors_are_checked():
    c = cpu_cache()
    assert (c.table == -1).all() and (c.lens == 0).all() and (c.refs == 0).all()
    with pytest.raises(ValueError, match="n_pages"):
        A.PagedCache(c.k, c.v[:4], c.table, c.lens, c.refs)
    with pytest.raises(TypeError, match="dtype"):
        A.PagedCache(c.k, c.v.half(), c.table, c.lens, c.refs)
    with pytest.raises(TypeError):
        A.PagedCache(c.k.float(), c.v.float(), c.table, c.lens, c.refs)
    with pytest.raises(ValueError, match="table must be"):
        A.PagedCache(c.k, c.v, c.table.long(), c.lens, c.refs)
    with pytest.raises(ValueError, match="table must be"):
        A.PagedCache(c.k, c.v, c.table.t(), c.lens, c.refs)
    with pytest.raises(ValueError, match="lens must be"):
        A.PagedCache(c.k, c.v, c.table, ints(0, 0), c.refs)
    with pytest.raises(ValueError, match="refs must be"):
        A.PagedCache(c.k, c.v, c.table, c.lens, ints(0))
    with pytest.raises(ValueError, match="k must be"):
        A.PagedCache(c.k.transpose(2, 3), c.v.transpose(2, 3), c.table, c.lens, c.refs)
    with pytest.raises(AttributeError):
        c.table = c.table


def test_decode_paged_arguments_are_checked():
    c = cpu_cache()
    q = torch.zeros(3, 4, 2, 64, dtype=BF)
    for bad, err, what in ((q[:2], ValueError, "mismatch"), (q.half(), TypeError, "dtype"),
                           (q[..., :32], ValueError, "mismatch"), (q[0], ValueError, "expected"),
                           (q.transpose(1, 2), ValueError, "contiguous")):
        with pytest.raises(err, match=what):
            A.decode_paged(bad, c)
    with pytest.raises(ValueError, match="out must be"):
        A.decode_paged(q, c, out=torch.zeros(3, 4, 2, 64, dtype=BF), out_f32=True)
    with pytest.raises(ValueError, match="lse must be"):
        A.decode_paged(q, c, lse=torch.zeros(3, 4))
    with pytest.raises(ValueError, match="shared_table must be"):
        A.decode_paged(q, c, shared_len=17, shared_table=ints(1))
    with pytest.raises(ValueError, match="negative"):
        A.decode_paged(q, c, shared_len=-1, shared_table=ints(1))
    with pytest.raises(ValueError, match="workspace must be"):
        A.decode_paged(q, c, workspace=torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        A.decode_paged(q, c)


def test_management_arguments_are_checked():
    c = cpu_cache()
    kn = torch.zeros(3, 2, 5, 64, dtype=BF)
    with pytest.raises(ValueError, match="k_new must be"):
        A.pages_append(c, kn[:, :1], kn)
    with pytest.raises(ValueError, match="k_new must be"):
        A.pages_append(c, kn.transpose(1, 2), kn)
    with pytest.raises(ValueError, match="v_new must be"):
        A.pages_append(c, kn, kn[:, :, :4])
    with pytest.raises(ValueError, match="counts"):
        A.pages_append(c, kn, kn, ints(1, 2))
    with pytest.raises(ValueError, match="counts"):
        A.pages_append(c, kn, kn, torch.tensor([1, 2, 3]))
    with pytest.raises(ValueError, match="one length"):
        A.pages_trim(c, ints(1, 2), ints(0))
    with pytest.raises(ValueError, match="for 3 sequences"):
        A.pages_trim(c, ints(1, 2, 3, 4))
    with pytest.raises(ValueError, match="one length"):
        A.pages_fork(c, ints(1, 2), ints(0))
    with pytest.raises(ValueError, match="table_out must be"):
        A.pages_compact(c, table_out=ints(1))
    with pytest.raises(ValueError, match="refs_out must be"):
        A.pages_compact(c, refs_out=ints(1))
    with pytest.raises(ValueError, match="one length"):
        A.pages_copy(c, ints(1, 2), ints(0))
    for call in (lambda x: A.pages_append(x, kn, kn), A.pages_trim, A.pages_compact,
                 lambda x: A.pages_fork(x, ints(1), ints(0)), lambda x: A.pages_copy(x, ints(1), ints(0))):
        with pytest.raises(ValueError, match="CUDA"):
            call(c)
        with pytest.raises(ValueError, match="refs"):
            call(cpu_cache(refs=False))


# ------------------------------------------------------------------ C ABI

M = 1 << 24   # arrays far enough apart for the sizes below
ADDR = dict(k=M, v=2 * M, table=3 * M, lens=4 * M, refs=5 * M)
SIZES = dict(n_pages=8, H_kv=2, page_size=16, d=64, B=3, max_pages=4, dtype=0)


def struct(**kw):
    return A._PagesStruct(**{**ADDR, **SIZES, **kw})


def decode(s=None, q=6 * M, o=7 * M, lse=8 * M, shared=None, n_shared=0, ws=9 * M, ws_bytes=M, H=4,
           N_q=2, causal=1, window=0, n_sink=0, scale=0.125, f32=0):
    s = struct() if s is None else s
    return A.load_library().attn_decode_paged(q, ctypes.addressof(s) if s else None, o, lse, shared,
                                              n_shared, ws, ws_bytes, H, N_q, causal, window, n_sink,
                                              scale, f32, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(s=0), INV), (dict(s=struct(k=None)), INV), (dict(s=struct(lens=None)), INV),
    (dict(s=struct(table=None)), INV), (dict(s=struct(n_pages=0)), INV), (dict(s=struct(n_pages=-1)), INV),
    (dict(s=struct(B=-1)), INV), (dict(s=struct(H_kv=0)), INV), (dict(s=struct(dtype=2)), INV),
    (dict(s=struct(dtype=A.ATTN_OUT_F32)), INV), (dict(s=struct(d=0)), INV), (dict(s=struct(page_size=0)), INV),
    (dict(s=struct(d=48)), UNS), (dict(s=struct(d=32)), UNS), (dict(s=struct(d=16)), UNS),
    (dict(s=struct(page_size=8)), UNS), (dict(s=struct(page_size=48)), UNS), (dict(s=struct(page_size=512)), UNS),
    (dict(s=struct(n_pages=1 << 30)), UNS), (dict(s=struct(max_pages=1 << 27)), UNS),
    (dict(s=struct(k=M + 8)), MIS), (dict(s=struct(table=3 * M + 2)), MIS),
    (dict(H=-1), INV), (dict(H=5), INV), (dict(N_q=-1), INV), (dict(causal=2), INV), (dict(f32=2), INV),
    (dict(window=-1), INV), (dict(n_sink=-1), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(n_shared=-1), INV), (dict(n_shared=16), INV),
    (dict(ws_bytes=-1), INV), (dict(ws_bytes=1000), INV), (dict(ws=None), INV), (dict(q=None), INV),
    (dict(o=None), INV), (dict(causal=0, window=4), UNS), (dict(N_q=513), UNS),
    (dict(q=6 * M + 8), MIS), (dict(lse=8 * M + 4), MIS), (dict(ws=9 * M + 16), MIS),
    (dict(o=6 * M), INV), (dict(o=M), INV), (dict(lse=7 * M), INV), (dict(ws=2 * M), INV),
    (dict(ws=7 * M), INV), (dict(o=3 * M), INV), (dict(lse=4 * M), INV),
    (dict(shared=7 * M, n_shared=16), INV),
])
def test_decode_paged_refusals(kw, expect):
    assert decode(**kw) == expect


@pytest.mark.parametrize("kw", [dict(N_q=0), dict(H=0), dict(s=struct(B=0)),
                                dict(N_q=0, q=None, o=None, lse=None, ws=None)])
def test_decode_paged_empty_problem_is_a_no_op(kw):
    assert decode(**kw) == A.ATTN_OK


def test_workspace_queries():
    need = A.decode_paged_workspace_bytes
    assert need(0, 4, 2, 1, 64) == 0 and need(3, 4, 2, 0, 64) == 0
    assert need(-1, 4, 2, 1, 64) == -1 and need(3, 5, 2, 1, 64) == -1 and need(3, 4, 0, 1, 64) == -1
    assert need(3, 4, 2, 1, 64, -1) == -1
    assert 0 < need(3, 4, 2, 1, 64) < need(3, 4, 2, 1, 128) < 16 << 20
    assert need(3, 4, 2, 1, 64, 127) == need(3, 4, 2, 1, 64) < need(3, 4, 2, 1, 64, 128)
    lib = A.load_library()
    assert lib.attn_pages_append_workspace_bytes(-1, 1, 16) == -1
    assert lib.attn_pages_append_workspace_bytes(4, 100, 16) >= 4 * (6 * 4 + 4 * 8)
    assert lib.attn_pages_compact_workspace_bytes(-1) == -1
    assert lib.attn_pages_compact_workspace_bytes(100) >= 4 * 303


def append(s=None, k=6 * M, v=7 * M, counts=8 * M, n=5, ws=9 * M, ws_bytes=M):
    s = struct() if s is None else s
    return A.load_library().attn_pages_append(ctypes.addressof(s), k, v, counts, n, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(s=struct(refs=None)), INV), (dict(s=struct(refs=3 * M)), INV), (dict(s=struct(v=M + 1024)), INV),
    (dict(n=-1), INV), (dict(k=None), INV), (dict(ws=None), INV), (dict(ws_bytes=8), INV),
    (dict(k=6 * M + 8), MIS), (dict(counts=8 * M + 2), MIS), (dict(ws=9 * M + 4), MIS),
    (dict(k=M), INV), (dict(v=5 * M), INV), (dict(ws=6 * M), INV), (dict(ws=3 * M), INV),
    (dict(counts=4 * M), INV), (dict(counts=9 * M), INV),
])
def test_append_refusals(kw, expect):
    assert append(**kw) == expect


def test_other_management_refusals():
    lib, s = A.load_library(), struct()
    p = ctypes.addressof(s)
    assert append(n=0) == 0 and append(s=struct(B=0)) == 0
    trim, fork, copy = lib.attn_pages_trim, lib.attn_pages_fork, lib.attn_pages_copy
    assert trim(p, None, None, -1, None) == INV and trim(p, None, None, 4, None) == INV
    assert trim(p, 6 * M, 7 * M + 1, 2, None) == MIS and trim(p, 4 * M, None, 2, None) == INV
    assert trim(p, 6 * M, 3 * M, 2, None) == INV and trim(p, None, None, 0, None) == 0
    for f in (fork, copy):
        assert f(p, 6 * M, 7 * M, -1, None) == INV and f(p, None, 7 * M, 2, None) == INV
        assert f(p, 6 * M, 7 * M + 2, 2, None) == MIS and f(p, 6 * M, 3 * M, 2, None) == INV
        assert f(p, 6 * M, 7 * M, 0, None) == 0
    compact = lib.attn_pages_compact
    assert compact(p, None, None, None, None, M, None) == INV
    assert compact(p, None, None, None, 6 * M, 16, None) == INV
    assert compact(p, None, None, None, 6 * M + 4, M, None) == MIS
    assert compact(p, 4 * M, None, None, 6 * M, M, None) == INV
    assert compact(p, 6 * M, None, None, 6 * M, M, None) == INV
    assert compact(p, 7 * M, 7 * M, None, 6 * M, M, None) == INV
    assert compact(p, None, None, 3 * M, 6 * M, M, None) == INV
    bad = struct(refs=None)
    assert compact(ctypes.addressof(bad), None, None, None, 6 * M, M, None) == INV


def test_a_cache_remembers_one_size_of_a_call():
    """A server's prompts and prefixes are of ever new lengths: the handle keeps the
    workspace bytes of the last ones only, and asks again when they change."""
    c = cpu_cache()
    asked = []

    def scratch(call, sizes, need):
        def query():
            asked.append(sizes)
            return need
        return A._scratch(None, c, call, sizes, query).numel()

    for n in range(100, 200):
        assert scratch("append", n, n) == n and scratch("append", n, n) == n
        assert scratch("decode", (4, 1, n), 2 * n) == 2 * n and scratch("decode", (4, 1, n), 0) == 2 * n
    assert asked == [x for n in range(100, 200) for x in (n, (4, 1, n))]
    assert set(c._need) == {"append", "decode"}
    assert scratch("decode", (4, 0, 0), 0) == 16 and scratch("decode", (4, -1, 0), -1) == 16
    own = torch.zeros(7, dtype=torch.uint8)
    assert A._scratch(own, c, "append", 1, None) is own


@pytest.mark.parametrize("name", ["window", "n_sink", "shared_len"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63, -2 ** 31, -2 ** 32 + 5])
def test_sizes_beyond_32_bits_are_refused(name, value):
    """ctypes keeps the lowest 32 bits of an int: 2^32 + 5 would be a window of 5."""
    with pytest.raises(ValueError, match="32 bits"):
        A.decode_paged(torch.zeros(3, 4, 2, 64, dtype=BF), cpu_cache(), **{name: value})
    with pytest.raises(ValueError, match="CUDA"):
        A.decode_paged(torch.zeros(3, 4, 2, 64, dtype=BF), cpu_cache(), **{name: 2 ** 31 - 1})


def test_workspace_queries_refuse_what_the_calls_refuse():
    need = A.decode_paged_workspace_bytes
    for bad in ((3, 4, 2, 513, 64), (3, 4, 2, 1, 32), (3, 4, 2, 1, 100), (2 ** 30, 4, 2, 1, 64),
                (2 ** 31 - 1, 2 ** 31 - 1, 1, 2 ** 31 - 1, 128)):
        assert need(*bad) == -1 and need(*bad, 128) == -1
    assert need(3, 4, 2, 512, 64) > 0
    most = (2 ** 31 - 1) // 2 // 8
    assert need(most, 8, 8, 1, 64) > 0 and need(most + 1, 8, 8, 1, 64) == -1
    pages = A.load_library().attn_pages_append_workspace_bytes
    for bad in ((4, 100, 8), (4, 100, 48), (4, 100, 0), (4, 100, 512), (2 ** 31 - 1, 2 ** 31 - 1, 16),
                (2 ** 31 - 1, 1, 256)):
        assert pages(*bad) == -1
    assert pages(1, 2 ** 31 - 1, 16) >= 4 * (2 ** 31 // 16) and pages(0, 5, 16) == 0
    # the call itself: refused for its size, however large the workspace
    big = struct(B=2 ** 24, max_pages=1, table=1 << 37, lens=1 << 38, refs=1 << 39)
    assert A.load_library().attn_pages_append(ctypes.addressof(big), 1 << 40, 1 << 41, None, 2 ** 15, 1 << 42,
                                              1 << 40, None) == UNS


def test_decode_workspace_of_the_longest_prefix():
    """The largest prefix and the most K/V heads that the sizes allow: no overflow on the way."""
    need, last = A.decode_paged_workspace_bytes, 2 ** 31 - 1
    assert need(1, 2 ** 26, 2 ** 26, 1, 64, last) >= 2 * (2 ** 26) * 8 * 64 * 4
    assert need(3, 64, 8, 1, 64, last) > need(3, 64, 8, 1, 64, 128) > need(3, 64, 8, 1, 64)
