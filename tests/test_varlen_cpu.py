"""Packed sequences and the paged cache, host side (no GPU): every refusal of the C ABI comes
before any launch, the torch helpers reject what the library would misread, and the
cache's books (pages, shares, forks, compaction) hold against a model that keeps every
sequence's tokens in a plain list."""
import random

import pytest
import torch

import causal_flash_attention_attn_b200 as fa

A = 0x10000  # an aligned fake device address: never dereferenced
BF, F32 = fa.FORGE_DTYPE_BF16, fa.FORGE_DTYPE_F32
INVALID, UNSUPPORTED, WORKSPACE = fa.FORGE_ERR_INVALID_ARG, fa.FORGE_ERR_UNSUPPORTED, fa.FORGE_ERR_WORKSPACE


# ------------------------------------------------------------------ C ABI
def varlen(backward, **kw):
    a = dict(q=A, k=A, v=A, o=A, res=None, lse=A, dO=A, dq=A, dk=A, dv=A, cu=A, n=3, rows=500, Hq=4, Hkv=2, D=128, qs=None,
             ks=None, vs=None, scale=0.1, window=0, softcap=0.0, sink=None, dsink=None, dtype=BF, ws=A, nbytes=None)
    a.update(kw)
    H, K, D = a["Hq"], a["Hkv"], a["D"]
    qs, ks, vs = a["qs"] or H * D, a["ks"] or K * D, a["vs"] or K * D
    size = fa.forge_attn_varlen_bwd_workspace_size if backward else fa.forge_attn_varlen_fwd_workspace_size
    nbytes = size(3, 500, 4, 2, 128, BF) if a["nbytes"] is None else a["nbytes"]
    if backward:
        return fa.forge_attn_varlen_bwd(a["q"], a["k"], a["v"], a["o"], a["res"], a["lse"], a["dO"], a["dq"], a["dk"],
                                        a["dv"], a["cu"], a["n"], a["rows"], H, K, D, qs, ks, vs, a["scale"], a["window"],
                                        a["softcap"], a["sink"], a["dsink"], 1, a["dtype"], a["ws"], nbytes, 0)
    return fa.forge_attn_varlen_fwd(a["q"], a["k"], a["v"], a["o"], a["res"], a["lse"], a["cu"], a["n"], a["rows"], H, K, D, qs,
                                    ks, vs, a["scale"], a["window"], a["softcap"], a["sink"], 1, a["dtype"], a["ws"],
                                    nbytes, 0)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(Hkv=3), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=63), INVALID), (dict(rows=0), INVALID),
    (dict(n=0), INVALID), (dict(n=(1 << 20) + 1), INVALID), (dict(rows=(1 << 30) + 1), INVALID),
    (dict(Hq=1 << 14, Hkv=1 << 14, rows=1 << 24), INVALID),        # grid
    (dict(window=-1), INVALID), (dict(scale=0.0), INVALID), (dict(softcap=float("nan")), INVALID),
    (dict(q=0), INVALID), (dict(k=A + 8), INVALID), (dict(cu=0), INVALID), (dict(cu=A + 2), INVALID),
    (dict(o=A + 4), INVALID), (dict(lse=A + 4), INVALID), (dict(sink=A + 1), INVALID), (dict(dtype=7), INVALID),
    (dict(res=A + 8), INVALID), (dict(res=A + 16), INVALID),
    (dict(qs=4 * 128 - 8), INVALID),                               # rows would overlap
    (dict(ks=2 * 128 + 4), INVALID),                               # not a multiple of 16 bytes
    (dict(vs=1 << 37), INVALID),
    (dict(ws=0), WORKSPACE), (dict(ws=A + 16), WORKSPACE), (dict(nbytes=511), WORKSPACE),
])
def test_varlen_rejects(backward, kw, code):
    assert varlen(backward, **kw) == code


def test_varlen_bwd_rejects_its_own():
    assert varlen(True, dq=A + 8) == INVALID
    assert varlen(True, dsink=A, sink=None) == INVALID
    assert varlen(True, dsink=A + 2, sink=A) == INVALID


def test_varlen_workspace_sizes():
    f, b = fa.forge_attn_varlen_fwd_workspace_size, fa.forge_attn_varlen_bwd_workspace_size
    assert f(3, 500, 4, 3, 128, BF) == 0 and b(0, 500, 4, 2, 128, BF) == 0
    # a tile per 256 rows and one more per sequence, 32 bytes each
    assert f(3, 500, 4, 2, 128, BF) >= 256 + 32 * (500 // 256 + 3)
    # never more tiles than rows: 64 sequences of one row each
    assert f(1 << 20, 64, 4, 2, 128, BF) <= 256 + 32 * 64 + 256
    # f32 has no accumulator; bf16 pads each sequence to 128 rows
    assert b(3, 500, 4, 2, 128, F32) < 256 + 32 * 11 + 256 + 4 * 4 * 500 + 512
    assert b(3, 500, 4, 2, 128, BF) >= 4 * 4 * 128 * (500 + 3 * 127)


def paged(fn, **kw):
    a = dict(q=A, k=A, v=A, kp=A, vp=A, o=A, lse=A, table=A, lens=A, cu=None, B=2, rows=2, Hq=8, Hkv=2, D=128, P=10,
             ps=64, width=4, ks=None, stride=None, scale=0.1, window=0, softcap=0.0, sink=None, dtype=BF, ws=A,
             nbytes=1 << 30)
    a.update(kw)
    stride = a["stride"] if a["stride"] is not None else a["Hkv"] * a["ps"] * a["D"]
    if fn == "decode":
        return fa.forge_attn_decode_paged(a["q"], a["kp"], a["vp"], a["o"], a["lse"], a["table"], a["lens"], a["B"],
                                          a["Hq"], a["Hkv"], a["D"], a["P"], a["ps"], a["width"], stride, a["scale"],
                                          a["window"], a["softcap"], a["sink"], a["dtype"], a["ws"], a["nbytes"], 0)
    ks = a["ks"] or a["Hkv"] * a["D"]
    return fa.forge_attn_paged_append(a["k"], a["v"], a["kp"], a["vp"], a["table"], a["lens"], a["cu"], a["B"],
                                      a["rows"], a["Hkv"], a["D"], a["P"], a["ps"], a["width"], ks, ks, stride,
                                      a["dtype"], 0)


@pytest.mark.parametrize("fn", ["decode", "append"])
@pytest.mark.parametrize("kw,code", [
    (dict(ps=24), UNSUPPORTED), (dict(ps=0), INVALID), (dict(P=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(B=0, rows=0), INVALID), (dict(width=0), INVALID), (dict(kp=0), INVALID), (dict(vp=A + 8), INVALID),
    (dict(table=0), INVALID), (dict(lens=A + 1), INVALID), (dict(stride=2 * 64 * 128 - 8), INVALID),
    (dict(stride=2 * 64 * 128 + 4), INVALID), (dict(dtype=3), INVALID),
])
def test_paged_calls_reject(fn, kw, code):
    assert paged(fn, **kw) == code


def test_paged_calls_reject_their_own():
    assert paged("decode", Hq=34) == UNSUPPORTED                      # 17 query heads a KV head
    assert paged("decode", Hq=7) == INVALID
    assert paged("decode", q=A + 4) == INVALID
    assert paged("decode", sink=A + 2) == INVALID
    assert paged("decode", width=1 << 25, ps=64) == INVALID           # 2^31 positions
    assert paged("decode", nbytes=16) == WORKSPACE
    assert paged("append", rows=3) == INVALID                         # three tokens, two sequences, no cu_seqlens
    assert paged("append", ks=2 * 128 + 2) == INVALID
    assert paged("append", k=0) == INVALID


@pytest.mark.parametrize("src,dst,code", [
    ([0, 10], [1, 2], INVALID), ([0, 1], [2, -1], INVALID), ([], [], fa.FORGE_OK), ([3], [3], fa.FORGE_OK),
])
def test_paged_copy_refuses_pages_outside_the_pool(src, dst, code):
    s, d = torch.tensor(src, dtype=torch.int32), torch.tensor(dst, dtype=torch.int32)
    assert fa.forge_attn_paged_copy(A, A, s, d, len(src), 1, 0, 10, 2, 64, 128, 2 * 64 * 128, BF, 0) == code


def test_paged_copy_rejects():
    s = torch.tensor([0], dtype=torch.int32)

    def call(n=1, layers=1, ls=0, src=s, ps=64):
        return fa.forge_attn_paged_copy(A, A, src, s, n, layers, ls, 10, 2, ps, 128, 2 * ps * 128, BF, 0)
    assert call(n=-1) == INVALID and call(layers=0) == INVALID and call(src=None) == INVALID
    assert call(ps=8) == UNSUPPORTED and call(layers=2, ls=12) == INVALID


# ---------------------------------------------------------------- torch helpers
def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


Q, K, CU = z(10, 4, 64), z(10, 2, 64), torch.tensor([0, 4, 10], dtype=torch.int32)
POOL, TABLE, LENS = z(5, 2, 16, 64), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)


def test_valid_host_tensors_fail_only_on_the_device_check():
    fused = z(10, 8 * 64).view(10, 8, 64)
    for q, k, v in ((Q, K, K), (fused[:, :4], fused[:, 4:6], fused[:, 6:])):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            fa.attention_varlen_fwd(q, k, v, CU)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fa.attention_varlen_bwd(Q, K, K, Q, z(4, 10, dtype=torch.float32), Q, CU)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fa.attention_decode_paged(z(3, 4, 64), POOL, POOL, TABLE, LENS)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fa.paged_append(K, K, POOL, POOL, TABLE, LENS, torch.tensor([0, 1, 2, 10], dtype=torch.int32))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fa.paged_copy(POOL, POOL, [0], [1])


@pytest.mark.parametrize("args,match", [
    ((Q[0], K, K, CU), r"q must be \[rows, H, D\]"),
    ((Q, K[:9], K[:9], CU), "k has shape"),
    ((Q, K, z(10, 2, 32), CU), "v has shape"),
    ((Q, K, z(10, 2, 64, dtype=torch.float32), CU), "v has dtype"),
    ((Q, z(10, 64, 2).transpose(1, 2), K, CU), "k's heads must be contiguous"),
    ((z(1, 4, 64).expand(10, 4, 64), K, K, CU), "q's rows must be at least"),
    ((z(10, 4 * 64 + 4).as_strided((10, 4, 64), (4 * 64 + 4, 64, 1)), K, K, CU), "multiple of 16 bytes"),
    ((Q, K, K, CU[:1]), "cu_seqlens must be"),
])
def test_varlen_helpers_reject(args, match):
    with pytest.raises(ValueError, match=match):
        fa.attention_varlen_fwd(*args)


def test_paged_helpers_reject():
    q = z(3, 4, 64)
    with pytest.raises(ValueError, match="pages must be contiguous"):
        fa.attention_decode_paged(q, POOL.transpose(1, 2), POOL.transpose(1, 2), TABLE, LENS)
    with pytest.raises(ValueError, match="v_pages has shape"):
        fa.attention_decode_paged(q, POOL, z(6, 2, 16, 64), TABLE, LENS)
    with pytest.raises(ValueError, match="page_table"):
        fa.attention_decode_paged(q, POOL, POOL, TABLE[0], LENS)
    with pytest.raises(ValueError, match="need cu_seqlens"):
        fa.paged_append(K, K, POOL, POOL, TABLE, LENS)
    with pytest.raises(ValueError, match="2 sources for 1 destinations"):
        fa.paged_copy(POOL, POOL, [0, 1], [2])
    with pytest.raises(ValueError, match="out of range"):
        fa.paged_copy(POOL, POOL, torch.tensor([1 << 33]), torch.tensor([0]))
    with pytest.raises(ValueError, match="list of page numbers"):
        fa.paged_copy(POOL, POOL, torch.tensor([0.5]), torch.tensor([0]))


# ------------------------------------------------------------------ the books
class Host(fa.PagedCache):
    """PagedCache over host pools whose copies are done by torch, in order."""

    def _copy(self, moves, stream):
        for a, b in moves:
            self.k_pages[:, b] = self.k_pages[:, a]
            self.v_pages[:, b] = self.v_pages[:, a]


def make(num_pages=24, ps=16, layers=2):
    pools = tuple(torch.zeros(layers, num_pages, 1, ps, 1) for _ in range(2))
    return Host(num_pages, 1, 1, page_size=ps, num_layers=layers, pages=pools)


def write(c, seq, start, values):
    for i, x in enumerate(values):
        t = start + i
        for pool, sign in ((c.k_pages, 1), (c.v_pages, -1)):
            pool[:, c.pages(seq)[t // c.page_size], 0, t % c.page_size, 0] = sign * x


def read(c, seq):
    out = []
    for t in range(c.length(seq)):
        p, r = c.pages(seq)[t // c.page_size], t % c.page_size
        k, v = c.k_pages[:, p, 0, r, 0], c.v_pages[:, p, 0, r, 0]
        assert torch.equal(k, -v) and bool((k == k[0]).all())
        out.append(int(k[0]))
    return out


def test_cache_books_against_a_model():
    rng = random.Random(3)
    c, model, stamp = make(), {}, 0
    for step in range(600):
        do = rng.choice(["new", "extend", "extend", "extend", "fork", "free", "compact"])
        if do == "new" and len(model) < 8:
            model[c.new()] = []
        elif do == "extend" and model:
            seqs = rng.sample(sorted(model), rng.randint(1, min(4, len(model))))
            counts = [rng.choice([0, 1, 1, 5, 16, 17, 40]) for _ in seqs]
            before = {s: (c.pages(s), c.length(s)) for s in model}, c.free_pages
            try:
                starts = c.extend(seqs, counts)
            except MemoryError:  # nothing has changed
                assert ({s: (c.pages(s), c.length(s)) for s in model}, c.free_pages) == before
                continue
            assert starts == [len(model[s]) for s in seqs]
            for s, n, start in zip(seqs, counts, starts):
                new = list(range(stamp + 1, stamp + 1 + n))
                stamp += n
                write(c, s, start, new)
                model[s] += new
        elif do == "fork" and model and len(model) < 8:
            s = rng.choice(sorted(model))
            model[c.fork(s)] = list(model[s])
        elif do == "free" and model:
            s = rng.choice(sorted(model))
            c.free(s)
            del model[s]
        elif do == "compact":
            c.compact()
            held = {p for s in model for p in c.pages(s)}
            assert held == set(range(len(held)))
        held = {p for s in model for p in c.pages(s)}
        assert len(held) + c.free_pages == c.num_pages
        for s, tokens in model.items():
            assert c.length(s) == len(tokens) and len(c.pages(s)) == -(-len(tokens) // c.page_size)
            assert read(c, s) == tokens, (step, do, s)


def test_cache_copies_a_shared_last_page_once_per_extra_holder():
    c = make()
    a = c.new()
    c.extend([a], [20])
    b, d = c.fork(a), c.fork(a)
    assert c.pages(a) == c.pages(b) == c.pages(d) and c.free_pages == 22
    c.extend([a, b, d], [1, 1, 1])      # two copies of the second page, the first stays shared
    assert c.free_pages == 20
    assert len({c.pages(s)[1] for s in (a, b, d)}) == 3 and len({c.pages(s)[0] for s in (a, b, d)}) == 1
    c.extend([a], [11])                 # fills its own page: nothing to copy
    e = c.fork(a)
    c.extend([e], [1])                  # the last page is full: a new one, no copy
    assert c.pages(e)[:2] == c.pages(a) and c.free_pages == 19


def test_cache_refusals():
    with pytest.raises(ValueError, match="multiple of 16"):
        fa.PagedCache(4, 1, 64, page_size=8, pages=(z(1), z(1)))
    with pytest.raises(ValueError, match="at least 1"):
        fa.PagedCache(0, 1, 64)
    with pytest.raises(ValueError, match="expected"):
        fa.PagedCache(4, 1, 64, page_size=16, pages=(z(1), z(1)))
    c = make()
    a = c.new()
    with pytest.raises(ValueError, match="each sequence once"):
        c.extend([a, a], [1, 1])
    with pytest.raises(ValueError, match="negative"):
        c.extend([a], [-1])
    with pytest.raises(KeyError):
        c.extend([99], [1])
    c.free(a)
    with pytest.raises(KeyError):
        c.free(a)


def state(c):
    return (sorted(c._free), list(c._refs), {s: list(p) for s, p in c._pages.items()}, dict(c._lens),
            c.k_pages.clone(), c.v_pages.clone())


def same(a, b):
    return a[:4] == b[:4] and torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])


class Failing(Host):
    fail = False

    def _copy(self, moves, stream):
        if self.fail and moves:
            raise fa.ForgeError(fa.FORGE_ERR_INVALID_ARG, "forge_attn_paged_copy")
        super()._copy(moves, stream)


def test_a_copy_that_fails_leaves_the_books_as_they_were():
    pools = tuple(torch.zeros(2, 12, 1, 16, 1) for _ in range(2))
    c = Failing(12, 1, 1, page_size=16, num_layers=2, pages=pools)
    gone, a = c.new(), c.new()
    c.extend([gone, a], [32, 20])
    write(c, a, 0, range(1, 21))
    b, d = c.fork(a), c.fork(a)
    before = state(c)
    c.fail = True
    with pytest.raises(fa.ForgeError):
        c.extend([a, b, d], [1, 30, 1])
    assert same(state(c), before)
    c.fail = False
    assert c.extend([a, b, d], [1, 30, 1]) == [20, 20, 20]
    assert read(c, b)[:20] == list(range(1, 21)) and len({c.pages(s)[1] for s in (a, b, d)}) == 3
    c.free(gone)
    before = state(c)
    c.fail = True
    with pytest.raises(fa.ForgeError):
        c.compact()
    assert same(state(c), before)
    c.fail = False
    assert c.compact() and read(c, b)[:20] == list(range(1, 21))
    assert {p for s in (a, b, d) for p in c.pages(s)} == set(range(c.num_pages - c.free_pages))


def test_cache_refuses_pools_that_its_calls_could_not_take():
    shape = (2, 4, 1, 16, 64)
    ok = z(*shape)

    def build(k, v, **kw):
        return fa.PagedCache(4, 1, 64, page_size=16, num_layers=2, pages=(k, v), **kw)
    assert build(ok, z(*shape)).num_pages == 4
    assert build(z(4, 2, 1, 16, 64).transpose(0, 1), z(4, 2, 1, 16, 64).transpose(0, 1)).num_pages == 4  # layers inside
    for k, v, kw, match in (
            (ok, z(*shape, dtype=torch.float32), {}, "torch.bfloat16 on cpu and torch.float32 on cpu"),
            (ok, z(*shape), dict(dtype=torch.float32), "expected torch.float32"),
            (z(*shape, dtype=torch.float16), z(*shape, dtype=torch.float16), {}, "unsupported dtype"),
            (ok, z(4, 2, 1, 16, 64).transpose(0, 1), {}, "expected the same"),
            (z(2, 4, 1, 64, 16).transpose(3, 4), z(2, 4, 1, 64, 16).transpose(3, 4), {}, "must be contiguous")):
        with pytest.raises(ValueError, match=match):
            build(k, v, **kw)
    with pytest.raises(ValueError, match="head_dim must be"):
        fa.PagedCache(4, 1, 96)
    with pytest.raises(ValueError, match="unsupported dtype"):
        fa.PagedCache(4, 1, 64, dtype=torch.float16)


def test_fork_of_an_unknown_sequence_changes_nothing():
    c = make()
    a = c.new()
    c.extend([a], [5])
    before = state(c)
    with pytest.raises(KeyError):
        c.fork(77)
    assert same(state(c), before) and c.new() == a + 1


@pytest.mark.parametrize("src,match", [([0.5], "list of page numbers"), ([2.0], "list of page numbers"), (["1"], "list of page"),
                                       ([1 << 33], "out of range"), ([-1 << 40], "out of range")])
def test_paged_copy_takes_whole_page_numbers_only(src, match):
    with pytest.raises(ValueError, match=match):
        fa.paged_copy(POOL, POOL, src, [0])
    with pytest.raises(ValueError, match=match):
        fa.paged_copy(POOL, POOL, [0], src)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):  # integers of any kind get on to the next check
        fa.paged_copy(POOL, POOL, [torch.tensor(1), 2], iter([True, 3]))


def test_cache_tables_are_the_books_and_serve_every_layer(monkeypatch):
    c = make()
    a, b, e = c.new(), c.new(), c.new()
    c.extend([a, b], [20, 40])
    table, lens = c.tables(iter([b, e, a]))
    assert table.tolist() == [c.pages(b), [0] * 3, c.pages(a) + [0]] and lens.tolist() == [40, 0, 20]
    assert table.dtype == lens.dtype == torch.int32 and table.is_contiguous() and lens.is_contiguous()
    assert c.tables([])[0].shape == (0, 1) and c.tables([])[1].shape == (0,)
    got = []
    monkeypatch.setattr(fa, "paged_append", lambda k, v, kp, vp, table, starts, cu, stream: got.append((table, starts)))
    monkeypatch.setattr(fa, "attention_decode_paged", lambda q, kp, vp, table, lens, stream=None, **o: got.append((table, lens)))
    # given tables are what the library gets, without being built again
    given, device_starts = (table, lens), torch.tensor([1, 2, 3], dtype=torch.int32)
    monkeypatch.setattr(c, "_rows", lambda seqs: pytest.fail("built again"))
    c.append(0, None, None, [b, e, a], device_starts, tables=given)
    c.append(1, None, None, None, [1, 2, 3], tables=given)
    c.decode(1, None, [b, e, a], tables=given)
    assert got[0][0] is table and got[0][1] is device_starts and got[1][0] is table and got[2] == given
    assert got[1][1].tolist() == [1, 2, 3] and got[1][1].dtype == torch.int32
    with pytest.raises(ValueError, match="tables of 3 sequences for 2"):
        c.decode(0, None, [a, b], tables=given)
    with pytest.raises(ValueError, match="tables of 3 sequences for 1"):
        c.append(0, None, None, [a], [0], tables=given)
    monkeypatch.undo()
    # and without, the books of the call's moment
    monkeypatch.setattr(fa, "paged_append", lambda k, v, kp, vp, table, starts, cu, stream: got.append((table, starts)))
    for starts in ([20, 40], device_starts[:2]):
        c.append(0, None, None, iter([a, b]), starts)
        assert got[-1][0].tolist() == [c.pages(a) + [0], c.pages(b)] and got[-1][1].tolist() == list(starts)


def test_the_raw_calls_keep_their_keyword_and_the_cache_takes_any_pair():
    import inspect
    for fn in (fa.forge_attn_varlen_fwd, fa.forge_attn_varlen_bwd):
        assert "clear_tail" in inspect.signature(fn).parameters
    pools = iter((z(1, 4, 1, 16, 64), z(1, 4, 1, 16, 64)))
    c = fa.PagedCache(4, 1, 64, page_size=16, pages=pools)
    assert c.k_pages.shape == c.v_pages.shape == (1, 4, 1, 16, 64)
