"""The paged KV cache on the GPU: decode against a plain f64 computation over the gathered pages,
append and copy bit for bit against loops over tokens and pages, and a serving run of all of
them together against attention over whole sequences. Decode tolerances are those of the other
parity tests (parity_util)."""
import math

import numpy as np
import pytest
import torch

import causal_flash_attention_attn_b200 as fa
from parity_util import check_close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}


def plain_decode(q, kp, vp, table, lens, W, C, sink):
    """f64: (o, lse), o = 0 and lse = -inf (or the sink) where nothing is visible."""
    q, kp, vp, table = q.double().cpu(), kp.double().cpu(), vp.double().cpu(), table.cpu()
    B, Hq, D = q.shape
    Hkv, ps = kp.shape[1:3]
    o, lse = torch.zeros_like(q), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(lens):
        lo = max(0, n - W) if W else 0
        at = torch.arange(lo, n)
        pages = table[b].long()[at // ps]
        for h in range(Hq):
            k, v = kp[pages, h // (Hq // Hkv), at % ps], vp[pages, h // (Hq // Hkv), at % ps]
            s = k @ q[b, h] / math.sqrt(D)
            s = C * torch.tanh(s / C) if C else s
            if sink is not None:
                s = torch.cat([s, sink[h].double().cpu()[None]])
            if len(s):
                lse[b, h] = torch.logsumexp(s, 0)
                o[b, h] = torch.exp(s - lse[b, h])[:len(at)] @ v
    return o, lse


def pool(dtype, lens, ps, Hkv, D, seed, spare=5, sigma=1.0):
    """Pools whose pages no query sees hold NaN, and a table of scattered pages (entries past a length: bad)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    P, width = sum(need) + spare, max(need + [1])
    order = torch.randperm(P, generator=g)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    kp, vp = (torch.full((P, Hkv, ps, D), float("nan")) for _ in range(2))
    at = 0
    for b, n in enumerate(lens):
        for i in range(need[b]):
            page = int(order[at])
            at += 1
            table[b, i] = page
            m = min(ps, n - i * ps)
            kp[page, :, :m] = torch.randn(Hkv, m, D, generator=g) * sigma
            vp[page, :, :m] = torch.randn(Hkv, m, D, generator=g)
    return kp.to(TDT[dtype]).to(DEV), vp.to(TDT[dtype]).to(DEV), table.to(DEV)


def check_decode(got, want, dtype):
    o, lse = got
    ro, rl = want
    check_close("o", o, ro.numpy(), dtype)
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse.cpu()), empty)
    if not bool(empty.all()):
        check_close("lse", lse.cpu()[~empty], rl[~empty].numpy(), dtype)


CASES = [
    # name, dtype, Hq, Hkv, D, page, lens, window, softcap, sink
    ("g4", "bf16", 8, 2, 128, 16, [1, 15, 16, 17, 63, 64, 65, 0, 1000], 0, 0.0, False),
    ("g7_sink", "bf16", 28, 4, 128, 64, [0, 300, 1, 129], 0, 0.0, True),
    ("g16_win", "bf16", 16, 1, 128, 48, [500, 97, 0, 12], 100, 0.0, False),
    ("g1_cap", "bf16", 3, 3, 64, 32, [5, 700, 64], 0, 30.0, True),
    ("d64_win1", "bf16", 8, 8, 64, 16, [5, 700, 64, 1], 1, 0.0, False),
    ("d256", "bf16", 8, 4, 256, 128, [1, 128, 900, 129], 0, 0.0, False),
    ("d256_g16_cap_win", "bf16", 16, 1, 256, 16, [400, 33], 300, 50.0, True),
    ("one", "bf16", 32, 8, 128, 16, [1000], 0, 0.0, False),
    ("empty_batch", "bf16", 4, 2, 128, 16, [0, 0, 0], 0, 0.0, False),
    ("empty_batch_sink", "bf16", 4, 2, 64, 16, [0], 0, 0.0, True),
    ("long", "bf16", 4, 2, 128, 64, [20000, 3], 0, 0.0, False),
    ("many", "bf16", 2, 1, 64, 16, [(37 * i) % 90 for i in range(300)], 0, 0.0, False),
    ("f32_g4", "f32", 8, 2, 128, 16, [1, 16, 17, 0, 333], 0, 0.0, False),
    ("f32_g1_d64_win", "f32", 3, 3, 64, 32, [5, 400], 37, 0.0, True),
    ("f32_g8_d256", "f32", 8, 1, 256, 16, [9, 130, 8], 0, 0.0, False),
    ("f32_g16_cap", "f32", 16, 1, 128, 16, [100, 31], 0, 30.0, False),
    ("f32_g16_d64", "f32", 32, 2, 64, 64, [700], 0, 0.0, True),
    ("f32_g12_d256", "f32", 12, 1, 256, 48, [200, 0, 1], 0, 0.0, True),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_decode_matches_f64(case):
    _, dtype, Hq, Hkv, D, ps, lens, W, C, use_sink = case
    kp, vp, table = pool(dtype, lens, ps, Hkv, D, seed=len(lens), sigma=2.0 if C else 1.0)
    if W:  # rows before the window are not read either
        for b, n in enumerate(lens):
            for t in range(0, max(0, n - W)):
                p = int(table[b, t // ps])
                kp[p, :, t % ps] = float("nan")
                vp[p, :, t % ps] = float("inf")
    g = torch.Generator().manual_seed(1)
    q = (torch.randn(len(lens), Hq, D, generator=g) * (2.0 if C else 1.0)).to(TDT[dtype]).to(DEV)
    sink = torch.tensor(np.linspace(-0.5, 3.0, Hq), dtype=torch.float32, device=DEV) if use_sink else None
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    first = fa.attention_decode_paged(q, kp, vp, table, sl, window=W, softcap=C, sink=sink)
    torch.cuda.synchronize()
    assert fa.forge_attn_check() == fa.FORGE_OK
    check_decode(first, plain_decode(q, kp, vp, table, lens, W, C, sink), dtype)
    again = fa.attention_decode_paged(q, kp, vp, table, sl, window=W, softcap=C, sink=sink)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_equals_the_contiguous_cache():
    B, Hq, Hkv, T, D = 3, 8, 2, 900, 128
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(B, Hkv, 960, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn(B, Hq, D, generator=g).to(torch.bfloat16).to(DEV)
    sl = torch.tensor([T, 1, 450], dtype=torch.int32, device=DEV)
    o, lse = fa.attention_decode(q, k, v, T=T, seq_lens=sl)
    # the same cache cut into pages of 64
    kp, vp = (x.view(B, Hkv, 15, 64, D).transpose(1, 2).reshape(B * 15, Hkv, 64, D) for x in (k, v))
    table = torch.arange(B * 15, dtype=torch.int32, device=DEV).view(B, 15)
    po, pl = fa.attention_decode_paged(q, kp, vp, table, sl)
    check_close("o", po, o.double().cpu().numpy(), "bf16")
    check_close("lse", pl, lse.double().cpu().numpy(), "bf16")


def test_pages_far_apart():
    # a pool whose page stride takes the last page's offset past 2^32 bytes and 2^31 elements
    P, Hkv, ps, D, stride = 5, 2, 16, 128, (1 << 29) + 64
    buf = torch.empty(4 * stride + 2 * Hkv * ps * D, dtype=torch.bfloat16, device=DEV)
    kp, vp = (buf[i * Hkv * ps * D:].as_strided((P, Hkv, ps, D), (stride, ps * D, D, 1)) for i in range(2))
    g = torch.Generator().manual_seed(6)
    rows = torch.randn(70, 2 * Hkv, D, generator=g).to(torch.bfloat16).to(DEV)
    table = torch.tensor([[4, 0, 3, 1, 2]], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 70], dtype=torch.int32, device=DEV)
    fa.paged_append(rows[:, :Hkv], rows[:, Hkv:], kp, vp, table, zero, cu)
    q = torch.randn(1, 8, D, generator=g).to(torch.bfloat16).to(DEV)
    sl = torch.tensor([70], dtype=torch.int32, device=DEV)
    near = [torch.stack([x[i] for i in range(P)]) for x in (kp, vp)]
    assert torch.equal(near[0][4], rows[:16, :Hkv].transpose(0, 1))
    check_decode(fa.attention_decode_paged(q, kp, vp, table, sl), plain_decode(q, *near, table, [70], 0, 0.0, None),
                 "bf16")
    fa.paged_copy(kp, vp, [4], [2])
    assert torch.equal(kp[2], near[0][4]) and torch.equal(vp[2], near[1][4]) and torch.equal(kp[3], near[0][3])


def test_bad_pages_and_lengths_are_reported():
    kp, vp, table = pool("bf16", [100, 40], 16, 2, 128, seed=1)
    q = torch.randn(2, 4, 128, device=DEV).to(torch.bfloat16)
    good = torch.tensor([100, 40], dtype=torch.int32, device=DEV)
    want = fa.attention_decode_paged(q, kp, vp, table, good)
    for page in (-1, kp.shape[0], 1 << 30):
        bad = table.clone()
        bad[0, 2] = page
        o, lse = fa.attention_decode_paged(q, kp, vp, bad, good)
        assert fa.forge_attn_check() == fa.FORGE_ERR_INVALID_ARG and fa.forge_attn_check() == fa.FORGE_OK
        assert torch.equal(o[1], want[0][1]) and bool(torch.isfinite(o).all())
    for n in (-1, table.shape[1] * 16 + 1, 1 << 30):
        o, lse = fa.attention_decode_paged(q, kp, vp, table, torch.tensor([n, 40], dtype=torch.int32, device=DEV))
        assert fa.forge_attn_check() == fa.FORGE_ERR_INVALID_ARG
        check_close("o", o[1], want[0][1].double().cpu().numpy(), "bf16")
        assert not bool(o[0].any()) and bool((lse[0] == -math.inf).all())


def test_decode_captured_follows_lengths_and_tables():
    kp, vp, table = pool("bf16", [500, 64, 300], 16, 2, 128, seed=2)
    q = torch.randn(3, 8, 128, device=DEV).to(torch.bfloat16)
    sl = torch.tensor([500, 64, 300], dtype=torch.int32, device=DEV)
    fa.attention_decode_paged(q, kp, vp, table, sl)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fa.attention_decode_paged(q, kp, vp, table, sl)
        graphs.append((g, out))
    for lens in ([500, 64, 300], [17, 0, 299], [0, 1, 2]):
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        want = fa.attention_decode_paged(q, kp, vp, table, sl)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


# ------------------------------------------------------------------ append
def loop_append(k, v, kp, vp, table, starts, lens):
    row = 0
    for b, n in enumerate(lens):
        for i in range(n):
            t, ps = starts[b] + i, kp.shape[2]
            page = int(table[b, t // ps])
            kp[page, :, t % ps], vp[page, :, t % ps] = k[row], v[row]
            row += 1


@pytest.mark.parametrize("dtype,Hkv,D,ps,lens,starts,fused,pad", [
    ("bf16", 4, 128, 16, [1] * 9, [0, 1, 15, 16, 17, 31, 100, 47, 48], False, 0),
    ("bf16", 2, 64, 48, [0, 1, 100, 7, 0], [5, 47, 0, 44, 3], True, 11),
    ("f32", 3, 128, 16, [33, 16], [16, 15], True, 0),
    ("bf16", 1, 256, 128, [700, 1], [1, 127], False, 1),
    ("bf16", 8, 128, 64, [3000, 1000], [0, 90], True, 0),
])
def test_append_matches_a_loop(dtype, Hkv, D, ps, lens, starts, fused, pad):
    dt, rows, n = TDT[dtype], sum(lens) + pad, len(lens)
    width = max(-(-(a + b) // ps) for a, b in zip(lens, starts)) + 1
    kp, vp = (torch.randn(n * width + 3, Hkv, ps, D, device=DEV).to(dt) for _ in range(2))
    table = torch.randperm(n * width + 3)[:n * width].to(torch.int32).view(n, width)
    kv = torch.randn(rows, 2 * Hkv + 1, D, device=DEV).to(dt)
    k, v = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    rk, rv = kp.clone(), vp.clone()
    loop_append(k, v, rk, rv, table, starts, lens)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    fa.paged_append(k, v, kp, vp, table.to(DEV), st, cu)
    assert fa.forge_attn_check() == fa.FORGE_OK
    assert torch.equal(kp, rk) and torch.equal(vp, rv)
    if all(x == 1 for x in lens) and not pad:  # the same without cu_seqlens
        kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
        rk, rv = torch.zeros_like(kp), torch.zeros_like(vp)
        loop_append(k, v, rk, rv, table, starts, lens)
        fa.paged_append(k, v, kp2, vp2, table.to(DEV), st)
        assert torch.equal(kp2, rk) and torch.equal(vp2, rv)


def test_append_skips_and_reports_bad_places():
    kp, vp = (torch.zeros(4, 2, 16, 64, device=DEV) for _ in range(2))
    k, v = (torch.ones(4, 2, 64, device=DEV) for _ in range(2))
    table = torch.tensor([[0, 1], [2, 9], [-1, 3], [3, 3]], dtype=torch.int32, device=DEV)
    starts = torch.tensor([32, 16, 0, -1], dtype=torch.int32, device=DEV)
    fa.paged_append(k, v, kp, vp, table, starts)
    assert fa.forge_attn_check() == fa.FORGE_ERR_INVALID_ARG
    assert not bool(kp.any()) and not bool(vp.any())
    starts = torch.tensor([31, 15, 16, 0], dtype=torch.int32, device=DEV)
    fa.paged_append(k, v, kp, vp, table, starts)
    # three distinct places (the last two tokens, of equal values, share page 3's first row), 2 heads of 64
    assert fa.forge_attn_check() == fa.FORGE_OK and int(kp.sum()) == 3 * 128


# -------------------------------------------------------------------- copy
@pytest.mark.parametrize("dtype,layers,P,Hkv,ps,D", [("bf16", 3, 40, 2, 16, 64), ("f32", 1, 9, 1, 32, 128),
                                                     ("bf16", 2, 1500, 1, 16, 64), ("bf16", 1, 12, 8, 128, 256)])
def test_copy_is_one_after_the_other(dtype, layers, P, Hkv, ps, D):
    # random pairs, so that pages are read after they are written and written again, and chains
    g = torch.Generator().manual_seed(P)
    kp, vp = (torch.randn(layers, P, Hkv, ps, D, generator=g).to(TDT[dtype]).to(DEV) for _ in range(2))
    n = min(P + 100, 1200)
    src, dst = torch.randint(P, (n,), generator=g), torch.randint(P, (n,), generator=g)
    src[:5], dst[:5] = torch.arange(5), torch.arange(1, 6)
    rk, rv = kp.clone(), vp.clone()
    for a, b in zip(src.tolist(), dst.tolist()):
        rk[:, b], rv[:, b] = rk[:, a].clone(), rv[:, a].clone()
    ck, cv = kp.clone(), vp.clone()
    fa.paged_copy(ck, cv, src, dst.tolist())
    assert torch.equal(ck, rk) and torch.equal(cv, rv)
    if layers == 1:
        fa.paged_copy(kp[0], vp[0], src.to(torch.int32), dst.to(torch.int32))
        assert torch.equal(kp, rk) and torch.equal(vp, rv)
    with pytest.raises(fa.ForgeError):
        fa.paged_copy(kp, vp, [0], [P])


def test_copy_of_many_distinct_pages_and_a_permutation_cycle():
    P = 1400
    kp = torch.arange(P, device=DEV, dtype=torch.float32).view(P, 1, 1, 1).expand(P, 1, 16, 64).contiguous()
    vp = -kp
    fa.paged_copy(kp, vp, list(range(700)), list(range(700, 1400)))
    want = torch.arange(700, device=DEV, dtype=torch.float32).repeat(2)
    assert torch.equal(kp[:, 0, 15, 63], want) and torch.equal(vp[:, 0, 0, 0], -want)
    fa.paged_copy(kp, vp, [3, 0, 1, 2], [9, 3, 0, 1])  # a shift through page 9
    assert kp[[9, 3, 0, 1], 0, 7, 7].tolist() == [3.0, 0.0, 1.0, 2.0]


# ------------------------------------------------------------------ together
def test_a_serving_run():
    """Prompts prefilled packed and appended, forks, tokens decoded one by one, a sequence freed, the pool
    compacted: every decoded token's output is that of attention over the whole sequence so far."""
    L, Hq, Hkv, D = 2, 8, 2, 128
    cache = fa.PagedCache(64, Hkv, D, page_size=16, num_layers=L, device=DEV)
    cache.k_pages.fill_(float("nan"))
    cache.v_pages.fill_(float("nan"))
    g = torch.Generator(device=DEV).manual_seed(9)

    def tokens(n):
        return torch.randn(L, n, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)

    def packed(x):
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    lens = [37, 1, 80]
    seqs = [cache.new() for _ in lens]
    text = dict(zip(seqs, tokens(sum(lens)).split(lens, 1)))
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    starts = cache.extend(seqs, lens)
    for layer in range(L):
        q, k, v = packed(torch.cat([text[s][layer] for s in seqs]))
        o, _ = fa.attention_varlen_fwd(q, k, v, cu)
        assert bool(torch.isfinite(o).all())
        cache.append(layer, k, v, seqs, starts, cu)

    def step(now):
        new = tokens(len(now))
        starts = cache.extend(now, [1] * len(now))
        for i, s in enumerate(now):
            text[s] = torch.cat([text[s], new[:, i:i + 1]], 1)
        for layer in range(L):
            q, k, v = packed(new[layer])
            cache.append(layer, k, v, now, starts)
            o, lse = cache.decode(layer, q.contiguous(), now, window=50)
            whole = torch.cat([text[s][layer] for s in now])
            ends = torch.tensor([0] + list(np.cumsum([text[s].shape[1] for s in now])), dtype=torch.int32, device=DEV)
            ro, rl = fa.attention_varlen_fwd(*packed(whole), ends, window=50)
            last = (ends[1:] - 1).long()
            check_close("o", o, ro[last].double().cpu().numpy(), "bf16")
            check_close("lse", lse, rl[:, last].t().double().cpu().numpy(), "bf16")
    for i in range(20):
        step(seqs)
        if i == 5:
            seqs.append(cache.fork(seqs[0]))
            text[seqs[-1]] = text[seqs[0]].clone()
            seqs.append(cache.fork(seqs[0]))
            text[seqs[-1]] = text[seqs[0]].clone()
        if i == 11:
            cache.free(seqs.pop(2))
            moves = cache.compact()
            assert moves
            cache.k_pages[:, cache.num_pages - cache.free_pages:] = float("nan")
        if i == 14:
            cache.free(seqs.pop(0))
    assert fa.forge_attn_check() == fa.FORGE_OK


def test_cache_calls_on_another_stream_keep_their_tables():
    # the tables that append and decode build must not be given away while the stream that reads
    # them is still busy; another tensor of their sizes would hold no page number
    side, Hkv, D, n = torch.cuda.Stream(), 2, 64, 5
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(n * 7, Hkv, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(n, 4, D, generator=g).bfloat16().to(DEV)
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV) * 7
    out = []
    for stream in (None, side):
        cache = fa.PagedCache(32, Hkv, D, page_size=16)
        seqs = [cache.new() for _ in range(n)]
        starts = cache.extend(seqs, [7] * n)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                torch.cuda._sleep(50_000_000)
        cache.append(0, k, v, seqs, starts, cu, stream=stream)
        junk = [torch.full((m,), 1 << 20, dtype=torch.int32, device=DEV) for m in (n, n) * 4]
        o, lse = cache.decode(0, q, seqs, stream=stream)
        junk += [torch.full((m,), 1 << 20, dtype=torch.int32, device=DEV) for m in (n, n) * 4]
        torch.cuda.synchronize()
        out.append((o, lse))
        del junk
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert fa.forge_attn_check() == fa.FORGE_OK


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 8, 2, 128), ("bf16", 3, 3, 64), ("bf16", 16, 1, 256),
                                            ("f32", 8, 2, 128), ("f32", 2, 2, 64), ("f32", 12, 1, 256)])
@pytest.mark.parametrize("W,C,use_sink", [(0, 0.0, False), (0, 0.0, True), (90, 30.0, True)])
def test_a_bad_page_holds_no_visible_key(dtype, Hq, Hkv, D, W, C, use_sink):
    # sequences with a bad page first, inside, last, everywhere, and none, against f64 without those keys
    lens, ps = [100, 300, 33, 70, 90, 1500], 16
    kp, vp, table = pool(dtype, lens, ps, Hkv, D, seed=7)
    bad = table.clone()
    gone = {0: [0], 1: [5, 6, 18], 2: [2], 3: list(range(5)), 5: [0, 40, 41, 93]}
    for b, pages in gone.items():
        for i, at in enumerate(pages):
            bad[b, at] = (-1, kp.shape[0], 1 << 30)[i % 3]
    g = torch.Generator().manual_seed(3)
    q = torch.randn(len(lens), Hq, D, generator=g).to(TDT[dtype]).to(DEV)
    sink = torch.tensor(np.linspace(-0.5, 3.0, Hq), dtype=torch.float32, device=DEV) if use_sink else None
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = fa.attention_decode_paged(q, kp, vp, bad, sl, window=W, softcap=C, sink=sink)
    assert fa.forge_attn_check() == fa.FORGE_ERR_INVALID_ARG
    o, lse = torch.zeros(len(lens), Hq, D, dtype=torch.float64), torch.zeros(len(lens), Hq, dtype=torch.float64)
    for b, n in enumerate(lens):
        at = torch.tensor([t for t in range(max(0, n - W) if W else 0, n) if t // ps not in gone.get(b, [])], dtype=torch.long)
        where = table[b].cpu().long()[at // ps], slice(None), at % ps
        k, v = (x.double().cpu()[where].repeat_interleave(Hq // Hkv, 1) for x in (kp, vp))
        s = torch.einsum("thd,hd->ht", k, q[b].double().cpu()) / math.sqrt(D)
        s = C * torch.tanh(s / C) if C else s
        if use_sink:
            s = torch.cat([s, sink.double().cpu()[:, None]], 1)
        if s.shape[1] == 0:
            lse[b] = -math.inf
            continue
        lse[b] = torch.logsumexp(s, 1)
        o[b] = torch.einsum("ht,thd->hd", torch.exp(s - lse[b][:, None])[:, :len(at)], v)
    check_decode(got, (o, lse), dtype)
    assert not bool(got[0][3].any())


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 8, 2, 128), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("use_sink", [False, True])
def test_a_nan_among_the_visible_keys_shows_in_o_and_lse(dtype, Hq, Hkv, D, use_sink):
    # in one KV head: a NaN key (one of many, all of a warp's step, the only one) makes o and lse NaN, a NaN
    # value o alone; the other head and the other sequences are as they were
    lens, ps, G = [300, 300, 1, 40, 300, 5000], 16, Hq // Hkv
    kp, vp, table = pool(dtype, lens, ps, Hkv, D, seed=11)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(len(lens), Hq, D, generator=g).to(TDT[dtype]).to(DEV)
    sink = torch.tensor(np.linspace(-0.5, 3.0, Hq), dtype=torch.float32, device=DEV) if use_sink else None
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = fa.attention_decode_paged(q, kp, vp, table, sl, sink=sink)
    for b, rows in ((0, [37]), (1, range(32, 48)), (2, [0]), (5, [4321])):
        for t in rows:
            kp[int(table[b, t // ps]), 0, t % ps, 3] = float("nan")
    vp[int(table[4, 2]), 0, 5] = float("nan")
    o, lse = fa.attention_decode_paged(q, kp, vp, table, sl, sink=sink)
    assert fa.forge_attn_check() == fa.FORGE_OK
    hit = torch.tensor([0, 1, 2, 5], device=DEV)
    assert bool(torch.isnan(lse[hit, :G]).all()) and bool(torch.isnan(o[hit, :G]).all())
    assert bool(torch.isnan(o[4, :G]).all()) and torch.equal(lse[4], want[1][4])
    assert torch.equal(o[3], want[0][3]) and torch.equal(lse[3], want[1][3])
    assert torch.equal(o[:, G:], want[0][:, G:]) and torch.equal(lse[:, G:], want[1][:, G:])


@pytest.mark.parametrize("cu", [[0, 5, 3], [0, 5, 3, 8], [1, 4, 8], [0, 4, 9], [0, -1, 8], [0, 1 << 30, 8], [0] * 300 + [9]])
def test_append_reports_lengths_that_do_not_ascend(cu):
    n, rows, ps = len(cu) - 1, 8, 16
    kp, vp = (torch.zeros(2 * n, 1, ps, 64, device=DEV) for _ in range(2))
    k = torch.ones(rows, 1, 64, device=DEV)
    table = torch.arange(2 * n, dtype=torch.int32, device=DEV).view(n, 2)
    starts = torch.zeros(n, dtype=torch.int32, device=DEV)
    fa.paged_append(k, k, kp, vp, table, starts, torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert fa.forge_attn_check() == fa.FORGE_ERR_INVALID_ARG and fa.forge_attn_check() == fa.FORGE_OK


@pytest.mark.parametrize("cu", [[0, 8], [0, 0, 3, 3, 8], [0, 2], [0, 0]])
def test_append_takes_empty_sequences_and_rows_behind_the_last(cu):
    n, rows, ps = len(cu) - 1, 8, 16
    kp, vp = (torch.zeros(n, 1, ps, 64, device=DEV) for _ in range(2))
    k = torch.arange(1, rows + 1, device=DEV, dtype=torch.float32).view(rows, 1, 1).expand(rows, 1, 64).contiguous()
    table = torch.arange(n, dtype=torch.int32, device=DEV).view(n, 1)
    starts = torch.zeros(n, dtype=torch.int32, device=DEV)
    fa.paged_append(k, -k, kp, vp, table, starts, torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert fa.forge_attn_check() == fa.FORGE_OK
    want = torch.zeros_like(kp)
    for b in range(n):
        want[b, 0, :cu[b + 1] - cu[b]] = k[cu[b]:cu[b + 1], 0]
    assert torch.equal(kp, want) and torch.equal(vp, -want)


def test_cache_calls_do_not_wait_for_the_device():
    Hkv, D, seqs_n = 2, 64, 3
    cache = fa.PagedCache(64, Hkv, D, page_size=16, num_layers=2, device=DEV)
    seqs = [cache.new() for _ in range(seqs_n)]
    k = torch.randn(60, Hkv, D, device=DEV).bfloat16()
    q = torch.randn(seqs_n + 1, 4, D, device=DEV).bfloat16()
    cu = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        starts = cache.extend(seqs, [20] * 3)
        cache.append(0, k, k, seqs, starts, cu)
        cache.append(1, k, k, seqs, starts, cu)
        seqs.append(cache.fork(seqs[1]))
        starts = cache.extend(seqs, [1] * 4)
        now = cache.tables(seqs)
        for layer in range(2):
            cache.append(layer, k[:4], k[:4], seqs, starts, tables=now)
            o, lse = cache.decode(layer, q, seqs, tables=now)
        o2, lse2 = cache.decode(1, q, seqs)
        side.wait_stream(torch.cuda.current_stream())
        o3, lse3 = cache.decode(1, q, seqs, stream=side)
        cache.free(seqs.pop(0))
        assert cache.compact()
    finally:
        torch.cuda.set_sync_debug_mode("default")
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(o, o3) and torch.equal(lse, lse3)
    assert fa.forge_attn_check() == fa.FORGE_OK


def test_a_captured_step_of_the_cache_follows_its_tables():
    # one graph for a step of two layers; before each replay the new step's tables, starts and tokens are
    # copied into the tensors that the graph reads. A second cache takes the same steps without a graph.
    L, Hq, Hkv, D, n, steps = 2, 4, 2, 64, 3, 40
    caches = [fa.PagedCache(40, Hkv, D, page_size=16, num_layers=L, device=DEV) for _ in range(2)]
    for c in caches:
        c.k_pages.zero_(), c.v_pages.zero_()
    seqs = [[c.new() for _ in range(n)] for c in caches]
    g = torch.Generator(device=DEV).manual_seed(8)
    width = 4
    table = torch.zeros(n, width, dtype=torch.int32, device=DEV)
    lens, starts = (torch.zeros(n, dtype=torch.int32, device=DEV) for _ in range(2))
    new = torch.zeros(L, n, Hq + 2 * Hkv, D, device=DEV, dtype=torch.bfloat16)

    def step(c, s, at, tables):
        out = []
        for layer in range(L):
            q, k, v = new[layer, :, :Hq], new[layer, :, Hq:Hq + Hkv], new[layer, :, Hq + Hkv:]
            c.append(layer, k, v, s, at, tables=tables)
            out += c.decode(layer, q.contiguous(), s, tables=tables)
        return out
    graph = torch.cuda.CUDAGraph()
    pool_before = caches[0].k_pages.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(caches[0], seqs[0], starts, (table, lens))
    assert torch.equal(caches[0].k_pages, pool_before)
    with pytest.raises(RuntimeError, match="build them before"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            caches[1].decode(0, new[0, :, :Hq].contiguous(), seqs[1])
    for i in range(steps):
        new.copy_(torch.randn(new.shape, generator=g, device=DEV))
        at = [c.extend(s, [1] * n) for c, s in zip(caches, seqs)]
        t, length = caches[0].tables(seqs[0])
        table[:, :t.shape[1]] = t
        lens.copy_(length)
        starts.copy_(length - 1)
        graph.replay()
        want = step(caches[1], seqs[1], at[1], None)
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
        if i == 17:
            for c, s in zip(caches, seqs):
                c.free(s[0])
                s[0] = c.fork(s[1])
    assert torch.equal(caches[0].k_pages, caches[1].k_pages) and torch.equal(caches[0].v_pages, caches[1].v_pages)
    assert fa.forge_attn_check() == fa.FORGE_OK
