"""Operators for packed sequences and the paged key/value cache, as cases to be timed.

Five operators, named by a case's "op":
  prompt  causal attention over a whole prompt batch: sequences of different lengths packed
          along the token axis, query heads sharing KV heads; forward only (serving)
  train   the same with its gradient: o, and dq, dk, dv (and dsink) for a given dO
  decode  attention of one new token per sequence over a paged KV cache
  append  new tokens' keys and values written into the pages of their sequences
  copy    pages copied to other pages of the pool in every layer (a fork's own last page,
          the moves of a compaction)

`own` False computes the plain form with elementary torch operations in 32 bits; True calls
causal_flash_attention_attn_b200.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------ the cases
def listed():
    return [
        # a scheduler's step with a few short prompts: latency counts
        dict(name="prompt_few", op="prompt", dtype="bf16", Hq=32, Hkv=8, D=128, lens="1,9,46,72", pad=0,
             window=0, softcap=0.0, sink=False, fused=True),
        # long prompts of a sliding-window layer, 16K tokens in all
        dict(name="prompt_long", op="prompt", dtype="bf16", Hq=32, Hkv=8, D=128, lens="9001,5000,2383", pad=0,
             window=4096, softcap=0.0, sink=False, fused=False),
        # a small model's batch of short documents (head dim 64, no shared heads)
        dict(name="train_short", op="train", dtype="bf16", Hq=6, Hkv=6, D=64,
             lens="512,77,300,512,129,64,411,256,33,500,190,1,345,512,222,128", pad=0,
             window=0, softcap=0.0, sink=False, fused=False),
        # ordinary documents of mixed lengths, grouped heads
        dict(name="train_mixed", op="train", dtype="bf16", Hq=28, Hkv=4, D=128,
             lens="4096,1531,1024,777,333,256,100,75", pad=0,
             window=0, softcap=0.0, sink=False, fused=False),
        # head dim 256 with the score cap
        dict(name="train_capped", op="train", dtype="bf16", Hq=8, Hkv=4, D=256, lens="3000,905,191", pad=0,
             window=0, softcap=50.0, sink=False, fused=False),
        # the f32 path, small
        dict(name="train_f32", op="train", dtype="f32", Hq=2, Hkv=2, D=64, lens="128,77,51", pad=0,
             window=0, softcap=0.0, sink=False, fused=False),
        # one sequence's next token: latency counts
        dict(name="decode_one", op="decode", dtype="bf16", Hq=32, Hkv=8, D=128, lens="1000", page=16,
             window=0, softcap=0.0, sink=False),
        # a full batch with long contexts of different lengths
        dict(name="decode_batch", op="decode", dtype="bf16", Hq=32, Hkv=8, D=128,
             lens="16384,9000,12001,16384,2048,15000,7777,16000,4096,11111,16384,1,13000,16383,8192,6000", page=64,
             window=0, softcap=0.0, sink=False),
        # one new token for each of 64 sequences
        dict(name="append_step", op="append", dtype="bf16", Hq=28, Hkv=4, D=128, lens=",".join(["1"] * 64),
             past=4096, page=16, fused=True),
        # whole prompts enter the cache
        dict(name="append_prompt", op="append", dtype="bf16", Hq=32, Hkv=8, D=128, lens="9001,5000,2383", past=0,
             page=64, fused=True),
        # forks: each gets a copy of its last, partly filled page, in every layer
        dict(name="copy_fork", op="copy", dtype="bf16", Hkv=8, D=128, page=64, layers=6, pages=64, moves=4),
        # a compaction that moves a good part of the pool
        dict(name="copy_compact", op="copy", dtype="bf16", Hkv=8, D=128, page=64, layers=6, pages=1024, moves=384),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _split(rng, total, n):
    """n lengths of at least 1 that add up to total."""
    w = [rng.random() ** 2 + 1e-3 for _ in range(n)]
    lens = [max(1, int(total * x / sum(w))) for x in w]
    lens[lens.index(max(lens))] += total - sum(lens)
    return lens if min(lens) >= 1 else [total]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "decode", "decode", "append", "copy"])
    if op == "copy":
        pages = _log_int(rng, 16, 1024)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), Hkv=rng.choice([1, 2, 4, 6, 8]),
                    D=rng.choice([64, 128]), page=rng.choice([16, 32, 64]), layers=rng.randint(1, 6),
                    pages=pages, moves=_log_int(rng, 1, max(1, pages * 3 // 8)))
    Hq, Hkv = rng.choice([(28, 4), (32, 8), (8, 4), (6, 6), (16, 1), (8, 8)])
    if op == "append":
        n = _log_int(rng, 1, 64)
        total = max(n, _log_int(rng, 1, 16384))
        lens = [1] * n if rng.random() < 0.4 else _split(rng, total, n)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128]),
                    lens=",".join(map(str, lens)), past=rng.choice([0, rng.randint(1, 4096)]),
                    page=rng.choice([16, 32, 64, 128]), fused=rng.random() < 0.5)
    sink = rng.random() < 0.3
    if op == "decode":
        D = rng.choice([64, 128, 128, 256])
        longest = _log_int(rng, 1, 16384)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        most = (160 if dtype == "bf16" else 80) * 10 ** 6  # cached values of K, as in the largest listed batch
        n = _log_int(rng, 1, min(64, max(1, most // (longest * Hkv * D))))
        lens = [_log_int(rng, 1, longest) for _ in range(n - 1)] + [longest]
        return dict(op=op, dtype=dtype, Hq=Hq, Hkv=Hkv, D=D,
                    lens=",".join(map(str, lens)), page=rng.choice([16, 32, 64, 128]),
                    window=rng.choice([0, 0, rng.randint(1, 4096)]), softcap=rng.choice([0.0, 0.0, 50.0]), sink=sink)
    D = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
    most = 640 if dtype == "f32" else 8192 if op == "train" or D == 256 else 16384
    total = _log_int(rng, 1, most)
    lens = _split(rng, total, min(total, _log_int(rng, 1, 32)))
    case = dict(op=op, dtype=dtype, Hq=Hq, Hkv=Hkv, D=D, lens=",".join(map(str, lens)),
                pad=rng.choice([0, 0, rng.randint(1, 200)]), window=rng.choice([0, 0, rng.randint(1, 4096)]),
                softcap=rng.choice([0.0, 0.0, 50.0]), sink=sink, fused=rng.random() < 0.5)
    # no more work than the largest listed case of its kind
    return case if work(case)["flops"] <= (7.1e11 if op == "prompt" else 5.2e11) else draw(rng)


# ------------------------------------------------------------------------ the inputs
def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * sigma).to(dt)

    state = dict(case=case)
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "copy":
        shape = (case["layers"], case["pages"], Hkv, case["page"], D)
        state["k_pages"], state["v_pages"] = normal(*shape), normal(*shape)
        # distinct pages, sources first: known on the host, where the bookkeeping is done
        order = torch.randperm(case["pages"], generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        state["src"], state["dst"] = order[:case["moves"]].clone(), order[case["moves"]:2 * case["moves"]].clone()
        return state
    lens, Hq = _lens(case), case["Hq"]
    n, total = len(lens), sum(lens)
    sigma = 2.0 if case.get("softcap") else 1.0  # capped layers see large scores
    if case["op"] in ("prompt", "train", "append"):
        cu = torch.zeros(n + 1, dtype=torch.int64)
        cu[1:] = torch.tensor(lens).cumsum(0)
        state["cu_seqlens"] = cu.to(torch.int32).to(dev)
        rows = total + case.get("pad", 0)
        if case["fused"]:  # views of one projection's output, token stride (Hq + 2 Hkv) * D
            qkv = normal(rows, Hq + 2 * Hkv, D)
            qkv[:, :Hq + Hkv] *= sigma
            state["q"], state["k"], state["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            state["q"], state["k"] = normal(rows, Hq, D, sigma=sigma), normal(rows, Hkv, D, sigma=sigma)
            state["v"] = normal(rows, Hkv, D)
    if case["op"] == "train":
        state["dO"] = normal(rows, Hq, D)
    if case.get("sink"):
        state["sink"] = torch.randn(Hq, generator=g, device=dev)
    if case["op"] in ("decode", "append"):
        page = case["page"]
        held = torch.tensor(lens) if case["op"] == "decode" else torch.tensor(lens) + case["past"]
        width = -(-int(held.max()) // page)
        used = n * width
        # the pages of the sequences lie scattered in a pool with some to spare
        table = torch.randperm(used + 16, generator=torch.Generator().manual_seed(seed))[:used]
        state["page_table"] = table.to(torch.int32).reshape(n, width).to(dev)
        shape = (used + 16, Hkv, page, D)
        if case["op"] == "decode":
            state["q"] = normal(n, Hq, D, sigma=sigma)
            state["k_pages"], state["v_pages"] = normal(*shape, sigma=sigma), normal(*shape)
            state["seq_lens"] = held.to(torch.int32).to(dev)
        else:
            state["k_pages"], state["v_pages"] = (torch.zeros(shape, dtype=dt, device=dev) for _ in range(2))
            state["starts"] = torch.full((n,), case["past"], dtype=torch.int32, device=dev)
    return state


# ------------------------------------------------------------------------ plain forms
def _visible(cu_seqlens, rows, window):
    """[rows, rows] truth values: key j is visible to query i."""
    at = torch.arange(rows, device=cu_seqlens.device)
    seq = torch.searchsorted(cu_seqlens[1:].long(), at, right=True)  # rows behind the last sequence: one past it
    i, j = at[:, None], at[None, :]
    see = (j <= i) & (seq[:, None] == seq[None, :]) & (at < cu_seqlens[-1])[:, None]
    return see & (j > i - window) if window else see


def _scores(q, k, scale, softcap):
    """q [Hkv, G, R, D], k [Hkv, 1, C, D] -> the scores, before the mask."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    return s.div_(softcap).tanh_().mul_(softcap) if softcap else s


def _softmax(s, hidden, sink):
    """exp(s - lse) in place, and lse; rows that see nothing give zeros and -inf."""
    s.masked_fill_(hidden, -math.inf)
    m = s.amax(-1, keepdim=True)
    if sink is not None:
        m = torch.maximum(m, sink)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m0).exp_()
    l = p.sum(-1, keepdim=True)
    if sink is not None:
        l = l + torch.exp(sink - m0)
    return p.div_(torch.where(l == 0, torch.ones_like(l), l)), m0 + torch.log(l)


def _heads(x, Hkv):
    """[rows, H, D] -> [Hkv, H / Hkv, rows, D] in 32 bits."""
    return x.float().reshape(x.shape[0], Hkv, -1, x.shape[2]).permute(1, 2, 0, 3)


def _rows(x, dtype):
    """[Hkv, G, rows, D] -> [rows, Hkv * G, D]"""
    return x.permute(2, 0, 1, 3).flatten(1, 2).to(dtype)


def _plain_packed(st):
    case, cu = st["case"], st["cu_seqlens"]
    Hkv, D, cap = case["Hkv"], case["D"], case["softcap"]
    dt, scale = st["q"].dtype, 1.0 / math.sqrt(D)
    q, k, v = (_heads(st[x], Hkv) for x in ("q", "k", "v"))
    rows = st["q"].shape[0]
    sink = st["sink"].view(Hkv, -1, 1, 1) if "sink" in st else None
    hidden = ~_visible(cu, rows, case["window"])
    padding = (torch.arange(rows, device=cu.device) >= cu[-1])[:, None]
    s = _scores(q, k, scale, cap)
    if case["op"] == "train" and cap:
        slope = 1 - (s / cap).square_()
    p, lse = _softmax(s, hidden, sink)
    lse = lse.masked_fill(padding, -math.inf)
    o = torch.matmul(p, v)
    out = dict(o=_rows(o, dt))
    if case["op"] == "prompt":
        out["lse"] = lse.flatten(0, 1).squeeze(-1)
        return out
    dO = _heads(st["dO"], Hkv).masked_fill(padding, 0.0)
    dv = torch.matmul(p.transpose(-1, -2), dO).sum(1, keepdim=True)
    delta = (dO * o).sum(-1, keepdim=True)
    ds = p.mul_(torch.matmul(dO, v.transpose(-1, -2)).sub_(delta))
    if cap:
        ds.mul_(slope)
    out["dq"] = _rows(torch.matmul(ds, k).mul_(scale), dt)
    out["dk"] = _rows(torch.matmul(ds.transpose(-1, -2), q).sum(1, keepdim=True).mul_(scale), dt)
    out["dv"] = _rows(dv, dt)
    if sink is not None:
        out["dsink"] = -(torch.exp(sink - lse).masked_fill(padding, 0.0) * delta).sum((2, 3)).flatten()
    return out


def _plain_decode(st):
    case = st["case"]
    Hkv, D = case["Hkv"], case["D"]
    q = st["q"].float().view(len(st["q"]), Hkv, -1, D)
    table = st["page_table"].long()
    k, v = (st[x][table].float().permute(0, 2, 1, 3, 4).flatten(2, 3) for x in ("k_pages", "v_pages"))
    at = torch.arange(k.shape[2], device=q.device)
    n = st["seq_lens"][:, None]
    hidden = at >= n
    if case["window"]:
        hidden |= at < n - case["window"]
    sink = st["sink"].view(1, Hkv, -1, 1) if "sink" in st else None
    p, lse = _softmax(_scores(q, k, 1.0 / math.sqrt(D), case["softcap"]), hidden[:, None, None, :], sink)
    return dict(o=torch.matmul(p, v).flatten(1, 2).to(st["q"].dtype), lse=lse.flatten(1))


def _plain_append(st):
    cu, page = st["cu_seqlens"].long(), st["case"]["page"]
    at = torch.arange(st["k"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], at, right=True)
    pos = st["starts"].long()[seq] + at - cu[seq]
    where = st["page_table"].long()[seq, pos // page], slice(None), pos % page
    st["k_pages"][where] = st["k"]
    st["v_pages"][where] = st["v"]
    return dict(k_pages=st["k_pages"], v_pages=st["v_pages"])


def _plain_copy(st):
    src, dst = (st[x].to(st["k_pages"].device).long() for x in ("src", "dst"))
    st["k_pages"][:, dst] = st["k_pages"][:, src]
    st["v_pages"][:, dst] = st["v_pages"][:, src]
    return dict(k_pages=st["k_pages"], v_pages=st["v_pages"])


# ------------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if not own:
        with torch.no_grad():
            if case["op"] in ("prompt", "train"):
                return _plain_packed(state)
            return {"decode": _plain_decode, "append": _plain_append, "copy": _plain_copy}[case["op"]](state)
    import causal_flash_attention_attn_b200 as fa
    sink = state.get("sink")
    if case["op"] == "prompt":
        o, lse = fa.attention_varlen_fwd(state["q"], state["k"], state["v"], state["cu_seqlens"],
                                         window=case["window"], softcap=case["softcap"], sink=sink)
        return dict(o=o, lse=lse)
    if case["op"] == "train":
        leaves = [x.detach().requires_grad_() for x in (state["q"], state["k"], state["v"], sink) if x is not None]
        o = fa.attention_varlen(*leaves[:3], state["cu_seqlens"], window=case["window"], softcap=case["softcap"],
                                sink=leaves[3] if sink is not None else None)
        grads = torch.autograd.grad(o, leaves, state["dO"])
        return dict(zip(("o", "dq", "dk", "dv", "dsink"), (o.detach(), *grads)))
    if case["op"] == "decode":
        o, lse = fa.attention_decode_paged(state["q"], state["k_pages"], state["v_pages"], state["page_table"],
                                           state["seq_lens"], window=case["window"], softcap=case["softcap"],
                                           sink=sink)
        return dict(o=o, lse=lse)
    if case["op"] == "append":
        fa.paged_append(state["k"], state["v"], state["k_pages"], state["v_pages"], state["page_table"],
                        state["starts"], cu_seqlens=state["cu_seqlens"])
    else:
        fa.paged_copy(state["k_pages"], state["v_pages"], state["src"], state["dst"])
    return dict(k_pages=state["k_pages"], v_pages=state["v_pages"])


# ------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size, D, Hkv = (2 if case["dtype"] == "bf16" else 4), case["D"], case["Hkv"]
    if case["op"] == "copy":
        return dict(bytes=2 * 2 * case["layers"] * case["moves"] * Hkv * case["page"] * D * size, flops=0)
    lens, Hq = _lens(case), case["Hq"]
    total, n, row = sum(lens), len(lens), D * size
    if case["op"] == "append":  # every new row read and written, tables read
        pages = sum(-(-(x + case["past"]) // case["page"]) - case["past"] // case["page"] for x in lens)
        return dict(bytes=2 * 2 * total * Hkv * row + 4 * (2 * n + 1 + pages), flops=0)
    W = case["window"] or max(lens)
    sinks = 4 * Hq if case["sink"] else 0
    if case["op"] == "decode":
        seen = sum(min(x, W) for x in lens)
        pages = sum(-(-x // case["page"]) - max(0, x - W) // case["page"] for x in lens)
        return dict(bytes=2 * seen * Hkv * row + 2 * n * Hq * row + 4 * n * Hq + 4 * n + 4 * pages + sinks,
                    flops=4 * D * Hq * seen)
    pairs = sum(x * (x + 1) // 2 if x <= W else W * (W + 1) // 2 + (x - W) * W for x in lens)
    if case["op"] == "prompt":
        return dict(bytes=2 * total * (Hq + Hkv) * row + 4 * total * Hq + 4 * (n + 1) + sinks,
                    flops=4 * D * Hq * pairs)
    return dict(bytes=4 * total * (Hq + Hkv) * row + 4 * (n + 1) + 2 * sinks, flops=14 * D * Hq * pairs)


# ------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "copy":
        for name in ("k_pages", "v_pages"):
            for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
                st[name][:, d] = st[name][:, s]
        return dict(k_pages=st["k_pages"].double(), v_pages=st["v_pages"].double())
    lens, Hkv, D, Hq = _lens(case), case["Hkv"], case["D"], case["Hq"]
    if case["op"] == "append":
        table, page, row = st["page_table"].tolist(), case["page"], 0
        for b, n in enumerate(lens):
            i = 0
            while i < n:
                pos = case["past"] + i
                take = min(n - i, page - pos % page)
                for new, pool in (("k", "k_pages"), ("v", "v_pages")):
                    there = st[pool][table[b][pos // page], :, pos % page:pos % page + take]
                    there.copy_(st[new][row:row + take].transpose(0, 1))
                i, row = i + take, row + take
        return dict(k_pages=st["k_pages"].double(), v_pages=st["v_pages"].double())
    G, W, cap = Hq // Hkv, case["window"], case["softcap"]

    def attend(q, k, v, sink, first):
        """Queries q [R, D] at positions first, first + 1, ... against k, v [C, D]: (o, lse)."""
        s = q @ k.T / math.sqrt(D)
        if cap:
            s = cap * torch.tanh(s / cap)
        back = first + torch.arange(len(q), device=q.device)[:, None] - torch.arange(len(k), device=q.device)[None, :]
        s = torch.where((back >= 0) & ((back < W) if W else True), s, -math.inf)
        if sink is not None:
            s = torch.cat([s, sink.expand(len(q), 1)], 1)
        lse = torch.logsumexp(s, 1)
        return torch.exp(s - lse[:, None])[:, :len(k)] @ v, lse

    sink = st["sink"].double() if "sink" in st else None
    if case["op"] == "decode":
        o = torch.zeros(len(lens), Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(len(lens), Hq, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            for h in range(Hkv):
                k, v = (st[x][st["page_table"][b].long(), h].flatten(0, 1)[:n].double() for x in ("k_pages", "v_pages"))
                for hq in range(h * G, (h + 1) * G):
                    a, c = attend(st["q"][b, hq:hq + 1].double(), k, v, None if sink is None else sink[hq], n - 1)
                    o[b, hq], lse[b, hq] = a[0], c[0]
        return dict(o=o, lse=lse)
    rows = st["q"].shape[0]
    train = case["op"] == "train"
    o = torch.zeros(rows, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, rows), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(o), *(torch.zeros(rows, Hkv, D, dtype=torch.float64, device="cuda") for _ in "kv")
    dsink = torch.zeros(Hq, dtype=torch.float64, device="cuda")
    row = 0
    for n in lens:
        here = slice(row, row + n)
        row += n
        for hq in range(Hq):
            h = hq // G
            leaves = [st["q"][here, hq], st["k"][here, h], st["v"][here, h]] + ([] if sink is None else [sink[hq]])
            leaves = [x.double().detach().requires_grad_(train) for x in leaves]
            a, c = attend(*leaves[:3], None if sink is None else leaves[3], 0)
            o[here, hq], lse[hq, here] = a.detach(), c.detach()
            if train:
                d = torch.autograd.grad(a, leaves, st["dO"][here, hq].double())
                dq[here, hq] = d[0]
                dk[here, h] += d[1]
                dv[here, h] += d[2]
                if sink is not None:
                    dsink[hq] += d[3]
    if not train:
        return dict(o=o, lse=lse)
    out = dict(o=o, dq=dq, dk=dk, dv=dv)
    if sink is not None:
        out["dsink"] = dsink
    return out
