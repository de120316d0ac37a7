"""Attention over packed sequences on the GPU, forward and backward, against the f64 oracle run on
each sequence by itself (the definition of the packed call). Tolerances are those of the other
parity tests (parity_util): 1e-4 for f32, 2e-2 + 1e-2 |ref| for bf16 with Delta from the bf16 o; where
many terms add up, the bf16 bar gives way to the sum of the roundings themselves (`roundings`)."""
import math

import numpy as np
import pytest
import torch

import causal_flash_attention_attn_b200 as fa
import oracle
from parity_util import check_close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}

EDGES = [0, 1, 127, 128, 129, 0, 255, 256, 257, 2, 385]
CASES = [
    # name, dtype, lens, pad, Hq, Hkv, D, window, softcap, sink, fused
    ("d128_edges", "bf16", EDGES, 0, 4, 2, 128, 0, 0.0, False, False),
    ("d128_fused_pad", "bf16", [300, 45, 130], 70, 14, 2, 128, 0, 0.0, False, True),
    ("d128_win_cap_sink", "bf16", [385, 3, 0, 260], 1, 4, 1, 128, 100, 5.0, True, True),
    ("d128_win1", "bf16", [130, 7], 0, 2, 2, 128, 1, 0.0, False, False),
    ("d128_long", "bf16", [2500, 60], 0, 2, 1, 128, 0, 0.0, False, False),
    ("d64_edges", "bf16", EDGES, 5, 3, 3, 64, 0, 0.0, True, False),
    ("d64_many_short", "bf16", [1 + 7 * i % 61 for i in range(150)], 0, 2, 1, 64, 0, 0.0, False, True),
    ("d64_win", "bf16", [700, 512, 90], 0, 6, 6, 64, 200, 0.0, False, False),
    ("d256_edges", "bf16", EDGES, 0, 2, 1, 256, 0, 0.0, False, False),
    ("d256_win_cap_sink", "bf16", [333, 64, 65], 9, 4, 2, 256, 150, 50.0, True, True),
    ("one_row", "bf16", [1], 0, 1, 1, 128, 0, 0.0, False, False),
    ("f32_d64_edges", "f32", [0, 1, 63, 64, 65, 130], 3, 4, 2, 64, 0, 0.0, True, True),
    ("f32_d128_win", "f32", [200, 31], 0, 4, 1, 128, 40, 0.0, False, False),
    ("f32_d256_cap", "f32", [100, 0, 33], 0, 2, 2, 256, 0, 5.0, False, False),
]


def make(dtype, lens, pad, Hq, Hkv, D, softcap, sink, fused, seed=0):
    g = torch.Generator().manual_seed(seed)
    rows, dt, sig = sum(lens) + pad, TDT[dtype], 2.0 if softcap else 1.0
    qkv = torch.randn(rows, Hq + 2 * Hkv, D, generator=g)
    qkv[:, :Hq + Hkv] *= sig
    qkv = qkv.to(dt).to(DEV)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    dO = torch.randn(rows, Hq, D, generator=g).to(dt).to(DEV)
    sk = torch.tensor(np.linspace(-0.5, 3.0, Hq), dtype=torch.float32, device=DEV) if sink else None
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    return q, k, v, dO, sk, cu


def raw(q, k, v, dO, sk, cu, W, C, clear, fill=float("nan"), res=False):
    """Both calls through the C ABI, outputs pre-filled, workspaces full of 0xFF; res: with o's residual."""
    rows, Hq, D = q.shape
    Hkv, n, dt, sc = k.shape[1], cu.numel() - 1, fa.dtype_code(q.dtype), 1.0 / math.sqrt(q.shape[2])

    def filled(*shape, dtype=q.dtype):
        return torch.full(shape, fill, dtype=dtype, device=DEV)
    o, lse = filled(rows, Hq, D), filled(Hq, rows, dtype=torch.float32)
    o_res = filled(rows, Hq, D) if res else None
    dq, dk, dv = filled(rows, Hq, D), filled(rows, Hkv, D), filled(rows, Hkv, D)
    ds = filled(Hq, dtype=torch.float32) if sk is not None else None
    st = (q.stride(0) if rows > 1 else Hq * D, *(x.stride(0) if rows > 1 else Hkv * D for x in (k, v)))
    for back in (False, True):
        size = fa.forge_attn_varlen_bwd_workspace_size if back else fa.forge_attn_varlen_fwd_workspace_size
        ws = torch.full((size(n, rows, Hq, Hkv, D, dt),), 255, dtype=torch.uint8, device=DEV)
        if back:
            s = fa.forge_attn_varlen_bwd(q, k, v, o, o_res, lse, dO, dq, dk, dv, cu, n, rows, Hq, Hkv, D, *st, sc, W, C,
                                         sk, ds, clear, dt, ws, ws.numel())
        else:
            s = fa.forge_attn_varlen_fwd(q, k, v, o, o_res, lse, cu, n, rows, Hq, Hkv, D, *st, sc, W, C, sk, clear, dt, ws,
                                         ws.numel())
        assert s == fa.FORGE_OK, fa.forge_attn_status_string(s)
    torch.cuda.synchronize()
    assert fa.forge_attn_check() == fa.FORGE_OK
    if res and dtype_is_bf16(q):  # hi + lo: what o's rounding lost is below half a unit of its last place
        total = int(cu[-1])
        assert bool((o_res[:total].float().abs() <= 2.0 ** -8 * o[:total].float().abs() + 1e-37).all())
    return o, lse, dq, dk, dv, ds


def dtype_is_bf16(x):
    return x.dtype == torch.bfloat16


def roundings(q, k, v, dO, sk, W, C):
    """Element-wise bounds on the bf16 call's error for one sequence ([T, H, D] tensors): a bf16 rounding
    is off by at most u = 2^-8 of the value, and the kernels round P and dS (scale included) before
    their products and each output once. With |.| the terms' absolute values,
      |err o|  <= u |o| + u sum_j P_ij |v_j|                                     (P)
      |err dv| <= u |dv| + u sum_i P_ij |dO_i|                                   (P)
      |err Delta_i| <= u sum_d |dO_id o_id|     (the reference's Delta is taken from o rounded to bf16; the
                       call's o is a rounding of a value that differs by the P term above)
                       + sum_d |dO_id| (u sum_j P_ij |v_jd| + u |o_id|)
      |err dS_ij| <= u |dS_ij| + scale P_ij t'_ij |err Delta_i|,  and dq, dk sum those against |k|, |q|,
    plus u of the output. f32 accumulation and the exponential (4e-6) are smaller by 2^-9 and are
    covered by the factor 1.05. Returns bounds for o, dq, dk, dv."""
    u, (T, Hq, D), Hkv = 2.0 ** -8, q.shape, k.shape[1]
    qh, kh, vh, dh = (x.double().transpose(0, 1) for x in (q, k, v, dO))
    kh, vh = (x.repeat_interleave(Hq // Hkv, 0) for x in (kh, vh))
    s = qh @ kh.transpose(1, 2) / math.sqrt(D)
    slope = torch.ones_like(s)
    if C:
        s = C * torch.tanh(s / C)
        slope = 1 - (s / C) ** 2
    i = torch.arange(T, device=q.device)
    see = (i[None] <= i[:, None]) & ((i[None] > i[:, None] - W) if W else True)
    s = s.masked_fill(~see, -math.inf)
    if sk is not None:
        s = torch.cat([s, sk.double()[:, None, None].expand(Hq, T, 1)], 2)
    p = torch.softmax(s, 2)[:, :, :T]
    o, pv = p @ vh, p @ vh.abs()
    ds = p * (dh @ vh.transpose(1, 2) - (dh * o).sum(2, keepdim=True)) * slope / math.sqrt(D)
    edelta = (dh.abs() * (2 * u * o.abs() + u * pv)).sum(2, keepdim=True)
    eds = u * ds.abs() + p * slope * edelta / math.sqrt(D)

    def group(x):
        return x.view(Hkv, Hq // Hkv, T, D).sum(1)
    bound = (u * o.abs() + u * pv, u * (ds @ kh).abs() + eds @ kh.abs(),
             u * group(ds.transpose(1, 2) @ qh).abs() + group(eds.transpose(1, 2) @ qh.abs()),
             u * group(p.transpose(1, 2) @ dh).abs() + u * group(p.transpose(1, 2) @ dh.abs()))
    return [1.05 * x.cpu().numpy() for x in bound]


def close(name, got, ref, dtype, bound):
    if dtype == "f32":
        return check_close(name, got, ref, dtype)
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), name
    err, tol = np.abs(got - ref), np.maximum(2e-2 + 1e-2 * np.abs(ref), bound)
    assert np.all(err <= tol), (name, float((err / tol).max()))


def compare(dtype, lens, q, k, v, dO, sk, W, C, got):
    o, lse, dq, dk, dv, ds = got
    Hq, D = q.shape[1:]
    sc, row = 1.0 / math.sqrt(D), 0
    rds, mag = np.zeros(Hq), np.zeros(Hq)
    host = None if sk is None else sk.cpu()
    for n in lens:
        if n == 0:
            continue
        at = slice(row, row + n)
        row += n
        qs, ks, vs, ds_ = (x[at].transpose(0, 1)[None].cpu() for x in (q, k, v, dO))
        ro, rl, _ = oracle.attn_fwd_ext(qs, ks, vs, sc, W, C, sink=host)
        rdq, rdk, rdv, rs, delta, rlse = oracle.attn_bwd_ext(qs, ks, vs, ds_, sc, W, C, sink=host, o_round=dtype)
        bounds = roundings(q[at], k[at], v[at], dO[at], sk, W, C) if dtype == "bf16" else [None] * 4
        for name, x, r, bound in zip(("o", "dq", "dk", "dv"), (o, dq, dk, dv), (ro, rdq, rdk, rdv), bounds):
            close(f"{name}[{at}]", x[at].transpose(0, 1), r[0], dtype, bound)
        check_close(f"lse[{at}]", lse[:, at][None].cpu(), rl, dtype)
        if sk is not None:
            rds += rs
            mag += np.abs(np.exp(host.double().numpy()[None, :, None] - rlse) * delta).sum(axis=(0, 2))
    if sk is not None:  # a sum of terms of both signs: the bar applies to their magnitude (test_ext_gpu.py)
        err = np.abs(ds.double().cpu().numpy() - rds)
        assert np.all(err <= (1e-4 * (1 + mag) if dtype == "f32" else 2e-2 + 1e-2 * mag)), (err, mag)


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_matches_oracle_per_sequence(case):
    _, dtype, lens, pad, Hq, Hkv, D, W, C, sink, fused = case
    q, k, v, dO, sk, cu = make(dtype, lens, pad, Hq, Hkv, D, C, sink, fused)
    total = sum(lens)
    if pad:  # rows behind the last sequence are not read
        for x in (q, k, v, dO):
            x[total:] = float("nan")
    got = raw(q, k, v, dO, sk, cu, W, C, clear=0)
    compare(dtype, lens, q, k, v, dO, sk, W, C, got)
    o, lse, dq, dk, dv, _ = got
    for x in (o, dq, dk, dv, lse.t()):  # ... and their outputs left as they were
        assert bool(torch.isnan(x[total:]).all())
    o, lse, dq, dk, dv, _ = raw(q, k, v, dO, sk, cu, W, C, clear=1)
    assert torch.equal(o[:total], got[0][:total]) and torch.equal(lse[:, :total], got[1][:, :total])
    assert torch.equal(dk[:total], got[3][:total]) and torch.equal(dv[:total], got[4][:total])
    for x in (o, dq, dk, dv):
        assert not bool(x[total:].any())
    assert bool((lse[:, total:] == -math.inf).all())


@pytest.mark.parametrize("case", [c for c in CASES if c[1] == "bf16"], ids=[c[0] for c in CASES if c[1] == "bf16"])
def test_the_residual_of_o_takes_its_rounding_out_of_the_gradients(case):
    """With o_res, Delta lacks o's rounding: dq and dk against the exact gradient, in the 2-norm. What is left is
    the rounding of dS (at most u = 2^-8 of each term: u |dS| |K| in the 2-norm of independent roundings) and of
    the outputs (u): 2 u relative, where the plain Delta may exceed it many times over (peaked rows). The
    residual's own rounding leaves |err Delta_i| <= u^2 sum_d |dO_id o_id|, which reaches dq_i times
    scale max |k| and dk times scale max |q| (`floor`, summed over the rows: all there is where the exact
    gradient is 0, as in rows that see one key)."""
    _, dtype, lens, pad, Hq, Hkv, D, W, C, sink, fused = case
    q, k, v, dO, sk, cu = make(dtype, lens, pad, Hq, Hkv, D, C, sink, fused)
    got = raw(q, k, v, dO, sk, cu, W, C, clear=0, res=True)
    if not sink:  # (with a sink the forward also splits P)
        plain = raw(q, k, v, dO, sk, cu, W, C, clear=0)
        assert torch.equal(got[0][:sum(lens)], plain[0][:sum(lens)])
        assert torch.equal(got[1][:, :sum(lens)], plain[1][:, :sum(lens)])
    host, row, off, floor = None if sk is None else sk.cpu(), 0, np.zeros((2, 2)), np.zeros(2)
    want, room = np.zeros(Hq), np.zeros(Hq)
    for n in lens:
        at = slice(row, row + n)
        row += n
        if n == 0:
            continue
        ref = oracle.attn_bwd_ext(*(x[at].transpose(0, 1)[None].cpu() for x in (q, k, v, dO)), 1.0 / math.sqrt(D), W, C,
                                  sink=host, o_round=None)
        part = 2.0 ** -16 / math.sqrt(D) * float((dO[at].double() * got[0][at].double()).abs().sum())
        if sink:
            # Delta = sum_d dO_d (o + o_res)_d: P in two terms and o in two terms leave 2 * 2^-17 of each
            # product |P| |dP| and |dO_d o_d|; tanh (1e-7 of the cap, 50 at most) and the f32
            # exponent (lse up to ~20, 2^-24 of it) move P by less than 8e-6. Each row's dsink term is
            # exp(sink - lse) Delta, summed.
            ps = np.exp(host.double().numpy()[None, :, None] - ref[5])
            qh, kh, vh, dh = (x[at].double().transpose(0, 1).cpu() for x in (q, k, v, dO))
            mag = (dh.abs() @ vh.abs().repeat_interleave(Hq // Hkv, 0).transpose(1, 2)).amax(2).numpy()
            want, room = want + ref[3], room + ((2 * 2.0 ** -17 + 8e-6) * ps[0] * mag).sum(1)
        floor += [part * float(x[at].double().norm(dim=2).max()) for x in (k, q)]
        for i in (0, 1):
            x = got[2 + i][at].transpose(0, 1).double().cpu().numpy()
            off[i] += ((x - ref[i][0]) ** 2).sum(), (ref[i][0] ** 2).sum()
    for i in (0, 1):
        err, size = np.sqrt(off[i])
        print(f"{case[0]} {'dq dk'.split()[i]}: {err / max(size, 1e-30):.2e} of its norm")
        assert err <= 2 * 2.0 ** -8 * size + floor[i], (i, err, size, floor[i])
    if sink:
        err = np.abs(got[5].double().cpu().numpy() - want)
        print(f"{case[0]} dsink: {np.linalg.norm(err) / np.linalg.norm(want):.2e} of its norm")
        assert np.all(err <= room), (err, room)


@pytest.mark.parametrize("dtype,D,Hq,Hkv", [("bf16", 128, 4, 2), ("bf16", 64, 3, 3), ("bf16", 256, 2, 1),
                                             ("f32", 64, 2, 1)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -3.0e38])
def test_one_sequences_values_stay_in_it(dtype, D, Hq, Hkv, poison):
    lens = [100, 200, 61, 300, 5]
    q, k, v, dO, _, cu = make(dtype, lens, 0, Hq, Hkv, D, 0.0, False, False)
    clean = raw(q, k, v, dO, None, cu, 0, 0.0, 0)
    rest = torch.ones(sum(lens), dtype=torch.bool, device=DEV)
    for b in (1, 3):  # between clean sequences whose tiles run into them
        rest[int(cu[b]):int(cu[b + 1])] = False
        for x in (q, k, v, dO):
            x[int(cu[b]):int(cu[b + 1])] = poison
    o, lse, dq, dk, dv, _ = raw(q, k, v, dO, None, cu, 0, 0.0, 0)
    assert torch.equal(o[rest], clean[0][rest]) and torch.equal(lse[:, rest], clean[1][:, rest])
    assert torch.equal(dk[rest], clean[3][rest]) and torch.equal(dv[rest], clean[4][rest])
    if dtype == "f32":
        assert torch.equal(dq[rest], clean[2][rest])
    else:  # f32 atomics in any order, then one rounding
        check_close("dq", dq[rest], clean[2][rest].double().cpu().numpy(), dtype)


@pytest.mark.parametrize("D,T", [(128, 700), (64, 512), (256, 300)])
def test_equal_lengths_give_the_dense_call(D, T):
    B, Hq, Hkv = 3, 4, 2
    q, k, v, dO, _, cu = make("bf16", [T] * B, 0, Hq, Hkv, D, 0.0, False, False)
    o, lse, dq, dk, dv, _ = raw(q, k, v, dO, None, cu, 0, 0.0, 0)

    def dense(x):
        return x.view(B, T, -1, D).transpose(1, 2).contiguous()
    do, dl = fa.attention_fwd(dense(q), dense(k), dense(v))
    ddq, ddk, ddv = fa.attention_bwd(dense(q), dense(k), dense(v), do, dl, dense(dO))
    # the packed forward at head dims 64 and 128 splits a tile's columns between two warps, which take
    # another exponential where only one half is masked; the packed backward may cut a key
    # tile's queries into parts, whose sums then add up in another order
    if D == 256:
        assert torch.equal(dense(o), do) and torch.equal(lse.view(Hq, B, T).transpose(0, 1), dl)
    check_close("o", dense(o), do.double().cpu().numpy(), "bf16")
    check_close("lse", lse.view(Hq, B, T).transpose(0, 1), dl.double().cpu().numpy(), "bf16")
    check_close("dk", dense(dk), ddk.double().cpu().numpy(), "bf16")
    check_close("dv", dense(dv), ddv.double().cpu().numpy(), "bf16")
    check_close("dq", dense(dq), ddq.double().cpu().numpy(), "bf16")


def test_window_of_the_longest_sequence_is_no_window():
    lens = [200, 90]
    q, k, v, dO, _, cu = make("bf16", lens, 0, 2, 1, 128, 0.0, False, False)
    a, b = raw(q, k, v, dO, None, cu, 0, 0.0, 0), raw(q, k, v, dO, None, cu, 1 << 30, 0.0, 0)
    c = raw(q, k, v, dO, None, cu, 200, 0.0, 0)
    for i in (0, 1, 3, 4):
        assert torch.equal(a[i], b[i]) and torch.equal(a[i], c[i])


@pytest.mark.parametrize("cu", [[1, 5, 10], [0, 6, 4, 10], [0, 5, 11], [0, -1, 10], [0, 10, 0, 10]])
def test_bad_lengths_are_reported_and_nothing_is_computed(cu):
    q, k, v, dO, _, _ = make("bf16", [10], 0, 2, 1, 128, 0.0, False, False)
    bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
    n, sc, dt = len(cu) - 1, 0.1, fa.FORGE_DTYPE_BF16
    o, lse = torch.full_like(q, 7.0), torch.full((2, 10), 7.0, device=DEV)
    ws = torch.empty(fa.forge_attn_varlen_fwd_workspace_size(n, 10, 2, 1, 128, dt), dtype=torch.uint8, device=DEV)
    assert fa.forge_attn_varlen_fwd(q, k, v, o, None, lse, bad, n, 10, 2, 1, 128, 256, 128, 128, sc, 0, 0.0, None, 0, dt, ws,
                                    ws.numel()) == fa.FORGE_OK
    assert fa.forge_attn_check() == fa.FORGE_ERR_INVALID_ARG and fa.forge_attn_check() == fa.FORGE_OK
    assert bool((o == 7.0).all()) and bool((lse == 7.0).all())
    dq, dk, dv = (torch.full_like(x, 7.0) for x in (q, k, v))
    ws = torch.empty(fa.forge_attn_varlen_bwd_workspace_size(n, 10, 2, 1, 128, dt), dtype=torch.uint8, device=DEV)
    assert fa.forge_attn_varlen_bwd(q, k, v, o, None, lse, dO, dq, dk, dv, bad, n, 10, 2, 1, 128, 256, 128, 128, sc, 0,
                                    0.0, None, None, 0, dt, ws, ws.numel()) == fa.FORGE_OK
    assert fa.forge_attn_check() == fa.FORGE_ERR_INVALID_ARG
    assert all(bool((x == 7.0).all()) for x in (dq, dk, dv))


def test_all_lengths_zero():
    q, k, v, dO, _, _ = make("bf16", [4], 0, 2, 1, 64, 0.0, False, False)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    o, lse = fa.attention_varlen_fwd(q, k, v, cu)
    assert not bool(o.any()) and bool((lse == -math.inf).all())
    assert all(not bool(x.any()) for x in fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu))
    assert fa.forge_attn_check() == fa.FORGE_OK


def test_more_sequences_than_the_schedule_holds_at_once():
    lens = [(i * 7) % 5 for i in range(2500)]
    q, k, v, dO, _, cu = make("bf16", lens, 0, 2, 1, 64, 0.0, False, False)
    compare("bf16", lens, q, k, v, dO, None, 0, 0.0, raw(q, k, v, dO, None, cu, 0, 0.0, 0))


def test_autograd_gradients_match_the_formula_and_differences():
    # f32: the library's gradient of sum(o * c) against f64 autograd of the definition and against
    # central differences; a step h has a truncation error ~h^2 and a rounding error ~eps |f| / h
    lens, Hq, Hkv, D, W, C = [30, 0, 70], 4, 2, 64, 20, 5.0
    q, k, v, c, sk, cu = make("f32", lens, 2, Hq, Hkv, D, 0.0, True, True)
    leaves = [x.clone().requires_grad_() for x in (q, k, v, sk)]
    o = fa.attention_varlen(*leaves[:3], cu, window=W, softcap=C, sink=leaves[3])
    grads = torch.autograd.grad(o, leaves, c.transpose(0, 1).contiguous().transpose(0, 1))  # a strided dO

    def definition(q, k, v, sk):
        out, row = torch.zeros_like(q), 0
        for n in lens:
            i = torch.arange(n, device=DEV)
            see = (i[None] <= i[:, None]) & (i[None] > i[:, None] - W)
            for h in range(Hq):
                s = C * torch.tanh(q[row:row + n, h] @ k[row:row + n, h // 2].T / math.sqrt(D) / C)
                s = torch.cat([s.masked_fill(~see, -math.inf), sk[h].expand(n, 1)], 1)
                out[row:row + n, h] = torch.softmax(s, 1)[:, :n] @ v[row:row + n, h // 2]
            row += n
        return out
    wide = [x.detach().double().requires_grad_() for x in leaves]
    for name, a, b in zip(("q", "k", "v", "sink"), grads, torch.autograd.grad(definition(*wide), wide, c.double())):
        check_close("d" + name, a, b.cpu().numpy(), "f32")
    h, g = 1e-4, torch.Generator(device=DEV).manual_seed(1)
    with torch.no_grad():
        for i, a in enumerate(grads):
            d = torch.randn(a.shape, generator=g, device=DEV, dtype=torch.float64)
            up, down = ([x + (s * h * d if j == i else 0) for j, x in enumerate(wide)] for s in (1, -1))
            diff = float(((definition(*up) - definition(*down)) * c.double()).sum() / (2 * h))
            got, size = float((a.double() * d).sum()), float((a.double().abs() * d.abs()).sum())
            assert abs(got - diff) <= 1e-4 * size + 1e-4, (i, got, diff)


def test_gradients_of_shared_heads_and_repeated_inputs():
    # k and v the same tensor, broadcast over query heads: both gradients land in one leaf
    q, k, _, dO, _, cu = make("f32", [50, 21], 0, 4, 1, 64, 0.0, False, False)
    x = k.clone().requires_grad_()
    (g,) = torch.autograd.grad(fa.attention_varlen(q, x, x, cu), x, dO)
    o, lse = fa.attention_varlen_fwd(q, k, k, cu)
    _, dk, dv = fa.attention_varlen_bwd(q, k, k, o, lse, dO, cu)
    assert torch.equal(g, dk + dv)


def test_captured_calls_follow_the_lengths():
    lens_a, lens_b = [100, 300, 112], [257, 1, 200]
    q, k, v, dO, _, cu = make("bf16", lens_a, 0, 4, 2, 128, 0.0, False, False)
    rows = 512

    def step():
        o, lse = fa.attention_varlen_fwd(q, k, v, cu)
        return (o, lse, *fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):  # two graphs, each with workspaces of its own pool
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for lens in (lens_a, lens_b):
        cu.copy_(torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32))
        want = step()
        for graph, out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        total = sum(lens)
        for graph, out in graphs:
            for i in (0, 3, 4):
                assert torch.equal(out[i], want[i]), i
            assert torch.equal(out[1], want[1])
            check_close("dq", out[2][:total], want[2][:total].double().cpu().numpy(), "bf16")
        assert total <= rows
    assert fa.forge_attn_check() == fa.FORGE_OK


def test_calls_on_two_streams_at_once():
    sets = [make("bf16", lens, 0, 4, 2, 128, 0.0, False, False, seed=i)
            for i, lens in enumerate(([900, 100], [33] * 20, [1200], [400, 1, 400]))]
    want = [fa.attention_varlen_fwd(q, k, v, cu) for q, k, v, dO, _, cu in sets]
    grads = [fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu) for (q, k, v, dO, _, cu), (o, lse) in zip(sets, want)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for _ in range(3):
        for s, (q, k, v, dO, _, cu) in zip(streams, sets):
            # one by the argument, one by the current stream, one by the raw handle
            o, lse = fa.attention_varlen_fwd(q, k, v, cu, stream=s)
            with torch.cuda.stream(s):
                got.append((o, lse, *fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu, stream=s.cuda_stream)))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        (o, lse), (dq, dk, dv) = want[i % 4], grads[i % 4]
        assert torch.equal(x[0], o) and torch.equal(x[1], lse) and torch.equal(x[3], dk) and torch.equal(x[4], dv)
    assert fa.forge_attn_check() == fa.FORGE_OK


def test_a_gradient_that_starts_anywhere_and_no_second_derivative():
    # o behind a single element: its gradient is a dense part of the whole one's, 2 bytes off
    q, k, v, dO, _, cu = make("bf16", [70, 33], 0, 4, 2, 64, 0.0, False, False)
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    one = torch.zeros(1, dtype=q.dtype, device=DEV)
    both = torch.cat([one, fa.attention_varlen(*x, cu).flatten()])
    got = torch.autograd.grad(both, x, torch.cat([one, dO.flatten()]))
    o, lse, o_res = fa.attention_varlen_fwd(q, k, v, cu, return_residual=True)
    want = fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu, o_res=o_res)
    check_close("dq", got[0], want[0].double().cpu().numpy(), "bf16")
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    g = torch.autograd.grad(fa.attention_varlen(*x, cu).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g[0].float().sum().backward()


def test_captured_autograd_step():
    q, k, v, dO, _, cu = make("bf16", [200, 1, 155], 0, 4, 2, 128, 0.0, False, False)
    x = [t.clone().requires_grad_() for t in (q, k, v)]

    def step():
        o = fa.attention_varlen(*x, cu, window=90)
        o.backward(dO)
        return o.detach()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t in x:
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for t, new in zip(x, (0.5 * q, k + 1, -v)):
        t.data.copy_(new)
        t.grad.zero_()  # the captured pass wrote its gradient here and adds nothing on a replay
    graph.replay()
    torch.cuda.synchronize()
    o, lse, o_res = fa.attention_varlen_fwd(*[t.detach() for t in x], cu, window=90, return_residual=True)
    want = fa.attention_varlen_bwd(*[t.detach() for t in x], o, lse, dO, cu, window=90, o_res=o_res)
    assert torch.equal(out, o)
    check_close("dq", x[0].grad, want[0].double().cpu().numpy(), "bf16")
    assert torch.equal(x[1].grad, want[1]) and torch.equal(x[2].grad, want[2])


def test_a_backward_that_takes_longer_than_a_wait_may():
    """2^20 rows of one sequence: about three seconds, with no tile that a sequence's end cuts, whose
    rows two warps of every CTA stand by to clear. Compared on the first 128 rows (which see only
    one another) and on the last 128 keys (which only the last 128 queries see), with the bounds of
    `roundings`: u of each term for P and dS and u for the output. lse is the call's (f32, up to ~20 in
    log2 units: P within 1e-5 of its value, u = 4e-3), and so is Delta, from o + o_res (u^2)."""
    T, n, Hq, D, u = 1 << 20, 128, 4, 128, 2.0 ** -8
    g = torch.Generator(device=DEV).manual_seed(2)
    q, dO = (torch.randn(T, Hq, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(T, 1, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    o, lse, o_res = fa.attention_varlen_fwd(q, k, v, cu, return_residual=True)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    dq, dk, dv = fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu, o_res=o_res)
    end.record()
    assert fa.forge_attn_check() == fa.FORGE_OK
    print(f"backward {start.elapsed_time(end) / 1e3:.2f} s")
    assert all(bool(torch.isfinite(x).all()) for x in (o, dq, dk, dv, lse))
    for at, names in ((slice(0, n), ("o", "dq")), (slice(T - n, T), ("dk", "dv"))):
        qh, dh = (x[at].double().transpose(0, 1) for x in (q, dO))
        kh, vh = (x[at].double().transpose(0, 1) for x in (k, v))
        p = (qh @ kh.transpose(1, 2) / math.sqrt(D) - lse[:, at].double()[:, :, None]).exp().tril()
        whole = (o[at].double() + o_res[at].double()).transpose(0, 1)
        ds = p * (dh @ vh.transpose(1, 2) - (dh * whole).sum(2, keepdim=True)) / math.sqrt(D)
        eds = u * ds.abs() + p * u * u * (dh * whole).abs().sum(2, keepdim=True) / math.sqrt(D)
        pt, dst = p.transpose(1, 2), ds.transpose(1, 2)
        want = dict(o=(o, p @ vh, p @ vh.abs()), dq=(dq, ds @ kh, eds @ kh.abs() / u),
                    dk=(dk, (dst @ qh).sum(0, True), (eds.transpose(1, 2) @ qh.abs()).sum(0, True) / u),
                    dv=(dv, (pt @ dh).sum(0, True), (pt @ dh.abs()).sum(0, True)))
        for name in names:
            got, ref, terms = want[name]
            err = (got[at].double().transpose(0, 1) - ref).abs()
            tol = 1.05 * u * (ref.abs() + terms) + 1e-30
            assert bool((err <= tol).all()), (name, float((err / tol).max()))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 3), (128, 4, 2), (256, 2, 1)])
@pytest.mark.parametrize("W,sink", [(0, False), (70, True)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -3.0e38, 300.0])
def test_one_sequences_values_stay_in_it_with_a_cap(D, Hq, Hkv, W, sink, poison):
    # a capped score takes one of two forms of the tanh (1e-7 apart), by its size and its
    # neighbours' in the tile: only scores of its own sequence may have a say
    lens = [100, 200, 61, 300, 5]
    q, k, v, dO, sk, cu = make("bf16", lens, 9, Hq, Hkv, D, 0.0, sink, False)
    clean = raw(q, k, v, dO, sk, cu, W, 50.0, 0, res=True)
    rest = torch.ones(sum(lens) + 9, dtype=torch.bool, device=DEV)
    rest[sum(lens):] = False
    for b in (1, 3):
        rest[int(cu[b]):int(cu[b + 1])] = False
    for x in (q, k, v, dO):
        x[~rest] = poison
    o, lse, dq, dk, dv, _ = raw_unchecked(q, k, v, dO, sk, cu, W, 50.0)
    assert torch.equal(o[rest], clean[0][rest]) and torch.equal(lse[:, rest], clean[1][:, rest])
    assert torch.equal(dk[rest], clean[3][rest]) and torch.equal(dv[rest], clean[4][rest])
    check_close("dq", dq[rest], clean[2][rest].double().cpu().numpy(), "bf16")


def raw_unchecked(q, k, v, dO, sk, cu, W, C):
    """As raw(.., res=True), through the helpers and without its check of o_res (poisoned rows have none)."""
    o, lse, o_res = fa.attention_varlen_fwd(q, k, v, cu, window=W, softcap=C, sink=sk, return_residual=True)
    g = fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu, window=W, softcap=C, sink=sk, o_res=o_res)
    torch.cuda.synchronize()
    assert fa.forge_attn_check() == fa.FORGE_OK
    return (o, lse, *g[:3], None)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 3), (128, 4, 2), (256, 2, 1)])
def test_without_grad_mode_the_call_is_the_plain_forward(D, Hq, Hkv):
    q, k, v, _, sk, cu = make("bf16", [130, 300, 7], 0, Hq, Hkv, D, 0.0, True, False)
    x = [t.clone().requires_grad_() for t in (q, k, v, sk)]
    want = fa.attention_varlen_fwd(q, k, v, cu, window=90, sink=sk)[0]
    for scope in (torch.no_grad, torch.inference_mode):
        with scope():
            o = fa.attention_varlen(*x[:3], cu, window=90, sink=x[3])
        assert not o.requires_grad and torch.equal(o, want)
    o = fa.attention_varlen(q, k, v, cu, window=90, sink=sk)
    assert not o.requires_grad and torch.equal(o, want)


@pytest.mark.parametrize("W,C", [(0, 0.0), (90, 50.0)])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 3), (128, 4, 2), (256, 2, 1)])
def test_a_sink_that_is_not_trained(D, Hq, Hkv, W, C):
    # the forward is the plain one (P in one term: its bits), the other gradients are those of the same
    # o, lse and residual, and no dsink is formed
    q, k, v, dO, sk, cu = make("bf16", [130, 300, 7], 5, Hq, Hkv, D, C, True, False)
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    o = fa.attention_varlen(*x, cu, window=W, softcap=C, sink=sk)
    got = torch.autograd.grad(o, x, dO)
    assert torch.equal(o, fa.attention_varlen_fwd(q, k, v, cu, window=W, softcap=C, sink=sk)[0])
    o, lse, o_res = fa.attention_varlen_fwd(q, k, v, cu, window=W, softcap=C, sink=sk, return_residual=True,
                                            sink_fixed=True)
    want = fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu, window=W, softcap=C, o_res=o_res)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    check_close("dq", got[0], want[0].double().cpu().numpy(), "bf16")
    assert not bool(o[-5:].any())  # the rows behind the last sequence are cleared as ever
    # a trained sink alone: the split forward, and its gradient
    s = sk.clone().requires_grad_()
    (ds,) = torch.autograd.grad(fa.attention_varlen(q, k, v, cu, window=W, softcap=C, sink=s), s, dO)
    o, lse, o_res = fa.attention_varlen_fwd(q, k, v, cu, window=W, softcap=C, sink=sk, return_residual=True)
    assert torch.equal(ds, fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu, window=W, softcap=C, sink=sk, o_res=o_res)[3])
    assert fa.forge_attn_check() == fa.FORGE_OK


@pytest.mark.parametrize("with_sink", [False, True])
def test_training_without_the_residual(with_sink):
    # the backward gets no o_res (the plain call's gradients), and the graph keeps one tensor of o's size less
    q, k, v, dO, sk, cu = make("bf16", [700, 300], 0, 8, 2, 128, 0.0, with_sink, False)
    x = [t.clone().requires_grad_() for t in (q, k, v, sk) if t is not None]
    held = []
    for residual in (True, False):
        # (counted on the graph: the allocator's figures depend on the blocks that earlier tests left)
        o = fa.attention_varlen(*x[:3], cu, sink=x[3] if with_sink else None, residual=residual)
        held.append(sum(t.numel() * t.element_size() for t in o.grad_fn.saved_tensors if t is not None))
    assert held[0] - held[1] == o.numel() * 2
    got = torch.autograd.grad(o, x, dO)
    po, lse = fa.attention_varlen_fwd(q, k, v, cu, sink=sk)
    want = fa.attention_varlen_bwd(q, k, v, po, lse, dO, cu, sink=sk)
    assert torch.equal(o, po) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    check_close("dq", got[0], want[0].double().cpu().numpy(), "bf16")
    if with_sink:
        assert torch.equal(got[3], want[3])
    assert fa.forge_attn_check() == fa.FORGE_OK


# every compiled variant of the bf16 kernels that the cases above leave out: with and without a cap (scores of
# standard deviation 4: a cap of 5 takes the exponential tanh, 50 the polynomial one), a window and a sink
VARIANTS = [
    ("d64_cap", "bf16", [300, 1, 129, 64], 3, 4, 2, 64, 0, 5.0, False, True),
    ("d64_cap50", "bf16", [257, 128, 40], 0, 3, 3, 64, 0, 50.0, False, False),
    ("d64_win_cap", "bf16", [385, 31, 200], 0, 4, 1, 64, 77, 50.0, False, True),
    ("d64_cap_sink", "bf16", [300, 0, 129], 0, 4, 2, 64, 0, 5.0, True, False),
    ("d64_win_cap_sink", "bf16", [300, 65], 2, 4, 2, 64, 90, 50.0, True, False),
    ("d64_win_sink", "bf16", [300, 65], 2, 4, 2, 64, 90, 0.0, True, False),
    ("d128_cap", "bf16", [300, 1, 129, 64], 3, 4, 2, 128, 0, 5.0, False, True),
    ("d128_cap50", "bf16", [513, 128, 40], 0, 3, 3, 128, 0, 50.0, False, False),
    ("d128_win_cap", "bf16", [385, 31, 200], 0, 4, 1, 128, 77, 50.0, False, True),
    ("d128_sink", "bf16", [300, 0, 129, 600], 0, 4, 2, 128, 0, 0.0, True, False),
    ("d128_win_sink", "bf16", [300, 65], 2, 7, 1, 128, 90, 0.0, True, False),
    ("d128_cap_sink", "bf16", [300, 130], 0, 4, 2, 128, 0, 50.0, True, False),
    ("d256_cap", "bf16", [300, 129, 64], 3, 4, 2, 256, 0, 5.0, False, True),
    ("d256_win", "bf16", [300, 129, 64], 0, 2, 2, 256, 100, 0.0, False, False),
    ("d256_sink", "bf16", [300, 0, 129], 0, 4, 2, 256, 0, 0.0, True, False),
    ("f32_d64_win_cap_sink", "f32", [150, 0, 65], 3, 4, 2, 64, 40, 50.0, True, True),
    ("f32_d128_cap_sink", "f32", [150, 33], 0, 4, 1, 128, 0, 5.0, True, False),
]


@pytest.mark.parametrize("case", VARIANTS, ids=[c[0] for c in VARIANTS])
def test_variants_match_oracle_per_sequence(case):
    test_matches_oracle_per_sequence(case)


@pytest.mark.parametrize("case", [c for c in VARIANTS if c[1] == "bf16"], ids=[c[0] for c in VARIANTS if c[1] == "bf16"])
def test_variants_with_the_residual(case):
    test_the_residual_of_o_takes_its_rounding_out_of_the_gradients(case)


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 32, 2, 128), ("bf16", 64, 1, 64), ("bf16", 16, 1, 256), ("f32", 64, 1, 64)])
def test_rows_whose_offsets_pass_32_bits(dtype, Hq, Hkv, D):
    # q, o, dO and dq of more than 2^32 elements, in 8200 short sequences: the last ones are what they are in
    # a call of their own, bit for bit, but for dk and dv (bf16) of the one of 300 rows: its first key tile has
    # three query tiles, and in the small call, where a CTA's share is less than that, it is cut into parts
    # (of two tiles at least, so that no other one is), whose sums add up in another order before they are rounded
    lens = [128] * 8190 + [77, 128, 1, 300, 129, 64, 0, 200, 33, 128]
    total = sum(lens)
    tail = sum(lens[8190:])
    assert total * Hq * D > 1 << 32
    g = torch.Generator(device=DEV).manual_seed(4)
    q, dO = (torch.randn(total, Hq, D, generator=g, device=DEV, dtype=TDT[dtype]) for _ in range(2))
    k, v = (torch.randn(total, Hkv, D, generator=g, device=DEV, dtype=TDT[dtype]) for _ in range(2))
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)

    def both(q, k, v, dO, cu):
        o, lse, o_res = fa.attention_varlen_fwd(q, k, v, cu, return_residual=True)
        return (o, lse.t(), *fa.attention_varlen_bwd(q, k, v, o, lse, dO, cu, o_res=o_res))
    got = [x[-tail:].clone() for x in both(q, k, v, dO, cu)]
    assert fa.forge_attn_check() == fa.FORGE_OK
    q, k, v, dO = (x[-tail:].clone() for x in (q, k, v, dO))
    torch.cuda.empty_cache()
    want = both(q, k, v, dO, (cu[8190:] - cu[8190]).contiguous())
    at = torch.ones(tail, dtype=torch.bool, device=DEV)
    at[77 + 128 + 1:][:300] = dtype == "f32"
    for i in (0, 1, 3, 4) if dtype == "bf16" else range(5):
        rows = slice(None) if i < 2 else at
        assert torch.equal(got[i][rows], want[i][rows]), i
        check_close(str(i), got[i], want[i].double().cpu().numpy(), dtype)
    check_close("dq", got[2], want[2].double().cpu().numpy(), dtype)
