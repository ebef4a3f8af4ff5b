"""GPU parity of the mixture-of-experts operators against the fp64 oracle, through the C ABI.

Tolerances, per element, derived from the arithmetic:
  * a tensor-core sum of K products errs by at most K * 2^-23 * S, S = sum |a_i b_i| (every add truncates
    to 24 bits; the number of adds is at most K);
  * an activation passes an input error d on as at most 1.2 d (GeLU and SiLU have slopes below 1.13;
    the derivatives, applied to an exact h_pre, do not see it) and adds a few binary32 roundings of its
    own: 2^-18 of |h| covers __expf's (2 + 1.2 |x|) * 2^-23 for |x| <= 24, erff and tanhf;
  * one rounding to bf16 is off by at most 2^-8 of the value, to fp32 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import synthetic as S
import tensor_sharded_matmul_b200 as tp
from gpu_util import f64
from oracle import mlp as OM
from oracle import moe as M

pytestmark = pytest.mark.gpu

ACT = {"none": tp.TP_ACT_NONE, "gelu": tp.TP_ACT_GELU, "gelu_tanh": tp.TP_ACT_GELU_TANH, "swiglu": tp.TP_ACT_SWIGLU}
GATE = {"softmax": tp.TP_GATE_SOFTMAX, "topk": tp.TP_GATE_TOPK}
DT = {"f32": (tp.TP_F32, torch.float32, 2.0 ** -24), "bf16": (tp.TP_BF16, torch.bfloat16, 2.0 ** -8)}
MARK = 123.0     # what untouched outputs hold


def dev(x, dtype=None):
    t = x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))
    return t.to("cuda", dtype) if dtype else t.to("cuda")


def settled():
    torch.cuda.synchronize()
    st, site = tp.tp_device_status(1)
    assert st == tp.TP_OK, f"device wait site {site}"


def within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}: "
                           f"{got[bad][0]} for {ref[bad][0]}, allowed {np.broadcast_to(bound, ref.shape)[bad][0]}")


def plan_of(counts, N, seed, tail=0):
    """Segments of the given row counts over random tokens, `tail` rows behind the last."""
    r = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1]) + tail
    return off, r.integers(0, N, R).astype(np.int32), R


# ------------------------------------------------------------------ router
def _route(logits, k, gate, dtype):
    N, E = logits.shape
    l = dev(logits, DT[dtype][1])
    o = dict(expert=torch.full((N, k), -9, dtype=torch.int32, device="cuda"), weight=torch.full((N, k), MARK, device="cuda"),
             slot=torch.full((N, k), -9, dtype=torch.int32, device="cuda"),
             offsets=torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"),
             row_token=torch.full((N * k,), -9, dtype=torch.int32, device="cuda"))
    nb = tp.tp_moe_route_ws_bytes(N, E, k)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    tp.tp_moe_route(l, DT[dtype][0], N, E, k, GATE[gate], o["expert"], o["weight"], o["slot"], o["offsets"], o["row_token"], ws, nb)
    settled()
    return l, o


def _logits(N, E, seed, dtype):
    r = np.random.default_rng(seed)
    v = torch.from_numpy(2 * r.standard_normal((N, E))).to(DT[dtype][1])      # bf16: ties are common
    if N > 3:
        v[N // 2, : E // 2] = -math.inf
        v[N - 1] = -math.inf                      # nothing left
        v[N - 2, 0] = math.nan
        v[N - 3, E - 1] = math.inf
        v[1] = 0.5                                # all tied
    return v


@pytest.mark.parametrize("gate", ["softmax", "topk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,E,k", [(1, 1, 1), (1, 64, 8), (5, 8, 2), (64, 33, 6), (65, 64, 6), (200, 130, 16), (1000, 257, 8),
                                   (129, 1024, 4), (2500, 8, 8)])
def test_route(N, E, k, gate, dtype):
    v = _logits(N, E, N + E, dtype)
    l, o = _route(v, k, gate, dtype)
    vv = f64(v)
    ref = M.route(vv, k, gate)
    for name in ("expert", "slot", "offsets"):
        assert np.array_equal(o[name].cpu().numpy(), ref[name]), name
    rows = int(ref["offsets"][-1])
    got = o["row_token"].cpu().numpy()
    assert np.array_equal(got[:rows], ref["row_token"]) and (got[rows:] == -9).all()
    # exp of a difference d in binary32: 2^-24 |d| from d's rounding, expf's 2 units; sums of E/32 + 5 adds; a division
    clean = np.where(np.isfinite(vv), vv, 0.0)
    span = np.minimum(clean.max(1) - clean.min(1), 110.0)[:, None]
    within(f64(o["weight"]), ref["weight"], ref["weight"] * (span + E / 32 + 24) * 2.0 ** -23 + 1e-38, "weight")
    # gradient; dweight of choices that are -1 must not matter
    dw = np.random.default_rng(N).standard_normal((N, k)).astype(np.float32)
    dw[ref["expert"] < 0] = np.nan
    dl = torch.full((N, E), MARK, dtype=l.dtype, device="cuda")
    tp.tp_moe_route_bwd(l, DT[dtype][0], N, E, k, GATE[gate], o["expert"], dev(dw), dl)
    settled()
    g = M.route_backward(vv, ref["expert"], np.nan_to_num(dw).astype(np.float64), gate)
    q = M.gate_softmax(vv, ref["expert"], gate)
    size = q * (np.abs(np.nan_to_num(dw)).max(1, keepdims=True) * 2)          # both terms of the difference
    within(f64(dl), g, size * (span + E / 16 + 32) * 2.0 ** -22 + DT[dtype][2] * np.abs(g) + 1e-38, "dlogits")


# ------------------------------------------------------------------ products
def _products_ref(x, idx, off, R, w, act):
    h = M.ragged_products(x, idx, off, R, w)
    S_ = M.ragged_products(np.abs(x), idx, off, R, np.abs(w))
    return h, S_, OM.activate(h, act)


COUNTS = {
    "one row": [0, 0, 1, 0], "one each": [1] * 5, "ragged": [3, 0, 17, 64, 65, 1], "empty": [0, 0, 0],
    "long": [300, 0, 257, 40], "very long": [700, 1, 129], "many": [i % 7 for i in range(100)],
}


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("counts,K,n", [
    ("one row", 64, 128), ("one each", 8, 8), ("ragged", 200, 136), ("empty", 64, 64), ("long", 136, 72), ("very long", 72, 264),
    ("many", 104, 40), ("ragged", 1160, 200), ("one row", 2056, 64),
])
def test_ragged_linear(counts, K, n, act):
    c = COUNTS[counts]
    E, N, wide = len(c), 50, 2 if act == "swiglu" else 1
    off, idx, R = plan_of(c, N, K + n, tail=5)
    d = S.Draw(K + n)
    x, w = d.normal((N, K), 1.0), d.normal((E, K, wide * n), 1.0 / math.sqrt(K))
    idx[off[-1]:] = 1 << 30                      # behind the last: never used
    h, size, ref = _products_ref(f64(x), idx, off, R, f64(w), act)
    used = ~np.isnan(ref[:, 0])
    dh = K * 2.0 ** -23 * size
    if act == "swiglu":
        g, u, dg, du = h[:, :n], h[:, n:], dh[:, :n], dh[:, n:]
        slack = 1.2 * dg * (np.abs(u) + du) + np.abs(OM.silu(g)) * du + 2.0 ** -18 * np.abs(g) * (np.abs(u) + du)
    else:
        slack = dh if act == "none" else 1.2 * dh + 2.0 ** -18 * np.abs(h)
    for out in ("bf16", "f32"):
        tpd, td, eps = DT[out]
        y = torch.full((R, n), MARK, dtype=td, device="cuda")
        pre = torch.full((R, wide * n), MARK, dtype=torch.bfloat16, device="cuda") if act != "none" else None
        tp.tp_ragged_linear(dev(x), N, dev(idx), dev(off), R, E, K, n, ACT[act], dev(w), y, tpd, pre)
        settled()
        got = f64(y)
        within(got[used], ref[used], (slack + eps * (np.abs(ref) + slack))[used] + 1e-37, f"{counts} {out}")
        assert (got[~used] == MARK).all()
        if pre is not None:
            got = f64(pre)
            within(got[used], h[used], (dh + 2.0 ** -8 * (np.abs(h) + dh))[used], f"{counts} pre")
            assert (got[~used] == MARK).all()


def test_ragged_linear_without_index_and_strange_offsets():
    """Rows of x itself; offsets that leave the buffer, run backwards or start late are taken as clamped, and rows of no
    segment (NaN here) reach no result."""
    E, K, n, R = 4, 72, 88, 90
    d = S.Draw(5)
    x, w = d.normal((R, K), 1.0), d.normal((E, K, n), 0.1)
    for off in ([7, 30, 30, 77, 80], [-5, 10, 4, 60, 1000], [90, 90, 90, 90, 90], [1 << 30] * 5):
        off = np.array(off, np.int32)
        owners = np.zeros(R, int)
        for a, b in M.segments(off, R):
            owners[a:b] += 1
        inside, once = owners > 0, owners == 1          # an element of two segments (forbidden) is either's product
        xx = x.clone()
        xx[torch.from_numpy(~inside)] = math.nan
        y = torch.full((R, n), MARK, device="cuda")
        tp.tp_ragged_linear(dev(xx), R, None, dev(off), R, E, K, n, tp.TP_ACT_NONE, dev(w), y, tp.TP_F32)
        settled()
        ref = M.ragged_products(f64(x), None, off, R, f64(w))
        size = M.ragged_products(np.abs(f64(x)), None, off, R, np.abs(f64(w)))
        got = f64(y)
        within(got[once], ref[once], ((K + 1) * 2.0 ** -23 * size)[once], str(off))
        for i in np.flatnonzero(owners > 1):
            at = [M.segments([a, b], R)[0] for a, b in zip(off[:-1], off[1:])]
            each = [f64(x)[i] @ f64(w)[e] for e, (a, b) in enumerate(at) if a <= i < b]
            assert (np.min([np.abs(got[i] - r) for r in each], axis=0) < 1e-3).all()
        assert (got[~inside] == MARK).all()


def test_rows_outside_x_read_as_zeros():
    E, K, n, N = 3, 64, 72, 20
    off, idx, R = plan_of([40, 3, 100], N, 1)
    idx[[0, 5, 41, 60, 142]] = [-1, N, 1 << 30, -(1 << 31), N + 7]
    d = S.Draw(6)
    x, w = d.normal((N, K), 1.0), d.normal((E, K, n), 0.1)
    dy = d.normal((R, n), 1.0)
    y = torch.full((R, n), MARK, device="cuda")
    tp.tp_ragged_linear(dev(x), N, dev(idx), dev(off), R, E, K, n, tp.TP_ACT_NONE, dev(w), y, tp.TP_F32)
    dw = torch.full((E, K, n), MARK, device="cuda")
    tp.tp_ragged_linear_dw(dev(x), N, dev(idx), dev(dy), dev(off), R, E, K, n, dw, tp.TP_F32)
    settled()
    within(f64(y), M.ragged_products(f64(x), idx, off, R, f64(w)),
           (K + 1) * 2.0 ** -23 * M.ragged_products(np.abs(f64(x)), idx, off, R, np.abs(f64(w))) + 1e-38, "y")
    assert (f64(y)[[0, 5, 41, 60, 142]] == 0).all()
    within(f64(dw), M.ragged_linear_dw(f64(x), idx, f64(dy), off, R, E),
           100 * 2.0 ** -23 * M.ragged_linear_dw(np.abs(f64(x)), idx, np.abs(f64(dy)), off, R, E) + 1e-38, "dw")


def test_infinities_stay_in_their_own_rows():
    """An infinity or NaN in one row of x changes that row alone, also inside the same tile."""
    E, K, n, N = 2, 128, 136, 30
    off, idx, R = plan_of([20, 9], N, 3)
    idx[:] = np.arange(R)
    d = S.Draw(7)
    x, w = d.normal((N, K), 1.0), d.normal((E, K, n), 0.1)
    clean = M.ragged_products(f64(x), idx, off, R, f64(w))
    size = M.ragged_products(np.abs(f64(x)), idx, off, R, np.abs(f64(w)))
    x[4, 7], x[25, 100] = math.inf, math.nan
    y = torch.full((R, n), MARK, device="cuda")
    tp.tp_ragged_linear(dev(x), N, dev(idx), dev(off), R, E, K, n, tp.TP_ACT_NONE, dev(w), y, tp.TP_F32)
    settled()
    got = f64(y)
    keep = [i for i in range(R) if i not in (4, 25)]
    within(got[keep], clean[keep], ((K + 1) * 2.0 ** -23 * size)[keep], "other rows")
    assert not np.isfinite(got[4]).any() and np.isnan(got[25]).all()


@pytest.mark.parametrize("act,out,counts,K,n", [
    ("swiglu", "bf16", [1300, 0, 1, 2211, 700, 500], 2056, 4400), ("none", "f32", [4000, 5000, 6500], 2056, 4104),
    ("gelu", "bf16", [4600, 500, 5000], 2048, 4352), ("swiglu", "f32", [3, 300, 260], 136, 2048)])
def test_gathered_rows_that_are_put_side_by_side(act, out, counts, K, n):
    """Wide products of many gathered rows copy them to the end of y's own rows first. Results are those of rows
    that the caller put side by side, bit for bit, and the formula's; rows in front of the segments and behind them
    are left as they were."""
    d = S.Draw(len(counts), "cuda")
    N, front, tail = 3000, 5, 7
    E, wide = len(counts), 2 * n if act == "swiglu" else n
    off = front + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1]) + tail
    idx = torch.from_numpy(np.random.default_rng(R).integers(0, N, R).astype(np.int32))
    idx[front], idx[R - tail - 1], idx[front + 1] = -1, N, idx[front + 2]
    x, w = d.normal((N, K)), d.normal((E, K, wide), 1 / math.sqrt(K))
    dt, tt, eps = DT[out]
    outside = (idx < 0) | (idx >= N)
    rows = torch.where(outside[:, None].cuda(), torch.zeros((), dtype=x.dtype, device="cuda"), x[idx.clamp(0, N - 1).long().cuda()])
    ys, pres = [], []
    for gathered in (True, False):
        y = torch.full((R, n), MARK, dtype=tt, device="cuda")
        pre = torch.full((R, wide), MARK, dtype=torch.bfloat16, device="cuda") if act != "none" else None
        tp.tp_ragged_linear(x if gathered else rows, N if gathered else R, dev(idx) if gathered else None, dev(off), R, E, K, n,
                            ACT[act], w, y, dt, pre)
        settled()
        ys.append(y), pres.append(pre)
    assert torch.equal(ys[0], ys[1])
    assert act == "none" or torch.equal(pres[0], pres[1])
    for keep in (slice(0, front), slice(R - tail, R)):
        assert (ys[0][keep] == MARK).all()
    for e in range(E):
        part = slice(int(off[e]), int(off[e + 1]))
        a, b = rows[part].double(), w[e].double()
        h, size = a @ b, a.abs() @ b.abs() * K * 2.0 ** -23
        if act == "swiglu":
            g, u = h[:, :n], h[:, n:]
            s = g * torch.sigmoid(g)
            ref = s * u
            slack = 1.2 * size[:, :n] * (u.abs() + size[:, n:]) + (s.abs() + 2.0 ** -18 * g.abs()) * size[:, n:] + 2.0 ** -18 * (g * u).abs()
        elif act == "gelu":
            ref, slack = 0.5 * h * (1 + torch.erf(h / math.sqrt(2))), 1.2 * size + 2.0 ** -18 * h.abs()
        else:
            ref, slack = h, size
        assert bool(((ys[0][part].double() - ref).abs() <= slack + eps * (ref.abs() + slack)).all()), e


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("counts,k,n", [("ragged", 136, 200), ("one row", 64, 2056), ("long", 72, 136), ("very long", 264, 72),
                                        ("many", 40, 104), ("one each", 8, 8)])
def test_ragged_linear_dx(counts, k, n, act):
    c = COUNTS[counts]
    E, wide = len(c), 2 if act == "swiglu" else 1
    off, _, R = plan_of(c, 1, k, tail=3)
    d = S.Draw(k * n)
    dy, w, hp = d.normal((R, n), 1.0), d.normal((E, k, n), 1.0 / math.sqrt(n)), d.normal((R, wide * k), 1.0)
    dy[off[-1]:] = math.nan
    dx = torch.full((R, wide * k), MARK, dtype=torch.bfloat16, device="cuda")
    tp.tp_ragged_linear_dx(dev(dy), dev(off), R, E, k, n, dev(w), ACT[act], dev(hp) if act != "none" else None, dx)
    settled()
    ref = M.ragged_linear_dx(f64(dy), off, R, f64(w), act, f64(hp))
    dz = n * 2.0 ** -23 * M.ragged_products(np.abs(f64(dy)), None, off, R, np.abs(np.swapaxes(f64(w), 1, 2)))
    dz2 = dz + 2.0 ** -18 * np.abs(M.ragged_products(f64(dy), None, off, R, np.swapaxes(f64(w), 1, 2)))
    if act == "swiglu":
        g, u = np.abs(f64(hp)[:, :k]), np.abs(f64(hp)[:, k:])
        slack = np.concatenate([1.2 * dz2 * u, dz2 * g], 1)
    else:
        slack = dz if act == "none" else 1.2 * dz2
    used = np.arange(R) < off[-1]
    got = f64(dx)
    within(got[used], ref[used], (slack + 2.0 ** -8 * (np.abs(ref) + slack))[used] + 1e-37, counts)
    assert (got[~used] == MARK).all()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,k,n", [("ragged", 136, 200), ("one row", 64, 2056), ("long", 72, 136), ("very long", 264, 520),
                                        ("many", 40, 104), ("one each", 8, 8), ("empty", 64, 64)])
def test_ragged_linear_dw(counts, k, n, out, gather):
    c = COUNTS[counts]
    E, N = len(c), 40
    off, idx, R = plan_of(c, N, k, tail=3)
    d = S.Draw(k + n)
    x, dy = d.normal((N if gather else R, k), 1.0), d.normal((R, n), 1.0)
    dy[off[-1]:] = math.nan
    if not gather:
        x[off[-1]:] = math.nan
        idx = None
    dw = torch.full((E, k, n), MARK, dtype=DT[out][1], device="cuda")
    tp.tp_ragged_linear_dw(dev(x), x.shape[0], dev(idx) if gather else None, dev(dy), dev(off), R, E, k, n, dw, DT[out][0])
    settled()
    ref = M.ragged_linear_dw(f64(x), idx, f64(dy), off, R, E)
    size = M.ragged_linear_dw(np.abs(f64(x)), idx, np.abs(f64(dy)), off, R, E)
    K = max(c) if max(c) < 512 else 512 + 4        # spans of 512 rows, then round-to-nearest adds
    slack = K * 2.0 ** -23 * size
    within(f64(dw), ref, slack + DT[out][2] * (np.abs(ref) + slack), counts)


def test_no_rows_at_all():
    dw = torch.full((3, 16, 24), MARK, device="cuda")
    off = dev(np.zeros(4, np.int32))
    tp.tp_ragged_linear_dw(None, 0, None, None, off, 0, 3, 16, 24, dw, tp.TP_F32)
    settled()
    assert (dw == 0).all()


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("ud", ["bf16", "f32"])
@pytest.mark.parametrize("yd", ["bf16", "f32"])
@pytest.mark.parametrize("N,k,h", [(1, 1, 8), (3, 2, 72), (70, 6, 264), (40, 16, 2056), (9, 3, 4096)])
def test_combine_and_gradient(N, k, h, ud, yd):
    r = np.random.default_rng(N * k)
    R = N * k + 3
    slot = r.permutation(R)[: N * k].reshape(N, k).astype(np.int32)
    slot[0, 0] = -1 if N > 1 else slot[0, 0]
    if N > 2:
        slot[1, k - 1], slot[2] = R + 5, -1
    d = S.Draw(N)
    u, dy = d.normal((R, h), 1.0, DT[ud][1]), d.normal((N, h), 1.0, DT[yd][1])
    w = r.standard_normal((N, k)).astype(np.float32)
    for weight in (w, None):
        y = torch.full((N, h), MARK, dtype=DT[yd][1], device="cuda")
        tp.tp_moe_combine(dev(u), DT[ud][0], R, None if weight is None else dev(weight), dev(slot), N, h, k, y, DT[yd][0])
        settled()
        ref = M.combine(f64(u), weight, slot)
        size = M.combine(np.abs(f64(u)), None if weight is None else np.abs(weight), slot) * (k + 1) * 2.0 ** -24
        within(f64(y), ref, size + DT[yd][2] * (np.abs(ref) + size) + 1e-38, "y")
    du = torch.full((R, h), MARK, dtype=torch.bfloat16, device="cuda")
    dwt = torch.full((N, k), MARK, device="cuda")
    tp.tp_moe_combine_bwd(dev(dy), DT[yd][0], dev(u), DT[ud][0], R, dev(w), dev(slot), N, h, k, du, dwt)
    settled()
    rdu, rdw = M.combine_backward(f64(dy), f64(u), w, slot)
    named = ~np.isnan(rdu[:, 0])
    within(f64(du)[named], rdu[named], (2.0 ** -8 + 2.0 ** -23) * np.abs(rdu[named]) + 1e-38, "du")
    assert (f64(du)[~named] == MARK).all()
    _, size = M.combine_backward(np.abs(f64(dy)), np.abs(f64(u)), np.abs(w), slot)
    within(f64(dwt), rdw, (h / 32 + 8) * 2.0 ** -24 * size + 1e-38, "dweight")


# ------------------------------------------------------------------ the MLP, as it is used
def _mlp(N, h, F, E, k, act, gate, seed, masked=0, stream=None):
    d = S.Draw(seed)
    wide = 2 if act == "swiglu" else 1
    b = dict(x=d.normal((N, h), 1.0), logits=d.normal((N, E), 1.0, torch.float32),
             w_in=d.normal((E, h, wide * F), 1.0 / math.sqrt(h)), w_down=d.normal((E, F, h), 1.0 / math.sqrt(F)),
             dy=d.normal((N, h), 1.0))
    if masked:
        b["logits"][N - masked:] = -math.inf
    host = {n: v for n, v in b.items()}
    b = {n: dev(v) for n, v in b.items()}
    R = N * k
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    b.update(expert=torch.zeros((N, k), **i32), weight=torch.zeros((N, k), device="cuda"), slot=torch.zeros((N, k), **i32),
             offsets=torch.zeros(E + 1, **i32), row_token=torch.zeros(R, **i32), h_pre=torch.zeros((R, wide * F), **bf),
             z=torch.zeros((R, F), **bf), u=torch.zeros((R, h), **bf), y=torch.zeros((N, h), device="cuda"),
             du=torch.zeros((R, h), **bf), dh=torch.zeros((R, wide * F), **bf), dweight=torch.zeros((N, k), device="cuda"),
             dw_in=torch.zeros((E, h, wide * F), device="cuda"), dw_down=torch.zeros((E, F, h), device="cuda"),
             dx=torch.zeros((N, h), device="cuda"), dlogits=torch.zeros((N, E), device="cuda"))
    nb = tp.tp_moe_mlp_ws_bytes(N, E, k)
    b["ws"] = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def forward(stream=None):
        tp.tp_moe_mlp_fwd(b["x"], N, h, F, E, k, GATE[gate], ACT[act], b["logits"], tp.TP_F32, b["w_in"], b["w_down"], b["expert"],
                          b["weight"], b["slot"], b["offsets"], b["row_token"], None if act == "none" else b["h_pre"], b["z"],
                          b["u"], b["y"], tp.TP_F32, b["ws"], nb, stream)

    def backward(stream=None):
        tp.tp_moe_mlp_bwd(b["x"], b["dy"], N, h, F, E, k, GATE[gate], ACT[act], b["logits"], tp.TP_F32, b["w_in"], b["w_down"],
                          b["expert"], b["weight"], b["slot"], b["offsets"], b["row_token"], None if act == "none" else b["h_pre"],
                          b["z"], b["u"], b["du"], b["dh"], b["dweight"], b["dw_in"], b["dw_down"], b["dx"], tp.TP_F32,
                          b["dlogits"], stream)
    return b, host, forward, backward


def rel(got, ref):
    return float(np.linalg.norm(f64(got) - ref) / max(np.linalg.norm(ref), 1e-30))


@pytest.mark.parametrize("N,h,F,E,k,act,gate,masked", [
    (1, 64, 128, 8, 2, "swiglu", "topk", 0),           # one token
    (33, 136, 72, 4, 2, "gelu", "softmax", 5),
    (300, 128, 200, 3, 2, "swiglu", "softmax", 0),     # long segments
    (150, 72, 64, 40, 6, "gelu_tanh", "topk", 20),
    (90, 64, 64, 5, 1, "none", "softmax", 90),         # every token masked
])
def test_mlp_forward_and_backward(N, h, F, E, k, act, gate, masked):
    """The whole MLP and its gradients. The intermediates z, u, du, dh and the rows of dx are rounded to bf16, a
    relative error of at most 2^-8 an element each and on average (uniform in half a step) about 2^-9.3;
    at most five of them, independent, lie on the way to an output, and softmax's dlogits subtract two
    such sums: 2-norm errors stay below 5 * 2^-8 of the output's norm."""
    b, host, forward, backward = _mlp(N, h, F, E, k, act, gate, seed=N + E, masked=masked)
    forward()
    backward()
    settled()
    ref = M.moe_mlp_backward(f64(host["x"]), f64(host["logits"]), f64(host["w_in"]), f64(host["w_down"]), k, gate, act, f64(host["dy"]))
    assert np.array_equal(b["expert"].cpu().numpy(), ref["expert"]) and np.array_equal(b["offsets"].cpu().numpy(), ref["offsets"])
    rows = len(ref["row_token"])
    assert rel(b["z"][:rows], ref["z"]) < 2.0 ** -8
    for name in ("y", "dx", "dw_in", "dw_down", "dweight"):
        assert rel(b[name], ref[name]) < 5 * 2.0 ** -8, name
    if not (gate == "topk" and k == 1):
        assert np.linalg.norm(f64(b["dlogits"]) - ref["dlogits"]) < 5 * 2.0 ** -8 * np.linalg.norm(
            M.gate_softmax(f64(host["logits"]), ref["expert"], gate) * np.abs(ref["dweight"]).max(initial=0) + 1e-30)


def test_mlp_of_many_rows_an_expert():
    """The composite puts gathered rows side by side in buffers that it does not need at that moment; its results are
    those of the operators called one by one on the rows' indices, bit for bit."""
    N, h, F, E, k = 2100, 512, 2048, 4, 2
    b, host, forward, backward = _mlp(N, h, F, E, k, "swiglu", "topk", seed=5, masked=11)
    R = N * k
    forward()
    backward()
    settled()
    d = {n: dev(host[n]) for n in ("x", "dy", "w_in", "w_down")}
    z, u, du = (torch.zeros((R, m), dtype=torch.bfloat16, device="cuda") for m in (F, h, h))
    pre, dh = (torch.zeros((R, 2 * F), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dweight = torch.zeros((N, k), device="cuda")
    dw_in = torch.zeros((E, h, 2 * F), device="cuda")
    tp.tp_ragged_linear(d["x"], N, b["row_token"], b["offsets"], R, E, h, F, tp.TP_ACT_SWIGLU, d["w_in"], z, tp.TP_BF16, pre)
    tp.tp_ragged_linear(z, R, None, b["offsets"], R, E, F, h, tp.TP_ACT_NONE, d["w_down"], u, tp.TP_BF16, None)
    tp.tp_moe_combine_bwd(d["dy"], tp.TP_BF16, u, tp.TP_BF16, R, b["weight"], b["slot"], N, h, k, du, dweight)
    tp.tp_ragged_linear_dx(du, b["offsets"], R, E, F, h, d["w_down"], tp.TP_ACT_SWIGLU, pre, dh)
    tp.tp_ragged_linear_dw(d["x"], N, b["row_token"], dh, b["offsets"], R, E, h, 2 * F, dw_in, tp.TP_F32)
    settled()
    rows = int(b["offsets"][-1])
    assert rows == R - 11 * k
    for name, got in (("z", z), ("u", u)):
        assert torch.equal(b[name][:rows], got[:rows]), name
    assert torch.equal(b["dw_in"], dw_in)


def test_a_captured_step_replays_on_new_routings():
    """Forward and backward captured once; new inputs in the same buffers, other segment sizes, other streams: the
    replay gives what the eager calls give, bit for bit, and two runs of either are the same."""
    b, _, forward, backward = _mlp(200, 136, 128, 8, 2, "swiglu", "topk", seed=11, masked=9)
    names = ("y", "dx", "dw_in", "dw_down", "dlogits", "weight", "offsets")
    forward(), backward()
    settled()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        forward(), backward()
    for seed in (21, 22):
        new, _, _, _ = _mlp(200, 136, 128, 8, 2, "swiglu", "topk", seed=seed, masked=seed - 15)
        b["x"].copy_(new["x"]), b["logits"].copy_(new["logits"]), b["dy"].copy_(new["dy"])
        g.replay()
        settled()
        first = {n: b[n].clone() for n in names}
        g.replay()
        settled()
        assert all(torch.equal(first[n], b[n]) for n in names)
        for n in names:
            b[n].fill_(7)
        with torch.cuda.stream(side):
            forward(), backward()
        settled()
        assert all(torch.equal(first[n], b[n]) for n in names)


def test_two_streams_at_once():
    """Two MLPs with their own buffers, interleaved on two streams, do not disturb each other."""
    runs = [_mlp(120 + 40 * i, 128, 96, 6, 2, "swiglu", "topk", seed=i) for i in range(2)]
    want = []
    for b, _, forward, backward in runs:
        forward(), backward()
        settled()
        want.append({n: b[n].clone() for n in ("y", "dx", "dw_in")})
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for s, (_, _, forward, backward) in zip(streams, runs):
            forward(s), backward(s)
    settled()
    for (b, _, _, _), w in zip(runs, want):
        assert all(torch.equal(b[n], w[n]) for n in w)


# ------------------------------------------------------------------ adapters
def _lora_case(N, k, n, t, L, rank, ids, seed, scale=True):
    d = S.Draw(seed)
    x, w = d.normal((N, k), 1.0), d.normal((t, k, n // t), 1.0 / math.sqrt(k))
    a, b = d.normal((L, k, rank), 1.0 / math.sqrt(k)), d.normal((t, L, rank, n // t), 0.5)
    sc = d.uniform((L,), 0.5, 1.5) if scale else None
    off = torch.full((L + 1,), -9, dtype=torch.int32, device="cuda")
    tok = torch.full((N,), -9, dtype=torch.int32, device="cuda")
    nb = tp.tp_lora_plan_ws_bytes(N, L)
    tp.tp_lora_plan(dev(ids), N, L, off, tok, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    ro, rt, _ = M.sort_rows(ids[:, None], L, rest=True)
    settled()
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(tok.cpu().numpy(), rt)
    y = torch.full((t, N, n // t), MARK, dtype=torch.bfloat16, device="cuda")
    nb = tp.tp_lora_ws_bytes(N, rank)
    ws = torch.full((nb // 4,), math.nan, device="cuda")
    tp.tp_lora_linear(dev(x), N, k, n, t, dev(w), L, rank, dev(a), dev(b), dev(sc) if scale else None, off, tok, y, ws, nb)
    settled()
    X, W, A, B = f64(x), f64(w), f64(a), f64(b)
    SC = None if sc is None else f64(sc)
    ref = M.lora(X, W, A, B, SC, ids)
    # v = x A: K adds; split into two bf16: 2^-16; then one sum of k + 2 rank products
    size = M.lora(np.abs(X), np.abs(W), np.abs(A), np.abs(B), SC, ids)
    slack = size * ((2 * k + 2 * rank) * 2.0 ** -23 + 2.0 ** -16)
    within(f64(y), ref, slack + 2.0 ** -8 * (np.abs(ref) + slack), "y")


@pytest.mark.parametrize("N,k,n,t,L,rank", [
    (1, 64, 128, 1, 1, 8), (1, 4096, 256, 2, 4, 16), (7, 136, 72, 1, 3, 24), (64, 264, 512, 4, 32, 16), (65, 200, 400, 2, 70, 8),
    (300, 128, 272, 1, 5, 64), (500, 72, 64, 8, 2, 128), (130, 64, 136, 1, 1024, 16),
    # pairs (tiles of 256 tokens by 256 columns that fill half of the GPU): partial tiles, an odd number of k-blocks
    # (a stage of x and v), few and very many adapters in a tile
    (600, 72, 3584, 16, 3, 24), (520, 136, 4160, 8, 200, 8), (1000, 512, 4096, 8, 1, 128), (257, 1160, 5120, 8, 4, 40),
    # few tokens: x A token by token (ranks that end inside sixteen, every adapter or one, very long contractions), and
    # the sizes from which it is a product
    (1, 4104, 128, 1, 1, 40), (5, 9000, 64, 1, 1024, 8), (64, 1000, 136, 1, 64, 32), (64, 2056, 128, 1, 1, 48), (64, 4096, 72, 1, 2, 24),
    (3, 200, 64, 1, 2, 264),
    # tiles of 192 and of 224 tokens
    (1152, 72, 16384, 16, 8, 16), (4000, 136, 6144, 8, 30, 24),
])
def test_lora(N, k, n, t, L, rank):
    ids = np.random.default_rng(N + L).integers(-1, L + (N > 5), N).astype(np.int32)     # L itself: no adapter
    _lora_case(N, k, n, t, L, rank, ids, N + k, scale=N % 2 == 1)


@pytest.mark.parametrize("ids", ["none", "all one", "last alone"])
def test_lora_uneven_batches(ids):
    N, L = 290, 6
    v = {"none": np.full(N, -1), "all one": np.full(N, 3), "last alone": np.r_[np.full(N - 1, -1), 5]}[ids].astype(np.int32)
    _lora_case(N, 136, 200, 1, L, 40, v, 9)


def test_lora_infinite_values_stay_with_their_token():
    """An infinite x row makes its own outputs non-finite and no other token's."""
    N, k, n, L, rank = 40, 64, 136, 2, 16
    d = S.Draw(3)
    x, w = d.normal((N, k), 1.0), d.normal((1, k, n), 0.1)
    a, b = d.normal((L, k, rank), 0.1), d.normal((1, L, rank, n), 0.5)
    ids = (np.arange(N) % 2).astype(np.int32)
    off, tok, _ = M.sort_rows(ids[:, None], L, rest=True)
    ref = M.lora(f64(x), f64(w), f64(a), f64(b), None, ids)
    size = M.lora(np.abs(f64(x)), np.abs(f64(w)), np.abs(f64(a)), np.abs(f64(b)), None, ids)[0]
    x[8, 3] = math.inf
    y = torch.full((1, N, n), MARK, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(N * rank, device="cuda")
    tp.tp_lora_linear(dev(x), N, k, n, 1, dev(w), L, rank, dev(a), dev(b), None, dev(off), dev(tok), y, ws, N * rank * 4)
    settled()
    got, keep = f64(y)[0], [i for i in range(N) if i != 8]
    assert not np.isfinite(got[8]).any()
    slack = size * ((2 * k + 2 * rank) * 2.0 ** -23 + 2.0 ** -16)
    within(got[keep], ref[0][keep], (slack + 2.0 ** -8 * (np.abs(ref[0]) + slack))[keep], "other tokens")


@pytest.mark.parametrize("N,n,t", [(3, 128, 1), (40, 272, 2), (130, 264, 1), (600, 3584, 16)])
def test_lora_infinities_of_an_adapter_stay_with_its_tokens(N, n, t):
    """An infinity and a NaN in one adapter's B reach its own tokens as the formula says, and no other token of
    the tile that they share; neither does a row of x that is all NaN."""
    k, L, rank = 72, 3, 24
    d = S.Draw(N)
    x, w = d.normal((N, k), 1.0), d.normal((t, k, n // t), 0.1)
    a, b = d.normal((L, k, rank), 0.1), d.normal((t, L, rank, n // t), 0.5)
    ids = ((np.arange(N) * 7 + 1) % (L + 1) - 1).astype(np.int32)
    assert ids[0] == 0 and (N < 40 or ids[1] == -1)
    size = M.lora(np.abs(f64(x)), np.abs(f64(w)), np.abs(f64(a)), np.abs(f64(b)), None, ids)
    b[0, 0, 5, 9] = math.inf
    b[t - 1, 0, rank - 1, 0] = math.nan
    x[1] = math.nan
    with np.errstate(invalid="ignore"):
        ref = M.lora(f64(x), f64(w), f64(a), f64(b), None, ids)
    off, tok, _ = M.sort_rows(ids[:, None], L, rest=True)
    y = torch.full((t, N, n // t), MARK, dtype=torch.bfloat16, device="cuda")
    nb = tp.tp_lora_ws_bytes(N, rank)
    ws = torch.full((nb // 4,), math.nan, device="cuda")
    tp.tp_lora_linear(dev(x), N, k, n, t, dev(w), L, rank, dev(a), dev(b), None, dev(off), dev(tok), y, ws, nb)
    settled()
    got, good = f64(y), np.isfinite(ref)
    own = ids == 0
    own[1] = True
    assert good[:, ~own].all() and not good.all()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    slack = size * ((2 * k + 2 * rank) * 2.0 ** -23 + 2.0 ** -16)
    within(got[good], ref[good], (slack + 2.0 ** -8 * (np.abs(ref) + slack))[good], "finite")


@pytest.mark.parametrize("N,n", [(1, 1024), (3, 1024), (40, 1024), (64, 1024), (100, 1024), (700, 6144)])
def test_lora_calls_back_to_back(N, n):
    """Many calls on one stream with nothing between them (each kernel begins beside the one before it), over several
    sets of buffers: every result is the one of a call by itself, bit for bit, and no wait runs out."""
    k, t, L, rank = 2048, 2, 4, 16
    nb = tp.tp_lora_ws_bytes(N, rank)
    sets = []
    for seed in range(3):
        d = S.Draw(seed, "cuda")
        ids = torch.randint(-1, L, (N,), generator=d.gen, device="cuda", dtype=torch.int32)
        off, tok, _ = M.sort_rows(ids.cpu().numpy()[:, None], L, rest=True)
        sets.append(dict(x=d.normal((N, k)), w=d.normal((t, k, n // t), 0.02), a=d.normal((L, k, rank), 0.02),
                         b=d.normal((t, L, rank, n // t), 0.5), off=dev(off), tok=dev(tok),
                         ws=torch.empty(nb // 4, device="cuda"), y=torch.zeros((t, N, n // t), dtype=torch.bfloat16, device="cuda")))

    def call(s):
        tp.tp_lora_linear(s["x"], N, k, n, t, s["w"], L, rank, s["a"], s["b"], None, s["off"], s["tok"], s["y"], s["ws"], nb)

    want = []
    for s in sets:
        call(s)
        settled()
        want.append(s["y"].clone())
        s["y"].zero_()
    for i in range(90):
        call(sets[i % 3])
    settled()
    for s, w in zip(sets, want):
        assert torch.equal(s["y"], w)


@pytest.mark.parametrize("rows", [1, 20, 64, 300])
def test_products_back_to_back(rows):
    """The same of the expert products: up (gathered), down, gradient, a chain of calls that read each other's
    outputs."""
    E, k, n = 4, 1024, 512
    d = S.Draw(rows, "cuda")
    off, idx, R = plan_of([rows] * E, 64, rows)
    off, idx = dev(off), dev(idx)
    x, w1, w2 = d.normal((64, k)), d.normal((E, k, 2 * n), 0.03), d.normal((E, n, k), 0.03)
    z, u = (torch.zeros((R, m), dtype=torch.bfloat16, device="cuda") for m in (n, k))
    pre, dh = (torch.zeros((R, 2 * n), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def chain(check=lambda: None):
        tp.tp_ragged_linear(x, 64, idx, off, R, E, k, n, tp.TP_ACT_SWIGLU, w1, z, tp.TP_BF16, pre)
        check()
        tp.tp_ragged_linear(z, R, None, off, R, E, n, k, tp.TP_ACT_NONE, w2, u, tp.TP_BF16)
        check()
        tp.tp_ragged_linear_dx(u, off, R, E, n, k, w2, tp.TP_ACT_SWIGLU, pre, dh)
        check()

    chain(settled)
    want = [v.clone() for v in (z, u, dh)]
    for _ in range(40):
        chain()
    settled()
    assert all(torch.equal(a, b) for a, b in zip((z, u, dh), want))
