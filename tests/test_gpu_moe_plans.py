"""Segments and row lists that the plans of this library do not make but its entry points take: the result is the
formula's, and does not depend on which kernel the sizes lead to."""
import math

import numpy as np
import pytest
import torch

import synthetic as S
import tensor_sharded_matmul_b200 as tp
from gpu_util import f64
from oracle import moe as M
from test_gpu_moe import MARK, dev, settled, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["backwards", "once back", "clamped", "late"])
@pytest.mark.parametrize("N,n,t", [(5, 128, 1), (40, 272, 2), (130, 264, 1), (600, 3584, 16), (1000, 4096, 8)])
def test_lora_with_a_callers_own_plan(N, n, t, form):
    """Segments of adapters in any order, disjoint; some tokens that no row names, and rows that name no token."""
    k, L, rank = 136, 4, 24
    off = np.array({"backwards": [N // 2, N, 0, N // 4, N // 4],      # the second ends before it begins: empty
                    "once back": [0, 5, 3, 3, 3], "clamped": [-7, 1, 1, N + 9, 1 << 30], "late": [N] * 5}[form], np.int32)
    d = S.Draw(N)
    x, w = d.normal((N, k), 1.0), d.normal((t, k, n // t), 0.1)
    a, b, sc = d.normal((L, k, rank), 0.1), d.normal((t, L, rank, n // t), 0.5), d.uniform((L,), 0.5, 1.5)
    tok = np.random.default_rng(N).permutation(N).astype(np.int32)
    unnamed = np.zeros(N, bool)
    for i, v in ((3, -1), (N - 1, N + 3)):
        unnamed[tok[i]] = True
        tok[i] = v
    ids = np.full(N, -1)
    for e, (lo, hi) in enumerate(M.segments(off, N)):
        named = tok[lo:hi]
        ids[named[(named >= 0) & (named < N)]] = e
    y = torch.full((t, N, n // t), MARK, dtype=torch.bfloat16, device="cuda")
    nb = tp.tp_lora_ws_bytes(N, rank)
    ws = torch.full((nb // 4,), math.nan, device="cuda")
    tp.tp_lora_linear(dev(x), N, k, n, t, dev(w), L, rank, dev(a), dev(b), dev(sc), dev(off), dev(tok), y, ws, nb)
    settled()
    ref = M.lora(f64(x), f64(w), f64(a), f64(b), f64(sc), ids)
    size = M.lora(np.abs(f64(x)), np.abs(f64(w)), np.abs(f64(a)), np.abs(f64(b)), f64(sc), ids)
    slack = size * ((2 * k + 2 * rank) * 2.0 ** -23 + 2.0 ** -16)      # as in test_lora
    got = f64(y)
    within(got[:, ~unnamed], ref[:, ~unnamed], (slack + 2.0 ** -8 * (np.abs(ref) + slack))[:, ~unnamed], form)
    assert (got[:, unnamed] == MARK).all()


def test_lora_of_very_many_tokens():
    """Every token's place and every tile's adapters, far beyond one tile; some places are not named and hold rubbish."""
    N, k, n, L, rank = 70001, 64, 512, 300, 8
    d = S.Draw(3, "cuda")
    x, w, a, b = d.normal((N, k)), d.normal((1, k, n), 0.1), d.normal((L, k, rank), 0.1), d.normal((1, L, rank, n), 0.5)
    ids = torch.randint(-1, L + 2, (N,), generator=d.gen, device="cuda", dtype=torch.int32)
    off, tok = torch.full((L + 1,), -9, dtype=torch.int32, device="cuda"), torch.full((N,), -9, dtype=torch.int32, device="cuda")
    pb, nb = tp.tp_lora_plan_ws_bytes(N, L), tp.tp_lora_ws_bytes(N, rank)
    tp.tp_lora_plan(ids, N, L, off, tok, torch.empty(pb, dtype=torch.uint8, device="cuda"), pb)
    lost = tok[::5003].clone().long()
    tok[::5003] = -1
    for rubbish in (0, 12345, -1):                       # what the workspace holds before
        ws = torch.full((nb // 4,), rubbish, dtype=torch.int32, device="cuda")
        y = torch.full((1, N, n), MARK, dtype=torch.bfloat16, device="cuda")
        tp.tp_lora_linear(x, N, k, n, 1, w, L, rank, a, b, None, off, tok, y, ws, nb)
        settled()
        assert (y[0, lost] == MARK).all()
        mine = (ids >= 0) & (ids < L)
        at = torch.where(mine, ids, 0).long()
        bad = 0
        for c in range(0, N, 10000):
            part = slice(c, c + 10000)
            A, B, X = a[at[part]].double(), b[0, at[part]].double(), x[part].double()
            A[~mine[part]] = 0
            v, sv = (torch.einsum("nk,nkr->nr", p, q) for p, q in ((X, A), (X.abs(), A.abs())))
            ref = X @ w[0].double() + torch.einsum("nr,nrm->nm", v, B)
            slack = (X.abs() @ w[0].double().abs() + torch.einsum("nr,nrm->nm", sv, B.abs())) * ((2 * k + 2 * rank) * 2.0 ** -23 + 2.0 ** -16)
            off_by = (y[0, part].double() - ref).abs() > slack + 2.0 ** -8 * (ref.abs() + slack)
            gone = lost[(lost >= c) & (lost < c + 10000)] - c
            off_by[gone] = False
            bad += int(off_by.sum())
        assert bad == 0


@pytest.mark.parametrize("counts,K,n,act", [
    ([3, 0, 1], 72, 136, "none"), ([40, 9], 136, 72, "swiglu"), ([1, 20], 2056, 64, "gelu"),      # tiles of few rows
    ([700, 300], 264, 2600, "none"), ([700, 300], 264, 1336, "swiglu"),                           # pairs, gathered rows
    ([2200, 1900], 2048, 5120, "none"),                                                           # put side by side first
])
def test_rows_outside_x_meet_infinities_in_w(counts, K, n, act):
    """A row that an index outside x names is a row of zeros for every kernel: it gives zeros, and NaN in the columns where
    its expert's w holds an infinity or NaN, as zeros do that lie in x. What row 0 of x holds does not matter."""
    E, N, wide = len(counts), 50, 2 if act == "swiglu" else 1
    d = S.Draw(K + n, "cuda")
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1])
    idx = torch.from_numpy(np.random.default_rng(R).integers(1, N - 1, R).astype(np.int32))
    at = [0, 1, R // 2, R - 1]
    outside, inside = idx.clone(), idx.clone()
    for i, v in zip(at, (-1, N, 1 << 30, -(1 << 31))):
        outside[i], inside[i] = v, N - 1
    x, w = d.normal((N, K)), d.normal((E, K, wide * n), 1 / math.sqrt(K))
    x[0] = math.nan
    x[N - 1] = 0
    w[0, 5, 3], w[E - 1, K - 1, wide * n - 1] = math.inf, math.nan
    ys = []
    for rows in (outside, inside):
        y = torch.full((R, n), MARK, device="cuda")
        tp.tp_ragged_linear(x, N, dev(rows), dev(off), R, E, K, n, {"none": tp.TP_ACT_NONE, "gelu": tp.TP_ACT_GELU, "swiglu": tp.TP_ACT_SWIGLU}[act],
                            w, y, tp.TP_F32)
        settled()
        ys.append(y)
    assert torch.equal(ys[0].isnan(), ys[1].isnan()) and torch.equal(ys[0].nan_to_num(7), ys[1].nan_to_num(7))
    for i in at:
        e = 0 if i < off[1] else E - 1
        z = torch.zeros(K, dtype=torch.float64, device="cuda") @ w[e].double()
        want = z[:n] + z[n:] if act == "swiglu" else z
        assert torch.equal(ys[0][i].isnan(), want.isnan()) and bool((ys[0][i].nan_to_num(0) == 0).all()), i
