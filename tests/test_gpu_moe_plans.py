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
