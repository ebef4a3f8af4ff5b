"""Calls of the mixture-of-experts operators and the adapters that follow one another on a stream with nothing between
them, over buffers that they share. Whatever a call leaves behind is wrong for the next one: inputs, indices and segments
change from call to call, and outputs, intermediates and workspaces are filled with NaN before each chain, so that a kernel
which reads before its predecessor has written, or does not write, is seen. Every result has to be, bit for bit, that of
the same calls waited for one by one in buffers of their own, and those are held to the 64-bit formula."""
import math

import pytest
import torch

import synthetic as S
import tensor_sharded_matmul_b200 as tp
from test_gpu_moe import settled

pytestmark = pytest.mark.gpu

NAN = math.nan


def same(a, b):
    """Bit for bit, NaN included."""
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("last", ["ids", "x"])           # what is written directly before the calls that read it
@pytest.mark.parametrize("N,n", [(1, 1024), (3, 1024), (40, 1024), (64, 1024), (100, 1024), (700, 5120)])
def test_lora_of_changing_batches(N, n, last):
    """Plan and projection in a chain over one set of buffers, other tokens and adapters each time."""
    k, t, L, rank, rounds = 2048, 2, 4, 16, 24
    d = S.Draw(N, "cuda")
    w, a, b = d.normal((t, k, n // t), 0.02), d.normal((L, k, rank), 0.02), d.normal((t, L, rank, n // t), 0.5)
    batches = [(d.normal((N, k)), torch.randint(-1, L, (N,), generator=d.gen, device="cuda", dtype=torch.int32)) for _ in range(3)]
    if N == 1:
        for i, (_, ids) in enumerate(batches):
            ids.fill_(i)
    pb, nb = tp.tp_lora_plan_ws_bytes(N, L), tp.tp_lora_ws_bytes(N, rank)

    def buffers():
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(x=torch.empty((N, k), dtype=torch.bfloat16, device="cuda"), ids=torch.empty(N, **i32), off=torch.empty(L + 1, **i32),
                    tok=torch.empty(N, **i32), pws=torch.empty(pb, dtype=torch.uint8, device="cuda"), ws=torch.empty(nb // 4, device="cuda"))

    def calls(o, x, ids, y, check=lambda: None):
        o["ws"].fill_(NAN)
        o["off"].fill_(0), o["tok"].fill_(0), y.fill_(NAN)
        if last == "ids":
            o["x"].copy_(x)
        o["ids"].copy_(ids)
        check()
        tp.tp_lora_plan(o["ids"], N, L, o["off"], o["tok"], o["pws"], pb)
        check()
        if last == "x":
            o["x"].copy_(x)
            check()
        tp.tp_lora_linear(o["x"], N, k, n, t, w, L, rank, a, b, None, o["off"], o["tok"], y, o["ws"], nb)
        check()

    want = []
    for x, ids in batches:
        y = torch.empty((t, N, n // t), dtype=torch.bfloat16, device="cuda")
        calls(buffers(), x, ids, y, settled)
        X, mine = x.double(), torch.nn.functional.one_hot((ids + 1).long(), L + 1)[:, 1:].double()
        v = torch.einsum("nk,lkr,nl->nlr", X, a.double(), mine)
        size_v = torch.einsum("nk,lkr,nl->nlr", X.abs(), a.double().abs(), mine)
        for r in range(t):
            ref = X @ w[r].double() + torch.einsum("nlr,lrm->nm", v, b[r].double())
            size = X.abs() @ w[r].double().abs() + torch.einsum("nlr,lrm->nm", size_v, b[r].double().abs())
            # as in test_lora: v's k adds and its split, then one sum of k + 2 rank products, and the rounding
            slack = size * ((2 * k + 2 * rank) * 2.0 ** -23 + 2.0 ** -16)
            assert bool(((y[r].double() - ref).abs() <= slack + 2.0 ** -8 * (ref.abs() + slack)).all())
        want.append(y)
    shared = buffers()
    ys = [torch.empty_like(want[0]) for _ in range(rounds)]
    for i, y in enumerate(ys):
        calls(shared, *batches[i % 3], y)
    settled()
    for i, y in enumerate(ys):
        assert same(y, want[i % 3]), i
