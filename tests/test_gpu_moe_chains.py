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
from test_gpu_moe import _mlp, dev, plan_of, settled

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


@pytest.mark.parametrize("rows,k,n", [
    (1, 1024, 512), (20, 1024, 512), (64, 1024, 512), (300, 1024, 512),
    (300, 2048, 1024),                                   # pairs, gathered rows
    (1000, 2048, 4096),                                  # pairs, gathered rows that are put side by side first
])
def test_products_over_shared_buffers(rows, k, n):
    """Up (gathered, SwiGLU), down, both gradients of down: each reads what the call before it wrote."""
    E, N, rounds = 4, 64, 8
    d = S.Draw(rows + n, "cuda")
    w1, w2 = d.normal((E, k, 2 * n), 1 / math.sqrt(k)), d.normal((E, n, k), 1 / math.sqrt(n))
    cases = []
    for i in range(3):
        counts = [rows, rows, rows, rows]
        counts[i], counts[(i + 1) % E] = 2 * rows - rows // 2, rows // 2
        off, idx, R = plan_of(counts, N, rows + i)
        cases.append((d.normal((N, k)), dev(off), dev(idx)))
    bf = dict(dtype=torch.bfloat16, device="cuda")

    def buffers():
        return dict(x=torch.empty((N, k), **bf), off=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                    idx=torch.empty(R, dtype=torch.int32, device="cuda"), z=torch.empty((R, n), **bf), u=torch.empty((R, k), **bf),
                    pre=torch.empty((R, 2 * n), **bf), dh=torch.empty((R, 2 * n), **bf), dw=torch.empty((E, n, k), device="cuda"))

    def chain(o, x, off, idx, check=lambda: None):
        for name in ("z", "u", "pre", "dh", "dw"):
            o[name].fill_(NAN)
        o["x"].copy_(x), o["off"].copy_(off), o["idx"].copy_(idx)
        check()
        tp.tp_ragged_linear(o["x"], N, o["idx"], o["off"], R, E, k, n, tp.TP_ACT_SWIGLU, w1, o["z"], tp.TP_BF16, o["pre"])
        check()
        tp.tp_ragged_linear(o["z"], R, None, o["off"], R, E, n, k, tp.TP_ACT_NONE, w2, o["u"], tp.TP_BF16)
        check()
        tp.tp_ragged_linear_dx(o["u"], o["off"], R, E, n, k, w2, tp.TP_ACT_SWIGLU, o["pre"], o["dh"])
        check()
        tp.tp_ragged_linear_dw(o["z"], R, None, o["u"], o["off"], R, E, n, k, o["dw"], tp.TP_F32)
        check()
        return [o[name].clone() for name in ("z", "u", "pre", "dh", "dw")]

    want = [chain(buffers(), *c, check=settled) for c in cases]
    for w in want:
        assert not any(v.isnan().any() for v in w)
    shared = buffers()
    got = [chain(shared, *cases[i % 3]) for i in range(rounds)]
    settled()
    for i, g in enumerate(got):
        assert all(same(a, b) for a, b in zip(g, want[i % 3])), i


KEPT = ("h_pre", "z", "u", "y", "du", "dh", "dweight", "dw_in", "dw_down", "dx", "dlogits", "weight")
OUT = ("y", "dx", "dw_in", "dw_down", "dlogits", "weight", "offsets")


@pytest.mark.parametrize("N,h,F,E", [(7, 136, 72, 6), (200, 128, 96, 6), (2100, 512, 2048, 4)])
def test_mlp_over_shared_buffers(N, h, F, E):
    """Forward and backward of other tokens and logits each time, on one stream and on two at once."""
    runs = [_mlp(N, h, F, E, 2, "swiglu", "topk", seed=N + i, masked=i) for i in range(3)]
    inputs = [{n: b[n].clone() for n in ("x", "logits", "dy")} for b, _, _, _ in runs]
    for b, _, _, _ in runs[1:]:
        for n in ("w_in", "w_down"):
            b[n].copy_(runs[0][0][n])
    want = []
    for b, _, forward, backward in runs:
        for n in KEPT:
            b[n].fill_(NAN)
        settled()
        forward(), settled()
        backward(), settled()
        want.append({n: b[n].clone() for n in OUT})
        assert not any(v.isnan().any() for v in want[-1].values())

    def step(run, i, stream):
        b, _, forward, backward = run
        for n in KEPT:
            b[n].fill_(NAN)
        for n, v in inputs[i].items():
            b[n].copy_(v)
        forward(stream), backward(stream)
        return {n: b[n].clone() for n in OUT}

    got = [(i % 3, step(runs[0], i % 3, None)) for i in range(7)]
    settled()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(6):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(((i + j) % 3, step(runs[j], (i + j) % 3, s)))
    settled()
    for at, (i, g) in enumerate(got):
        for n in OUT:
            assert same(g[n], want[i][n]), (at, n)


@pytest.mark.parametrize("N,n,t", [(100, 136, 1), (700, 5120, 2)])        # (700: the adapters' pairs)
def test_captured_with_copies_and_a_fork(N, n, t):
    """A captured step whose calls follow copies, a cleared buffer and a join of two streams instead of kernels: its replays on
    new inputs are the eager calls'."""
    h, F, E, L, rank = 128, 96, 6, 4, 16
    runs = [_mlp(N, h, F, E, 2, "swiglu", "topk", seed=70 + i, masked=3) for i in range(2)]
    d = S.Draw(5, "cuda")
    source = [dict(x=d.normal((N, h)), logits=d.normal((N, E), 1.0, torch.float32), dy=d.normal((N, h)),
                   ids=torch.randint(-1, L, (N,), generator=d.gen, device="cuda", dtype=torch.int32)) for _ in range(3)]
    feed = {name: v.clone() for name, v in source[0].items()}
    w, a, b = d.normal((t, h, n // t), 0.1), d.normal((L, h, rank), 0.1), d.normal((t, L, rank, n // t), 0.5)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, off, tok = torch.zeros(N, **i32), torch.zeros(L + 1, **i32), torch.zeros(N, **i32)
    pb, nb = tp.tp_lora_plan_ws_bytes(N, L), tp.tp_lora_ws_bytes(N, rank)
    pws, ws = torch.empty(pb, dtype=torch.uint8, device="cuda"), torch.empty(nb // 4, device="cuda")
    out = torch.zeros((t, N, n // t), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):                    # the other stream: its own copies, forward, backward
            for name in ("x", "logits", "dy"):
                runs[1][0][name].copy_(feed[name])
            runs[1][2](side), runs[1][3](side)
        ids.copy_(feed["ids"])
        tp.tp_lora_plan(ids, N, L, off, tok, pws, pb)    # directly behind a copy
        out.zero_()
        tp.tp_lora_linear(feed["x"], N, h, n, t, w, L, rank, a, b, None, off, tok, out, ws, nb)
        runs[0][0]["dy"].copy_(feed["dy"])
        for name in ("x", "logits"):
            runs[0][0][name].copy_(feed[name])
        runs[0][2](here)
        here.wait_stream(side)
        runs[0][3](here)                                 # directly behind the join

    def results():
        settled()
        return [out.clone()] + [run[0][name].clone() for run in runs for name in OUT]

    want = []
    for src in source:
        for name, v in src.items():
            feed[name].copy_(v)
        step()
        want.append(results())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in (1, 0, 2, 1):
        for name, v in source[i].items():
            feed[name].copy_(v)
        for run in runs:
            for name in KEPT:
                run[0][name].fill_(NAN)
        ws.fill_(NAN)
        g.replay()
        for x, y in zip(results(), want[i]):
            assert same(x, y)
