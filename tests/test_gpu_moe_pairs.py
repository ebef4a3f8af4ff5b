"""What the CTA-pair kernels compute, and the whole MLP in every type, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import synthetic as S
import tensor_sharded_matmul_b200 as tp
from gpu_util import f64
from oracle import moe as M
from test_gpu_moe import ACT, DT, GATE, MARK, _lora_case, dev, rel, settled

pytestmark = pytest.mark.gpu


def _act_back(h, dz, act):
    """act'(h) dz in 64 bits, from the derivatives' definitions; SwiGLU: [dgate | dup]."""
    if act == "swiglu":
        g, u = h.chunk(2, dim=1)
        s = torch.sigmoid(g)
        return torch.cat([dz * u * (s + g * s * (1 - s)), dz * g * s], 1)
    if act == "gelu":
        return dz * (torch.special.ndtr(h) + h * torch.exp(-h * h / 2) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c, a = math.sqrt(2 / math.pi), 0.044715
        s = torch.sigmoid(2 * c * (h + a * h ** 3))                    # (1 + tanh) / 2
        return dz * (s + h * s * (1 - s) * 2 * c * (1 + 3 * a * h * h))
    return dz


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("counts,k,n", [
    ([700, 0, 1, 600, 290], 2056, 136),          # uneven tiles, an odd number of k-blocks, partial column tiles
    ([513, 31, 0, 1025], 2600, 72),              # a last tile of one row in front of a low one
])
def test_dx_on_pairs(counts, k, n, act):
    """Tolerances as in test_ragged_linear_dx: dz is a sum of n products, off by at most n * 2^-23 * sum |dy w|; the derivative
    passes it on with a slope below 1.2 and adds 2^-18 of dz; one rounding to bf16."""
    E, wide, front, tail = len(counts), 2 if act == "swiglu" else 1, 3, 5
    off = front + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1]) + tail
    d = S.Draw(k + n, "cuda")
    dy, w, hp = d.normal((R, n)), d.normal((E, k, n), 1 / math.sqrt(n)), d.normal((R, wide * k))
    hp[:, ::7] *= 8                              # gates far from zero too
    dy[:front], dy[R - tail:] = math.nan, math.nan
    dx = torch.full((R, wide * k), MARK, dtype=torch.bfloat16, device="cuda")
    tp.tp_ragged_linear_dx(dy, dev(off), R, E, k, n, w, ACT[act], hp if act != "none" else None, dx)
    settled()
    assert (dx[:front] == MARK).all() and (dx[R - tail:] == MARK).all()
    for e in range(E):
        part = slice(int(off[e]), int(off[e + 1]))
        dz = dy[part].double() @ w[e].double().t()
        size = n * 2.0 ** -23 * (dy[part].double().abs() @ w[e].double().abs().t())
        h = hp[part].double()
        ref = _act_back(h, dz, act)
        if act == "none":
            slack = size
        else:
            size = size + 2.0 ** -18 * dz.abs()
            slack = 1.2 * size
            if act == "swiglu":
                g, u = h.abs().chunk(2, dim=1)
                slack = torch.cat([1.2 * size * u, size * g], 1)
        bad = ~((dx[part].double() - ref).abs() <= slack + 2.0 ** -8 * (ref.abs() + slack) + 1e-37)
        assert not bad.any(), (e, int(bad.sum()), torch.nonzero(bad)[0].tolist())


@pytest.mark.parametrize("N,L,rank", [(4001, 30, 24), (2501, 45, 136)])
def test_lora_whose_first_product_takes_pairs(N, L, rank):
    """x A of so many adapters goes to the pair kernel, which applies each adapter's scale to its own rows."""
    ids = np.random.default_rng(N).integers(-1, L, N).astype(np.int32)
    _lora_case(N, 136, 6144, 8, L, rank, ids, N, scale=True)


@pytest.mark.parametrize("types", ["f32 bf16 bf16", "bf16 f32 bf16", "bf16 bf16 f32", "f32 f32 f32"])
@pytest.mark.parametrize("N,h,F,E,k,act,gate,masked", [
    (37, 136, 72, 6, 2, "swiglu", "topk", 3), (300, 72, 200, 3, 2, "gelu", "softmax", 0),
    (2100, 512, 2048, 4, 2, "swiglu", "topk", 11),           # pairs, rows put side by side, spans of weight gradients
    (2100, 512, 2048, 4, 1, "gelu_tanh", "softmax", 1),
])
def test_mlp_in_every_type(N, h, F, E, k, act, gate, masked, types):
    """Logits (and their gradient), y and dx in fp32 and bf16. z, u, du, dh and the rows of dx are rounded to bf16, each by at
    most 2^-8 of the value; at most five of them lie on the way to an output, whose own rounding is a sixth: 2-norms of
    the errors stay below 6 * 2^-8 of the output's."""
    ld, yd, xd = (DT[v] for v in types.split())
    d = S.Draw(N + F, "cuda")
    wide, R = 2 if act == "swiglu" else 1, N * k
    x, dy, logits = d.normal((N, h)), d.normal((N, h)), d.normal((N, E), 1.0, ld[1])
    w_in, w_down = d.normal((E, h, wide * F), 1 / math.sqrt(h)), d.normal((E, F, h), 1 / math.sqrt(F))
    logits[N - masked:] = -math.inf
    new = lambda shape, dt=torch.bfloat16: torch.full(shape, math.nan, dtype=dt, device="cuda")           # noqa: E731
    whole = lambda *shape: torch.full(shape, -9, dtype=torch.int32, device="cuda")                       # noqa: E731
    expert, slot, offsets, row_token = whole(N, k), whole(N, k), whole(E + 1), whole(R)
    weight, dweight, y, dx, dlogits = new((N, k), torch.float32), new((N, k), torch.float32), new((N, h), yd[1]), new((N, h), xd[1]), new((N, E), ld[1])
    h_pre, z, u, du, dh = new((R, wide * F)), new((R, F)), new((R, h)), new((R, h)), new((R, wide * F))
    dw_in, dw_down = new((E, h, wide * F), torch.float32), new((E, F, h), torch.float32)
    nb = tp.tp_moe_mlp_ws_bytes(N, E, k)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    tp.tp_moe_mlp_fwd(x, N, h, F, E, k, GATE[gate], ACT[act], logits, ld[0], w_in, w_down, expert, weight, slot, offsets, row_token,
                      h_pre, z, u, y, yd[0], ws, nb)
    tp.tp_moe_mlp_bwd(x, dy, N, h, F, E, k, GATE[gate], ACT[act], logits, ld[0], w_in, w_down, expert, weight, slot, offsets,
                      row_token, h_pre, z, u, du, dh, dweight, dw_in, dw_down, dx, xd[0], dlogits)
    settled()
    ref = M.moe_mlp_backward(f64(x), f64(logits), f64(w_in), f64(w_down), k, gate, act, f64(dy))
    rows = len(ref["row_token"])
    assert np.array_equal(expert.cpu().numpy(), ref["expert"]) and np.array_equal(offsets.cpu().numpy(), ref["offsets"])
    assert np.array_equal(row_token[:rows].cpu().numpy(), ref["row_token"]) and np.array_equal(slot.cpu().numpy(), ref["slot"])
    got = dict(y=y, dx=dx, dw_in=dw_in, dw_down=dw_down, dweight=dweight, z=z[:rows])
    for name, v in got.items():
        assert rel(v, ref[name]) < 6 * 2.0 ** -8, (name, rel(v, ref[name]))
    if not (gate == "topk" and k == 1):
        size = np.linalg.norm(M.gate_softmax(f64(logits), ref["expert"], gate) * np.abs(ref["dweight"]).max(initial=0))
        assert np.linalg.norm(f64(dlogits) - ref["dlogits"]) < 6 * 2.0 ** -8 * size
