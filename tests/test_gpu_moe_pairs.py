"""What the CTA-pair kernels compute, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import synthetic as S
import tensor_sharded_matmul_b200 as tp
from test_gpu_moe import ACT, MARK, _lora_case, dev, settled

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
