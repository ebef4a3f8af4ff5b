"""Refusals and empty calls of the mixture-of-experts and adapter entry points, on the host (no call here
reaches the GPU)."""
import pytest

import tensor_sharded_matmul_b200 as tp

FAKE = 1 << 20   # 16-byte aligned, never dereferenced: the calls fail validation first
BIG = 1 << 31


def _expect(status, fn, *args):
    with pytest.raises(tp.TPError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


def _route(N=4, E=8, k=2, gate=tp.TP_GATE_TOPK, dtype=tp.TP_F32, logits=FAKE, expert=FAKE, ws=FAKE, ws_bytes=1 << 30):
    tp.tp_moe_route(logits, dtype, N, E, k, gate, expert, FAKE, FAKE, FAKE, FAKE, ws, ws_bytes, 0)


def _linear(x=FAKE, x_rows=64, index=FAKE, offsets=FAKE, R=64, E=4, k=64, n=64, act=tp.TP_ACT_NONE, w=FAKE, y=FAKE,
            y_dtype=tp.TP_BF16, pre=None):
    tp.tp_ragged_linear(x, x_rows, index, offsets, R, E, k, n, act, w, y, y_dtype, pre, 0)


def _lora(x=FAKE, N=64, k=64, n=64, t=2, L=4, rank=16, a=FAKE, ws=FAKE, ws_bytes=1 << 30):
    tp.tp_lora_linear(x, N, k, n, t, FAKE, L, rank, a, FAKE, FAKE, FAKE, FAKE, FAKE, ws, ws_bytes, 0)


@pytest.mark.parametrize("status,kw", [
    (tp.TP_EINVAL, dict(N=-1)), (tp.TP_EINVAL, dict(E=0)), (tp.TP_EINVAL, dict(k=0)), (tp.TP_EINVAL, dict(gate=2)),
    (tp.TP_EINVAL, dict(dtype=tp.TP_BF16_RING)), (tp.TP_EUNSUPPORTED, dict(E=1025)), (tp.TP_EUNSUPPORTED, dict(E=64, k=17)),
    (tp.TP_ESHAPE, dict(E=2, k=3)), (tp.TP_ESHAPE, dict(N=BIG)), (tp.TP_EINVAL, dict(logits=0)), (tp.TP_EINVAL, dict(expert=0)),
    (tp.TP_EALIGN, dict(logits=FAKE + 2)), (tp.TP_EALIGN, dict(expert=FAKE + 1)),
    (tp.TP_ENOSPACE, dict(N=65, ws=0)), (tp.TP_ENOSPACE, dict(N=65, ws_bytes=8 * 3 * 4 - 1)),
])
def test_route_refusals(status, kw):
    _expect(status, lambda: _route(**kw))


def test_route_bwd_refusals():
    b = lambda N=4, E=8, k=2, g=0, d=tp.TP_F32, l=FAKE, dl=FAKE: tp.tp_moe_route_bwd(l, d, N, E, k, g, FAKE, FAKE, dl, 0)  # noqa: E731
    _expect(tp.TP_EINVAL, lambda: b(l=0))
    _expect(tp.TP_EINVAL, lambda: b(g=-1))
    _expect(tp.TP_EALIGN, lambda: b(dl=FAKE + 2))
    _expect(tp.TP_ESHAPE, lambda: b(k=9))
    b(N=0, l=0, dl=0)


@pytest.mark.parametrize("status,kw", [
    (tp.TP_EINVAL, dict(R=-1)), (tp.TP_EINVAL, dict(k=0)), (tp.TP_EINVAL, dict(E=0)), (tp.TP_EUNSUPPORTED, dict(E=1025)),
    (tp.TP_ESHAPE, dict(R=BIG)), (tp.TP_ESHAPE, dict(n=BIG)), (tp.TP_ESHAPE, dict(index=None, x_rows=63)),
    (tp.TP_ESHAPE, dict(x_rows=0)), (tp.TP_EALIGN, dict(k=60)), (tp.TP_EALIGN, dict(n=4)), (tp.TP_EALIGN, dict(x=FAKE + 8)),
    (tp.TP_EALIGN, dict(w=FAKE + 8)), (tp.TP_EALIGN, dict(y=FAKE + 4)), (tp.TP_EALIGN, dict(offsets=FAKE + 2)),
    (tp.TP_EALIGN, dict(index=FAKE + 1)), (tp.TP_EINVAL, dict(w=0)), (tp.TP_EINVAL, dict(act=7)), (tp.TP_EINVAL, dict(y_dtype=2)),
    (tp.TP_EINVAL, dict(pre=FAKE)), (tp.TP_EALIGN, dict(act=tp.TP_ACT_GELU, pre=FAKE + 8)),
])
def test_ragged_linear_refusals(status, kw):
    _expect(status, lambda: _linear(**kw))


def test_ragged_gradient_refusals():
    dx = lambda R=64, n=64, act=tp.TP_ACT_NONE, h=None, dy=FAKE: tp.tp_ragged_linear_dx(dy, FAKE, R, 4, 64, n, FAKE, act, h, FAKE, 0)  # noqa: E731
    _expect(tp.TP_EINVAL, lambda: dx(act=tp.TP_ACT_GELU))             # no h_pre
    _expect(tp.TP_EINVAL, lambda: dx(h=FAKE))                         # h_pre without an activation
    _expect(tp.TP_EALIGN, lambda: dx(n=12))
    _expect(tp.TP_EINVAL, lambda: dx(dy=0))
    dx(R=0, dy=0)
    dw = lambda x=FAKE, xr=64, i=None, R=64, dt=tp.TP_F32, o=FAKE, g=FAKE: tp.tp_ragged_linear_dw(x, xr, i, FAKE, o, R, 4, 64, 64, g, dt, 0)  # noqa: E731
    _expect(tp.TP_EINVAL, lambda: dw(dt=tp.TP_BF16_RING))
    _expect(tp.TP_EINVAL, lambda: dw(o=0))
    _expect(tp.TP_EINVAL, lambda: dw(x=0))
    _expect(tp.TP_ESHAPE, lambda: dw(xr=10))
    _expect(tp.TP_EALIGN, lambda: dw(g=FAKE + 8))


def test_combine_refusals():
    c = lambda u=FAKE, R=8, w=FAKE, N=4, h=64, k=2, ud=tp.TP_BF16, y=FAKE: tp.tp_moe_combine(u, ud, R, w, FAKE, N, h, k, y, tp.TP_F32, 0)  # noqa: E731
    _expect(tp.TP_EALIGN, lambda: c(h=12))
    _expect(tp.TP_EINVAL, lambda: c(h=0))
    _expect(tp.TP_EINVAL, lambda: c(u=0))
    _expect(tp.TP_EINVAL, lambda: c(ud=2))
    _expect(tp.TP_EALIGN, lambda: c(y=FAKE + 8))
    _expect(tp.TP_EUNSUPPORTED, lambda: c(k=17))
    _expect(tp.TP_ESHAPE, lambda: c(N=BIG))
    c(N=0, u=0, y=0)
    b = lambda w=FAKE, k=2, du=FAKE, N=4: tp.tp_moe_combine_bwd(FAKE, tp.TP_BF16, FAKE, tp.TP_BF16, 8, w, FAKE, N, 64, k, du, FAKE, 0)  # noqa: E731
    _expect(tp.TP_EINVAL, lambda: b(w=None))
    _expect(tp.TP_EINVAL, lambda: b(du=0))
    _expect(tp.TP_EALIGN, lambda: b(du=FAKE + 2))
    b(N=0)


@pytest.mark.parametrize("status,kw", [
    (tp.TP_EINVAL, dict(t=0)), (tp.TP_EINVAL, dict(t=17)), (tp.TP_EINVAL, dict(N=-1)), (tp.TP_EINVAL, dict(rank=0)),
    (tp.TP_EINVAL, dict(L=0)), (tp.TP_EUNSUPPORTED, dict(L=1025)), (tp.TP_EDIVIS, dict(n=72, t=5)), (tp.TP_EALIGN, dict(n=72, t=2)),
    (tp.TP_EALIGN, dict(rank=12)), (tp.TP_EALIGN, dict(a=FAKE + 8)), (tp.TP_EINVAL, dict(x=0)), (tp.TP_ESHAPE, dict(N=BIG)),
    (tp.TP_ENOSPACE, dict(ws=0)), (tp.TP_ENOSPACE, dict(ws_bytes=64 * 16 * 4 - 1)),
])
def test_lora_refusals(status, kw):
    _expect(status, lambda: _lora(**kw))


def test_plan_refusals_and_sizes():
    p = lambda id=FAKE, N=65, L=4, o=FAKE, ws=FAKE, b=1 << 20: tp.tp_lora_plan(id, N, L, o, FAKE, ws, b, 0)  # noqa: E731
    _expect(tp.TP_EINVAL, lambda: p(id=0))
    _expect(tp.TP_EINVAL, lambda: p(L=0))
    _expect(tp.TP_EUNSUPPORTED, lambda: p(L=1025))
    _expect(tp.TP_EALIGN, lambda: p(o=FAKE + 2))
    _expect(tp.TP_ENOSPACE, lambda: p(ws=0))
    p(N=0, id=0, o=0, ws=0)
    assert tp.tp_moe_route_ws_bytes(64, 128, 8) == 0 and tp.tp_moe_route_ws_bytes(65, 128, 8) == 128 * 3 * 4
    assert tp.tp_moe_mlp_ws_bytes(1000, 16, 2) == tp.tp_moe_route_ws_bytes(1000, 16, 2) == 16 * 17 * 4
    assert tp.tp_lora_plan_ws_bytes(128, 7) == (8 * 3 + 128) * 4 and tp.tp_lora_ws_bytes(64, 24) == 64 * 24 * 4
    assert tp.tp_lora_ws_bytes(300, 24) == 300 * 24 * 4 + 300 * 4 + 2 * 257 * 4
    assert tp.tp_moe_route_ws_bytes(-1, 8, 2) == tp.tp_lora_ws_bytes(0, 8) == 0


def test_mlp_refusals_and_empty_calls():
    f = lambda N=4, act=tp.TP_ACT_GELU, x=FAKE, h_pre=None, F=64, ws=FAKE, wb=0: tp.tp_moe_mlp_fwd(  # noqa: E731
        x, N, 64, F, 8, 2, 0, act, FAKE, tp.TP_F32, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, h_pre, FAKE, FAKE, FAKE, tp.TP_F32,
        ws, wb, 0)
    _expect(tp.TP_EINVAL, lambda: f(x=0))
    _expect(tp.TP_EINVAL, lambda: f(act=tp.TP_ACT_NONE, h_pre=FAKE))
    _expect(tp.TP_EALIGN, lambda: f(F=60))
    _expect(tp.TP_ENOSPACE, lambda: f(N=100))
    f(N=0, x=0)
    _expect(tp.TP_EINVAL, tp.tp_moe_mlp_bwd, FAKE, FAKE, 4, 64, 64, 8, 2, 0, tp.TP_ACT_GELU, FAKE, tp.TP_F32, *[FAKE] * 7, None,
            *[FAKE] * 8, tp.TP_F32, FAKE, 0)
    _linear(R=0, x=0, x_rows=0, index=None, offsets=0, w=0, y=0)
    _route(N=0, logits=0, expert=0, ws=0, ws_bytes=0)
    _lora(N=0, x=0, a=0, ws=0, ws_bytes=0)


_BWD = ("x", "dy", "N", "h", "F", "E", "k", "gate", "act", "logits", "logits_dtype", "w_in", "w_down", "expert", "weight", "slot",
        "offsets", "row_token", "h_pre", "z", "u", "du_ws", "dh_ws", "dweight_ws", "dw_in", "dw_down", "dx", "dx_dtype", "dlogits")


def _mlp_bwd(**kw):
    a = dict({n: FAKE for n in _BWD}, N=4, h=64, F=64, E=8, k=2, gate=tp.TP_GATE_TOPK, act=tp.TP_ACT_GELU, logits_dtype=tp.TP_F32,
             dx_dtype=tp.TP_F32)
    a.update(kw)
    tp.tp_moe_mlp_bwd(*[a[n] for n in _BWD], 0)


@pytest.mark.parametrize("N", [4, 4096])           # few rows an expert; many, which are put side by side
def test_mlp_bwd_refuses_a_row_token_off_its_elements(N):
    _expect(tp.TP_EALIGN, lambda: _mlp_bwd(N=N, row_token=FAKE + 2))


@pytest.mark.parametrize("status,kw", [
    *[(tp.TP_EALIGN, {n: FAKE + 2}) for n in ("expert", "weight", "slot", "offsets", "dweight_ws", "logits", "dlogits")],
    (tp.TP_EALIGN, dict(logits=FAKE + 1, logits_dtype=tp.TP_BF16)), (tp.TP_EALIGN, dict(dlogits=FAKE + 1, logits_dtype=tp.TP_BF16)),
    (tp.TP_ESHAPE, dict(act=tp.TP_ACT_SWIGLU, F=(1 << 28) + 8)),       # its 2 F columns are too many
])
def test_mlp_bwd_refuses_before_it_launches(status, kw):
    _expect(status, lambda: _mlp_bwd(**kw))


def test_mlp_bwd_of_no_tokens_checks_what_it_writes():
    _expect(tp.TP_EALIGN, lambda: _mlp_bwd(N=0, offsets=FAKE + 2))
    _expect(tp.TP_ESHAPE, lambda: _mlp_bwd(N=0, act=tp.TP_ACT_SWIGLU, F=(1 << 28) + 8))
