"""The operators beside the layer's forward pass on the GPU: tokens sorted by
expert and back with their gradients, the router's gradient, and the experts'
products in 8-bit integers, against their 64-bit forms."""
import numpy as np
import pytest
import torch

import oracle
import operator_refs as R
from mixture_experts_ffn_token_b200 import abi

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def randn(seed, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


# ------------------------------------------------------------------- rows
ROWS = [  # T, H, E, k, drop
    (1, 8, 1, 1, 0.0), (1, 4096, 64, 8, 0.0), (3, 16, 4, 3, 0.4), (33, 264, 5, 2, 0.0), (130, 1000, 40, 9, 0.2),
    (65, 2056, 3, 1, 0.5), (17, 520, 33, 32, 0.1), (257, 2048, 128, 6, 0.0), (5, 72, 20, 17, 0.0), (9, 8200, 16, 4, 1.0),
    (2, 24, 7, 5, 0.0),
]


@pytest.mark.parametrize("weighted", [True, False], ids=["w", "no_w"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,drop", ROWS)
def test_rows_forward(T, H, E, k, drop, dtype, weighted):
    cfg = abi.config(T, H, E, k, 8)
    _, off, inv = R.routing(T, E, k, seed=T + H, drop=drop)
    x, rows = randn(1, T, H, dtype=dtype), randn(2, T * k, H, dtype=dtype)
    w = randn(3, T, k) if weighted else None
    before = randn(4, T * k, H, dtype=dtype)
    got = before.cuda()
    abi.moe_dispatch(cfg, x.cuda(), inv.cuda(), got, expert_weights=cuda(w))
    ref = R.spread(x, inv.view(T, k), w, before)
    tol = R.tol_spread(ref, dtype)
    tol[int(off[-1]):] = 0                              # rows of no slot stay as they were
    if w is None:
        tol[:] = 0
    R.assert_within(got, ref, tol, "dispatch")
    out = torch.full((T, H), float("nan"), dtype=dtype, device="cuda")
    abi.moe_combine(cfg, rows.cuda(), inv.cuda(), out, expert_weights=cuda(w))
    ref, mag = R.gather(rows, inv.view(T, k), w)
    R.assert_within(out, ref, R.tol_gather(ref, mag, k, dtype), "combine")


@pytest.mark.parametrize("weighted", [True, False], ids=["w", "no_w"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,drop", ROWS)
def test_rows_backward(T, H, E, k, drop, dtype, weighted):
    cfg = abi.config(T, H, E, k, 8)
    _, off, inv = R.routing(T, E, k, seed=T + H, drop=drop)
    inv2 = inv.view(T, k)
    tok, rows = randn(1, T, H, dtype=dtype), randn(2, T * k, H, dtype=dtype)
    w = randn(3, T, k) if weighted else None
    before = randn(4, T * k, H, dtype=dtype)
    d_dot, m_dot = R.dots(tok, rows, inv2)
    for with_dw in (True, False):
        d_w = torch.full((T, k), float("nan"), device="cuda") if with_dw else None
        d_x = torch.full((T, H), float("nan"), dtype=dtype, device="cuda")
        abi.moe_dispatch_backward(cfg, rows.cuda(), inv.cuda(), d_x, x=tok.cuda() if with_dw else None,
                                  expert_weights=cuda(w), d_expert_weights=d_w)
        ref, mag = R.gather(rows, inv2, w)
        R.assert_within(d_x, ref, R.tol_gather(ref, mag, k, dtype), "d_x")
        if with_dw:
            R.assert_within(d_w, d_dot, R.tol_dots(m_dot, H), "dispatch d_w")
            d_w.fill_(float("nan"))
        d_rows = before.cuda()
        abi.moe_combine_backward(cfg, tok.cuda(), inv.cuda(), d_rows, rows=rows.cuda() if with_dw else None,
                                 expert_weights=cuda(w), d_expert_weights=d_w)
        ref = R.spread(tok, inv2, w, before)
        tol = R.tol_spread(ref, dtype)
        tol[int(off[-1]):] = 0
        R.assert_within(d_rows, ref, tol, "d_rows")
        if with_dw:
            R.assert_within(d_w, d_dot, R.tol_dots(m_dot, H), "combine d_w")


def test_rows_of_no_slot_do_not_leak():
    """NaN in the rows and weights of dropped slots reaches nothing."""
    T, H, E, k = 20, 136, 4, 3
    cfg = abi.config(T, H, E, k, 8)
    _, off, inv = R.routing(T, E, k, seed=3, drop=0.5)
    rows = randn(1, T * k, H)
    rows[int(off[-1]):] = float("nan")
    w = randn(2, T, k)
    w[inv.view(T, k) < 0] = float("nan")
    out, d_w = torch.empty(T, H, device="cuda"), torch.empty(T, k, device="cuda")
    abi.moe_combine(cfg, rows.cuda(), inv.cuda(), out, expert_weights=w.cuda())
    assert torch.isfinite(out).all()
    abi.moe_dispatch_backward(cfg, rows.cuda(), inv.cuda(), out, x=randn(3, T, H).cuda(), expert_weights=w.cuda(),
                              d_expert_weights=d_w)
    assert torch.isfinite(out).all() and torch.isfinite(d_w).all()
    assert (d_w.cpu()[inv.view(T, k) < 0] == 0).all()


def test_positions_out_of_range_are_skipped():
    T, H, E, k = 6, 64, 4, 2
    cfg = abi.config(T, H, E, k, 8)
    _, _, inv = R.routing(T, E, k, seed=5)
    bad = inv.clone()
    bad[3], bad[7] = T * k, 2 ** 31 - 1
    gone = inv.clone()
    gone[3] = gone[7] = -1
    x, rows, w = randn(1, T, H).cuda(), randn(2, T * k, H).cuda(), randn(3, T, k).cuda()
    for a, b in zip(*[[t for t in _all_rows(cfg, x, rows, w, i.cuda(), T, H, k)] for i in (bad, gone)]):
        assert torch.equal(a, b)


def _all_rows(cfg, x, rows, w, inv, T, H, k):
    spread, out = torch.zeros_like(rows), torch.empty_like(x)
    abi.moe_dispatch(cfg, x, inv, spread, expert_weights=w)
    abi.moe_combine(cfg, rows, inv, out, expert_weights=w)
    d_x, d_rows = torch.empty_like(x), torch.zeros_like(rows)
    d_w1, d_w2 = torch.empty(T, k, device="cuda"), torch.empty(T, k, device="cuda")
    abi.moe_dispatch_backward(cfg, rows, inv, d_x, x=x, expert_weights=w, d_expert_weights=d_w1)
    abi.moe_combine_backward(cfg, x, inv, d_rows, rows=rows, expert_weights=w, d_expert_weights=d_w2)
    return spread, out, d_x, d_w1, d_rows, d_w2


@pytest.mark.parametrize("T,H,E,k,drop,dtype", [
    (5003, 1544, 128, 6, 0.0, BF16), (5003, 1544, 128, 6, 0.0, F32), (8209, 4104, 8, 2, 0.0, BF16),
    (1100, 2056, 40, 3, 0.3, F32), (1025, 1000, 30, 16, 0.1, BF16), (4097, 2184, 16, 8, 0.2, BF16),
    (12007, 264, 9, 4, 0.1, BF16), (16500, 24, 3, 1, 0.0, F32),
    (3001, 2056, 12, 7, 0.1, BF16), (5000, 128, 20, 19, 0.1, BF16), (2500, 256, 40, 32, 0.1, F32), (3000, 480, 9, 5, 0.2, BF16)])
def test_rows_large(T, H, E, k, drop, dtype):
    """Tokens by the thousand, ragged, the same bits on every run."""
    cfg = abi.config(T, H, E, k, 8)
    _, off, inv = R.routing(T, E, k, seed=11, drop=drop)
    x, rows, w = randn(1, T, H, dtype=dtype), randn(2, T * k, H, dtype=dtype), randn(3, T, k)
    a = _all_rows(cfg, x.cuda(), rows.cuda(), w.cuda(), inv.cuda(), T, H, k)
    b = _all_rows(cfg, x.cuda(), rows.cuda(), w.cuda(), inv.cuda(), T, H, k)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    inv2 = inv.view(T, k)
    ref = R.spread(x, inv2, w, torch.zeros_like(rows))
    R.assert_within(a[0], ref, R.tol_spread(ref, dtype), "dispatch")
    R.assert_within(a[4], ref, R.tol_spread(ref, dtype), "d_rows")
    ref, mag = R.gather(rows, inv2, w)
    for got in (a[1], a[2]):
        R.assert_within(got, ref, R.tol_gather(ref, mag, k, dtype), "gather")
    ref, mag = R.dots(x, rows, inv2)
    for got in (a[3], a[5]):
        R.assert_within(got, ref, R.tol_dots(mag, H), "d_w")


# ------------------------------------------------------------ router gradient
def route_inputs(T, E, S, k, dtype, pad, seed, std=2.0):
    logits = randn(seed, T, E + S + pad, dtype=dtype, std=std)
    idx = torch.rand(T, E, generator=torch.Generator().manual_seed(seed + 1)).argsort(1)[:, :k].to(torch.int32)
    return logits, idx, randn(seed + 2, T, k), (randn(seed + 3, T, S) if S else None)


def route_backward(logits, idx, d_w, d_s, E, S, dtype, scale=None, fill=5.0, d_scale=False):
    T, k = idx.shape
    cfg = abi.config(T, 8, E, k, 8, router="sigmoid_sink" if scale is not None else "softmax_topk", num_sink=S,
                     logits_dtype=dtype, logits_row_stride=logits.shape[1],
                     route_scale=scale[0] if scale is not None else 1.0)
    out = torch.full(logits.shape, fill, dtype=dtype, device="cuda")
    gs = torch.tensor([scale[1]], device="cuda") if scale is not None and scale[1] is not None else None
    d_gs = torch.full((1,), float("nan"), device="cuda") if d_scale else None
    ws = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda") if d_scale else None
    abi.moe_route_backward(cfg, logits.cuda(), idx.cuda(), d_w.cuda(), out, d_sink_weights=cuda(d_s), global_scale=gs,
                           d_global_scale=d_gs, workspace=ws)
    return out.cpu(), (None if d_gs is None else float(d_gs))


@pytest.mark.parametrize("dtype,pad", [(F32, 0), (F32, 3), (BF16, 0), (BF16, 5)])
@pytest.mark.parametrize("T,E,S,k", [(1, 1, 0, 1), (1, 8, 0, 2), (7, 33, 0, 32), (130, 128, 0, 4), (5, 1024, 0, 8),
                                     (3, 2, 0, 2)])
def test_softmax_router_gradient(T, E, S, k, dtype, pad):
    logits, idx, d_w, _ = route_inputs(T, E, S, k, dtype, pad, seed=T + E)
    got, _ = route_backward(logits, idx, d_w, None, E, S, dtype)
    ref, tol, _, _ = R.route_grad(logits, idx, d_w, None, E, S, False)
    R.assert_within(got[:, :E], ref, tol + ref.abs() * R.HALF[dtype] + 1e-38, "d_logits")
    assert (got[:, E:] == 5.0).all()


@pytest.mark.parametrize("dtype,pad", [(F32, 0), (BF16, 2)])
@pytest.mark.parametrize("T,E,S,k", [(1, 4, 1, 1), (9, 128, 2, 6), (130, 40, 0, 8), (3, 64, 31, 1), (2, 1024, 16, 16),
                                     (4500, 12, 1, 3)])
def test_sink_router_gradient(T, E, S, k, dtype, pad):
    logits, idx, d_w, d_s = route_inputs(T, E, S, k, dtype, pad, seed=T + E)
    for scale, sink_grad in (((2.5, 0.7), True), ((1.5, None), False)):
        ds = d_s if sink_grad else None
        got, d_gs = route_backward(logits, idx, d_w, ds, E, S, dtype, scale=scale, d_scale=True)
        ref, tol, ref_gs, tol_gs = R.route_grad(logits, idx, d_w, ds, E, S, True, scale[0],
                                                float(torch.tensor(scale[1] if scale[1] else 1.0)))
        R.assert_within(got[:, :E + S], ref, tol + ref.abs() * R.HALF[dtype] + 1e-38, "d_logits")
        assert (got[:, E + S:] == 5.0).all()
        assert abs(d_gs - ref_gs) <= tol_gs + abs(ref_gs) * 2 * R.F32


def test_router_gradient_extremes():
    """Logits whose sigmoids underflow, saturate or are minus infinity."""
    E, S, k = 6, 2, 2
    logits = torch.tensor([[-800.0, -801.0, 3, 4, 5, 6, -802.0, -799.5], [90.0, 88.0, 0, 0, 0, 0, 91.0, 60.0],
                           [-1e30, -1e30, 0, 0, 0, 0, -1e30, -1e30], [float("-inf"), 1.0, 0, 0, 0, 0, 2.0, -3.0]])
    idx = torch.tensor([[0, 1]] * 4, dtype=torch.int32)
    d_w, d_s = randn(1, 4, k), randn(2, 4, S)
    got, _ = route_backward(logits, idx, d_w, d_s, E, S, F32, scale=(2.0, 1.0))
    ref, tol, _, _ = R.route_grad(logits[:3], idx[:3], d_w[:3], d_s[:3], E, S, True, 2.0, 1.0)
    R.assert_within(got[:3], ref, tol + 1e-38, "d_logits")
    # an expert whose logit is minus infinity has no weight and no gradient
    ref, tol, _, _ = R.route_grad(logits[3:].clamp(min=-1e4), idx[3:], d_w[3:], d_s[3:], E, S, True, 2.0, 1.0)
    assert got[3, 0] == 0
    # (the bound counts steps of the largest |l|, here of the finite ones: at most 4)
    R.assert_within(got[3:], ref, tol / 100 + 1e-38, "d_logits")


def test_router_gradient_of_repeated_and_missing_experts():
    E, k = 8, 4
    logits, _, d_w, _ = route_inputs(3, E, 0, k, F32, 0, seed=9)
    idx = torch.tensor([[1, 1, 1, 5], [-1, 8, 2, 3], [-1, -1, 100, -5]], dtype=torch.int32)
    got, _ = route_backward(logits, idx, d_w, None, E, 0, F32)
    ref, tol, _, _ = R.route_grad(logits, idx, d_w, None, E, 0, False)
    R.assert_within(got, ref, tol + ref.abs() * R.F32, "d_logits")
    assert (got[2] == 0).all()


@pytest.mark.parametrize("sink", [False, True])
def test_router_gradient_against_differences(sink):
    """Central differences of the oracle's 64-bit weights: steps of 2^-8 in fp32
    logits, whose h^2/6 times the third derivative (below 8 max|dw| c) bounds the error."""
    T, E, S, k = 2, 10, (2 if sink else 0), (6 if sink else 4)
    logits, _, d_w, d_s = route_inputs(T, E, S, k, F32, 0, seed=21, std=1.0)
    logits = (logits * 256).round() / 256
    rs, gs = (2.5, 0.5) if sink else (1.0, 1.0)
    if sink:
        idx, _, _ = oracle.route_sigmoid_sink(logits.numpy(), E, S, k, None, rs, gs)
    else:
        idx, _ = oracle.route_softmax_topk(logits.numpy(), E, k)
    idx = torch.from_numpy(np.array(idx)).int()

    def loss(z):  # the selection held fixed, as the gradient holds it
        cols = torch.cat([idx.long(), torch.arange(E, E + S).expand(T, S)], 1)
        v = z.double().gather(1, cols)
        w = torch.softmax(torch.nn.functional.logsigmoid(v) if sink else v, 1) * rs * gs
        return float((w * torch.cat([d_w, d_s] if sink else [d_w], 1).double()).sum())

    got, _ = route_backward(logits, idx, d_w, d_s, E, S, F32, scale=(rs, gs) if sink else None)
    h = 2.0 ** -8
    worst = 8 * rs * gs * float(max(d_w.abs().max(), d_s.abs().max() if sink else 0.0))
    for t in range(T):
        for c in range(E + S):
            up, down = logits.clone(), logits.clone()
            up[t, c] += h
            down[t, c] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - float(got[t, c])) <= worst * h * h / 6 + 1e-6


def test_no_tokens():
    """A batch of no tokens enqueues nothing; the global scale's gradient is the empty sum."""
    E, S, k = 4, 1, 3
    cfg = abi.config(0, 64, E, k, 64, router="sigmoid_sink", num_sink=S)
    ws = torch.full((abi.moe_operator_workspace_size(cfg),), 255, dtype=torch.uint8, device="cuda")
    e = lambda *s, dtype=F32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    i32, i8 = torch.int32, torch.int8
    d_gs = torch.full((1,), 7.0, device="cuda")
    abi.moe_route_backward(cfg, e(0, E + S), e(0, k, dtype=i32), e(0, k), e(0, E + S), d_sink_weights=e(0, S),
                           d_global_scale=d_gs, workspace=ws)
    assert float(d_gs) == 0.0
    abi.moe_dispatch(cfg, e(0, 64), e(0, dtype=i32), e(0, 64))
    abi.moe_combine_backward(cfg, e(0, 64), e(0, dtype=i32), e(0, 64), rows=e(0, 64), d_expert_weights=e(0, k))
    abi.moe_dispatch_int8(cfg, e(0, 64, dtype=BF16), e(0, dtype=i32), e(0, 64, dtype=i8), e(0))
    abi.moe_quantize_rows(cfg, e(0, 64, dtype=BF16), None, e(0, 64, dtype=i8), e(0))
    abi.moe_grouped_linear_int8(cfg, "down", e(0, 64, dtype=i8), e(0), e(E, 64, 64, dtype=i8), e(E, 64),
                                torch.zeros(E + 1, dtype=i32, device="cuda"), e(0, 64, dtype=BF16), ws)
    torch.cuda.synchronize()


def test_rows_past_32_bits():
    """Rows whose offsets pass 2^32 bytes and 2^31 values, in every row operator."""
    T, H, E, k = 140000, 8192, 4, 2
    cfg = abi.config(T, H, E, k, 8)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=BF16)
    inv = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    rows, out, d_w = torch.zeros(T * k, H, dtype=BF16, device="cuda"), torch.zeros_like(x), torch.zeros(T, k, device="cuda")
    abi.moe_dispatch(cfg, x, inv, rows, expert_weights=w)
    p2 = inv.view(T, k).long()
    some = torch.cat([torch.arange(50), torch.arange(T - 50, T)]).cuda()
    ref = (w[some][:, :, None].double() * x[some][:, None].double())
    assert ((rows[p2[some]].double() - ref).abs() <= ref.abs() * (R.HALF[BF16] + 2 * R.F32)).all()
    assert T * k * H > 2 ** 31 and int(p2[some].max()) * H > 2 ** 31
    terms = w[some][:, :, None].double() * rows[p2[some]].double()
    ref, mag = terms.sum(1), terms.abs().sum(1)
    dot = (x[some][:, None].double() * rows[p2[some]].double())
    for grad in (False, True):
        if grad:
            abi.moe_dispatch_backward(cfg, rows, inv, out, x=x, expert_weights=w, d_expert_weights=d_w)
            assert ((d_w[some].double() - dot.sum(2)).abs() <= R.tol_dots(dot.abs().sum(2), H)).all()
        else:
            abi.moe_combine(cfg, rows, inv, out, expert_weights=w)
        assert ((out[some].double() - ref).abs() <= R.tol_gather(ref, mag, k, BF16)).all()
    d_rows = torch.zeros_like(rows)
    abi.moe_combine_backward(cfg, x, inv, d_rows, rows=rows, expert_weights=w, d_expert_weights=d_w)
    assert torch.equal(d_rows, rows)                       # the same products as the dispatch's
    assert ((d_w[some].double() - dot.sum(2)).abs() <= R.tol_dots(dot.abs().sum(2), H)).all()


def test_int8_past_32_bits():
    """8-bit rows and weights past 2^31 bytes, a product past 2^31 values."""
    T, H, D, E = 270000, 8192, 8200, 16
    cfg = abi.config(T, H, E, 1, D)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=BF16)
    inv = torch.randperm(T, generator=g, device="cuda").to(torch.int32)
    q, s = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    abi.moe_dispatch_int8(cfg, x, inv, q, s)
    some = torch.cat([torch.arange(40), torch.arange(T - 40, T)]).cuda()
    token = torch.empty_like(inv)
    token[inv.long()] = torch.arange(T, dtype=torch.int32, device="cuda")
    rq, rs = R.quantize(x[token[some].long()].cpu())
    assert torch.equal(q[some].cpu().double(), rq) and torch.equal(s[some].cpu(), rs)
    w = (torch.randn(E, H, 2 * D, generator=g, device="cuda", dtype=BF16) * 0.02)
    w_q, w_s = torch.empty(E, 2 * D, H, dtype=torch.int8, device="cuda"), torch.empty(E, 2 * D, device="cuda")
    abi.moe_quantize_weights(cfg, "gate_up", w, w_q, w_s)
    assert E * 2 * D * H > 2 ** 31
    rq, rs = R.quantize(w[-1, :, -30:].T.contiguous().cpu())
    assert torch.equal(w_q[-1, -30:].cpu().double(), rq) and torch.equal(w_s[-1, -30:].cpu(), rs)
    del w
    bounds = torch.linspace(0, T, E + 1).to(torch.int32)
    out = torch.zeros(T, D, dtype=BF16, device="cuda")
    ws = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_grouped_linear_int8(cfg, "gate_up", q, s, w_q, w_s, bounds.cuda(), out, ws)
    assert abi.moe_device_status(ws) == 0
    for rows, e in ((some[:40], 0), (some[40:], E - 1)):
        ref, tol = R.linear_int8(q[rows].cpu(), s[rows].cpu(), w_q[e][None].cpu(), w_s[e][None].cpu(), None,
                                 torch.tensor([0, 40]), "gate_up", "concatenated", "silu", 0.0, 0.0,
                                 torch.zeros(40, D, dtype=BF16))
        R.assert_within(out[rows], ref, tol, f"expert {e}")


# ------------------------------------------------------------------ 8-bit
QUANT = [(1, 8, 1), (3, 24, 2), (5, 520, 3), (2, 4096, 8), (7, 16400, 2), (4, 2880, 1), (600, 1000, 2), (450, 2888, 4),
         (333, 33000, 1)]


@pytest.mark.parametrize("T,H,k", QUANT)
def test_dispatch_int8(T, H, k):
    E = 9
    cfg = abi.config(T, H, E, k, 8)
    _, off, inv = R.routing(T, E, k, seed=T + H, drop=0.3)
    x = randn(H, T, H, dtype=BF16)
    x[0] = (x[0].float() * 1e-38).to(BF16)              # denormal maxima
    if T > 1:
        x[1] = 0
        x[1, H // 2] = 2.0 ** -133                      # the smallest value
    if T > 2:
        x[2] = 0
    q = torch.full((T * k, abi.int8_pitch(H)), 77, dtype=torch.int8, device="cuda")
    s = torch.full((T * k,), -3.0, device="cuda")
    abi.moe_dispatch_int8(cfg, x.cuda(), inv.cuda(), q, s)
    rq, rs = R.quantize(x)
    want_q = torch.full((T * k, abi.int8_pitch(H)), 77.0, dtype=torch.float64)
    want_s = torch.full((T * k,), -3.0)
    for slot, p in enumerate(inv.tolist()):
        if p >= 0:
            want_q[p], want_s[p] = 0, rs[slot // k]
            want_q[p, :H] = rq[slot // k]
    assert torch.equal(q.cpu().double(), want_q)
    assert torch.equal(s.cpu(), want_s)


@pytest.mark.parametrize("rows", [1, 70, 400])
@pytest.mark.parametrize("n", [8, 264, 1536, 33000])
def test_quantize_rows(rows, n):
    cfg = abi.config(rows, 8, 3, 1, n)
    h = randn(n, rows, n, dtype=BF16)
    h[-1] = (torch.arange(n) % 2 * 2 - 1).to(BF16) * 0.5  # every value a tie at half of the largest
    h[-1, 0] = -1.0
    live = rows - rows // 3
    off = torch.tensor([0, live // 2, live // 2, live], dtype=torch.int32)
    rq, rs = R.quantize(h)
    for offsets, m in ((off, live), (None, rows)):
        q = torch.full((rows, abi.int8_pitch(n)), 77, dtype=torch.int8, device="cuda")
        s = torch.full((rows,), -3.0, device="cuda")
        abi.moe_quantize_rows(cfg, h.cuda(), cuda(offsets), q, s)
        assert torch.equal(q[:m, :n].cpu().double(), rq[:m]) and torch.equal(s[:m].cpu(), rs[:m])
        assert (q[:m, n:] == 0).all()
        assert (q[m:] == 77).all() and (s[m:] == -3.0).all()


def test_quantize_every_value():
    """All finite bf16 values of a binade and every tie, under every maximum's significand."""
    tops = (torch.arange(128, 256).float() / 128).to(BF16)
    vals = torch.cat([torch.arange(0, 256).float() / 128 * 2.0 ** -e for e in range(0, 9)]).to(BF16)
    h = vals[None, :].expand(128, -1).clone()
    h = torch.where(h.float().abs() <= tops[:, None].float(), h, torch.zeros((), dtype=BF16))
    h[:, 1::2] *= -1
    h[:, 0] = tops
    n = h.shape[1]
    cfg = abi.config(128, 8, 1, 1, n)
    q = torch.empty(128, abi.int8_pitch(n), dtype=torch.int8, device="cuda")
    s = torch.empty(128, device="cuda")
    abi.moe_quantize_rows(cfg, h.cuda(), None, q, s)
    rq, rs = R.quantize(h)
    assert torch.equal(q[:, :n].cpu().double(), rq) and torch.equal(s.cpu(), rs)


def test_rows_with_nan_or_infinity_get_nan_scales():
    cfg = abi.config(4, 8, 1, 1, 64)
    h = randn(1, 4, 64, dtype=BF16)
    h[1, 5], h[2, 7], h[3, 0] = float("nan"), float("inf"), float("-inf")
    q, s = torch.empty(4, 64, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    abi.moe_quantize_rows(cfg, h.cuda(), None, q, s)
    assert torch.isfinite(s[0]) and torch.isnan(s[1:]).all()


@pytest.mark.parametrize("part", ["gate_up", "down"])
@pytest.mark.parametrize("E,H,D", [(1, 8, 8), (3, 264, 40), (2, 136, 520), (1, 1000, 72), (1, 4104, 24), (1, 16, 12304), (2, 40, 1288)])
def test_quantize_weights(E, H, D, part):
    cfg = abi.config(2, H, E, 1, D)
    K, N = (H, 2 * D) if part == "gate_up" else (D, H)
    w = randn(K + N, E, K, N, dtype=BF16, std=0.02)
    w[0, :, 0] = 0
    w[0, :, 1] = 2.0 ** -130
    q = torch.full((E, N, abi.int8_pitch(K)), 77, dtype=torch.int8, device="cuda")
    s = torch.full((E, N), -1.0, device="cuda")
    abi.moe_quantize_weights(cfg, part, w.cuda(), q, s)
    rq, rs = R.quantize(w.transpose(1, 2))
    assert torch.equal(q[..., :K].cpu().double(), rq) and torch.equal(s.cpu(), rs)
    assert (q[..., K:] == 0).all()


def int8_case(T, H, D, E, k, part, fmt="concatenated", act="silu", bias=False, drop=0.0, one=None, limit=None, seed=0):
    alpha = R.ALPHA if act == "swigluoai" else 0.0
    limit = (R.LIMIT if act == "swigluoai" else 0.0) if limit is None else limit
    cfg = abi.config(T, H, E, k, D, gate_up_format=fmt, activation=act, alpha=alpha, limit=limit, has_bias=bias)
    _, off, inv = R.routing(T, E, k, seed=T + H + seed, drop=drop, one_expert=one)
    K, N = (H, 2 * D) if part == "gate_up" else (D, H)
    g = torch.Generator().manual_seed(seed + K)
    # the padding of the rows holds anything: it is not read
    q = torch.randint(-127, 128, (T * k, abi.int8_pitch(K)), generator=g, dtype=torch.int8)
    w_q = torch.randint(-127, 128, (E, N, abi.int8_pitch(K)), generator=g, dtype=torch.int8)
    s = torch.rand(T * k, generator=g) * 0.02 + 0.005
    w_s = (torch.rand(E, N, generator=g) + 0.5) * 0.02 / K ** 0.5
    b = randn(seed, E, N, dtype=BF16, std=0.3) if bias else None
    before = randn(seed + 1, T * k, D if part == "gate_up" else H, dtype=BF16)
    out = before.cuda()
    ws = torch.full((abi.moe_operator_workspace_size(cfg),), 255, dtype=torch.uint8, device="cuda")
    abi.moe_grouped_linear_int8(cfg, part, q.cuda(), s.cuda(), w_q.cuda(), w_s.cuda(), off.cuda(), out, ws, bias=cuda(b))
    assert abi.moe_device_status(ws) == 0
    ref, tol = R.linear_int8(q[:, :K], s, w_q[..., :K], w_s, b, off, part, fmt, act, alpha, limit, before)
    R.assert_within(out, ref, tol, f"{part} {fmt} {act}")


INT8 = [  # T, H, D, E, k, drop, all on one expert
    (1, 8, 8, 1, 1, 0.0, None), (1, 264, 136, 8, 2, 0.0, None), (64, 128, 128, 1, 1, 0.0, 0), (65, 144, 256, 2, 1, 0.0, 1),
    (128, 392, 264, 3, 2, 0.0, 0), (129, 256, 128, 4, 1, 0.3, 2), (300, 520, 200, 40, 6, 0.1, None), (33, 1000, 96, 5, 3, 1.0, None),
    (700, 136, 72, 3, 2, 0.0, None), (300, 264, 1048, 30, 2, 0.1, None), (31, 1544, 2056, 40, 3, 0.0, 7),
    (1300, 2576, 2568, 5, 2, 0.1, 1), (2000, 3080, 1544, 3, 1, 0.0, 2), (900, 2312, 2600, 9, 1, 0.0, None),
]


@pytest.mark.parametrize("part", ["gate_up", "down"])
@pytest.mark.parametrize("T,H,D,E,k,drop,one", INT8)
def test_grouped_linear_int8(T, H, D, E, k, drop, one, part):
    int8_case(T, H, D, E, k, part, drop=drop, one=one)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("fmt", ["concatenated", "interleaved"])
@pytest.mark.parametrize("act,limit", [("silu", 0.0), ("silu", 1.5), ("swigluoai", 7.0), ("swigluoai", 0.0), ("gelu_tanh", 0.0)])
@pytest.mark.parametrize("T,H,D,E,k", [(150, 264, 328, 6, 2), (300, 264, 328, 40, 2), (1200, 264, 1288, 5, 1)],
                         ids=["few_tiles", "few_rows", "many_rows"])
def test_grouped_linear_int8_activations(T, H, D, E, k, act, limit, fmt, bias):
    int8_case(T, H, D, E, k, "gate_up", fmt=fmt, act=act, limit=limit, bias=bias, seed=7)
    if act == "silu" and limit == 0:
        int8_case(T, 8 * D, H, E, k, "down", fmt=fmt, bias=bias, seed=8)


@pytest.mark.parametrize("K", [1016, 1032, 2184, 4104, 8200])
@pytest.mark.parametrize("T,N,E,k,drop,one", [
    (1, 128, 1, 1, 0.0, None), (17, 136, 2, 1, 0.0, None), (100, 264, 3, 2, 0.2, None), (128, 512, 4, 1, 0.0, 2),
    (130, 128, 2, 1, 0.0, 0), (12, 1040, 5, 2, 1.0, None), (300, 520, 6, 1, 0.0, None)])
def test_grouped_linear_int8_long_k_few_tiles(K, T, N, E, k, drop, one):
    """A K that several blocks share: from two parts to eight, equal and not, with one
    row and with two pieces, empty experts and no row at all."""
    int8_case(T, N, K, E, k, "down", drop=drop, one=one, seed=11, bias=T % 2 == 1)
    int8_case(T, K, N // 16 * 8, E, k, "gate_up", drop=drop, one=one, seed=12, fmt="concatenated" if T % 2 else "interleaved",
              act="swigluoai", bias=T % 2 == 0)


@pytest.mark.parametrize("part", ["gate_up", "down"])
@pytest.mark.parametrize("rows", [1, 16, 31, 100, 128])
def test_grouped_linear_int8_same_bits_however_k_is_shared(rows, part):
    """The same rows and weights in batches of other sizes, which share K otherwise or not at all."""
    K, N, E = 4104, 256, 2
    H, D = (K, N // 2) if part == "gate_up" else (N, K)
    g = torch.Generator().manual_seed(rows)
    w_q = torch.randint(-127, 128, (E, N, abi.int8_pitch(K)), generator=g, dtype=torch.int8).cuda()
    w_s = (torch.rand(E, N, generator=g) * 0.002).cuda()
    q = torch.randint(-127, 128, (7000, abi.int8_pitch(K)), generator=g, dtype=torch.int8).cuda()
    s = (torch.rand(7000, generator=g) * 0.02).cuda()
    off = torch.tensor([0, 0, rows], dtype=torch.int32, device="cuda")
    outs = []
    for T in (rows, 600, 1400, 7000):  # 4, 12 (or 4), 24 and 112 tiles at most
        cfg = abi.config(T, H, E, 1, D)
        out = torch.zeros(T, D if part == "gate_up" else H, dtype=BF16, device="cuda")
        ws = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        abi.moe_grouped_linear_int8(cfg, part, q[:T], s[:T], w_q, w_s, off, out, ws)
        assert abi.moe_device_status(ws) == 0 and not out[rows:].any()
        outs.append(out[:rows])
    assert outs[0].any() and all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("H,D", [(2056, 64), (72, 2504)], ids=["shared_k", "whole_k"])
def test_grouped_linear_int8_offsets_written_just_before(H, D):
    """Offsets that the kernel right before writes: the product may have begun when they
    were still those of the call before, and goes by the new ones."""
    T, E, k = 40, 6, 2
    cfg = abi.config(T, H, E, k, D)
    R_ = T * k
    idx = [R.routing(T, E, k, seed=i, drop=0.3 * i, one_expert=4 if i == 2 else None)[0].cuda() for i in range(3)]
    g = torch.Generator().manual_seed(9)
    q = torch.randint(-127, 128, (R_, abi.int8_pitch(H)), generator=g, dtype=torch.int8).cuda()
    w_q = torch.randint(-127, 128, (E, 2 * D, abi.int8_pitch(H)), generator=g, dtype=torch.int8).cuda()
    s, w_s = (torch.rand(R_, generator=g) * 0.02).cuda(), (torch.rand(E, 2 * D, generator=g) * 0.002).cuda()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    perm, inv = torch.zeros(R_, dtype=torch.int32, device="cuda"), torch.zeros(R_, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(abi.moe_workspace_size(cfg), abi.moe_operator_workspace_size(cfg)), dtype=torch.uint8, device="cuda")
    ows = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    want = []
    for i in range(3):
        out = torch.zeros(R_, D, dtype=BF16, device="cuda")
        abi.moe_create_indices(cfg, idx[i], off, perm, inv, ws)
        torch.cuda.synchronize()
        abi.moe_grouped_linear_int8(cfg, "gate_up", q, s, w_q, w_s, off, out, ows)
        torch.cuda.synchronize()
        want.append(out)
    assert not torch.equal(want[0], want[1]) and not torch.equal(want[0], want[2])
    outs = [torch.zeros(R_, D, dtype=BF16, device="cuda") for _ in range(60)]
    for i, out in enumerate(outs):
        abi.moe_create_indices(cfg, idx[i % 3], off, perm, inv, ws)
        abi.moe_grouped_linear_int8(cfg, "gate_up", q, s, w_q, w_s, off, out, ows)
    assert all(torch.equal(out, want[i % 3]) for i, out in enumerate(outs))


def test_grouped_linear_int8_same_bits_in_every_tile_shape():
    """A row's product does not depend on how many rows its expert has, nor on the
    kernel that takes them."""
    H, D, E = 392, 1288, 4
    g = torch.Generator().manual_seed(5)
    w_q = torch.randint(-127, 128, (E, 2 * D, abi.int8_pitch(H)), generator=g, dtype=torch.int8).cuda()
    w_s = (torch.rand(E, 2 * D, generator=g) * 0.002).cuda()
    q = torch.randint(-127, 128, (2000, abi.int8_pitch(H)), generator=g, dtype=torch.int8).cuda()
    s = (torch.rand(2000, generator=g) * 0.02).cuda()
    outs = []
    for T in (2000, 60, 5):
        cfg = abi.config(T, H, E, 1, D, activation="swigluoai", alpha=R.ALPHA, limit=R.LIMIT)
        out = torch.zeros(T, D, dtype=BF16, device="cuda")
        ws = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        off = torch.tensor([0, T, T, T, T], dtype=torch.int32, device="cuda")   # all rows to expert 0
        abi.moe_grouped_linear_int8(cfg, "gate_up", q[:T], s[:T], w_q, w_s, off, out, ws)
        outs.append(out)
    assert torch.equal(outs[0][:60], outs[1]) and torch.equal(outs[0][:5], outs[2])


def test_grouped_linear_int8_largest_sums():
    """Every product 127 * 127 (and its negative) over the longest K: 2,114,060,288 in 32 bits."""
    K = 131072
    cfg = abi.config(2, 16, 1, 1, K)
    q = torch.full((2, K), 127, dtype=torch.int8, device="cuda")
    q[1] = -127
    w = torch.full((1, 16, K), 127, dtype=torch.int8, device="cuda")
    s, w_s = torch.ones(2, device="cuda"), torch.ones(1, 16, device="cuda")
    out = torch.zeros(2, 16, dtype=BF16, device="cuda")
    ws = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    abi.moe_grouped_linear_int8(cfg, "down", q, s, w, w_s, off, out, ws)
    want = torch.tensor([127.0 * 127 * K, -127.0 * 127 * K]).to(BF16)[:, None].expand(2, 16)
    assert torch.equal(out.cpu(), want)


def test_grouped_linear_int8_non_finite_scales():
    T, H, D, E = 5, 128, 64, 1
    cfg = abi.config(T, H, E, 1, D)
    q = torch.randint(-127, 128, (T, D), dtype=torch.int8)
    w = torch.randint(-127, 128, (E, H, D), dtype=torch.int8)
    s, w_s = torch.ones(T), torch.ones(E, H)
    s[2], w_s[0, 7] = float("nan"), 0.0
    out = torch.zeros(T, H, dtype=BF16, device="cuda")
    ws = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_grouped_linear_int8(cfg, "down", q.cuda(), s.cuda(), w.cuda(), w_s.cuda(),
                                torch.tensor([0, T], dtype=torch.int32).cuda(), out, ws)
    assert torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 3, 4]]).all() and (out[[0, 1, 3, 4], 7] == 0).all()


@pytest.mark.parametrize("act,limit", [("silu", 0.0), ("silu", 2.0), ("swigluoai", 7.0), ("gelu_tanh", 0.0)])
def test_grouped_linear_int8_nan_rows_stay_nan(act, limit):
    """A row with a NaN scale gives a row of NaN through every activation and clamp."""
    T, H, D, E = 70, 64, 40, 1
    cfg = abi.config(T, H, E, 1, D, activation=act, alpha=R.ALPHA if act == "swigluoai" else 0.0, limit=limit)
    q, w = torch.ones(T, H, dtype=torch.int8, device="cuda"), torch.ones(E, 2 * D, H, dtype=torch.int8, device="cuda")
    s, w_s = torch.full((T,), 0.1, device="cuda"), torch.full((E, 2 * D), 0.1, device="cuda")
    s[3] = s[69] = float("nan")
    out = torch.zeros(T, D, dtype=BF16, device="cuda")
    ws = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_grouped_linear_int8(cfg, "gate_up", q, s, w, w_s, torch.tensor([0, T], dtype=torch.int32).cuda(), out, ws)
    nan = torch.isnan(out).cpu()
    want = torch.zeros(T, D, dtype=torch.bool)
    want[[3, 69]] = True
    assert torch.equal(nan, want)


def test_grouped_linear_int8_largest_expert_count():
    int8_case(700, 64, 72, 1024, 2, "gate_up", seed=3)
    int8_case(700, 64, 72, 1024, 2, "down", drop=0.3, seed=4)


@pytest.mark.parametrize("offsets", [[0, 9, 8, 10], [0, 4, 8, 11], [1, 4, 8, 10], [0, -3, 8, 10], [0, 2 ** 30, 5, 10]])
def test_grouped_linear_int8_bad_offsets(offsets):
    """Offsets that are no CSR of at most R rows are recorded and nothing is written."""
    T, H, D, E = 10, 64, 64, 3
    cfg = abi.config(T, H, E, 1, D)
    q, w = torch.ones(T, D, dtype=torch.int8, device="cuda"), torch.ones(E, H, D, dtype=torch.int8, device="cuda")
    s, w_s = torch.ones(T, device="cuda"), torch.ones(E, H, device="cuda")
    out = torch.full((T, H), 3.0, dtype=BF16, device="cuda")
    ws = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_grouped_linear_int8(cfg, "down", q, s, w, w_s, torch.tensor(offsets, dtype=torch.int32).cuda(), out, ws)
    assert abi.moe_device_status(ws) == abi.DEVICE_ERR_CSR
    assert (out == 3.0).all()
    abi.moe_grouped_linear_int8(cfg, "down", q, s, w, w_s, torch.tensor([0, 4, 4, 10], dtype=torch.int32).cuda(), out, ws)
    assert abi.moe_device_status(ws) == 0 and (out == 64.0).all()


def test_create_indices_marks_skipped_slots():
    """A slot whose expert index is out of range has inverse -1, in each form of the build."""
    for T, E, k, form in ((10, 8, 2, "1"), (10, 8, 2, "0"), (5000, 64, 3, "1"), (5000, 64, 3, "0")):
        with pytest.MonkeyPatch.context() as mp:
            mp.setenv("MOE_B200_CSR_FUSED", form)
            cfg = abi.config(T, 8, E, k, 8)
            idx, off, inv = R.routing(T, E, k, seed=T, drop=0.3)
            ws = torch.empty(abi.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
            o = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            p, i = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.full((T * k,), 12345, dtype=torch.int32, device="cuda")
            abi.moe_create_indices(cfg, idx.cuda(), o, p, i, ws)
            assert torch.equal(o.cpu(), off) and torch.equal(i.cpu(), inv)


# --------------------------------------------------------------- together
def test_training_step_through_the_routing():
    """moe_route -> moe_create_indices -> moe_dispatch -> experts (a matrix each)
    -> moe_combine and back, in fp32, against autograd in 64 bits."""
    T, H, E, S, k = 60, 64, 8, 2, 6
    cfg = abi.config(T, H, E, k, 8, router="sigmoid_sink", num_sink=S, route_scale=2.5)
    x, logits, W = randn(1, T, H), randn(2, T, E + S), randn(3, E, H, H, std=H ** -0.5)
    gs, d_out = torch.tensor([0.8]), randn(4, T, H)
    dev = {n: t.cuda() for n, t in dict(x=x, logits=logits, W=W, gs=gs, d_out=d_out).items()}
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, w, sw = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda"), torch.empty(T, S, device="cuda")
    off, perm, inv = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T * k, **i32)
    ws = torch.empty(abi.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_route(cfg, dev["logits"], idx, w, sink_weights=sw, global_scale=dev["gs"])
    abi.moe_create_indices(cfg, idx, off, perm, inv, ws)
    rows, y = torch.empty(T * k, H, device="cuda"), torch.empty(T * k, H, device="cuda")
    abi.moe_dispatch(cfg, dev["x"], inv, rows)
    o = off.tolist()
    for e in range(E):
        y[o[e]:o[e + 1]] = rows[o[e]:o[e + 1]] @ dev["W"][e]
    out = torch.empty(T, H, device="cuda")
    abi.moe_combine(cfg, y, inv, out, expert_weights=w)
    d_y, d_w, d_rows = torch.empty_like(y), torch.empty_like(w), torch.empty_like(rows)
    abi.moe_combine_backward(cfg, dev["d_out"], inv, d_y, rows=y, expert_weights=w, d_expert_weights=d_w)
    for e in range(E):
        d_rows[o[e]:o[e + 1]] = d_y[o[e]:o[e + 1]] @ dev["W"][e].T
    d_x, d_logits, d_gs = torch.empty_like(dev["x"]), torch.empty_like(dev["logits"]), torch.empty(1, device="cuda")
    abi.moe_dispatch_backward(cfg, d_rows, inv, d_x)
    ows = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_route_backward(cfg, dev["logits"], idx, d_w, d_logits, global_scale=dev["gs"], d_global_scale=d_gs,
                           workspace=ows)
    # 64 bits, the same selection
    X, Z, G = x.double().requires_grad_(), logits.double().requires_grad_(), gs.double().requires_grad_()
    cols = torch.cat([idx.cpu().long(), torch.arange(E, E + S).expand(T, S)], 1)
    p = torch.softmax(torch.nn.functional.logsigmoid(Z.gather(1, cols)), 1) * 2.5 * G
    experts = torch.einsum("th,tkhi->tki", X, W.double()[idx.cpu().long()])
    ref = (p[:, :k, None] * experts).sum(1)
    ref.backward(d_out.double())
    # sums of H products of H-term sums in fp32 against 64 bits: H + k + 40 steps of the
    # terms' size, which random signs keep within sqrt(H) of the result's
    for got, want, n in ((out, ref, H), (d_x, X.grad, H * k), (d_logits, Z.grad, H * k), (d_gs, G.grad, H * k * T)):
        scale = float(want.detach().abs().max()) * n ** 0.5
        assert float((got.cpu().double() - want.detach()).abs().max()) <= scale * (H + k + 40) * R.F32


@pytest.mark.parametrize("fmt,act,bias", [("concatenated", "silu", False), ("interleaved", "swigluoai", True)])
def test_int8_layer(fmt, act, bias):
    """The 8-bit layer from bf16 weights to the combined output: each step
    against its 64-bit form on the step before's output, and the whole near
    the bf16 layer (moe_forward)."""
    T, H, D, E, k = 200, 264, 328, 8, 2
    alpha, limit = (R.ALPHA, R.LIMIT) if act == "swigluoai" else (0.0, 0.0)
    cfg = abi.config(T, H, E, k, D, gate_up_format=fmt, activation=act, alpha=alpha, limit=limit, has_bias=bias)
    x, logits = randn(1, T, H, dtype=BF16).cuda(), randn(2, T, E).cuda()
    W = {"gate_up": randn(3, E, H, 2 * D, dtype=BF16, std=0.05).cuda(), "down": randn(4, E, D, H, dtype=BF16, std=0.05).cuda()}
    B = {"gate_up": randn(5, E, 2 * D, dtype=BF16, std=0.1).cuda(), "down": randn(6, E, H, dtype=BF16, std=0.1).cuda()} if bias else {}
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
    off, perm, inv = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T * k, **i32)
    ws = torch.empty(abi.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_route(cfg, logits, idx, w)
    abi.moe_create_indices(cfg, idx, off, perm, inv, ws)
    q, s = {}, {}
    for part, K, N in (("gate_up", H, 2 * D), ("down", D, H)):
        q[part] = torch.empty(E, N, abi.int8_pitch(K), dtype=torch.int8, device="cuda")
        s[part] = torch.empty(E, N, device="cuda")
        abi.moe_quantize_weights(cfg, part, W[part], q[part], s[part])
    rq = torch.empty(T * k, abi.int8_pitch(H), dtype=torch.int8, device="cuda")
    hq = torch.empty(T * k, abi.int8_pitch(D), dtype=torch.int8, device="cuda")
    rs, hs = torch.empty(T * k, device="cuda"), torch.empty(T * k, device="cuda")
    h, y = (torch.empty(T * k, n, dtype=BF16, device="cuda") for n in (D, H))
    out = torch.empty(T, H, dtype=BF16, device="cuda")
    ows = torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")

    def layer():
        abi.moe_dispatch_int8(cfg, x, inv, rq, rs)
        abi.moe_grouped_linear_int8(cfg, "gate_up", rq, rs, q["gate_up"], s["gate_up"], off, h, ows, bias=B.get("gate_up"))
        abi.moe_quantize_rows(cfg, h, off, hq, hs)
        abi.moe_grouped_linear_int8(cfg, "down", hq, hs, q["down"], s["down"], off, y, ows, bias=B.get("down"))
        abi.moe_combine(cfg, y, inv, out, expert_weights=w)

    layer()
    assert abi.moe_device_status(ows) == 0
    c = lambda t: None if t is None else t.cpu()  # noqa: E731
    for part, aq, a_s, dst, K in (("gate_up", rq, rs, h, H), ("down", hq, hs, y, D)):
        ref, tol = R.linear_int8(aq[:, :K].cpu(), a_s.cpu(), q[part][..., :K].cpu(), s[part].cpu(), c(B.get(part)), off.cpu(),
                                 part, fmt, act, alpha, limit, dst.cpu())
        R.assert_within(dst, ref, tol, part)
    tq, ts = R.quantize(h.cpu())
    assert torch.equal(hq[:, :D].cpu().double(), tq) and torch.equal(hs.cpu(), ts)
    ref, mag = R.gather(y.cpu(), inv.cpu().view(T, k), w.cpu())
    R.assert_within(out, ref, R.tol_gather(ref, mag, k, BF16), "combine")
    # against the bf16 layer: each of the four quantised operands errs by at most
    # half a step of its row's largest value, about 1/64 of the row's rms at
    # these sizes and independent over K, twice through a product of two: 5%
    full = torch.empty_like(out)
    abi.moe_forward(cfg, x, logits, W["gate_up"], W["down"], full, ws, gate_up_b=B.get("gate_up"), down_b=B.get("down"))
    err = (out.double() - full.double()).norm() / full.double().norm()
    assert float(err) < 0.05, float(err)
    # captured and replayed on another stream, the same bits
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            layer()
    out.zero_(), h.zero_(), y.zero_(), rq.zero_(), hq.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_row_gradients_against_differences():
    """Dispatch and combine are linear in rows and weights, so a difference of the
    forward pass is the gradient up to rounding: along random directions, fp32
    outputs summed in 64 bits."""
    T, H, E, k = 37, 136, 6, 3
    cfg = abi.config(T, H, E, k, 8)
    _, _, inv = R.routing(T, E, k, seed=4, drop=0.2)
    inv = inv.cuda()
    x, rows, w = randn(1, T, H).cuda(), randn(2, T * k, H).cuda(), randn(3, T, k).cuda()
    dx, drows, dw = randn(4, T, H).cuda(), randn(5, T * k, H).cuda(), randn(6, T, k).cuda()
    g_rows, g_out = randn(7, T * k, H).cuda(), randn(8, T, H).cuda()

    def dispatch(x, w):
        out = torch.zeros(T * k, H, device="cuda")
        abi.moe_dispatch(cfg, x, inv, out, expert_weights=w)
        return out.double()

    def combine(rows, w):
        out = torch.zeros(T, H, device="cuda")
        abi.moe_combine(cfg, rows, inv, out, expert_weights=w)
        return out.double()

    b_x, b_w = torch.empty_like(x), torch.empty_like(w)
    abi.moe_dispatch_backward(cfg, g_rows, inv, b_x, x=x, expert_weights=w, d_expert_weights=b_w)
    c_rows, c_w = torch.zeros_like(rows), torch.empty_like(w)
    abi.moe_combine_backward(cfg, g_out, inv, c_rows, rows=rows, expert_weights=w, d_expert_weights=c_w)
    for f, a, da, grad, g in ((lambda v: dispatch(v, w), x, dx, b_x, g_rows), (lambda v: dispatch(x, v), w, dw, b_w, g_rows),
                              (lambda v: combine(v, w), rows, drows, c_rows, g_out), (lambda v: combine(rows, v), w, dw, c_w, g_out)):
        up, down = f(a + da), f(a - da)
        diff = float(((up - down) / 2 * g.double()).sum())
        along = float((grad.double() * da.double()).sum())
        # each of the T*k*H terms of up and down rounds k + 3 times; the gradient sums H / 32 + 24 deep
        size = float(((up.abs() + down.abs()) * g.double().abs()).sum()) + float((grad.double() * da.double()).abs().sum())
        assert abs(diff - along) <= size * (k + 3 + H / 32 + 24) * R.F32


def test_two_calls_at_once():
    """The same operators on two streams at the same time, a workspace each."""
    T, H, D, E, k = 500, 520, 264, 12, 2
    cfg = abi.config(T, H, E, k, D)
    jobs = []
    for i in range(2):
        _, off, inv = R.routing(T, E, k, seed=30 + i)
        g = torch.Generator().manual_seed(i)
        jobs.append(dict(
            off=off.cuda(), inv=inv.cuda(), x=randn(i, T, H, dtype=BF16).cuda(),
            w_q=torch.randint(-127, 128, (E, 2 * D, abi.int8_pitch(H)), generator=g, dtype=torch.int8).cuda(),
            w_s=(torch.rand(E, 2 * D, generator=g) * 0.01).cuda(), stream=torch.cuda.Stream(),
            q=torch.zeros(T * k, abi.int8_pitch(H), dtype=torch.int8, device="cuda"), s=torch.zeros(T * k, device="cuda"),
            h=torch.zeros(T * k, D, dtype=BF16, device="cuda"),
            ws=torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")))

    def run(j, stream=None):
        abi.moe_dispatch_int8(cfg, j["x"], j["inv"], j["q"], j["s"], stream=stream)
        abi.moe_grouped_linear_int8(cfg, "gate_up", j["q"], j["s"], j["w_q"], j["w_s"], j["off"], j["h"], j["ws"],
                                    stream=stream)

    want = []
    for j in jobs:
        run(j)
        torch.cuda.synchronize()
        want.append(j["h"].clone())
    for j in jobs:
        j["h"].zero_(), j["q"].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            run(j, j["stream"])
    torch.cuda.synchronize()
    for j, w in zip(jobs, want):
        assert torch.equal(j["h"], w) and abi.moe_device_status(j["ws"]) == 0


def test_calls_from_threads():
    """Four threads, a stream each, make the same kinds of calls at once."""
    import threading
    T, H, D, E, k = 40, 264, 136, 6, 2
    cfg = abi.config(T, H, E, k, D)
    g = torch.Generator().manual_seed(3)
    w_q = torch.randint(-127, 128, (E, 2 * D, abi.int8_pitch(H)), generator=g, dtype=torch.int8).cuda()
    w_s = (torch.rand(E, 2 * D, generator=g) * 0.01).cuda()
    jobs = []
    for i in range(4):
        _, off, inv = R.routing(T, E, k, seed=60 + i, drop=0.1 * i)
        jobs.append(dict(off=off.cuda(), inv=inv.cuda(), x=randn(60 + i, T, H, dtype=BF16).cuda(), stream=torch.cuda.Stream(),
                         q=torch.zeros(T * k, abi.int8_pitch(H), dtype=torch.int8, device="cuda"),
                         s=torch.zeros(T * k, device="cuda"), h=torch.zeros(T * k, D, dtype=BF16, device="cuda"),
                         rows=torch.zeros(T * k, H, dtype=BF16, device="cuda"), out=torch.zeros(T, H, dtype=BF16, device="cuda"),
                         ws=torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda")))

    def run(j):
        abi.moe_dispatch(cfg, j["x"], j["inv"], j["rows"])
        abi.moe_combine(cfg, j["rows"], j["inv"], j["out"])
        abi.moe_dispatch_int8(cfg, j["x"], j["inv"], j["q"], j["s"])
        abi.moe_grouped_linear_int8(cfg, "gate_up", j["q"], j["s"], w_q, w_s, j["off"], j["h"], j["ws"])

    want = []
    for j in jobs:
        run(j)
        torch.cuda.synchronize()
        want.append((j["out"].clone(), j["h"].clone()))
        j["out"].zero_(), j["h"].zero_()
    torch.cuda.synchronize()
    errors = []

    def thread(j):
        try:
            with torch.cuda.stream(j["stream"]):
                for _ in range(50):
                    run(j)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for j, (out, h) in zip(jobs, want):
        assert torch.equal(j["out"], out) and torch.equal(j["h"], h) and abi.moe_device_status(j["ws"]) == 0


def test_int8_shared_k_captured_and_at_once():
    """A K shared by blocks, captured: two graphs (a workspace each) replayed on two
    streams at the same time, on inputs that change between the replays."""
    T, H, D, E, k = 6, 4104, 136, 4, 2
    cfg = abi.config(T, H, E, k, D)
    g = torch.Generator().manual_seed(8)
    w_q = torch.randint(-127, 128, (E, 2 * D, abi.int8_pitch(H)), generator=g, dtype=torch.int8).cuda()
    w_s = (torch.rand(E, 2 * D, generator=g) * 0.002).cuda()
    xs = [randn(40 + i, T, H, dtype=BF16).cuda() for i in range(4)]
    routes = [[t.cuda() for t in R.routing(T, E, k, seed=50 + i, drop=0.2)[1:]] for i in range(4)]

    def job():
        return dict(x=xs[0].clone(), off=routes[0][0].clone(), inv=routes[0][1].clone(),
                    q=torch.zeros(T * k, abi.int8_pitch(H), dtype=torch.int8, device="cuda"), s=torch.zeros(T * k, device="cuda"),
                    h=torch.zeros(T * k, D, dtype=BF16, device="cuda"),
                    ws=torch.empty(abi.moe_operator_workspace_size(cfg), dtype=torch.uint8, device="cuda"))

    def run(j):
        j["h"].zero_()
        abi.moe_dispatch_int8(cfg, j["x"], j["inv"], j["q"], j["s"])
        abi.moe_grouped_linear_int8(cfg, "gate_up", j["q"], j["s"], w_q, w_s, j["off"], j["h"], j["ws"])

    def load(j, i):
        j["x"].copy_(xs[i]), j["off"].copy_(routes[i][0]), j["inv"].copy_(routes[i][1])

    plain, want = job(), []
    for i in range(4):
        load(plain, i)
        run(plain)
        torch.cuda.synchronize()
        want.append(plain["h"].clone())
    assert all(w.any() for w in want) and not torch.equal(want[0], want[1])
    jobs, graphs, streams = [job(), job()], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for j, st in zip(jobs, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            run(j)
        graphs.append(gr)
    torch.cuda.synchronize()
    for i in range(12):
        got = []
        for n, (j, st) in enumerate(zip(jobs, streams)):
            with torch.cuda.stream(st):
                load(j, (i + n) % 4)
                graphs[n].replay()
                got.append(j["h"].clone())
        torch.cuda.synchronize()
        for n, h in enumerate(got):
            assert torch.equal(h, want[(i + n) % 4]) and abi.moe_device_status(jobs[n]["ws"]) == 0


def test_backward_captured_and_on_a_given_stream():
    T, H, E, k = 300, 520, 16, 3
    cfg = abi.config(T, H, E, k, 8, logits_dtype=F32)
    _, _, inv = R.routing(T, E, k, seed=2)
    idx, _, _ = R.routing(T, E, k, seed=2)
    x, rows, w, inv = randn(1, T, H).cuda(), randn(2, T * k, H).cuda(), randn(3, T, k).cuda(), inv.cuda()
    logits, idx = randn(4, T, E).cuda(), idx.cuda()
    d_x, d_rows, d_w, d_l = torch.empty_like(x), torch.empty_like(rows), torch.empty_like(w), torch.empty_like(logits)

    def step(stream=None):
        abi.moe_combine_backward(cfg, x, inv, d_rows, rows=rows, expert_weights=w, d_expert_weights=d_w, stream=stream)
        abi.moe_dispatch_backward(cfg, d_rows, inv, d_x, stream=stream)
        abi.moe_route_backward(cfg, logits, idx, d_w, d_l, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (d_x, d_rows, d_w, d_l)]
    side = torch.cuda.Stream()
    for run in ("stream", "graph"):
        for t in (d_x, d_rows, d_w, d_l):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        if run == "stream":
            step(side)
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (d_x, d_rows, d_w, d_l))), run


# ---------------------------------------------------------------- refusals
def _calls():
    """Every operator with arguments that are as they should be, by name."""
    T, H, D, E, k, S = 5, 64, 48, 4, 2, 2
    R_ = T * k
    cfg = abi.config(T, H, E, k, D, router="sigmoid_sink", num_sink=S)
    z = lambda *shape, dt=F32: torch.zeros(shape, dtype=dt, device="cuda")  # noqa: E731
    i8, u8, i32 = torch.int8, torch.uint8, torch.int32
    ws = z(abi.moe_operator_workspace_size(cfg), dt=u8)
    inv = torch.arange(R_, dtype=i32, device="cuda")
    off = torch.tensor([0, 4, 4, 6, 10], dtype=i32, device="cuda")
    x, rows, w, dw = z(T, H, dt=BF16), z(R_, H, dt=BF16), z(T, k), z(T, k)
    q = dict(gate_up=z(R_, abi.int8_pitch(H), dt=i8), down=z(R_, abi.int8_pitch(D), dt=i8))
    lin = lambda part, K, N, n: dict(  # noqa: E731
        cfg=cfg, contraction=part, rows_q=q[part], row_scales=z(R_), w_q=z(E, N, abi.int8_pitch(K), dt=i8), w_scales=z(E, N),
        expert_offsets=off, out=z(R_, n, dt=BF16), workspace=ws)
    return {
        "moe_dispatch": [dict(cfg=cfg, x=x, inverse=inv, rows=rows, expert_weights=w)],
        "moe_dispatch_backward": [dict(cfg=cfg, d_rows=rows, inverse=inv, d_x=z(T, H, dt=BF16), x=x, expert_weights=w,
                                       d_expert_weights=dw)],
        "moe_combine": [dict(cfg=cfg, rows=rows, inverse=inv, out=x, expert_weights=w)],
        "moe_combine_backward": [dict(cfg=cfg, d_out=x, inverse=inv, d_rows=z(R_, H, dt=BF16), rows=rows, expert_weights=w,
                                      d_expert_weights=dw)],
        "moe_route_backward": [dict(cfg=cfg, logits=z(T, E + S), expert_indices=z(T, k, dt=i32), d_expert_weights=w,
                                    d_logits=z(T, E + S), d_sink_weights=z(T, S), global_scale=z(1), d_global_scale=z(1),
                                    workspace=ws)],
        "moe_dispatch_int8": [dict(cfg=cfg, x=x, inverse=inv, rows_q=q["gate_up"], row_scales=z(R_))],
        "moe_quantize_rows": [dict(cfg=cfg, h=z(R_, D, dt=BF16), expert_offsets=off, rows_q=q["down"], row_scales=z(R_))],
        "moe_grouped_linear_int8": [lin("gate_up", H, 2 * D, D), lin("down", D, H, H)],
    }


@pytest.mark.parametrize("name", ["moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward",
                                  "moe_route_backward", "moe_dispatch_int8", "moe_quantize_rows", "moe_grouped_linear_int8"])
def test_each_tensor_that_is_not_as_it_should_be_is_refused(name):
    call = getattr(abi, name)
    for good in _calls()[name]:
        call(**good)
        call(**good, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        outputs = {n: t.clone() for n, t in good.items() if isinstance(t, torch.Tensor)}
        for arg, t in good.items():
            if not isinstance(t, torch.Tensor):
                continue
            bad = [t.cpu(), t.double(), t.to(torch.int16)]
            if arg != "workspace":  # (any size, which the library checks)
                bad.append(torch.cat([t.reshape(-1), t.reshape(-1)[:1]]))
                if t.numel() > 1:
                    bad.append(torch.stack([t, t], -1)[..., 0])
            else:
                bad.append(torch.stack([t, t], -1)[..., 0])
            for b in bad:
                with pytest.raises(ValueError, match=arg if t.dtype is not BF16 else "bfloat16|float32|" + arg):
                    call(**{**good, arg: b})
        with pytest.raises((ValueError, abi.MoEError)):
            call(**{**good, next(n for n, t in good.items() if isinstance(t, torch.Tensor)): None})
        with pytest.raises(AttributeError):
            call(**good, stream=7)
        torch.cuda.synchronize()
        assert all(torch.equal(good[n], t) for n, t in outputs.items())
    if name == "moe_grouped_linear_int8":
        with pytest.raises(ValueError, match="contraction"):
            call(**{**good, "contraction": "up"})
        with pytest.raises(abi.MoEError):
            call(**{**good, "workspace": good["workspace"][:16]})
        with pytest.raises(abi.MoEError):
            call(**{**good, "bias": torch.zeros(4, 64, dtype=BF16, device="cuda")})  # (cfg.has_bias is 0)
