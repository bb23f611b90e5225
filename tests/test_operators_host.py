"""What the row, router-gradient and 8-bit operators refuse, on the host: the C
entry points by status code before anything is enqueued, the Python binding
by ValueError before the call.  No GPU needed."""
import ctypes

import pytest
import torch

import operator_refs as R
from mixture_experts_ffn_token_b200 import abi
from mixture_experts_ffn_token_b200.build import build

INVALID, UNSUPPORTED, SMALL = 1, 2, 3
FAKE, ODD = 0x10000, 0x10008  # aligned and misaligned non-null addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build()
    return abi.load_library()


def cfg(T=4, H=64, E=8, k=2, D=32, **kw):
    return abi.config(T, H, E, k, D, **kw)


def sink():
    return cfg(router="sigmoid_sink", num_sink=2)


BF16, F32 = 0, 1
ROWS = {  # entry point -> its pointers in order: (name, required)
    "moe_dispatch": (("x", 1), ("inverse", 1), ("w", 0), ("rows", 1)),
    "moe_combine": (("rows", 1), ("inverse", 1), ("w", 0), ("out", 1)),
    "moe_dispatch_backward": (("d_rows", 1), ("x", 2), ("inverse", 1), ("w", 0), ("d_x", 1), ("d_w", 0)),
    "moe_combine_backward": (("d_out", 1), ("rows", 2), ("inverse", 1), ("w", 0), ("d_rows", 1), ("d_w", 0)),
}


@pytest.mark.parametrize("name", sorted(ROWS))
def test_row_operators_refuse(lib, name):
    fn, args = getattr(lib, name), ROWS[name]
    c = cfg()
    full = [FAKE + 0x1000 * i for i in range(len(args))]
    assert fn(ctypes.byref(c), 2, *full, None) == INVALID                     # no such row type
    for i, (arg, required) in enumerate(args):
        call = list(full)
        call[i] = None
        if required:                                                          # 2: for the weights' gradient
            assert fn(ctypes.byref(c), BF16, *call, None) == INVALID, arg
        call[i] = ODD
        if arg not in ("inverse", "w", "d_w"):
            assert fn(ctypes.byref(c), F32, *call, None) == INVALID, arg
    assert fn(None, BF16, *full, None) == INVALID
    names = [a for a, _ in args]
    out = full[names.index({"moe_dispatch": "rows", "moe_combine": "out", "moe_dispatch_backward": "d_x",
                            "moe_combine_backward": "d_rows"}[name])]
    for i, arg in enumerate(names):                                           # no output in place of an input
        if full[i] != out and arg not in ("inverse", "w", "d_w"):
            assert fn(ctypes.byref(c), BF16, *[out if j == i else p for j, p in enumerate(full)], None) == INVALID
    assert fn(ctypes.byref(cfg(H=60)), BF16, *full, None) == UNSUPPORTED
    assert fn(ctypes.byref(cfg(T=0)), BF16, *([None] * len(args)), None) == 0  # no tokens: nothing to do


def test_route_backward_refuses(lib):
    by, need = ctypes.byref, abi.moe_operator_workspace_size(cfg())
    f = lib.moe_route_backward

    def call(c, logits=FAKE, gs=None, idx=FAKE, dw=FAKE, ds=None, out=FAKE + 0x1000, dgs=None, ws=None, n=0):
        return f(by(c), logits, gs, idx, dw, ds, out, dgs, ws, n, None)

    for kw in ({"logits": None}, {"idx": None}, {"dw": None}, {"out": None}, {"out": FAKE}):
        assert call(cfg(), **kw) == INVALID
        assert call(sink(), **kw) == INVALID
    assert call(cfg(), gs=FAKE) == INVALID                 # the softmax router has no global scale
    assert call(cfg(), dgs=FAKE, ws=FAKE, n=need) == INVALID
    assert call(cfg(), ds=FAKE) == INVALID                 # and no sink lanes
    assert call(sink(), dgs=FAKE) == INVALID               # the scale's gradient needs a workspace
    assert call(sink(), dgs=FAKE, ws=FAKE, n=need - 1) == SMALL
    assert call(sink(), dgs=FAKE, ws=ODD, n=need) == INVALID
    assert call(cfg(T=0), logits=None, idx=None, dw=None, out=None) == 0


def test_int8_refuses(lib):
    by, c = ctypes.byref, cfg()
    need = abi.moe_operator_workspace_size(c)
    assert lib.moe_dispatch_int8(by(c), None, FAKE, FAKE, FAKE, None) == INVALID
    assert lib.moe_dispatch_int8(by(c), FAKE, None, FAKE, FAKE, None) == INVALID
    assert lib.moe_dispatch_int8(by(c), FAKE, FAKE, ODD, FAKE, None) == INVALID
    assert lib.moe_dispatch_int8(by(c), FAKE, FAKE, FAKE, None, None) == INVALID
    assert lib.moe_quantize_rows(by(c), ODD, None, FAKE, FAKE, None) == INVALID
    assert lib.moe_quantize_rows(by(c), FAKE, None, None, FAKE, None) == INVALID
    assert lib.moe_quantize_weights(by(c), 2, FAKE, FAKE, FAKE, None) == INVALID
    assert lib.moe_quantize_weights(by(c), 0, ODD, FAKE, FAKE, None) == INVALID
    assert lib.moe_quantize_weights(by(c), 0, FAKE, FAKE, None, None) == INVALID

    def linear(c, which=0, a=FAKE, s=FAKE, w=FAKE, ws=FAKE, b=None, off=FAKE, out=FAKE, wk=FAKE, n=need):
        return lib.moe_grouped_linear_int8(by(c), which, a, s, w, ws, b, off, out, wk, n, None)

    for kw in ({"a": None}, {"a": ODD}, {"s": None}, {"w": None}, {"w": ODD}, {"ws": None}, {"ws": ODD}, {"off": None},
               {"out": None}, {"out": ODD}, {"wk": None}, {"wk": ODD}, {"which": 5}, {"b": FAKE}):
        assert linear(c, **kw) == INVALID, kw
    assert linear(c, n=need - 1) == SMALL
    assert linear(cfg(has_bias=True)) == INVALID and linear(cfg(has_bias=True), b=ODD) == INVALID
    # sums of K products of 127 * 127 have to stay in 32 bits
    assert linear(cfg(H=131080)) == UNSUPPORTED and linear(cfg(D=131080), which=1) == UNSUPPORTED
    assert lib.moe_dispatch_int8(by(cfg(H=131080)), FAKE, FAKE, FAKE, FAKE, None) == UNSUPPORTED
    assert lib.moe_quantize_rows(by(cfg(D=131080)), FAKE, None, FAKE, FAKE, None) == UNSUPPORTED
    assert linear(cfg(T=0), a=None, out=None) == 0


def test_workspace_size(lib):
    n = abi.moe_operator_workspace_size(cfg())
    assert 256 <= n <= 1 << 24 and n % 256 == 0
    assert lib.moe_operator_workspace_size(None, None) == INVALID
    assert lib.moe_operator_workspace_size(ctypes.byref(cfg()), None) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors stand in for device tensors")
def test_binding_refuses_tensors(lib):
    c = cfg()
    x, rows = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    inv, w = torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2)
    for bad in (dict(x=x.half()), dict(x=x[:3]), dict(x=None), dict(inverse=inv.long()), dict(inverse=inv[:7]),
                dict(rows=rows.float()), dict(rows=torch.zeros(64, 8, dtype=torch.bfloat16).T), dict(rows=rows[:, :32]),
                dict(expert_weights=w.double()), dict(expert_weights=torch.zeros(2, 4).T)):
        kw = dict(x=x, inverse=inv, rows=rows, expert_weights=w) | bad
        with pytest.raises(ValueError):
            abi.moe_dispatch(c, kw["x"], kw["inverse"], kw["rows"], expert_weights=kw["expert_weights"])
        if "x" not in bad:
            with pytest.raises(ValueError):
                abi.moe_combine(c, kw["rows"], kw["inverse"], x, expert_weights=kw["expert_weights"])
    d_w = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="x is required"):
        abi.moe_dispatch_backward(c, rows, inv, x, d_expert_weights=d_w)
    with pytest.raises(ValueError, match="rows is required"):
        abi.moe_combine_backward(c, x, inv, rows, d_expert_weights=d_w)
    with pytest.raises(ValueError, match="contraction"):
        abi.moe_quantize_weights(c, "up", x, x, x)
    with pytest.raises(ValueError, match="d_logits"):
        abi.moe_route_backward(c, torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), w, torch.zeros(4, 9))
    q, s = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError, match="rows_q"):
        abi.moe_dispatch_int8(c, x, inv, q.to(torch.uint8), s)
    with pytest.raises(ValueError, match="h must"):
        abi.moe_quantize_rows(c, torch.zeros(8, 32), None, torch.zeros(8, 32, dtype=torch.int8), s)
    w_q, w_s = torch.zeros(8, 64, 64, dtype=torch.int8), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="workspace is required"):
        abi.moe_grouped_linear_int8(c, "gate_up", q, s, w_q, w_s, torch.zeros(9, dtype=torch.int32),
                                    torch.zeros(8, 32, dtype=torch.bfloat16), None)


def test_reference_forms():
    """The 64-bit forms that the GPU tests compare with, against autograd and by hand."""
    T, H, E, k, S = 6, 16, 5, 3, 1
    _, off, inv = R.routing(T, E, k, seed=1, drop=0.2)
    inv = inv.view(T, k)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, H, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(T, k, generator=g, dtype=torch.float64, requires_grad=True)
    d_rows = torch.randn(T * k, H, generator=g, dtype=torch.float64)
    live = (inv >= 0).view(-1)
    rows = torch.zeros(T * k, H, dtype=torch.float64).index_put(
        (inv.view(-1)[live].long(),), (w[:, :, None] * x[:, None]).reshape(T * k, H)[live])
    assert torch.allclose(rows, R.spread(x, inv, w, torch.zeros(T * k, H)))
    rows.backward(d_rows)
    assert torch.allclose(x.grad, R.gather(d_rows, inv, w)[0]) and torch.allclose(w.grad, R.dots(x, d_rows, inv)[0])
    # the router's gradient
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].int()
    for sink in (False, True):
        s = S if sink else 0
        z = torch.randn(T, E + s, generator=g).double().requires_grad_()
        d_w, d_s = torch.randn(T, k, generator=g), torch.randn(T, S, generator=g)
        gs = torch.tensor(0.75, dtype=torch.float64, requires_grad=True)
        v = z.gather(1, torch.cat([idx.long(), torch.arange(E, E + s).expand(T, s)], 1))
        p = torch.softmax(torch.nn.functional.logsigmoid(v) if sink else v, 1) * (2.5 * gs if sink else 1.0)
        p.backward(torch.cat([d_w, d_s], 1).double() if sink else d_w.double())
        ref, _, d_gs, _ = R.route_grad(z.detach(), idx, d_w, d_s if sink else None, E, s, sink, 2.5, 0.75)
        assert torch.allclose(z.grad, ref)
        assert not sink or abs(float(gs.grad) - d_gs) < 1e-9
    # ties of the rounding go to the even value, and the largest to 127
    q, s = R.quantize(torch.tensor([[127.0, 0.5, 1.5, -63.5, -127.0, 2.5]], dtype=torch.bfloat16))
    assert q.tolist() == [[127, 0, 2, -64, -127, 2]] and float(s) == 1.0


def test_missing_binding_is_reported(monkeypatch):
    """Without _binding.so the operators say so; there is no other way in."""
    import sys

    import mixture_experts_ffn_token_b200 as pkg
    monkeypatch.setattr(abi, "_binding", None)
    monkeypatch.delattr(pkg, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, pkg.__name__ + "._binding", None)
    x, inv = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(OSError, match="_binding.so"):
        abi.moe_dispatch(abi.config(3, 64, 2, 1, 8), x, inv, torch.zeros(3, 64, dtype=torch.bfloat16))
