"""Combine and dispatch's gradient at sizes that go through the ring in shared
memory, for every number of terms that it is built for, in both types."""
import pytest
import torch

import operator_refs as R
from mixture_experts_ffn_token_b200 import abi

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def inputs(T, H, E, k, drop, dtype):
    _, _, inv = R.routing(T, E, k, seed=T + k, drop=drop)
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s, dt=F32: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    return inv.cuda(), n(T, H, dt=dtype), n(T * k, H, dt=dtype), n(T, k)


def terms(rows, inv, t):
    """The rows of tokens t's slots in 64 bits [n, k, H], zero for a slot of no expert."""
    p = inv[t].long()
    return torch.where((p >= 0)[:, :, None], rows[p.clamp(min=0)].double(), 0.0)


def check(T, H, E, k, drop, dtype, run):
    inv, tok, rows, w = inputs(T, H, E, k, drop, dtype)
    out = torch.full((T, H), float("nan"), dtype=dtype, device="cuda")
    cfg = abi.config(T, H, E, k, 8)
    d_w = run(cfg, inv.view(-1), tok, rows, w, out)
    inv = inv.view(T, k)
    for t0 in range(0, T, 2048):
        t = slice(t0, min(T, t0 + 2048))
        y = terms(rows, inv, t)
        prod = y * w[t].double()[:, :, None]
        R.assert_within(out[t], prod.sum(1).cpu(), R.tol_gather(prod.sum(1), prod.abs().sum(1), k, dtype).cpu(), "sums")
        if d_w is not None:
            dots = y * tok[t].double()[:, None]
            R.assert_within(d_w[t], dots.sum(2).cpu(), R.tol_dots(dots.abs().sum(2), H).cpu(), "d_w")


# 128 MB of rows and more, without the weights' gradient
@pytest.mark.parametrize("T,H,E,k,drop,dtype", [
    (70001, 1000, 7, 1, 0.0, BF16), (8501, 2056, 128, 2, 0.1, F32), (11003, 2056, 128, 6, 0.0, BF16),
    (13001, 1048, 40, 5, 0.2, BF16), (8009, 2888, 128, 3, 0.1, BF16), (8209, 2888, 128, 4, 0.0, BF16),
    (6007, 1544, 16, 4, 0.0, F32), (6007, 2056, 9, 3, 0.3, F32), (4099, 1160, 40, 8, 0.1, F32), (4801, 1032, 40, 7, 0.0, F32),
    (9001, 1544, 20, 7, 0.1, BF16)])
def test_combine(T, H, E, k, drop, dtype):
    assert T * k * H * (2 if dtype is BF16 else 4) >= 128 << 20

    def run(cfg, inv, tok, rows, w, out):
        abi.moe_combine(cfg, rows, inv, out, expert_weights=w)

    check(T, H, E, k, drop, dtype, run)


# 1024 tokens and 24 MB of rows, rows of more than 64 vectors, with the weights' gradient
@pytest.mark.parametrize("T,H,E,k,drop,dtype", [
    (4099, 1032, 16, 3, 0.1, BF16), (4001, 808, 128, 4, 0.0, BF16), (1025, 2888, 20, 5, 0.2, BF16), (1031, 2056, 128, 6, 0.0, BF16),
    (2003, 1000, 9, 7, 0.1, BF16), (1033, 1544, 40, 8, 0.0, BF16), (1409, 1000, 40, 9, 0.1, BF16),
    (1601, 1000, 16, 4, 0.1, F32), (1301, 1032, 40, 5, 0.0, F32), (1027, 1000, 40, 7, 0.1, F32), (1129, 776, 9, 8, 0.0, F32),
    (1063, 648, 40, 12, 0.2, F32), (1201, 520, 33, 16, 0.0, F32)])
def test_dispatch_backward(T, H, E, k, drop, dtype):
    size = 2 if dtype is BF16 else 4
    assert T >= 1024 and T * k * H * size >= 24 << 20 and H * size > 64 * 16

    def run(cfg, inv, tok, rows, w, out):
        d_w = torch.full((cfg.num_tokens, cfg.top_k), float("nan"), device="cuda")
        abi.moe_dispatch_backward(cfg, rows, inv, out, x=tok, expert_weights=w, d_expert_weights=d_w)
        return d_w

    check(T, H, E, k, drop, dtype, run)
