"""The status word that the two 8-bit products of a layer share in one workspace."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_token_b200 import abi

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
GEMM1, GEMM2, CSR = abi.DEVICE_ERR_TIMEOUT_GEMM1, abi.DEVICE_ERR_TIMEOUT_GEMM2, abi.DEVICE_ERR_CSR


class Products:
    """gate_up and down on one workspace, which holds anything at the start."""

    def __init__(self, T, H=64, D=72, E=3, fill=255):
        self.cfg = abi.config(T, H, E, 1, D)
        z = lambda *s, dt=torch.int8: torch.ones(s, dtype=dt, device="cuda")  # noqa: E731
        self.q = dict(gate_up=z(T, abi.int8_pitch(H)), down=z(T, abi.int8_pitch(D)))
        self.w = dict(gate_up=z(E, 2 * D, abi.int8_pitch(H)), down=z(E, H, abi.int8_pitch(D)))
        self.ws = dict(gate_up=z(E, 2 * D, dt=torch.float32), down=z(E, H, dt=torch.float32))
        self.out = dict(gate_up=z(T, D, dt=BF16), down=z(T, H, dt=BF16))
        self.scales = z(T, dt=torch.float32)
        bounds = torch.linspace(0, T, E + 1).to(I32)
        self.good, self.bad = bounds.cuda(), bounds.flip(0).contiguous().cuda()
        self.workspace = torch.full((abi.moe_operator_workspace_size(self.cfg),), fill, dtype=torch.uint8, device="cuda")

    def run(self, part, bad=False, workspace=None):
        abi.moe_grouped_linear_int8(self.cfg, part, self.q[part], self.scales, self.w[part], self.ws[part],
                                    self.bad if bad else self.good, self.out[part],
                                    self.workspace if workspace is None else workspace)

    def layer(self, bad=False):
        self.run("gate_up", bad)
        self.run("down")

    def record(self, bits):
        """As a kernel that gave up a wait records it."""
        word = self.workspace[:4].view(I32)
        word.copy_(word | bits)

    def status(self):
        return abi.moe_device_status(self.workspace)


@pytest.mark.parametrize("T", [5, 300], ids=["few_rows", "many_rows"])
def test_down_keeps_what_gate_up_recorded(T):
    p = Products(T)
    p.layer(bad=True)                                  # gate_up wrote nothing: down's result is no layer's
    assert p.status() == CSR
    p.layer()
    assert p.status() == 0                             # the next layer starts anew
    p.run("gate_up")
    p.record(GEMM1)
    p.run("down")
    assert p.status() == GEMM1
    v = ctypes.c_int32(0)
    assert abi.load_library().moe_device_status(p.workspace.data_ptr(), ctypes.byref(v), None) == abi.MOE_ERR_DEVICE_TIMEOUT
    p.run("gate_up")
    p.record(GEMM1)
    p.run("down", bad=True)
    assert p.status() == GEMM1 | CSR                   # both
    p.layer()
    assert p.status() == 0


@pytest.mark.parametrize("T", [5, 300], ids=["few_rows", "many_rows"])
def test_down_resets_its_own(T):
    """What a down product recorded is not kept by the next one, with or without a gate_up in between."""
    p = Products(T)
    for bits in (GEMM2, GEMM1, CSR, -1):               # (a workspace may hold anything)
        p.run("down")
        p.record(bits)
        p.run("down")
        assert p.status() == 0
        p.record(bits)
        p.run("gate_up")
        assert p.status() == 0
        p.run("down")
        assert p.status() == 0
    p.run("down", bad=True)
    assert p.status() == CSR
    p.run("down")
    assert p.status() == 0


def test_status_of_a_captured_layer():
    """gate_up by offsets that change between the replays, down by good ones."""
    p = Products(200)
    bad = p.bad.clone()
    p.bad.copy_(p.good)
    p.layer(bad=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.layer(bad=True)
    for offsets, want in ((bad, CSR), (p.good, 0), (bad, CSR), (bad, CSR), (p.good, 0)):
        p.bad.copy_(offsets)
        graph.replay()
        assert p.status() == want


@pytest.mark.parametrize("part", ["gate_up", "down"])
@pytest.mark.parametrize("captured", [False, True])
def test_status_of_no_tokens(part, captured):
    """A batch of no tokens is a success: its status is not what the memory held before."""
    for fill in (255, 2, 0):
        p = Products(0, fill=fill)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                p.run(part)
            graph.replay()
        else:
            p.run(part)
        assert p.status() == 0


def test_no_tokens_follow_the_same_rule():
    full, empty = Products(300), Products(0)
    full.run("gate_up", bad=True)
    empty.run("down", workspace=full.workspace)        # keeps what gate_up recorded
    assert full.status() == CSR
    empty.run("gate_up", workspace=full.workspace)     # starts anew
    assert full.status() == 0
    full.run("gate_up")
    full.record(GEMM1)
    empty.run("gate_up", workspace=full.workspace)
    full.run("down")
    assert full.status() == 0


def test_no_tokens_without_a_workspace():
    """From C, a batch of no tokens needs no pointer."""
    cfg = abi.config(0, 64, 3, 1, 72)
    fn = abi.load_library().moe_grouped_linear_int8
    for which in (0, 1):
        assert fn(ctypes.byref(cfg), which, None, None, None, None, None, None, None, None, 0, None) == 0
