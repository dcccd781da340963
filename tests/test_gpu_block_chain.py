"""The operators around a quantised projection, run together as a block uses them: the norm of
the stream, transform + quantise, the FP4 product, the requests' adapters on its output, and the
block's close with the next norm; and the 3-bit projection's decode step in the same way."""
import numpy as np
import pytest

import synth
from oracle import block as B
from oracle import gemm as G
from oracle import itq3 as I
from oracle import quant as Q
from tests.test_gpu_itq3 import pack_codes

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def np64(t):
    return t.double().cpu().numpy()


def _rel(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


class Block:
    """Buffers of one block of width d at M tokens, with an MXFP4 projection d -> d."""

    def __init__(self, lib, m, d, n, rank, seed=5):
        torch.manual_seed(seed)
        dev = dict(device="cuda")
        self.lib, self.m, self.d = lib, m, d
        self.stream = torch.randn(m, d, **dev).bfloat16()
        self.w = torch.rand(d, **dev).bfloat16() + 0.5
        self.w2 = torch.rand(d, **dev).bfloat16() + 0.5
        self.gate = torch.randn(d, **dev)
        weight = (torch.randn(d, d, **dev) * 0.05).bfloat16()
        self.t = torch.linalg.qr(torch.randn(d // 32, 32, 32, **dev))[0].contiguous()     # T_W = T^-T = T
        self.wc, self.ws = lib.alloc_quant_outputs(d, d, "mxfp4")
        lib.wush_transform_quant(weight, self.t, "wush", "mxfp4", self.wc, self.ws)
        self.weight = weight
        self.a = (torch.randn(n, rank, d, **dev) / d ** 0.5).bfloat16()
        self.b = torch.randn(n, d, rank, **dev).bfloat16()
        self.scale = torch.rand(n, **dev) + 0.5
        self.adapter = torch.randint(-1, n, (m,), **dev, dtype=torch.int32)
        self.h = torch.empty(m, d, **dev, dtype=torch.bfloat16)
        self.xc, self.xs = lib.alloc_quant_outputs(m, d, "mxfp4")
        self.y = torch.empty(m, d, **dev)
        self.out, self.h2 = torch.empty_like(self.stream), torch.empty_like(self.h)
        self.work = torch.empty(max(16, lib.wush_lora_workspace_bytes(m, d, d, n, rank)), dtype=torch.uint8, **dev)

    def run(self):
        lib, m, d = self.lib, self.m, self.d
        lib.wush_norm(self.stream, self.h, "rms", self.w)
        lib.wush_transform_quant(self.h, self.t, "wush", "mxfp4", self.xc, self.xs)
        lib.wush_qgemm(self.xc, self.xs, self.wc, self.ws, m, d, d, "mxfp4", 1.0, self.y)
        lib.wush_lora_add(self.h, self.adapter, self.a, self.b, self.y, self.y, self.work, scale=self.scale)
        lib.wush_residual_norm(self.y, self.stream, self.out, self.h2, post="rms", gate=self.gate, gate_act="sigmoid",
                               residual_scale=0.5, pre="rms", pre_weight=self.w2)


@pytest.mark.parametrize("m, d, n, rank", [(128, 512, 3, 16), (384, 1024, 5, 40)])
def test_a_block_matches_the_oracle(lib, m, d, n, rank):
    k = Block(lib, m, d, n, rank)
    k.run()
    torch.cuda.synchronize()
    assert lib.wush_check_device_status() == 0
    # each step against the oracle on the step's own inputs (the codes are decided by h's bits)
    h = B.norm(np64(k.stream), "rms", np64(k.w))
    assert _rel(np64(k.h), h) <= 2.0 ** -8
    t = k.t.cpu().numpy()
    dq = lambda x: Q.transform_quantize(x.float().cpu().numpy(), t, "mxfp4")["dq"]  # noqa: E731
    base = G.gemm_dequantized(dq(k.h), dq(k.weight))
    y, _ = B.lora_add(np64(k.h), k.adapter.cpu().numpy(), np64(k.a), np64(k.b), base, None, np64(k.scale))
    # A transformed value within fp32 rounding of a code's boundary can go the other way on the GPU.
    # A step of E2M1 is at most 2 where the codes' rms is above 2, so one such code among m * d moves
    # the product by at most 1 / sqrt(m d) of its norm (one of the d * d weights by less: d >= m); a
    # value lies that near a boundary with a chance of some 1e-6, so of 1.5 million sixteen are not
    # reached, and sixteen add up in squares to 4 / sqrt(m d).
    assert _rel(np64(k.y), y) <= 1e-4 + 4 / (m * d) ** 0.5
    # the adapters alone, on the GPU's own product
    lib.wush_qgemm(k.xc, k.xs, k.wc, k.ws, m, d, d, "mxfp4", 1.0, k.y)
    own = np64(k.y)
    y, _ = B.lora_add(np64(k.h), k.adapter.cpu().numpy(), np64(k.a), np64(k.b), own, None, np64(k.scale))
    k.run()
    torch.cuda.synchronize()
    assert _rel(np64(k.y), y) <= 4e-6
    _, out, h2 = B.residual_norm(np64(k.y), np64(k.stream), "rms", None, None, np64(k.gate), "sigmoid", 0.5, 1.0, "rms",
                                 np64(k.w2))
    assert _rel(np64(k.out), out) <= 2.0 ** -8 and _rel(np64(k.h2), h2) <= 2.0 ** -8


@pytest.mark.parametrize("m", [128, 384])
def test_a_captured_block_replays_on_new_inputs(lib, m):
    k = Block(lib, m, 512, 4, 24)
    k.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):                           # a stack: each block reads what the one before wrote
            k.run()
            k.stream.copy_(k.out)
    start = k.stream.clone()
    for seed in (1, 2):
        torch.manual_seed(seed)
        start.normal_()
        k.adapter.copy_(torch.randint(-1, 4, (m,), device="cuda"))
        k.stream.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (k.out, k.h2, k.y)]
        k.stream.copy_(start)
        for _ in range(3):
            k.run()
            k.stream.copy_(k.out)
        torch.cuda.synchronize()
        for a, b in zip(got, (k.out, k.h2, k.y)):
            assert torch.equal(a, b)
    assert lib.wush_check_device_status() == 0


@pytest.mark.parametrize("tokens", [1, 4, 16])
def test_a_decode_step_beside_the_three_bit_projection(lib, tokens):
    d_out, d_in, n, rank = 1024, 2048, 6, 16
    c, s = I.quantize(synth.itq3_weights(d_out, d_in))
    torch.manual_seed(tokens)
    stream = torch.randn(tokens, d_in, device="cuda")
    x = torch.empty(tokens, d_in, device="cuda", dtype=torch.float16)
    a = (torch.randn(n, rank, d_in, device="cuda") / d_in ** 0.5).half()
    b = torch.randn(n, d_out, rank, device="cuda").half()
    adapter = torch.arange(tokens, device="cuda", dtype=torch.int32) % (n + 1) - 1
    y = torch.empty(tokens, d_out, device="cuda")
    ws = torch.empty(tokens, d_in, device="cuda")
    lib.wush_norm(stream, x, "layer")
    lib.itq3_dequant_gemv(torch.from_numpy(pack_codes(c)).cuda(), torch.from_numpy(s).cuda(), x, d_out, 1, y, ws)
    lib.wush_lora_add(x, adapter, a, b, y, y)
    torch.cuda.synchronize()
    want, _ = B.lora_add(np64(x), adapter.cpu().numpy(), np64(a), np64(b), I.gemv(c, s, np64(x)))
    assert _rel(np64(y), want) <= 1e-5               # the 3-bit product's own tolerance
    assert _rel(np64(x), B.norm(np64(stream), "layer")) <= 2.0 ** -11
