"""Waits of the norms' and adapters' kernels that run out: the call ends, its status says so, and the next
call is right.  (The test hook leaves the operands out, so that the first waits see nothing arrive.)"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TIMEOUT = -5


def times_out(lib, call):
    """call() with a short limit, then without one; both statuses."""
    lib.wush_debug_set_wait_limit(64)
    try:
        call()
        first = lib.wush_check_device_status()
    finally:
        lib.wush_debug_set_wait_limit(0)
    call()
    return first, lib.wush_check_device_status()


@pytest.mark.parametrize("d, pad", [(2304, 0), (2305, 0), (2304, 1)])     # aligned, shifted, single elements
@pytest.mark.parametrize("rows", [300, 1300])
def test_norms(lib, rows, d, pad):
    y, gate = torch.randn(rows, d, device="cuda"), torch.randn(rows, d, device="cuda")
    r = torch.randn(rows, d + pad, device="cuda").bfloat16()[:, :d]
    o, h, o2, h2 = (torch.zeros(rows, d, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    lib.wush_residual_norm(y, r, o, h, post="rms", pre="layer", gate=gate)
    got = times_out(lib, lambda: lib.wush_residual_norm(y, r, o2, h2, post="rms", pre="layer", gate=gate))
    assert got == (TIMEOUT, 0)
    assert torch.equal(o, o2) and torch.equal(h, h2)
    lib.wush_norm(r, h, "rms")
    assert times_out(lib, lambda: lib.wush_norm(r, h2, "rms")) == (TIMEOUT, 0)
    assert torch.equal(h, h2)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens, d_in, d_out, n, rank", [(600, 2048, 1024, 5, 16), (600, 64, 72, 2, 128), (300, 512, 256, 3, 256),
                                                          (3000, 512, 4096, 8, 32)])
def test_adapters(lib, dt, tokens, d_in, d_out, n, rank):
    x, adapter = torch.randn(tokens, d_in, device="cuda").to(dt), torch.randint(-1, n, (tokens,), device="cuda").int()
    a, b = torch.randn(n, rank, d_in, device="cuda").to(dt), torch.randn(n, d_out, rank, device="cuda").to(dt)
    base = torch.randn(tokens, d_out, device="cuda")
    y, y2 = torch.empty_like(base), torch.empty_like(base)
    ws = torch.empty(lib.wush_lora_workspace_bytes(tokens, d_in, d_out, n, rank), dtype=torch.uint8, device="cuda")
    lib.wush_lora_add(x, adapter, a, b, base, y, ws)
    assert times_out(lib, lambda: lib.wush_lora_add(x, adapter, a, b, base, y2, ws)) == (TIMEOUT, 0)
    assert torch.equal(y, y2)


def test_calls_without_waits_do_not_care(lib):
    x = torch.randn(5, 512, device="cuda").bfloat16()
    h, h2 = torch.empty_like(x), torch.empty_like(x)
    lib.wush_norm(x, h, "rms")
    assert times_out(lib, lambda: lib.wush_norm(x, h2, "rms")) == (0, 0)
    assert torch.equal(h, h2)
