"""The norms and adapters where an element lies more than 2^31 elements, or 2^32 bytes, from the first, and
pools too large to be sorted by with more than 512 tokens."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = 2.0 ** -24


def lora_close(lib, x, adapter, a, b, base, y, ws=None):
    """y against the formula in fp64, only with the adapters in use.  With u = 2^-24 a token's sums take at most
    32 cuts of 2 u, 16 roundings, 17 cuts and 2 roundings of what their sizes add up to (all magnitudes)."""
    lib.wush_lora_add(x, adapter, a, b, base, y, ws)
    assert lib.wush_check_device_status() == 0
    want, size = base.double(), torch.zeros_like(base, dtype=torch.float64)
    for g in adapter.unique().tolist():
        if g < 0:
            continue
        m = adapter == g
        xa, ag, bg = x[m].double(), a[g].double(), b[g].double()
        want[m] += (xa @ ag.T) @ bg.T
        size[m] = (xa.abs() @ ag.abs().T) @ bg.abs().T
    err = (y.double() - want).abs()
    assert bool((err <= 120 * U * size + U * want.abs()).all()), float(err.max())


@pytest.mark.parametrize("tokens", [20, 300, 600])
@pytest.mark.parametrize("dt", [BF, HF])
def test_adapters_far_into_their_pool(lib, tokens, dt):
    # a and b hold 2^31 elements and more each
    n, rank, d_in, d_out = 2100, 256, 4096, 4096
    a, b = (torch.zeros(n, *s, dtype=dt, device="cuda") for s in ((rank, d_in), (d_out, rank)))
    last = [0, 1000, n - 2, n - 1]
    for g in last:
        a[g], b[g] = torch.randn(rank, d_in, device="cuda").to(dt) / 64, torch.randn(d_out, rank, device="cuda").to(dt)
    adapter = torch.tensor(last + [-1], device="cuda")[torch.arange(tokens, device="cuda") % 5].int()
    x, base = torch.randn(tokens, d_in, device="cuda").to(dt), torch.randn(tokens, d_out, device="cuda")
    size = lib.wush_lora_workspace_bytes(tokens, d_in, d_out, n, rank)
    lora_close(lib, x, adapter, a, b, base, torch.empty_like(base), torch.empty(max(size, 16), dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("tokens, wide", [(40, 1 << 26), (300, 1 << 23)])
def test_adapters_rows_far_apart(lib, tokens, wide):
    n, rank, d_in, d_out = 3, 16, 256, 136
    x = torch.empty(tokens, wide, dtype=BF, device="cuda")[:, :d_in]
    y, base = (torch.empty(tokens, wide, device="cuda")[:, :d_out] for _ in range(2))
    x.copy_(torch.randn(tokens, d_in, device="cuda"))
    base.copy_(torch.randn(tokens, d_out, device="cuda"))
    a, b = torch.randn(n, rank, d_in, device="cuda").to(BF), torch.randn(n, d_out, rank, device="cuda").to(BF)
    adapter = (torch.arange(tokens, device="cuda") % 4 - 1).int()
    ws = torch.empty(max(16, lib.wush_lora_workspace_bytes(tokens, d_in, d_out, n, rank)), dtype=torch.uint8, device="cuda")
    lora_close(lib, x, adapter, a, b, base, y, ws)


@pytest.mark.parametrize("tokens", [513, 1000, 4096])
@pytest.mark.parametrize("dt", [BF, HF])
def test_pools_too_large_to_sort_by(lib, tokens, dt):
    n, rank, d_in, d_out = 60000, 8, 64, 72
    assert lib.wush_lora_workspace_bytes(tokens, d_in, d_out, n, rank) == 0
    a, b = torch.randn(n, rank, d_in, device="cuda").to(dt), torch.randn(n, d_out, rank, device="cuda").to(dt)
    x, base = torch.randn(tokens, d_in, device="cuda").to(dt), torch.randn(tokens, d_out, device="cuda")
    t = torch.arange(tokens, device="cuda")
    for adapter in (t % 7 * 9999, torch.where(t % 3 == 0, -1, n - 1 - t // 40), torch.full_like(t, n - 1),
                    torch.where(t % 2 == 0, n, 5)):
        adapter = adapter.int()
        adapter[adapter >= n] = -1
        lora_close(lib, x, adapter, a, b, base, torch.empty_like(base))
    outside = torch.where(t % 2 == 0, n, 5).int()
    y, y2 = torch.empty_like(base), base.clone()
    lib.wush_lora_add(x, outside, a, b, base, y)
    lib.wush_lora_add(x, outside, a, b, y2, y2)
    assert torch.equal(y, y2) and torch.equal(y[::2], base[::2])


@pytest.mark.parametrize("rows, d, wide", [(40, 512, 1 << 26), (300, 2304, 1 << 23), (300, 2305, (1 << 23) + 1),
                                           (300, 2304, (1 << 23) + 3)])
def test_norms_rows_far_apart(lib, rows, d, wide):
    # an RMS norm with gate and residual; F and the other bounds as in fp32 sums of d squares: 160 u of the norm
    y, g = (torch.empty(rows, wide, device="cuda")[:, :d] for _ in range(2))
    r, o, h = (torch.empty(rows, wide, dtype=BF, device="cuda")[:, :d] for _ in range(3))
    for t in (y, g, r):
        t.copy_(torch.randn(rows, d, device="cuda"))
    lib.wush_residual_norm(y, r, o, h, post="rms", gate=g, pre="rms", eps=1e-6)
    assert lib.wush_check_device_status() == 0
    yd, rd, gd = y.double(), r.double(), g.double()
    u = yd / (yd.square().mean(1, keepdim=True) + 1e-6).sqrt() * gd
    want = rd + u
    e = 165 * U * u.abs() + U * want.abs()
    assert bool(((o.double() - want).abs() <= 2.0 ** -8 * (want.abs() + e) + e).all())
    n = want / (want.square().mean(1, keepdim=True) + 1e-6).sqrt()
    e = 165 * U * n.abs() + 4 * e.amax(1, keepdim=True) * (1 + n.abs())          # (the rows' deviation is above 1 / 2)
    assert bool(((h.double() - n).abs() <= 2.0 ** -8 * (n.abs() + e) + e).all())
