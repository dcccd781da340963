"""wush_lora_add where nothing cancels: positive factors, so that every cut of a sum goes the same way.

With u = 2^-24, relative to the result: a matrix instruction's addition of 16 products to a sum cuts at most
2 u of it.  s takes d_in / 16 = 16 of them at most and 16 sums of parts (u each); y takes 16 at rank 256 for a
term that is all of s but 2^-7, 32 more on sums 2^-7 as large, and two roundings: 2 * 16 + 16 + 2 * 16.25 + 2 < 83 u.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rank", [16, 64, 128, 256])
@pytest.mark.parametrize("tokens", [9, 300])
def test_positive_factors(lib, dt, rank, tokens):
    torch.manual_seed(rank + tokens)
    n, d_in, d_out = 2, 256, 2048
    rand = lambda *s: torch.rand(*s, device="cuda").to(dt)  # noqa: E731
    x, a, b = rand(tokens, d_in), rand(n, rank, d_in), rand(n, d_out, rank)
    adapter = (torch.arange(tokens, device="cuda") % n).int()
    ws = torch.empty(max(16, lib.wush_lora_workspace_bytes(tokens, d_in, d_out, n, rank)), dtype=torch.uint8, device="cuda")
    y = torch.empty(tokens, d_out, device="cuda")
    lib.wush_lora_add(x, adapter, a, b, None, y, ws)
    for g in range(n):
        mine = adapter == g
        want = (x[mine].double() @ a[g].double().T) @ b[g].double().T
        assert float(((y[mine].double() - want).abs() / want).max()) <= 83 * 2.0 ** -24
