"""GPU parity of wush_lora_add against the oracle in fp64.

Tolerance, derived from the arithmetic.  The products are exact in fp32; every sum rounds or
truncates by at most 2^-23 of its partial sum, and no value passes more than 64 such steps
(at most 32 MMA steps in one chain, the sums of the parts, the second product's terms), and
the split of s drops at most 2^-22 of the token's largest s.  So an element is within
80 * 2^-23 of ``size``, the bound on the magnitudes behind it, and the last sum with y_in rounds
once.  In norm, errors are bounded by the same 32 steps on partial sums that grow to the
result: 4e-6 of the adapters' part.
"""
import numpy as np
import pytest

from oracle import block as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = 2.0 ** -24


def pool(n, rank, d_in, d_out, dt, seed=0, ranks=None, garbage=float("nan")):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1000 * n + rank)
    a = (torch.randn(n, rank, d_in, generator=g, device="cuda") / d_in ** 0.5).to(dt)
    b = torch.randn(n, d_out, rank, generator=g, device="cuda").to(dt)
    if ranks is not None:                                      # what lies behind a rank may be anything
        for i, k in enumerate(ranks):
            k = min(max(k, 0), rank)
            a[i, k:] = garbage
            b[i, :, k:] = garbage
    return a, b


def compare(y, x, adapter, a, b, y_in, ranks, scale):
    n64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want, size = B.lora_add(n64(x), adapter.cpu().numpy(), n64(a), n64(b), n64(y_in),
                            None if ranks is None else ranks.cpu().numpy(), n64(scale))
    got = n64(y)
    err = np.abs(got - want)
    bad = ~(err <= 80 * 2 * U * size + U * (np.abs(want) + size * 1e-4) + 1e-37)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), float(np.nanmax(err)))
    part = want - (0 if y_in is None else n64(y_in))
    assert np.linalg.norm(err) <= 4e-6 * np.linalg.norm(part) + U * np.linalg.norm(want)


def check(lib, tokens, d_in, d_out, n, rank, dt=BF, ranks=None, scale=True, y_in=True, adapter=None, in_place=False,
          scale_x=1.0, seed=0, stream=None):
    torch.manual_seed(tokens * 7 + d_in + seed)
    x = (torch.randn(tokens, d_in, device="cuda") * scale_x).to(dt)
    a, b = pool(n, rank, d_in, d_out, dt, seed, ranks)
    if adapter is None:
        adapter = torch.randint(-1, n, (tokens,), device="cuda")
    adapter = torch.as_tensor(adapter, device="cuda").to(torch.int32)
    kt = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
    st = torch.randn(n, device="cuda") if scale else None
    base = torch.randn(tokens, d_out, device="cuda") if y_in else None
    y = base.clone() if in_place else torch.full((tokens, d_out), float("nan"), device="cuda")
    ws = torch.full((max(16, lib.wush_lora_workspace_bytes(tokens, d_in, d_out, n, rank)),), 255, dtype=torch.uint8,
                    device="cuda")                             # whatever an earlier call left
    torch.cuda.synchronize()
    lib.wush_lora_add(x, adapter, a, b, y if in_place else base, y, ws, kt, st, stream)
    torch.cuda.synchronize()
    assert lib.wush_check_device_status() == 0
    compare(y, x, adapter, a, b, base, kt, st)
    return x, adapter, a, b, base, y, ws, kt, st


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 120, 128, 136, 256])
@pytest.mark.parametrize("tokens", [1, 9, 300])
def test_ranks(lib, dt, rank, tokens):
    check(lib, tokens, 256, 264, 3, rank, dt)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("tokens, d_in, d_out", [(1, 32, 8), (1, 4096, 4096), (2, 64, 24), (7, 96, 4104), (8, 12288, 40),
                                                 (17, 2048, 1032), (63, 160, 72), (64, 512, 512), (65, 512, 520),
                                                 (129, 1056, 328), (200, 4096, 96), (513, 64, 1288), (1000, 320, 136),
                                                 (2049, 96, 64)])
def test_sizes(lib, dt, tokens, d_in, d_out):
    check(lib, tokens, d_in, d_out, 5, 16, dt)
    check(lib, tokens, d_in, d_out, 2, 48, dt, ranks=[48, 33])


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("tokens", [5, 70, 400])
def test_ranks_of_their_own(lib, dt, tokens):
    # padding behind each rank is NaN; 0 and negative ranks add nothing, one beyond the pool's is clamped
    ranks = [64, 0, 1, 5, 16, 17, 63, -4, 99, 31]
    check(lib, tokens, 192, 200, 10, 64, dt, ranks=ranks)
    check(lib, tokens, 192, 200, 2, 8, dt, ranks=[3, 7])


@pytest.mark.parametrize("tokens", [1, 6, 90, 700])
def test_forms(lib, tokens):
    for kw in (dict(scale=False), dict(y_in=False), dict(in_place=True), dict(scale=False, y_in=False)):
        check(lib, tokens, 128, 136, 4, 16, **kw)
        check(lib, tokens, 128, 136, 4, 40, HF, **kw)


@pytest.mark.parametrize("tokens", [4, 100, 900])
def test_who_has_which_adapter(lib, tokens):
    n = 6
    for name, ad in {"all one": [3] * tokens, "none": [-1] * tokens, "outside": [n, -7, 2 ** 31 - 1, -2 ** 31] * tokens,
                     "in turn": list(range(n)) * tokens, "runs": [i * 5 // tokens for i in range(tokens)],
                     "last only": [-1] * (tokens - 1) + [n - 1]}.items():
        for in_place in (False, True):
            check(lib, tokens, 64, 72, n, 16, adapter=ad[:tokens], in_place=in_place)


def test_many_adapters_few_tokens_each(lib):
    check(lib, 700, 64, 64, 1000, 8, adapter=torch.randperm(1000)[:700])
    check(lib, 40, 64, 64, 5000, 8, adapter=torch.randperm(5000)[:40])


@pytest.mark.parametrize("dt, scale_x", [(HF, 3000.0), (HF, 1e-4), (BF, 1e30), (BF, 1e-25)])
def test_magnitudes(lib, dt, scale_x):
    # s far beyond fp16's range, or far below it
    for tokens in (3, 300):
        check(lib, tokens, 1024, 64, 2, 16, dt, scale_x=scale_x, y_in=False, scale=False)


@pytest.mark.parametrize("tokens", [12, 320])
@pytest.mark.parametrize("dt", [BF, HF])
def test_strided_rows_and_their_surroundings(lib, tokens, dt):
    # x, y_in and y are columns of wider tensors; nothing outside y's columns is written
    d_in, d_out, n, rank = 96, 72, 3, 24
    x0, adapter, a, b, base, y0, ws, _, st = check(lib, tokens, d_in, d_out, n, rank, dt)
    xw = torch.full((tokens, d_in + 40), float("nan"), dtype=dt, device="cuda")
    xw[:, 8:8 + d_in] = x0
    iw = torch.full((tokens, d_out + 12), float("nan"), device="cuda")
    iw[:, 4:4 + d_out] = base
    yw = torch.full((tokens + 2, 3 * d_out), 7.0, device="cuda")
    lib.wush_lora_add(xw[:, 8:8 + d_in], adapter, a, b, iw[:, 4:4 + d_out], yw[1:-1, d_out:2 * d_out], ws, None, st)
    assert torch.equal(yw[1:-1, d_out:2 * d_out], y0)
    yw[1:-1, d_out:2 * d_out] = 7.0
    assert bool((yw == 7.0).all())


@pytest.mark.parametrize("tokens", [20, 400])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_with_their_token_and_adapter(lib, tokens, bad):
    x, adapter, a, b, base, y, ws, _, st = check(lib, tokens, 128, 64, 4, 16)
    adapter[0], adapter[1], adapter[5] = 2, 2, 3
    y0, y1 = torch.empty_like(y), torch.empty_like(y)
    lib.wush_lora_add(x, adapter, a, b, base, y0, ws, None, st)
    x2, a2 = x.clone(), a.clone()
    x2[1, 77] = bad
    a2[3, 4, 9] = bad
    lib.wush_lora_add(x2, adapter, a2, b, base, y1, ws, None, st)
    hit = adapter == 3
    hit[1] = True
    assert torch.equal(y0[~hit], y1[~hit])
    assert not bool(torch.isfinite(y1[hit]).all(1).any())


@pytest.mark.parametrize("tokens", [30, 600])
def test_equal_calls_give_equal_bits(lib, tokens):
    x, adapter, a, b, base, y, ws, _, st = check(lib, tokens, 2048, 256, 7, 32)
    for _ in range(5):
        y2 = torch.empty_like(y)
        lib.wush_lora_add(x, adapter, a, b, base, y2, ws, None, st)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("tokens", [3, 500])
def test_streams_and_graphs(lib, tokens):
    side = torch.cuda.Stream()
    check(lib, tokens, 256, 128, 4, 16, stream=side)
    x, adapter, a, b, base, y, ws, _, st = check(lib, tokens, 256, 128, 4, 16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.wush_lora_add(x, adapter, a, b, base, y, ws, None, st)
    for seed in (1, 2, 3):                                     # replays read new inputs and new adapters
        torch.manual_seed(seed)
        x.normal_()
        adapter.copy_(torch.randint(-1, 4, (tokens,), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        compare(y, x, adapter, a, b, base, None, st)
    # two calls at once, each with a workspace of its own
    other = torch.empty_like(ws)
    y1, y2 = torch.empty_like(y), torch.empty_like(y)
    torch.cuda.synchronize()
    for _ in range(20):
        lib.wush_lora_add(x, adapter, a, b, base, y1, ws, None, st)
        lib.wush_lora_add(x, adapter, a, b, base, y2, other, None, st, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y1) and torch.equal(y, y2)


def test_zero_tokens(lib):
    a, b = pool(2, 8, 64, 64, BF)
    lib.wush_lora_add(torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), a, b,
                      None, torch.empty(0, 64, device="cuda"))


def test_sizes_of_the_listed_projections(lib):
    # the widths of the framework's own workloads
    check(lib, 16, 4096, 4096, 4, 64, HF, ranks=[64, 32, 16, 61])
    check(lib, 260, 5120, 17408, 3, 16)
    check(lib, 300, 12288, 4096, 3, 64)


def test_requests_side_by_side_and_apart(lib):
    # rows of a tile that follow one another are fetched in blocks, the others one by one; pools of
    # more than 1024 adapters leave the order to chance
    t = torch.arange(900)
    for n in (3, 1500):
        for ad in (t // 300, t // 7 % n, (t * 7919) % n, torch.where(t % 50 < 43, t // 450, t % n)):
            check(lib, 900, 384, 136, n, 16, adapter=ad)
    check(lib, 3000, 64, 64, 2, 8, adapter=torch.zeros(3000))    # one adapter with many tiles


def test_a_long_row_of_blocks(lib):
    # enough column blocks that they are drawn from a counter, call after call
    x, adapter, a, b, base, y, ws, _, st = check(lib, 2500, 64, 4096, 9, 16)
    for _ in range(3):
        y2 = torch.empty_like(y)
        lib.wush_lora_add(x, adapter, a, b, base, y2, ws, None, st)
        assert torch.equal(y, y2)


def test_more_tokens_than_one_look_of_the_plan(lib):
    check(lib, 20000, 32, 16, 5, 8)


def test_a_pool_too_large_to_count_in_shared_memory(lib):
    assert lib.wush_lora_workspace_bytes(500, 64, 64, 60000, 8) == 0
    check(lib, 500, 64, 64, 60000, 8, adapter=torch.cat([torch.randperm(60000)[:300], torch.full((200,), 59999)]))
    check(lib, 400, 32, 64, 57344, 8, adapter=torch.cat([torch.randperm(57344)[:300], torch.full((100,), 57343)]))


@pytest.mark.parametrize("tokens", [2, 300])
def test_a_long_reduction(lib, tokens):
    check(lib, tokens, 1 << 17, 64, 2, 8)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("tokens", [3, 300])
def test_an_infinity_in_a_factor_counts_as_the_formula_says(lib, tokens, dt):
    # s of rank 0 is an infinity, the others' are beyond fp16's range: y is the infinity's sign times b's
    torch.manual_seed(tokens)
    x = torch.rand(tokens, 64, device="cuda").to(dt) + 0.5
    a, b = pool(2, 16, 64, 40, dt)
    a[1, 0, 5] = float("inf")
    adapter = (torch.arange(tokens, device="cuda") % 2).to(torch.int32)
    sc = torch.tensor([1.0, 1e6], device="cuda")
    ws = torch.empty(max(16, lib.wush_lora_workspace_bytes(tokens, 64, 40, 2, 16)), dtype=torch.uint8, device="cuda")
    y = torch.empty(tokens, 40, device="cuda")
    lib.wush_lora_add(x, adapter, a, b, None, y, ws, None, sc)
    assert bool(torch.isfinite(y[::2]).all())
    assert torch.equal(y[1::2], (float("inf") * torch.sign(b[1, :, 0].float())).expand_as(y[1::2]))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("tokens", [5, 300])
def test_small_ranks_beside_large_ones(lib, tokens, dt):
    # Rank j's s is some 2^-j of rank 0's, and row o of b uses rank o % 15 alone.  All terms of a
    # sum are positive, so that every rounding is relative to the result itself: the 80 steps of
    # 2^-23 above, the split of s (2^-24 down to 2^-14 of the largest) among them.
    torch.manual_seed(tokens)
    x = torch.rand(tokens, 256, device="cuda").to(dt) + 0.5
    a = ((torch.rand(1, 16, 256, device="cuda") + 0.5) * 2.0 ** -torch.arange(16, device="cuda")[:, None]).to(dt)
    o = torch.arange(120, device="cuda")
    b = torch.zeros(1, 120, 16, device="cuda", dtype=dt)
    b[0, o, o % 15] = (torch.rand(120, device="cuda") + 0.5).to(dt)
    ws = torch.empty(max(16, lib.wush_lora_workspace_bytes(tokens, 256, 120, 1, 16)), dtype=torch.uint8, device="cuda")
    y = torch.empty(tokens, 120, device="cuda")
    lib.wush_lora_add(x, torch.zeros(tokens, dtype=torch.int32, device="cuda"), a, b, None, y, ws)
    want = (x.double() @ a[0].double().T) @ b[0].double().T
    err = (y.double() - want).abs()
    assert bool((err <= 80 * 2 * U * want).all()), float((err / want).max())


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("tokens", [256, 257, 300, 511, 512, 513])
def test_two_tokens_a_thread(lib, tokens, dt):
    # pools with an adapter for every eight tokens stay in one launch up to 512 tokens
    assert (lib.wush_lora_workspace_bytes(tokens, 256, 136, 70, 24) == 0) == (tokens <= 512)
    t = torch.arange(tokens)
    for ad in (torch.full((tokens,), 69), t % 70, t * 7 // tokens, torch.where(t % 3 == 0, -1, t % 64)):
        check(lib, tokens, 256, 136, 70, 24, dt, adapter=ad)
    check(lib, tokens, 256, 136, 70, 24, dt, adapter=torch.where(t % 3 == 0, -1, t % 64), in_place=True)
