"""GPU parity of wush_norm and wush_residual_norm against the oracle in fp64.

Tolerances, derived from the arithmetic.  With u = 2^-24 (fp32's half step):
  * a row's statistic sums at most 32 values in a thread, 5 shuffle steps and 32 warps,
    each rounded once, on squares (2 more): 71 u relative, doubled for the square root's
    argument holding a rounded mean; F = 160 u covers it with the division and the root;
  * centring a layer norm's values loses u-sized parts of the row's largest value, which
    the division by the row's deviation magnifies: F * max|v| / sigma absolute;
  * each further product or sum rounds once; and the output to its type: half its step.
"""
import numpy as np
import pytest

from oracle import block as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24
F = 160 * U
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-38}       # half the subnormal step


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def norm_error(v, e, kind, weight, bias, eps, offset):
    """Bound on the error of a norm's fp32 output, given the bound ``e`` on its input's."""
    if kind == "none":
        return e
    c = v - v.mean(1, keepdims=True) if kind == "layer" else v
    sigma = np.sqrt((c * c).mean(1, keepdims=True) + eps)
    top = (np.abs(v).max(1, keepdims=True) * (F if kind == "layer" else 0) + e.max(1, keepdims=True) * 2) / sigma
    w = 1.0 if weight is None else np.abs(weight) + abs(offset)
    b = 0.0 if bias is None else np.abs(bias)
    n = np.abs(c) / sigma
    return (top * (1 + n) + F * n) * w + 4 * U * (n * w + b)


def close(got, want, dt, e):
    got = np64(got)
    step = float(torch.finfo(DT[dt]).eps) / 2
    bad = ~(np.abs(got - want) <= step * (np.abs(want) + e) + e + TINY[dt])       # (a NaN is bad)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want).max()))


def check(lib, rows, d, y="fp32", r="bf16", h="bf16", w="bf16", post="rms", pre="rms", gate=None, act="linear",
          a=1.0, b=1.0, offset=0.0, bias=False, eps=1e-6, weights=True, scale=1.0, in_place=False, give_r=True,
          want_r=True, want_h=True, make=None, stream=None, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * rows + d + seed)
    make = make or (lambda t, name: t)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ty = make((rand(rows, d) * scale + 0.25).to(DT[y]), "y")
    tr = make((rand(rows, d) * 2 * scale).to(DT[r]), "r") if give_r else None
    tg = None if gate is None else make(rand(rows, d) * 2, "gate").to(DT[y]) if gate == "element" else (rand(d) * 2).to(DT[y])
    vec = lambda: (rand(d) * 0.5 + 1).to(DT[w]) if weights else None  # noqa: E731
    bia = lambda: rand(d).to(DT[w]) if bias else None  # noqa: E731
    pw, pb, qw, qb = vec(), bia(), vec(), bia()
    nan = lambda dt: torch.full((rows, d), float("nan"), dtype=DT[dt], device="cuda")  # noqa: E731
    ins = [np64(t) for t in (ty, tr, tg, pw, pb, qw, qb)]
    out = (tr if in_place else make(nan(r), "r_out")) if want_r else None
    th = make(nan(h), "h") if want_h else None
    lib.wush_residual_norm(ty, tr, out, th, post=post, post_weight=pw, post_bias=pb, gate=tg, gate_act=act,
                           residual_scale=a, branch_scale=b, pre=pre, pre_weight=qw, pre_bias=qb, eps=eps,
                           weight_offset=offset, stream=stream)
    torch.cuda.synchronize()
    y64, r64, g64, pw, pb, qw, qb = ins
    u, o, hh = B.residual_norm(y64, r64, post, pw, pb, g64, act, a, b, pre, qw, qb, eps, offset)
    e = norm_error(y64, np.zeros_like(y64), post, pw, pb, eps, offset)
    if g64 is not None:
        # exp(-g) is 2^t with t = fp32(-g log2 e): t is off by u |g| log2 e, which is u |g| of the
        # exponential, and 2^t by 2 ulp (4 u); the sum rounds once, the quotient is within 2 ulp (4 u) and
        # two products round once each
        e = e * np.abs(B.activate(g64, act)) + (11 + np.abs(g64)) * U * np.abs(u)
    e = abs(b) * e + 3 * U * (np.abs(b * u) + (0 if r64 is None else np.abs(a * r64)))
    if want_r:
        close(out, o, r, e)
    if want_h:
        close(th, hh, h, norm_error(o, e, pre, qw, qb, eps, offset))
    return ty, tr, out, th


@pytest.mark.parametrize("rows, d", [(1, 1), (1, 8), (3, 5), (2, 256), (9, 100), (5, 1000), (1, 4096), (299, 4096),
                                     (301, 1024), (700, 136), (2, 12288), (3, 8200), (1, 32768), (2, 32767),
                                     (310, 4100), (4, 16392), (1531, 257), (900, 40), (1000, 2048), (400, 8192), (333, 12288), (310, 20000),
                                     (320, 32768), (305, 32767), (600, 6145), (597, 4094), (400, 8191), (311, 12289), (303, 16385), (301, 24571),
                                     (300, 2), (3000, 3), (2048, 1023)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_sizes(lib, rows, d, kind):
    check(lib, rows, d, post=kind, pre=kind, bias=kind == "layer", gate="element", act="silu")


@pytest.mark.parametrize("y", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("r", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("h", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("d", [520, 77])
def test_types(lib, y, r, h, d):
    for w in DT:
        check(lib, 6, d, y, r, h, w, gate="channel", act="sigmoid", bias=True)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate, act", [(None, "linear"), ("channel", "linear"), ("channel", "silu"),
                                       ("element", "linear"), ("element", "sigmoid"), ("element", "silu")])
def test_forms(lib, post, pre, gate, act):
    for d in (264, 263):
        check(lib, 5, d, post=post, pre=pre, gate=gate, act=act, a=0.5, b=-1.75, offset=1.0, r="fp32")
        check(lib, 5, d, post=post, pre=pre, gate=gate, act=act, weights=False, bias=True)


def test_absent_parts(lib):
    check(lib, 4, 512, give_r=False)
    check(lib, 4, 512, want_r=False)
    check(lib, 4, 512, want_h=False)
    check(lib, 4, 512, in_place=True)
    check(lib, 400, 333, in_place=True)
    check(lib, 4, 512, give_r=False, want_h=False, post="none")
    check(lib, 4, 512, a=0.0, b=0.0, eps=1e-5)                   # a row of zeros: norm 0
    check(lib, 4, 512, scale=1e-12, y="fp32", r="fp32")          # far below eps
    check(lib, 4, 512, scale=1e15, y="fp32", r="fp32", h="fp32")  # squares near 1e30


@pytest.mark.parametrize("d, wide, at", [(256, 768, 256), (256, 771, 256), (255, 600, 8), (64, 100, 3)])
def test_strided_rows_and_their_surroundings(lib, d, wide, at):
    # every tensor is a block of columns of a wider one; nothing outside it is written
    kept = {}

    def make(t, name):
        big = torch.full((t.shape[0] + 2, wide), 7.0, dtype=t.dtype, device="cuda")
        view = big[1:-1, at:at + d]
        view.copy_(t)
        kept[name] = big
        return view

    for rows in (3, 500):
        check(lib, rows, d, gate="element", act="sigmoid", make=make)
        for big in kept.values():
            edge = big.clone()
            edge[1:-1, at:at + d] = 7.0
            assert bool((edge == 7.0).all())


@pytest.mark.parametrize("rows", [7, 700])
@pytest.mark.parametrize("d", [256, 257, 1030])
def test_tensors_whose_rows_begin_apart(lib, rows, d):
    # row strides and first columns that agree in nothing
    at = {"y": 1, "r": 2, "r_out": 3, "h": 5, "gate": 0}

    def make(t, name):
        big = torch.full((t.shape[0] + 1, d + 8 + at[name]), 7.0, dtype=t.dtype, device="cuda")
        view = big[:-1, at[name]:at[name] + d]
        view.copy_(t)
        return view

    for kw in (dict(), dict(post="layer", pre="layer", bias=True, gate="element", act="silu"), dict(gate="channel")):
        check(lib, rows, d, make=make, **kw)


def test_outputs_side_by_side_in_one_buffer(lib):
    # r_out and h as columns of one wide tensor: they interleave but do not overlap
    rows, d = 33, 128
    buf = torch.zeros(rows, 2 * d, dtype=torch.bfloat16, device="cuda")
    y, r = torch.randn(rows, d, device="cuda"), torch.randn(rows, d, device="cuda").bfloat16()
    lib.wush_residual_norm(y, r, buf[:, :d], buf[:, d:], pre="rms")
    o, h = torch.empty_like(r), torch.empty_like(r)
    lib.wush_residual_norm(y, r, o, h, pre="rms")
    assert torch.equal(buf, torch.cat([o, h], 1))
    # one row only: a stride beyond the row plays no part
    lib.wush_residual_norm(y[:1], r[:1], buf[:1, :d], buf[:1, d:], pre="rms")
    assert torch.equal(buf[0, :d], o[0])


def test_norm_alone_equals_the_fused_one(lib):
    for rows, d in ((3, 4096), (500, 4096), (7, 33)):
        x = torch.randn(rows, d, device="cuda").bfloat16()
        w = torch.rand(d, device="cuda").bfloat16()
        h, h2, o = torch.empty(rows, d, device="cuda", dtype=torch.float16), None, None
        lib.wush_norm(x, h, "rms", w, eps=1e-5, weight_offset=1.0)
        want = B.norm(np64(x), "rms", np64(w), None, 1e-5, 1.0)
        close(h, want, "fp16", norm_error(np64(x), np.zeros(x.shape), "rms", np64(w), None, 1e-5, 1.0))
        z = torch.zeros_like(x)
        o, h2 = torch.empty_like(x), torch.empty_like(h)
        lib.wush_residual_norm(z, x, o, h2, pre="rms", pre_weight=w, eps=1e-5, weight_offset=1.0)
        assert torch.equal(h, h2) and torch.equal(o, x)
        lib.wush_norm(x, x, "rms", w, eps=1e-5, weight_offset=1.0)       # in place
        close(x, want, "bf16", norm_error(np64(o), np.zeros(x.shape), "rms", np64(w), None, 1e-5, 1.0))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [512, 61])
def test_a_bad_row_stays_its_own(lib, bad, d):
    y, r = torch.randn(6, d, device="cuda"), torch.randn(6, d, device="cuda")
    o, h = torch.empty_like(r), torch.empty_like(r)
    lib.wush_residual_norm(y, r, o, h, post="rms", pre="layer")
    y2 = y.clone()
    y2[2, d // 2] = bad
    o2, h2 = torch.empty_like(r), torch.empty_like(r)
    lib.wush_residual_norm(y2, r, o2, h2, post="rms", pre="layer")
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(o[keep], o2[keep]) and torch.equal(h[keep], h2[keep])
    assert bool(torch.isnan(h2[2]).all())


def test_zero_rows_launch_nothing(lib):
    x = torch.empty(0, 64, device="cuda")
    lib.wush_norm(x, torch.empty_like(x), "rms")
    lib.wush_residual_norm(x, x, x.clone(), torch.empty_like(x))


def test_streams_and_graphs(lib):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    check(lib, 40, 1024, stream=side)
    y, r = torch.randn(20, 4096, device="cuda"), torch.randn(20, 4096, device="cuda").bfloat16()
    o, h = torch.empty_like(r), torch.empty_like(r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.wush_residual_norm(y, r, o, h, post="rms", pre="rms")
    for seed in (1, 2):                                           # replays read the buffers' new contents
        torch.manual_seed(seed)
        y.normal_()
        g.replay()
        o2, h2 = torch.empty_like(r), torch.empty_like(r)
        lib.wush_residual_norm(y, r, o2, h2, post="rms", pre="rms")
        assert torch.equal(o, o2) and torch.equal(h, h2)


def test_results_do_not_depend_on_the_batch(lib):
    # a row's sums are in one order for a launch shape; across shapes only rounding may differ
    x = torch.randn(600, 4096, device="cuda")
    full, few = torch.empty_like(x), torch.empty(3, 4096, device="cuda")
    lib.wush_norm(x, full, "rms")
    again = torch.empty_like(x)
    lib.wush_norm(x, again, "rms")
    assert torch.equal(full, again)
    lib.wush_norm(x[:3], few, "rms")
    e = norm_error(np64(x[:3]), np.zeros((3, 4096)), "rms", None, None, 1e-6, 0.0)
    assert (np.abs(np64(few) - np64(full[:3])) <= 2 * (e + U * np.abs(np64(few)))).all()
