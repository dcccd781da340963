"""The ring kernel of wush_norm and wush_residual_norm (more than 296 rows wider than 2048) against the
formulas in fp64, over the types, forms and layouts that it tells apart.

Tolerances, derived from the arithmetic, with u = 2^-24 (fp32's half step):
  * a row's statistic sums at most 32 values in a thread, 5 shuffle steps and 32 warps, each rounded once,
    on squares (2 more): 71 u relative, doubled for the rounded mean; F = 160 u covers it with the division
    and the root;
  * centring loses u-sized parts of the row's largest value, which the division by the row's deviation
    magnifies: F max|v| / sigma absolute;
  * exp(-g) is off by u |g| and two ulp (4 u), the quotient by two ulp (4 u), three roundings more: (11 + |g|) u;
  * each further product or sum rounds once, and the output to its type: half its step.
"""
import itertools

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24
F = 160 * U
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-38}       # half the subnormal step


def norm64(v, e, kind, weight, bias, eps, offset):
    """N(v) in fp64 and a bound on the error of its fp32 form, given the bound ``e`` on its input's."""
    if kind == "none":
        return v, e
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    sigma = (c.square().mean(1, keepdim=True) + eps).sqrt()
    top = (v.abs().amax(1, keepdim=True) * (F if kind == "layer" else 0) + e.amax(1, keepdim=True) * 2) / sigma
    n = c / sigma
    w = torch.ones_like(v[0]) if weight is None else weight.double() + offset
    b = torch.zeros_like(v[0]) if bias is None else bias.double()
    size = w.abs() + (0 if weight is None else 2 * abs(offset))
    bound = (top * (1 + n.abs()) + F * n.abs()) * size + 4 * U * (n.abs() * size + b.abs())
    return n * w + b, bound


def close(got, want, dt, e):
    step = float(torch.finfo(DT[dt]).eps) / 2
    err = (got.double() - want).abs()
    bad = ~(err <= step * (want.abs() + e) + e + TINY[dt])       # (a NaN is bad)
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), float(err.max()))


def check(lib, rows, d, y="fp32", r="bf16", h="bf16", post="rms", pre="rms", gate=None, act="linear", a=1.0, b=1.0,
          offset=0.0, eps=1e-6, post_w="bf16", post_b=None, pre_w="bf16", pre_b=None, gate_t=None, r_out="own",
          want_h=True, view=lambda t, name: t):
    """post_w, post_b, pre_w, pre_b: a type, or None for an absent vector; r_out: own, in place or None."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * rows + d)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    vec = lambda t, one: None if t is None else (rand(d) * 0.5 + one).to(DT[t])  # noqa: E731
    ty = view((rand(rows, d) + 0.25).to(DT[y]), "y")
    tr = None if r is None else view((rand(rows, d) * 2).to(DT[r]), "r")
    gt = gate_t or y
    tg = None if gate is None else view((rand(rows, d) * 2).to(DT[gt]), "gate") if gate == "element" else \
        (rand(d) * 2).to(DT[gt])
    pw, pb, qw, qb = vec(post_w, 1), vec(post_b, 0), vec(pre_w, 1), vec(pre_b, 0)
    y64, r64 = ty.double(), None if tr is None else tr.double()
    out_t = r or "bf16"
    nan = lambda dt, name: view(torch.full((rows, d), float("nan"), dtype=DT[dt], device="cuda"), name)  # noqa: E731
    to = tr if r_out == "in place" else nan(out_t, "r_out") if r_out else None
    th = nan(h, "h") if want_h else None
    lib.wush_residual_norm(ty, tr, to, th, post=post, post_weight=pw, post_bias=pb, gate=tg, gate_act=act,
                           residual_scale=a, branch_scale=b, pre=pre, pre_weight=qw, pre_bias=qb, eps=eps,
                           weight_offset=offset)
    assert lib.wush_check_device_status() == 0
    u, e = norm64(y64, torch.zeros_like(y64), post, pw, pb, eps, offset)
    if tg is not None:
        g64 = tg.double()
        f = g64 if act == "linear" else g64.sigmoid() if act == "sigmoid" else g64 * g64.sigmoid()
        u, e = u * f, e * f.abs() + (11 + g64.abs()) * U * (u * f).abs()
    o = b * u if r64 is None else a * r64 + b * u
    e = abs(b) * e + 3 * U * ((b * u).abs() + (0 if r64 is None else (a * r64).abs()))
    if r_out:
        close(to, o, out_t, e)
    if want_h:
        want, e = norm64(o, e, pre, qw, qb, eps, offset)
        close(th, want, h, e)


TYPES = ("bf16", "fp16", "fp32")


@pytest.mark.parametrize("gate_t", TYPES)
@pytest.mark.parametrize("post_t", TYPES)
@pytest.mark.parametrize("pre_t", TYPES)
@pytest.mark.parametrize("d", [2560, 2561])
def test_types_of_the_vectors(lib, d, post_t, pre_t, gate_t):
    # every pairing of the types of a gate per channel and of both norms' vectors, each there or not
    for pw, pb, qw, qb in itertools.product((0, 1), repeat=4):
        check(lib, 298, d, gate="channel", gate_t=gate_t, post_w=post_t if pw else None, post_b=post_t if pb else None,
              pre_w=pre_t if qw else None, pre_b=pre_t if qb else None)
    for pw, pb in ((1, 0), (0, 1), (1, 1)):
        check(lib, 298, d, gate="channel", gate_t=gate_t, post_w=post_t if pw else None, post_b=post_t if pb else None,
              pre="none", pre_w=None)
        check(lib, 298, d, gate="channel", gate_t=gate_t, post="none", post_w=None, pre_w=pre_t if pw else None,
              pre_b=pre_t if pb else None)
        check(lib, 298, d, gate="channel", gate_t=gate_t, post_w=post_t if pw else None,
              post_b=post_t if pb else None, pre="none", pre_w=None, want_h=False)


@pytest.mark.parametrize("d", [2304, 3584, 5120])
def test_a_block_that_closes_with_a_scaled_norm_and_leaves_the_next_out(lib, d):
    for post_t, gate_t in itertools.product(TYPES, TYPES):
        check(lib, 400, d, gate="channel", gate_t=gate_t, post_w=post_t, pre="none", pre_w=None, want_h=False)
        check(lib, 400, d, gate="channel", gate_t=gate_t, post_w=post_t, pre="rms", pre_w=None, r="fp32", h="fp16")


@pytest.mark.parametrize("y", TYPES)
@pytest.mark.parametrize("r", TYPES + (None,))
@pytest.mark.parametrize("d", [2560, 2051])
def test_types_of_the_rows(lib, y, r, d):
    for h in TYPES:
        check(lib, 310, d, y, r, h, gate="element", gate_t="fp32" if h == "fp16" else "fp16", act="silu")
        check(lib, 310, d, y, r, h, post="layer", pre="layer", post_b="bf16", pre_b="bf16")


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("d", [2304, 2307])
def test_forms(lib, post, pre, d):
    # (1300 rows: every CTA's stages are refilled)
    for gate, act in ((None, "linear"), ("channel", "silu"), ("element", "sigmoid"), ("element", "linear")):
        for r_out, want_h in (("own", True), ("in place", True), (None, True), ("own", False), ("in place", False)):
            check(lib, 1300, d, post=post, pre=pre, gate=gate, act=act, r_out=r_out, want_h=want_h, a=0.5, b=-1.75,
                  offset=1.0)
        check(lib, 1300, d, post=post, pre=pre, gate=gate, act=act, r=None)


@pytest.mark.parametrize("d", [2560, 4097, 5124, 8200, 12288, 16390, 32765])
def test_wide_rows_in_place(lib, d):
    # (4 CTAs an SM at most: 1500 narrow rows and 700 wide ones come to each CTA's stages again)
    rows = 1500 if d < 6000 else 700
    check(lib, rows, d, gate="element", act="silu", r_out="in place")
    check(lib, rows, d, "bf16", "fp16", "fp32", r_out="in place", post="none", post_w=None)
    check(lib, rows, d, "fp32", "fp32", "bf16", post="layer", pre="layer", post_b="bf16", pre_b="bf16", gate="channel")


def columns(rows_more, wide, at, kept):
    """Tensors as columns of wider ones full of sevens (first column ``at[name]``), kept to be looked at."""
    def view(t, name):
        big = torch.full((t.shape[0] + rows_more, wide[name]), 7.0, dtype=t.dtype, device="cuda")
        out = big[1:1 + t.shape[0], at[name]:at[name] + t.shape[1]]
        out.copy_(t)
        kept.append((big, at[name], t.shape))
        return out
    return view


NAMES = ("y", "r", "r_out", "h", "gate")


@pytest.mark.parametrize("rows", [300, 1300])
@pytest.mark.parametrize("d, more, at", [(2304, 256, 128), (2304, 8, 8), (2304, 7, 3), (2305, 3, 2), (2307, 1, 0), (4101, 11, 5),
                                         (2304, 4, 4), (8193, 2, 1)])
def test_strided_rows_and_their_surroundings(lib, rows, d, more, at):
    # every tensor is a block of columns of a wider one; nothing outside it is written
    for kw in (dict(gate="element", act="sigmoid"), dict(r_out="in place", gate="channel"),
               dict(y="bf16", r="fp32", h="fp16", post="layer", pre="layer"), dict(post="none", post_w=None, want_h=False)):
        kept = []
        check(lib, rows, d, view=columns(2, dict.fromkeys(NAMES, d + more), dict.fromkeys(NAMES, at), kept), **kw)
        for big, first, (n, m) in kept:
            big[1:1 + n, first:first + m] = 7.0
            assert bool((big == 7.0).all())


@pytest.mark.parametrize("rows", [300, 1300])
@pytest.mark.parametrize("d", [2304, 2305, 4098, 6150])
def test_tensors_whose_rows_begin_apart(lib, rows, d):
    # row strides and first columns that agree in nothing: single elements
    at = {"y": 1, "r": 2, "r_out": 3, "h": 5, "gate": 0}
    wide = {k: d + 8 + v for k, v in at.items()}
    for kw in (dict(), dict(post="layer", pre="layer", post_b="bf16", pre_b="bf16", gate="element", act="silu"),
               dict(gate="channel", gate_t="fp32", r_out="in place"), dict(pre="none", pre_w=None, post_w="fp32", gate="channel")):
        kept = []
        check(lib, rows, d, view=columns(2, wide, at, kept), **kw)
        for big, first, (n, m) in kept:
            big[1:1 + n, first:first + m] = 7.0
            assert bool((big == 7.0).all())


@pytest.mark.parametrize("d", [2304, 2305])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_stays_its_own(lib, d, bad):
    rows = 1300
    y, r, gate = (torch.randn(rows, d, device="cuda") for _ in range(3))

    def run(y, r, gate):
        o, h = torch.empty_like(r), torch.empty_like(r)
        lib.wush_residual_norm(y, r, o, h, post="rms", pre="layer", gate=gate, gate_act="silu")
        return o, h

    o, h = run(y, r, gate)
    for which in range(3):
        ins = [y.clone(), r.clone(), gate.clone()]
        for row, col in ((0, 0), (7, d - 1), (650, d // 2), (rows - 1, d - 1)):
            ins[which][row, col] = bad
        o2, h2 = run(*ins)
        keep = torch.ones(rows, dtype=torch.bool, device="cuda")
        keep[[0, 7, 650, rows - 1]] = False
        assert torch.equal(o[keep], o2[keep]) and torch.equal(h[keep], h2[keep])
        assert not bool(torch.isfinite(h2[~keep]).any())


@pytest.mark.parametrize("d", [2304, 2305])
def test_two_streams_and_a_graph(lib, d):
    rows = 1300
    side = torch.cuda.Stream()
    y, r = torch.randn(rows, d, device="cuda"), torch.randn(rows, d, device="cuda").bfloat16()
    outs = [[torch.empty_like(r) for _ in range(2)] for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        lib.wush_residual_norm(y, r, *outs[0], post="rms", pre="rms")
        lib.wush_residual_norm(y, r, *outs[1], post="rms", pre="rms", stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.wush_residual_norm(y, r, *outs[2], post="rms", pre="rms")
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(outs[0], o))
    y.normal_()
    g.replay()
    lib.wush_residual_norm(y, r, *outs[0], post="rms", pre="rms")
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[2]))


def test_a_weight_between_an_outputs_rows(lib):
    # it shares no byte with them
    rows, d = 300, 2304
    x = torch.randn(rows, d, device="cuda").bfloat16()
    big = torch.ones(rows, 2 * d, dtype=torch.bfloat16, device="cuda")
    w = big[3, d:]
    w.copy_(torch.rand(d, device="cuda"))
    h = torch.empty_like(x)
    lib.wush_norm(x, h, "rms", w)
    lib.wush_norm(x, big[:, :d], "rms", w)
    assert torch.equal(big[:, :d], h)


@pytest.mark.parametrize("rows, d", [(3, 8), (3, 4096), (300, 2304), (300, 2305), (300, 32768)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_the_ends_of_the_range_of_squares(lib, rows, d, kind):
    # the root of the sum of squares just below 1.8e19; eps = 0 and the root of their mean just above 1.1e-19
    x = torch.randn(rows, d, device="cuda", dtype=torch.float64)
    if kind == "layer":
        x -= x.mean(1, keepdim=True)
    for v in (x / x.square().sum(1, keepdim=True).sqrt() * 1.7e19, x / x.square().mean(1, keepdim=True).sqrt() * 2e-19):
        v = v.float()
        h = torch.empty_like(v)
        lib.wush_norm(v, h, kind, eps=0.0)
        want, e = norm64(v.double(), torch.zeros_like(x), kind, None, None, 0.0, 0.0)
        close(h, want, "fp32", e)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("d", [4, 2304])
def test_gates_over_their_whole_range(lib, act, d):
    rows = 400
    g = torch.linspace(-110, 110, rows * d, device="cuda").view(rows, d)
    g[0, :3] = torch.tensor([0.0, float("inf"), -3e38], device="cuda")
    one, u = torch.ones(rows, d, device="cuda"), torch.empty(rows, d, device="cuda")
    lib.wush_residual_norm(one, None, u, gate=g, gate_act=act)
    want = 1 / (1 + (-g.double()).exp()) * (g.double() if act == "silu" else 1)
    # the bound on the sigmoid, silu's product, and what is below 1.2e-38 as 0
    bound = (11 + g.double().abs()) * U * want.abs() + 1.2e-38 * (g.double().abs() if act == "silu" else 1)
    ok = ((u.double() - want).abs() <= bound) | (u.double() == want)
    assert bool(ok.all()), torch.nonzero(~ok)[:4].tolist()
