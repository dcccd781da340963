"""What wush_norm and wush_residual_norm refuse, without a GPU: made-up pointers that are
never dereferenced for the C calls, CPU tensors for the binding."""
import pytest

aq = pytest.importorskip("activation_quantization_b200")
torch = pytest.importorskip("torch")
lib = aq._lib

OK, INVALID, UNSUPPORTED = 0, -1, -2
BF16, F32, F16 = 0, 1, 2
NAN, INF = float("nan"), float("inf")
MB = 1 << 20


def spec(kind=1, dtype=BF16, weight=64 * MB, bias=None, offset=0.0, eps=1e-6):
    return kind, dtype, weight or 0, bias or 0, offset, eps


def residual(**kw):
    # rows = 0 passes every check that does not depend on the rows, and launches nothing
    a = dict(y=1 * MB, yd=F32, ys=64, post=spec(), gate=2 * MB, gd=BF16, gs=64, act=1, r=3 * MB, rd=BF16, rs=64, a=1.0,
             b=1.0, rows=0, d=64, pre=spec(), o=4 * MB, os=64, h=5 * MB, hd=BF16, hs=64)
    a.update(kw)
    p = lambda k: a[k] or 0  # noqa: E731
    return lib.wush_residual_norm(aq._RESIDUAL_NORM_ARGS.pack(
        p("y"), p("gate"), p("r"), p("o"), p("h"), a["ys"], a["gs"], a["rs"], a["os"], a["hs"], a["rows"], a["d"],
        *a["post"], *a["pre"], a["yd"], a["gd"], a["rd"], a["hd"], a["act"], a["a"], a["b"]), None)


def test_residual_norm_refusals():
    assert residual() == OK
    assert lib.wush_residual_norm(None, None) == INVALID
    assert residual(post=spec(kind=0), pre=spec(kind=0), gate=None, r=None) == OK
    assert residual(y=None) == INVALID and residual(o=None, h=None) == INVALID
    assert residual(o=None) == OK and residual(h=None) == OK
    assert residual(d=0) == INVALID and residual(rows=-1) == INVALID
    assert residual(d=32769, ys=32769, gs=0, rs=32769, os=32769, hs=32769) == UNSUPPORTED
    assert residual(rows=1 << 31) == UNSUPPORTED
    for k in ("yd", "gd", "rd", "hd"):
        assert residual(**{k: 3}) == UNSUPPORTED and residual(**{k: -1}) == UNSUPPORTED, k
    for k in ("ys", "rs", "os", "hs"):
        assert residual(**{k: 63}) == INVALID and residual(**{k: 0}) == INVALID, k
        assert residual(**{k: -64}) == INVALID, k
    assert residual(gs=0) == OK and residual(gs=63) == INVALID
    assert residual(act=3) == UNSUPPORTED and residual(act=-1) == UNSUPPORTED
    assert residual(gate=None, act=9) == OK                               # no gate: its arguments are unused
    for k in ("y", "gate", "r", "o", "h"):
        assert residual(**{k: 4097}) == INVALID, k                        # not aligned to its element
    assert residual(y=4098) == INVALID                                    # fp32 at a 2-byte boundary
    assert residual(r=3 * MB + 2, gate=2 * MB + 2) == OK                  # bf16 needs no more than its element
    for bad in (NAN, INF, -INF):
        assert residual(a=bad) == INVALID and residual(b=bad) == INVALID
        assert residual(post=spec(eps=bad)) == INVALID and residual(pre=spec(offset=bad)) == INVALID
    assert residual(pre=spec(eps=-1e-6)) == INVALID and residual(pre=spec(eps=0.0)) == OK
    assert residual(post=spec(kind=3)) == UNSUPPORTED and residual(pre=spec(dtype=5)) == UNSUPPORTED
    assert residual(pre=spec(weight=4097)) == INVALID and residual(pre=spec(bias=4097)) == INVALID
    assert residual(pre=spec(kind=0, dtype=9, weight=4097, eps=NAN)) == OK   # kind none: the rest is unused
    assert residual(pre=spec(dtype=7, weight=None, bias=None)) == OK      # no vectors: their type is unused


def test_overlapping_outputs_are_refused():
    rows = dict(rows=4)
    assert residual(o=3 * MB, rs=64, os=64, rows=0) == OK
    # every one of these would launch if it were accepted, so all of them must be refused
    assert residual(o=1 * MB, **rows) == INVALID                          # r_out on y
    assert residual(h=1 * MB, **rows) == INVALID                          # h on y
    assert residual(h=3 * MB, **rows) == INVALID                          # h on r
    assert residual(h=4 * MB, **rows) == INVALID                          # h on r_out
    assert residual(o=3 * MB, os=72, **rows) == INVALID                   # r_out on r with another stride
    assert residual(o=3 * MB + 64, **rows) == INVALID                     # r_out half a row into r
    assert residual(o=2 * MB, **rows) == INVALID and residual(h=2 * MB, gs=0, **rows) == INVALID   # on the gate
    assert residual(o=2 * MB - 128 * 3, gs=0, **rows) == INVALID          # r_out's last row on a gate per channel
    # columns of one buffer: 64 columns at 0 and at 63 of rows of 128 share one column
    assert residual(o=4 * MB, os=128, h=4 * MB + 2 * 63, hs=128, **rows) == INVALID
    assert residual(o=4 * MB, os=128, h=4 * MB + 2 * 65, hs=128, **rows) == INVALID   # the last column wraps


def test_norm_refusals():
    def call(**kw):
        a = dict(x=1 * MB, xd=F32, xs=64, rows=0, d=64, n=spec(), h=2 * MB, hd=F16, hs=64)
        a.update(kw)
        return lib.wush_norm(a["x"], a["xd"], a["xs"], a["rows"], a["d"],
                             None if a["n"] is None else aq._NORM_SPEC.pack(*a["n"]), a["h"], a["hd"], a["hs"], None)

    assert call() == OK and call(n=None) == INVALID and call(x=None) == INVALID and call(h=None) == INVALID
    assert call(d=0) == INVALID and call(rows=-3) == INVALID and call(d=1 << 16, xs=1 << 16, hs=1 << 16) == UNSUPPORTED
    assert call(xd=4) == UNSUPPORTED and call(hd=4) == UNSUPPORTED and call(n=spec(kind=-1)) == UNSUPPORTED
    assert call(xs=63) == INVALID and call(hs=63) == INVALID and call(x=4099) == INVALID and call(h=4099) == INVALID
    assert call(rows=4, h=1 * MB) == INVALID                              # in place needs one type and stride
    assert call(rows=4, h=1 * MB + 256, hd=F32) == INVALID


def test_binding_checks():
    x, h = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        aq.wush_norm(x, h, "rms", w)                                      # all else is right
    with pytest.raises(ValueError, match="h must be"):
        aq.wush_norm(x, h[:, :63], "rms", w)
    with pytest.raises(ValueError, match="bf16, fp32 or fp16"):
        aq.wush_norm(x.double(), h, "rms", w)
    with pytest.raises(ValueError, match="weight must be"):
        aq.wush_norm(x, h, "rms", w[:63])
    with pytest.raises(ValueError, match="weight must be"):
        aq.wush_norm(x, h, "rms", torch.ones(128)[::2])
    with pytest.raises(ValueError, match="one type"):
        aq.wush_norm(x, h, "layer", w, w.half())
    with pytest.raises(ValueError, match="contiguous"):
        aq.wush_norm(torch.zeros(64, 4).T, h, "rms", w)
    with pytest.raises(ValueError, match="overlap"):
        aq.wush_norm(x[:1].expand(4, 64), h, "rms", w)
    with pytest.raises(KeyError):
        aq.wush_norm(x, h, "batch", w)
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        aq.wush_residual_norm(x, h, h, h.clone(), post="rms", pre="layer", gate=w, gate_act="silu")
    with pytest.raises(ValueError, match="r_out must have r's type"):
        aq.wush_residual_norm(x, h, x.clone())
    with pytest.raises(ValueError, match="gate per channel"):
        aq.wush_residual_norm(x, h, h, gate=w[:5])
    with pytest.raises(ValueError, match="gate must be"):
        aq.wush_residual_norm(x, h, h, gate=x[:2])
