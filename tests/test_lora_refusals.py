"""What wush_lora_add refuses, without a GPU: made-up pointers that are never dereferenced
for the C call, CPU tensors for the binding."""
import pytest

aq = pytest.importorskip("activation_quantization_b200")
torch = pytest.importorskip("torch")
lib = aq._lib

OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, -1, -2, -6
BF16, F32, F16 = 0, 1, 2
MB = 1 << 20


def call(**kw):
    # every call below either has no tokens or must be refused: nothing is launched
    v = dict(x=1 * MB, xd=BF16, xs=256, tokens=1000, d_in=256, d_out=512, adapter=2 * MB, a=3 * MB, b=4 * MB, n=4,
             rank=16, ranks=5 * MB, scale=6 * MB, yi=16 * MB, yis=512, y=32 * MB, ys=512, ws=64 * MB, wn=1 << 40)
    v.update(kw)
    p = lambda k: v[k] or 0  # noqa: E731
    return lib.wush_lora_add(aq._LORA_ARGS.pack(
        p("x"), p("adapter"), p("a"), p("b"), p("ranks"), p("scale"), p("yi"), p("y"), p("ws"), v["xs"], v["yis"],
        v["ys"], v["tokens"], v["d_in"], v["d_out"], v["n"], v["rank"], v["wn"], v["xd"]), None)


def test_shapes_and_types():
    assert call(tokens=0) == OK and lib.wush_lora_add(None, None) == INVALID
    assert call(tokens=-1) == INVALID
    for k, bad in (("d_in", (0, -32, 16, 48)), ("d_out", (0, 4, 12)), ("rank", (0, 4, 12, -8)), ("n", (0, -1))):
        for v in bad:
            assert call(**{k: v}) == INVALID, (k, v)
    assert call(xd=F32) == UNSUPPORTED and call(xd=5) == UNSUPPORTED
    assert call(rank=264) == UNSUPPORTED and call(d_in=1 << 25, xs=1 << 25) == UNSUPPORTED
    assert call(d_out=1 << 25, ys=1 << 25, yis=1 << 25) == UNSUPPORTED and call(tokens=1 << 27) == UNSUPPORTED
    assert call(n=(1 << 20) + 1) == UNSUPPORTED
    assert call(ys=1 << 58) == UNSUPPORTED and call(xs=1 << 39) == UNSUPPORTED
    # pools too large to sort by
    assert call(n=60000, tokens=4097) == UNSUPPORTED and call(n=50000, d_out=1 << 16, ys=1 << 16, yis=1 << 16,
                                                              tokens=4097) == UNSUPPORTED


def test_pointers_and_strides():
    for k in ("x", "adapter", "a", "b", "y"):
        assert call(**{k: None}) == INVALID, k
    for k in ("x", "a", "b", "y", "yi"):
        assert call(**{k: 64 * MB + 8}) == INVALID, k
    for k in ("adapter", "ranks", "scale"):
        assert call(**{k: 64 * MB + 2}) == INVALID, k
    assert call(xs=255) == INVALID and call(xs=260) == INVALID
    assert call(ys=511) == INVALID and call(ys=514) == INVALID and call(yis=511) == INVALID and call(yis=513) == INVALID


def test_overlaps():
    assert call(y=16 * MB + 2048) == INVALID                   # one row into y_in
    assert call(y=16 * MB, ys=516) == INVALID                  # y_in itself with another stride
    assert call(y=1 * MB) == INVALID                           # on x
    assert call(yis=1024, ys=1024, y=16 * MB + 511 * 4 + 4 - 16) == INVALID   # columns that share one place


def test_workspace():
    need = aq.wush_lora_workspace_bytes(1000, 256, 512, 4, 16)
    assert need > 0 and aq.wush_lora_workspace_bytes(256, 256, 512, 4, 16) == 0
    assert call(wn=need - 1) == TOO_SMALL and call(ws=None) == INVALID and call(ws=64 * MB + 8) == INVALID
    for at in (1 * MB, 16 * MB, 32 * MB, 32 * MB - 512):                  # on x, y_in and y
        assert call(ws=at) == INVALID, at
    for bad in ((-1, 256, 512, 4, 16), (0, 256, 512, 4, 16), (10, 0, 512, 4, 16), (10, 256, 512, 0, 16)):
        assert aq.wush_lora_workspace_bytes(*bad) == 0


def test_binding_checks():
    bf = torch.bfloat16
    x, a, b = torch.zeros(3, 64, dtype=bf), torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 24, 8, dtype=bf)
    g, y = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 24)

    def refused(match, **kw):
        v = dict(x=x, adapter=g, a=a, b=b, y_in=y, y=y, workspace=None, ranks=None, scale=None)
        v.update(kw)
        with pytest.raises(ValueError, match=match):
            aq.wush_lora_add(**v)

    refused("expected a CUDA tensor")                          # all else is right
    refused("expected a CUDA tensor", y_in=None, ranks=torch.zeros(2, dtype=torch.int32), scale=torch.zeros(2))
    refused("adapter must be", adapter=g.long())
    refused("adapter must be", adapter=g[:2])
    refused("a must be", a=a.half())
    refused("a must be", a=a[:, :, :32])
    refused("b must be", b=torch.zeros(2, 48, 8, dtype=bf)[:, ::2])
    refused("b must be", b=b.half())
    refused("y must be torch.float32", y=y.bfloat16())
    refused("y_in must be", y_in=y[:, :16])
    refused("ranks must be", ranks=torch.zeros(2))
    refused("scale must be", scale=torch.zeros(3))
    refused("bf16, fp32 or fp16", x=x.double())
