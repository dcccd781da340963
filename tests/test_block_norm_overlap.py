"""wush_norm and wush_residual_norm refuse outputs that lie on a norm's weight or bias, or on a gate per
channel, without a GPU: made-up pointers that are never dereferenced, every call below has rows and is refused."""
import pytest

aq = pytest.importorskip("activation_quantization_b200")
lib = aq._lib

INVALID, MB = -1, 1 << 20
BF16, F32 = 0, 1


def spec(weight=0, bias=0, dtype=BF16, kind=1):
    return kind, dtype, weight, bias, 0.0, 1e-6


def residual(post=spec(), pre=spec(), gate=0, rows=4, d=64, stride=64, o=4 * MB, h=5 * MB):
    return lib.wush_residual_norm(aq._RESIDUAL_NORM_ARGS.pack(
        1 * MB, gate, 3 * MB, o, h, d, 0, d, stride, stride, rows, d, *post, *pre, F32, BF16, BF16, BF16, 0, 1.0, 1.0), None)


# (rows of 64 bf16 are 128 bytes) on the first row, on its last byte's element, on the last row, over all of
# them, and just before the first
ON = [0, 126, 3 * 128, 3 * 128 + 126, -126]


@pytest.mark.parametrize("at", ON)
@pytest.mark.parametrize("out", [4 * MB, 5 * MB])
def test_residual_norm(at, out):
    v = out + at
    assert residual(post=spec(weight=v)) == INVALID and residual(post=spec(bias=v)) == INVALID
    assert residual(pre=spec(weight=v)) == INVALID and residual(pre=spec(bias=v)) == INVALID
    assert residual(gate=v) == INVALID


@pytest.mark.parametrize("at", ON)
def test_norm(at):
    for s in (spec(weight=5 * MB + at), spec(bias=5 * MB + at)):
        assert lib.wush_norm(1 * MB, F32, 64, 4, 64, aq._NORM_SPEC.pack(*s), 5 * MB, BF16, 64, None) == INVALID


def test_between_rows_too_close():
    # rows of 128 bytes every 256: a vector of 128 bytes from 130 on runs into the next row
    for v in (126, 130, 254):
        assert residual(post=spec(weight=4 * MB + v), stride=128) == INVALID
        assert residual(gate=4 * MB + v, stride=128) == INVALID
    # an fp32 vector is twice as long
    assert residual(post=spec(weight=4 * MB + 128, dtype=F32), stride=128) == INVALID
