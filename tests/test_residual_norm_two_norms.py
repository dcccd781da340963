"""wush_residual_norm's two norms can differ in everything, through the binding too."""
import pytest

aq = pytest.importorskip("activation_quantization_b200")
torch = pytest.importorskip("torch")


def packed(monkeypatch, **kw):
    """(post, pre) as (kind, weight_offset, eps) of the C call's arguments; nothing is launched."""
    calls = []
    monkeypatch.setattr(aq, "_launch", lambda fn, name, args, dev, stream: calls.append(args[0]))
    y = torch.zeros(2, 64)
    aq.wush_residual_norm(y, y, y.clone(), y.clone(), post="rms", pre="layer", **kw)
    f = aq._RESIDUAL_NORM_ARGS.unpack(calls[0])
    post, pre = f[12:18], f[18:24]
    return [(s[0], pytest.approx(s[4]), pytest.approx(s[5])) for s in (post, pre)]


def test_arguments(monkeypatch):
    assert packed(monkeypatch) == [(1, 0.0, 1e-6), (2, 0.0, 1e-6)]
    assert packed(monkeypatch, eps=1e-5, weight_offset=1.0) == [(1, 1.0, 1e-5), (2, 1.0, 1e-5)]
    assert packed(monkeypatch, eps=1e-5, weight_offset=1.0, pre_eps=0.0, pre_weight_offset=0.0) == \
        [(1, 1.0, 1e-5), (2, 0.0, 0.0)]
    assert packed(monkeypatch, pre_eps=0.5, pre_weight_offset=-2.0) == [(1, 0.0, 1e-6), (2, -2.0, 0.5)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows, d", [(3, 64), (300, 2304), (300, 2305)])
def test_results(lib, rows, d):
    # With u = 2^-24: an RMS norm of up to 2305 values loses at most 160 u of its result, here below 5 (the
    # largest of the normal values) times 5 (w + 1) = 25, and the sum rounds twice: o is within 162 u * 30.
    # h is below 30 / 2 * 5 (v - 1) = 75 and loses 160 u of it, and o's error, twice over, comes through times 5 / 2.
    y, r = torch.randn(rows, d, device="cuda"), torch.randn(rows, d, device="cuda")
    w, v = torch.randn(d, device="cuda"), torch.randn(d, device="cuda")
    o, h = torch.empty_like(r), torch.empty_like(r)
    lib.wush_residual_norm(y, r, o, h, post="rms", post_weight=w, pre="rms", pre_weight=v, eps=0.5, weight_offset=1.0,
                           pre_eps=2.0, pre_weight_offset=-1.0)
    y, r, w, v = y.double(), r.double(), w.double(), v.double()
    want = r + y / (y.square().mean(1, keepdim=True) + 0.5).sqrt() * (w + 1)
    assert bool(((o - want).abs() <= 2 ** -24 * 162 * 30).all())
    want = want / (want.square().mean(1, keepdim=True) + 2).sqrt() * (v - 1)
    assert bool(((h - want).abs() <= 2 ** -24 * (160 * 75 + 2 * 162 * 30 * 2.5)).all())
