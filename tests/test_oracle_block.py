"""The oracle's block operators against closed forms and torch's own fp64 norms."""
import numpy as np
import pytest

from oracle import block as B
from oracle._checks import NonFiniteInput

torch = pytest.importorskip("torch")


def test_norms_match_torch_fp64():
    rng = np.random.default_rng(1)
    v, w, b = rng.standard_normal((5, 37)) * 3 + 1, rng.standard_normal(37), rng.standard_normal(37)
    t = [torch.from_numpy(a) for a in (v, w, b)]
    want = torch.nn.functional.layer_norm(t[0], (37,), t[1], t[2], 1e-5).numpy()
    assert np.allclose(B.norm(v, "layer", w, b, 1e-5), want, rtol=1e-13, atol=1e-13)
    want = torch.nn.functional.rms_norm(t[0], (37,), t[1], 1e-5).numpy()
    assert np.allclose(B.norm(v, "rms", w - 1.0, None, 1e-5, 1.0), want, rtol=1e-12, atol=1e-12)
    # closed forms: a constant row has rms norm 1 and layer norm 0
    assert np.allclose(B.norm(np.full((1, 8), -3.0), "rms", eps=0.0), -1.0)
    assert np.all(B.norm(np.full((1, 8), -3.0), "layer", eps=1e-6) == 0.0)


def test_activations():
    g = np.array([[0.0, 800.0, -800.0, 1.5]])
    assert np.allclose(B.activate(g, "sigmoid"), [[0.5, 1.0, 0.0, 1 / (1 + np.exp(-1.5))]])
    assert np.allclose(B.activate(g, "silu"), g * B.activate(g, "sigmoid"))
    assert np.array_equal(B.activate(g, "linear"), g)


def test_residual_norm_is_its_parts():
    rng = np.random.default_rng(2)
    y, r, g = rng.standard_normal((3, 16)), rng.standard_normal((3, 16)), rng.standard_normal(16)
    w = rng.standard_normal(16)
    u, out, h = B.residual_norm(y, r, "rms", w, None, g, "silu", 0.5, 2.0, "layer", w)
    assert np.allclose(u, B.norm(y, "rms", w) * B.activate(g, "silu"))
    assert np.allclose(out, 0.5 * r + 2.0 * u) and np.allclose(h, B.norm(out, "layer", w))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_non_finite_inputs_are_refused(bad):
    ok, x = np.ones((2, 4)), np.ones((2, 4))
    x[1, 2] = bad
    for call in (lambda: B.norm(x, "rms"), lambda: B.residual_norm(x, ok), lambda: B.residual_norm(ok, x),
                 lambda: B.residual_norm(ok, ok, gate=x), lambda: B.activate(x, "silu"),
                 lambda: B.norm(ok, "rms", x[1])):
        with pytest.raises(NonFiniteInput):
            call()
