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


def test_lora_add_is_the_per_token_formula():
    rng = np.random.default_rng(3)
    x, a, b = rng.standard_normal((6, 8)), rng.standard_normal((3, 4, 8)), rng.standard_normal((3, 5, 4))
    a[1, 2:] = np.nan                                    # padding is never read
    b[1, :, 2:] = np.inf
    y_in, adapter, ranks = rng.standard_normal((6, 5)), np.array([2, -1, 0, 1, 3, 1]), np.array([4, 2, 0])
    scale = np.array([0.5, -2.0, 3.0])
    y, size = B.lora_add(x, adapter, a, b, y_in, ranks, scale)
    want = y_in.copy()
    want[2] += 0.5 * b[0] @ (a[0] @ x[2])
    for t in (3, 5):
        want[t] += -2.0 * b[1][:, :2] @ (a[1][:2] @ x[t])
    assert np.allclose(y, want, rtol=1e-13) and np.array_equal(y[[0, 1, 4]], y_in[[0, 1, 4]])
    assert np.all(size >= np.abs(y - y_in) * (1 - 1e-12))
    with pytest.raises(NonFiniteInput):
        B.lora_add(np.full((6, 8), np.nan), adapter, a, b)
