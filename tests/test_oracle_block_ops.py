"""The float64 oracle of layer norm and linear attention: gradients against central differences, and
the recurrence against its closed form."""
import numpy as np
import pytest

from oracle import block_ops as ref


def _central(f, x, eps=1e-6):
    """Gradient of the scalar f at x by central differences: their error is eps^2 / 6 times the third
    derivative (1e-12 here) plus rounding, |f| 2^-53 / eps (1e-9 for |f| of about 10)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + eps
        hi = f()
        x[i] = old - eps
        lo = f()
        x[i] = old
        g[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_gradient(affine):
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    w, b = (rng.standard_normal(7), rng.standard_normal(7)) if affine else (None, None)

    def loss():
        return float((ref.layer_norm(x, w, b)[0] * g).sum())
    _, mean, rstd = ref.layer_norm(x, w, b)
    dx, dw, db = ref.layer_norm_backward(x, g, mean, rstd, w)
    assert np.max(np.abs(dx - _central(loss, x))) < 1e-7
    if affine:
        assert np.max(np.abs(dw - _central(loss, w))) < 1e-7
        assert np.max(np.abs(db - _central(loss, b))) < 1e-7


@pytest.mark.parametrize("T", [1, 2, 6])
@pytest.mark.parametrize("with_state", [True, False])
def test_linear_attention_gradient(T, with_state):
    rng = np.random.default_rng(10 + T)
    q, k, v = rng.standard_normal((T, 3)), rng.standard_normal((T, 3)), rng.standard_normal((T, 2))
    g = -rng.uniform(0.05, 1.5, T)
    go = rng.standard_normal((T, 2))
    s0 = rng.standard_normal((3, 2)) if with_state else None
    gf = rng.standard_normal((3, 2)) if with_state else None

    def loss():
        o, S = ref.linear_attention(q, k, v, g, s0, 0.7)
        return float((o * go).sum() + (0.0 if gf is None else (S[-1] * gf).sum()))
    dq, dk, dv, dg, ds = ref.linear_attention_backward(q, k, v, g, go, s0, gf, 0.7)
    for got, x in ((dq, q), (dk, k), (dv, v), (dg, g)) + (((ds, s0),) if with_state else ()):
        assert np.max(np.abs(got - _central(loss, x))) < 1e-7


def test_linear_attention_closed_form():
    # o_t = scale sum_{j <= t} exp(g_{j+1} + .. + g_t) (q_t . k_j) v_j
    rng = np.random.default_rng(5)
    T = 9
    q, k, v = rng.standard_normal((T, 4)), rng.standard_normal((T, 4)), rng.standard_normal((T, 3))
    g = -rng.uniform(0.0, 1.0, T)
    g[4] = -np.inf
    o, _ = ref.linear_attention(q, k, v, g, None, 0.5)
    for t in range(T):
        want = sum(np.exp(g[j + 1:t + 1].sum()) * (q[t] @ k[j]) * v[j] for j in range(t + 1)) * 0.5
        assert np.allclose(o[t], want, rtol=1e-12, atol=1e-12)


def test_a_reset_forgets_and_has_no_gradient():
    rng = np.random.default_rng(6)
    q, k, v, go = (rng.standard_normal((6, 3)) for _ in range(4))
    g = np.full(6, -0.1)
    g[3] = -np.inf
    whole = ref.linear_attention(q, k, v, g, rng.standard_normal((3, 3)))[0]
    assert np.allclose(whole[3:], ref.linear_attention(q[3:], k[3:], v[3:], g[3:])[0])
    assert ref.linear_attention_backward(q, k, v, g, go)[3][3] == 0.0
