"""The 64-bit forms of the training operators against what fixes them: the
generator's published answers, closed forms, and gradients by differences."""
import numpy as np
import pytest

from oracle import training as O


@pytest.mark.parametrize(
    "counter,key,want",
    [  # the known answers published with the generator
        ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
        ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
        ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
         [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
    ],
)
def test_philox_known_answers(counter, key, want):
    assert O.philox4x32_10(np.array(counter), key).tolist() == want


def test_dropout_keeps_its_share_and_its_mean():
    p = 0.1
    keep = O.dropout_keep(np.arange(512), 1024, p, 5, 9)
    n = keep.size
    q = O.dropout_steps(p) / 65536
    assert abs(keep.mean() - (1 - q)) < 5 * np.sqrt(q * (1 - q) / n)  # five standard deviations
    assert O.dropout_scale(p) * (1 - q) == pytest.approx(1, abs=1e-15)
    assert O.dropout_keep(np.arange(4), 64, 0.0, 1, 1).all() and not O.dropout_keep(np.arange(4), 64, 1.0, 1, 1).any()
    for other in (O.dropout_keep(np.arange(512), 1024, p, 6, 9), O.dropout_keep(np.arange(512), 1024, p, 5, 10)):
        # independent masks agree in q^2 + (1 - q)^2 of the places
        a = q * q + (1 - q) ** 2
        assert abs((other == keep).mean() - a) < 5 * np.sqrt(a * (1 - a) / n)


@pytest.mark.parametrize("name", ["none", "silu", "gelu", "gelu_tanh"])
def test_groupnorm_gradients_by_differences(name):
    rng = np.random.default_rng(3)
    B, S, C, G = 2, 5, 6, 3
    x, dy = rng.normal(size=(B, S, C)) + 0.5, rng.normal(size=(B, S, C))
    w, b = 1 + 0.2 * rng.normal(size=C), 0.1 * rng.normal(size=C)
    dx, dw, db, _, _ = O.groupnorm_act_backward(x, dy, G, w, b, 1e-5, name)
    h = 1e-5  # central differences: an error of h^2 times the third derivative, and 1e-16 / h

    def slope(v, at, f):
        old = v[at]
        v[at] = old + h
        up = f()
        v[at] = old - h
        down = f()
        v[at] = old
        return (up - down) / (2 * h)

    f = lambda: (O.groupnorm_act(x, G, w, b, 1e-5, name) * dy).sum()  # noqa: E731
    for at in np.ndindex(x.shape):
        assert slope(x, at, f) == pytest.approx(dx[at], abs=1e-7)
    for c in range(C):
        assert slope(w, c, f) == pytest.approx(dw[c], abs=1e-7)
        assert slope(b, c, f) == pytest.approx(db[c], abs=1e-7)


def test_groupnorm_closed_forms():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(2, 7, 8)) * 3 + 1
    y = O.groupnorm_act(x, 4, eps=0.0, name="none").reshape(2, 7, 4, 2)
    assert np.allclose(y.mean(axis=(1, 3)), 0, atol=1e-12) and np.allclose((y**2).mean(axis=(1, 3)), 1, atol=1e-12)
    assert np.allclose(O.groupnorm_act(x + 5, 4, eps=0.0, name="none").reshape(y.shape), y, atol=1e-12)


def test_balance_gradient_by_differences_and_even_load():
    rng = np.random.default_rng(5)
    T, E, K = 6, 5, 2
    logits, experts = rng.normal(size=(T, E)), rng.integers(0, E, size=(T, K))
    mask = np.array([1, 1, 0, 1, 1, 1], dtype=bool)
    loss, counts = O.router_balance_loss(logits, experts, 0.3, mask)
    d, _ = O.router_balance_loss_backward(logits, counts, K, 1.7, 0.3, mask)
    h = 1e-5
    for at in np.ndindex(logits.shape):
        v = logits.copy()
        v[at] += h
        up = O.router_balance_loss(v, experts, 0.3, mask)[0]
        v[at] -= 2 * h
        down = O.router_balance_loss(v, experts, 0.3, mask)[0]
        assert 1.7 * (up - down) / (2 * h) == pytest.approx(d[at], abs=1e-9)
    # even counts and even probabilities: the loss is the coefficient
    even = np.arange(T * K).reshape(T, K) % 4
    assert O.router_balance_loss(np.zeros((T, 4)), even, 0.3)[0] == pytest.approx(0.3)
