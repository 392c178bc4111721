"""The tests' own 64-bit forms of the gradients against differences, and of the 8-bit conversion on
blocks whose result is known."""
import numpy as np

import _train as ref


def _differences(f, x, h=1e-5):
    """Central differences of the number f(x) at x."""
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        lo, hi = x.copy(), x.copy()
        lo[i] -= h
        hi[i] += h
        d[i] = (f(hi) - f(lo)) / (2 * h)
    return d


def _same(a, b):
    # central differences of smooth functions of order one: h^2 and 1e-16 / h
    assert np.abs(a - b).max() < 1e-8 * max(1.0, np.abs(b).max()), np.abs(a - b).max()


def test_norms_gradients():
    rng = np.random.default_rng(0)
    x, dy, w = rng.standard_normal((3, 8)), rng.standard_normal((3, 8)), rng.standard_normal(8)
    for mean in (False, True):
        f = lambda x, w, b: ((ref.norm(x, 1e-2, mean)[0] * w + b) * dy).sum()        # noqa: E731
        (dx, dw, db), _ = ref.norm_backward(dy, x, w, 1e-2, mean)
        _same(dx, _differences(lambda v: f(v, w, 0.0), x))
        _same(dw, _differences(lambda v: f(x, v, 0.0), w))
        _same(db, _differences(lambda v: f(x, w, v), np.zeros(8)))


def test_swiglu_gradient():
    rng = np.random.default_rng(1)
    gu, d = 2 * rng.standard_normal((3, 12)), rng.standard_normal((3, 6))
    _same(ref.swiglu_backward(d, gu)[0], _differences(lambda v: (ref.swiglu(v)[0] * d).sum(), gu))


def test_routing_gradient():
    """Of the gates, the balance loss (its loads are constants) and the z loss, with padding, a masked
    expert and an expert picked twice."""
    rng = np.random.default_rng(2)
    T, E, K, n = 6, 5, 3, 2
    logits, d_gate = rng.standard_normal((T, E)), rng.standard_normal((T, K))
    idx = np.argsort(-logits, 1)[:, :K]
    idx[0, 1] = idx[0, 0]
    seq = np.array([0, 1, 1, -1, 0, 2])              # 2 is no sequence either
    dl, bc, zc = (3.0, -2.0), 0.7, 0.3
    _, _, _, tokens, load = ref.balance_loss(logits, idx, seq, n, None, bc, zc)
    assert tokens.tolist() == [2, 2, 4]

    def f(v):
        p, _, lse, _ = ref.softmax(v)
        inside = np.isin(seq, (0, 1))
        s = np.where(inside, seq, 0)
        gates = np.take_along_axis(p, idx, 1)
        return ((gates * d_gate).sum() + dl[0] * bc / 4 * (p * load[s])[inside].sum() +
                dl[1] * zc / 4 * (lse[inside] ** 2).sum())

    _same(ref.route_backward(logits, idx, d_gate, seq, n, tokens, load, dl, bc, zc)[0],
          _differences(f, logits))
    losses = ref.balance_loss(logits, idx, seq, n, None, bc, zc)[0]
    none = np.zeros((T, K))
    _same(dl[0] * losses[0] + dl[1] * losses[1], f(logits) - (np.take_along_axis(
        ref.softmax(logits)[0], idx, 1) * (d_gate - none)).sum())


def test_loads_of_an_even_routing_are_one():
    idx = np.arange(24).reshape(8, 3) % 6
    counts, tokens, load = ref.loads(idx, None, 1, 6, None)
    assert (counts == 4).all() and (load == 1).all() and tokens.tolist() == [8, 8]
    group = np.array([0, 0, 3, 3, 3, -1])
    load = ref.loads(np.array([[0, 2, 5]]), None, 1, 6, group)[2]
    assert np.allclose(load, [[1, 1, 2 / 3, 2 / 3, 2 / 3, 0]])


def test_eight_bit_blocks_of_known_values():
    """Every code comes back from its value at any scale, and the scale is the least that clips nothing."""
    assert len(ref.E4M3) == 127 and ref.E4M3[-1] == 448 and ref.E4M3[8] == 2.0 ** -6
    x = np.zeros((5, 32))
    for i in range(4):
        x[i] = ref.E4M3[i * 32:i * 32 + 32][:32] if i < 3 else np.append(ref.E4M3[96:], 448.0)
    x[:, -1] = 448.0                                 # so that every block has scale 1
    x[4, :4] = 16.5, 17.5, 0.5 / 512, 1.5 / 512      # in the middle of two: to the even one
    codes, scales = ref.mx8_quantize(x)
    assert (scales == 127).all()
    v = ref.mx8_values(codes, scales)
    assert np.array_equal(v[:4], x[:4]) and v[4, :4].tolist() == [16, 18, 0, 2 / 512]
    assert np.array_equal(ref.mx8_quantize(-x)[0][:4], codes[:4] | 128)
    for top, scale in ((448.0, 127), (449.0, 128), (512.0, 128), (896.0, 128), (897.0, 129),
                       (2.0 ** -140, 0), (0.0, 0)):
        assert ref.mx8_quantize(np.full((1, 32), top))[1][0, 0] == scale, top
    x = np.full((1, 64), 1.0)
    x[0, 40] = np.inf
    codes, scales = ref.mx8_quantize(x)
    assert scales.tolist() == [[119, 255]] and np.isnan(ref.mx8_values(codes, scales)[0, 32:]).all()
