"""Plain 64-bit forms of the routing losses, the norms' backward passes and the
8-bit activations for the tests, with how far fp32 arithmetic may be from each,
written from the definitions: nothing of the package is used."""
import numpy as np
import torch

EPS_BF16 = torch.finfo(torch.bfloat16).eps / 2      # one rounding to bf16, relative
U = torch.finfo(torch.float32).eps                  # one fp32 operation, relative (twice half a step)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, bound, what=""):
    got = f64(got) if torch.is_tensor(got) else got
    d = np.abs(got - want) - bound
    assert np.isfinite(got).all() and d.max() <= 0, (what, float(d.max()), int(d.argmax()))


def rounded(v, e, dtype):
    """e and the rounding of a value to dtype (1e-37: where values are subnormal)."""
    return e + (EPS_BF16 if dtype is torch.bfloat16 else U) * (np.abs(v) + e) + 1e-37


# -------------------------------------------------------------- MXFP8 --

E4M3 = np.array([m / 512.0 for m in range(8)] +
                [(8 + m) / 8.0 * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])   # codes 0..126


def mx8_quantize(x):
    """(codes, scales) of float64 x [.., C]; blocks that hold a NaN or an infinity: scale 255, NaN codes."""
    b = x.reshape(*x.shape[:-1], -1, 32).astype(np.float64)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    ok = np.where(bad | (top == 0), 1.0, top)
    m, e = np.frexp(ok / 448.0)                      # ok / 448 = m 2^e, m in [1/2, 1)
    exp = np.where(m == 0.5, e - 1, e)               # the least power of two not below it
    exp = np.where(top == 0, -127, np.maximum(exp, -127))
    a = np.abs(np.where(bad[..., None], 0.0, b)) * np.exp2(-exp.astype(np.float64))[..., None]
    hi = np.minimum(np.searchsorted(E4M3, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    code = code | np.where(np.signbit(b), np.uint8(128), np.uint8(0))
    code = np.where(bad[..., None], np.uint8(127), code)
    return code.reshape(x.shape), np.where(bad, 255, exp + 127).astype(np.uint8)


def mx8_values(codes, scales):
    c = codes & 127
    v = np.where(c == 127, np.nan, E4M3[np.minimum(c, 126)]) * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


# -------------------------------------------------------------- the norms --

SUMS = 30      # additions of a row's sum one after the other: 32 of a thread's, 6 of a wave's, 16 of the
               # waves', so 54 half steps, and 3 steps for the products


def norm(x, eps, mean, ex=0.0):
    """(n, e_n, r, rel_r): the normed rows and their roots; ex: how far x may be from the values in fp32."""
    H = x.shape[-1]
    e = np.zeros_like(x) + ex
    if mean:
        e_m = (SUMS * U * np.abs(x)).mean(-1, keepdims=True) + e.mean(-1, keepdims=True)
        x = x - x.mean(-1, keepdims=True)
        e = e + e_m + U * np.abs(x)
    ms = (x * x).mean(-1, keepdims=True) + eps
    r = 1.0 / np.sqrt(ms)
    # squares off by 2 |x| e + e^2, their sum by SUMS steps; the root halves it and has 4 steps of its own
    rel = 0.5 * ((2 * np.abs(x) * e + e * e).mean(-1, keepdims=True) / ms + SUMS * U) + 4 * U
    return x * r, r * e + np.abs(x * r) * (rel + U), r, rel


def layer_norm(x, w, b, eps):
    n, e, _, _ = norm(x, eps, True)
    w, b = (1.0 if w is None else w), (0.0 if b is None else b)
    return n * w + b, e * np.abs(w) + U * (np.abs(n * w) + np.abs(n * w + b))


def norm_backward(dy, x, w, eps, mean, res=None):
    """dx, d_weight, d_bias and their bounds, of x's values themselves."""
    H = x.shape[-1]
    n, e_n, r, rel = norm(x, eps, mean)
    w = np.ones(H) if w is None else w
    g = dy * w
    e_g = U * np.abs(g)
    c = (g * n).mean(-1, keepdims=True)
    e_c = (np.abs(g) * e_n + e_g * np.abs(n) + SUMS * U * np.abs(g * n)).mean(-1, keepdims=True) + \
        3 * U * np.abs(c)
    m, e_m = 0.0, 0.0
    if mean:
        m = g.mean(-1, keepdims=True)
        e_m = (e_g + SUMS * U * np.abs(g)).mean(-1, keepdims=True)
    q = g - m - n * c
    e_q = e_g + e_m + np.abs(n) * e_c + np.abs(c) * e_n + 4 * U * (np.abs(g) + np.abs(m) + np.abs(n * c))
    dx = r * q
    e = r * e_q + np.abs(dx) * (rel + 3 * U)
    if res is not None:
        e = e + U * (np.abs(res) + np.abs(dx))
        dx = dx + res
    T = x.shape[0]
    dw, db = (dy * n).sum(0), dy.sum(0)
    any_order = (T / 2 + 4) * U                      # T additions in any order
    e_w = (np.abs(dy) * e_n + any_order * np.abs(dy * n)).sum(0)
    return (dx, dw, db), (e, e_w, any_order * np.abs(dy).sum(0))


# -------------------------------------------------------------- SwiGLU --

def sigmoid(g):
    return np.where(g > 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def swiglu(gu):
    """(hh, bound): 8 steps for the sigmoid (exp, sum, quotient), 2 for the products; a sigmoid below
    2^-126 may be lost."""
    g, u = np.split(gu, 2, axis=-1)
    h = g * sigmoid(g) * u
    return h, 12 * U * np.abs(h) + 2.0 ** -126 * np.abs(g * u)


def swiglu_backward(d, gu):
    """(d_gu, bound)."""
    g, u = np.split(gu, 2, axis=-1)
    s, o = sigmoid(g), sigmoid(-g)
    a = g * s
    tiny = 2.0 ** -126 * (1 + np.abs(g))
    dg, du = d * u * (s + a * o), d * a
    # 1 - s is off by a step of 1 and by s's 8; the rest is relative
    eg = np.abs(d * u) * (10 * U * s + np.abs(a) * (9 * U * s + U + 10 * U * o) + 6 * U * np.abs(s + a * o) + tiny)
    return np.concatenate((dg, du), -1), np.concatenate((eg, 12 * U * np.abs(du) + np.abs(d) * tiny), -1)


# -------------------------------------------------------------- the routing losses --

def softmax(logits):
    """(p, rel, lse, e_lse); rows of -inf alone: zeros."""
    top = logits.max(-1, keepdims=True)
    some = np.isfinite(top)
    with np.errstate(invalid="ignore"):
        d = np.where(np.isfinite(logits) & some, logits - np.where(some, top, 0.0), -np.inf)
    ex = np.exp(d)
    s = ex.sum(-1, keepdims=True)
    p = np.where(some, ex / np.where(some, s, 1.0), 0.0)
    lse = np.where(some, np.where(some, top, 0.0) + np.log(np.where(some, s, 1.0)), 0.0)[..., 0]
    # the difference's rounding grows by exp to |d| steps; exp 2, the sum of 16 + 6 additions 11, quotient 3
    rel = (np.where(np.isfinite(d), np.abs(d), 0.0) + 20) * U
    e_lse = 2 * U * (np.abs(np.where(some, top, 0.0))[..., 0] + np.abs(lse)) + 20 * U
    return p, rel, lse, e_lse


def sequences(seq, T, n_seq):
    return np.zeros(T, int) if seq is None else np.where((seq >= 0) & (seq < n_seq), seq, -1)


def loads(idx, seq, n_seq, E, group=None):
    """counts [n_seq, E], tokens [n_seq + 1], load [n_seq, E]."""
    T, K = idx.shape
    seq = sequences(seq, T, n_seq)
    counts = np.zeros((n_seq, E), np.int64)
    tokens = np.zeros(n_seq + 1, np.int64)
    for t in range(T):
        if seq[t] < 0:
            continue
        tokens[seq[t]] += 1
        for e in idx[t]:
            if 0 <= e < E:
                counts[seq[t], e] += 1
    tokens[n_seq] = tokens[:n_seq].sum()
    load = counts * E / (K * np.maximum(tokens[:n_seq, None], 1))
    if group is not None:
        out = np.zeros_like(load)
        for g in range(E):
            if (group == g).any():
                out[:, group == g] = load[:, group == g].mean(1, keepdims=True)
        load = out
    return counts, tokens, load


def balance_loss(logits, idx, seq=None, n_seq=1, group=None, bc=1.0, zc=0.0):
    """(losses, bounds, counts, tokens, load)."""
    T, E = logits.shape
    counts, tokens, load = loads(idx, seq, n_seq, E, group)
    seq = sequences(seq, T, n_seq)
    p, rel, lse, e_lse = softmax(logits)
    inside = seq >= 0
    N = max(int(tokens[n_seq]), 1)
    f = load[np.maximum(seq, 0)]
    b, e_b = (p * f)[inside].sum(), (p * f * (rel + 30 * U))[inside].sum()
    z, e_z = (lse ** 2)[inside].sum(), (2 * np.abs(lse) * e_lse + e_lse ** 2)[inside].sum()
    losses = np.array([bc * b, zc * z]) / N
    e = np.array([abs(bc) * e_b, abs(zc) * e_z]) / N + 4 * U * np.abs(losses)
    return losses, e, counts, tokens, load


def route_backward(logits, idx=None, d_gate=None, seq=None, n_seq=1, tokens=None, load=None, dl=None,
                   bc=1.0, zc=0.0):
    """(d_logits, bound)."""
    T, E = logits.shape
    p, rel, lse, e_lse = softmax(logits)
    g, e_g = np.zeros((T, E)), np.zeros((T, E))
    if d_gate is not None:
        K = idx.shape[1]
        for t in range(T):
            for k in range(K):
                if 0 <= idx[t, k] < E and p[t, idx[t, k]] > 0:
                    g[t, idx[t, k]] += d_gate[t, k]
                    e_g[t, idx[t, k]] += K * U * abs(d_gate[t, k])
    more, e_more = np.zeros((T, 1)), np.zeros((T, 1))
    if load is not None:
        seq = sequences(seq, T, n_seq)
        inside = (seq >= 0)[:, None]
        N = max(int(tokens[n_seq]), 1)
        dl = (1.0, 1.0) if dl is None else dl
        b = np.where(inside, bc * dl[0] / N * load[np.maximum(seq, 0)], 0.0)
        g, e_g = g + b, e_g + 6 * U * np.abs(b) + U * np.abs(g + b)
        c = 2 * zc * dl[1] / N
        more = np.where(inside, c * lse[:, None], 0.0)
        e_more = np.where(inside, abs(c) * e_lse[:, None] + 6 * U * np.abs(more), 0.0)
    dot = (p * g).sum(1, keepdims=True)
    e_dot = (p * np.abs(g) * (rel + 14 * U) + p * e_g).sum(1, keepdims=True)
    d = p * (g - dot + more)
    e = p * (e_g + e_dot + e_more + 4 * U * (np.abs(g) + np.abs(dot) + np.abs(more))) * (1 + rel) + \
        np.abs(d) * (rel + U)
    return d, e
