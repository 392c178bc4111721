"""Plain 64-bit forms of the 4-bit expert weights and the block norms for the
tests, written from the definitions: nothing of the package is used."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EPS_BF16 = torch.finfo(torch.bfloat16).eps / 2      # one rounding to bf16, relative
EPS_F32 = torch.finfo(torch.float32).eps            # one fp32 operation, relative (twice half a step)


def quantize(x):
    """(codes [.., C/2], scales [.., C/32]) of float64 x [.., C] with finite blocks or blocks that
    hold a NaN or an infinity (scale 255; their codes are returned as 0)."""
    b = x.reshape(*x.shape[:-1], -1, 32).astype(np.float64)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    ok = np.where(bad | (top == 0), 1.0, top)
    exp = np.frexp(ok)[1] - 1 - 2                    # floor(log2 m) - 2
    exp = np.where((top == 0) & ~bad, -127, np.maximum(exp, -127))
    v = np.where(bad[..., None], 0.0, b) * np.exp2(-exp.astype(np.float64))[..., None]
    a = np.abs(v)
    code = np.zeros(a.shape, np.uint8)
    for i in range(7):                               # on a middle the neighbour with an even code
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        code = np.where(a > mid if i % 2 == 0 else a >= mid, np.uint8(i + 1), code)
    code = code | np.where(np.signbit(v), np.uint8(8), np.uint8(0))
    code = code.reshape(*x.shape[:-1], -1, 2)
    scale = np.where(bad, 255, exp + 127).astype(np.uint8)
    return (code[..., 0] | (code[..., 1] << 4)).astype(np.uint8), scale


def values(codes, scales):
    """The float64 values of packed codes and scale bytes (255: NaN)."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def product(a, w, swiglu, out_bf16, a_err=0.0):
    """(c, bound) of rows a [m, D] and weights w [N, D] in float64: the product and how far fp32
    sums in any order and the output's rounding may be from it.  a_err: how far a itself may be."""
    D = a.shape[1]
    c = a @ w.T
    # D exact products summed with at most one relative step per addition
    e = D * EPS_F32 * (np.abs(a) @ np.abs(w).T)
    if np.ndim(a_err):
        e = e + a_err @ np.abs(w).T
    if swiglu:
        n = w.shape[0] // 2
        g, u, eg, eu = c[:, :n], c[:, n:], e[:, :n], e[:, n:]
        c = silu(g) * u
        # |silu'| < 1.1; exp, sum, quotient and product: 8 fp32 steps in all
        e = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 8 * EPS_F32 * np.abs(c)
    if out_bf16:
        e = e + EPS_BF16 * (np.abs(c) + e)
    return c, e + 1e-37


def spans(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
