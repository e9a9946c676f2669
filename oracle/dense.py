"""Dense-expert operators in 64 bits (numpy): E4M3 blocks with a scale for each 128 values, the
block-scaled product, the SwiGLU block and its gradient.  Written from the definitions;
shares no code with the CUDA path."""
import numpy as np

BLOCK = 128


def e4m3_round(y):
    """float64 -> the nearest E4M3 value (ties to even, 448 the largest; inf and NaN -> NaN)."""
    y = np.asarray(y, dtype=np.float64)
    fine = np.isfinite(y)
    z = np.where(fine, y, 0.0)
    _, e = np.frexp(z)                                     # |z| in [2^(e-1), 2^e)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    q = np.clip(np.rint(z / step) * step, -448.0, 448.0)   # np.rint: ties to even
    return np.where(fine, np.copysign(q, y), np.nan)


def e4m3_half_step(y):
    """Largest rounding error of E4M3 at y: half a step of y's binade."""
    _, e = np.frexp(np.asarray(y, dtype=np.float64))
    return np.exp2(np.maximum(e - 1, -6) - 4.0)


def block_scales(x, block_rows=1):
    """2^e of every block, e the smallest integer >= -126 with max|finite x| <= 448 * 2^e."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    out = np.ones((-(-R // block_rows), -(-C // BLOCK)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            b = x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            b = np.abs(b[np.isfinite(b)])
            top = b.max() if b.size else 0.0
            if top > 0:
                e = -126
                while top > 448.0 * 2.0 ** e:
                    e += 1
                out[i, j] = 2.0 ** e
    return out


def spread(scales, R, C, block_rows=1):
    """One scale for each value of an [R, C] matrix."""
    return np.repeat(np.repeat(scales, block_rows, axis=0)[:R], BLOCK, axis=1)[:, :C]


def quantize(x, block_rows=1):
    """(E4M3 values, scales)."""
    x = np.asarray(x, dtype=np.float64)
    s = block_scales(x, block_rows)
    return e4m3_round(x / spread(s, *x.shape, block_rows)), s


def block_product(q_x, s_x, q_w, s_w):
    """sum_b s_x s_w sum_{k in b} q_x q_w, and the same of magnitudes (for error bounds)."""
    M, K = q_x.shape
    N = q_w.shape[0]
    x = q_x * spread(s_x, M, K)
    w = q_w * spread(s_w, N, K, BLOCK)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def swiglu(x, w_gate, w_up):
    """h, g, u."""
    g, u = x @ w_gate.T, x @ w_up.T
    return g * sigmoid(g) * u, g, u


def swiglu_factor_grads(g, u, dh):
    """dg, du of h = silu(g) u."""
    s = sigmoid(g)
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s


def swiglu_grads(dg, du, x, w_gate, w_up):
    """dx, dw_gate, dw_up."""
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x
