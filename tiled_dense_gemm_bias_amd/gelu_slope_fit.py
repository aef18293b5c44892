"""Fits the polynomial of the GELU derivative that the kernels use.

gelu'(z) = Phi(z) + z phi(z). With m(x) = Phi(-x) / phi(x) (the Mills ratio) and x = |z|,

    q(x) = e^(-x^2/2) P(x),   P(x) = (m(x) - x) / sqrt(2 pi),

is gelu'(z) for z <= 0 and 1 - gelu'(z) for z > 0. P is smooth, and the exponential
bounds what an error of P does, so P is fitted by weighted least squares whose
weights are raised where the error is largest (Lawson's method) until the
weighted error is level.

    python -m tiled_dense_gemm_bias_amd.gelu_slope_fit
"""
import numpy as np

DEGREE, X_MAX, CLAMP = 7, 7.0, 8.0
COEFFS = (0.49999603629112244, -0.7976623773574829, 0.2479596585035324, -0.12582695484161377,
          0.049940045922994614, -0.013923607766628265, 0.002319070976227522, -0.00016855745343491435)


def target(x):
    from scipy.special import erfcx
    return (np.sqrt(np.pi / 2) * erfcx(x / np.sqrt(2)) - x) / np.sqrt(2 * np.pi)


def fit(degree=DEGREE, x_max=X_MAX, nodes=6000, rounds=400):
    """Coefficients, lowest first, and the largest weighted error."""
    x = (1 - np.cos(np.linspace(0, np.pi, nodes))) / 2 * x_max
    w, powers, want = np.exp(-x * x / 2), np.vander(x, degree + 1, increasing=True), target(x)
    lawson, best = np.ones_like(x), None
    for _ in range(rounds):
        s = w * np.sqrt(lawson)
        c = np.linalg.lstsq(powers * s[:, None], want * s, rcond=None)[0]
        e = np.abs((powers @ c - want) * w)
        if best is None or e.max() < best[1]:
            best = (c, e.max())
        lawson *= (e / e.max() + 1e-3) ** 0.5
        lawson /= lawson.max()
    return best


def slope(z, coeffs=COEFFS):
    """gelu'(z) in the kernels' fp32 steps."""
    f = np.float32
    z = np.asarray(z, f)
    a = np.minimum(np.abs(z), f(CLAMP))
    p = np.full_like(z, f(coeffs[-1]))
    for k in coeffs[-2::-1]:
        p = (p * a + f(k)).astype(f)
    q = (p * np.exp2((z * z).astype(f) * f(-0.7213475204444817)).astype(f)).astype(f)
    return np.where(z > 0, f(1) - q, q)


if __name__ == "__main__":
    c, e = fit()
    print("weighted error %.3g" % e)
    for v in c:
        print("%.17g" % np.float32(v))
