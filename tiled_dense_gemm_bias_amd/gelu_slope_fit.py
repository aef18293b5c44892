"""Fits the polynomial of the GELU derivative that the kernels use.

gelu'(z) = Phi(z) + z phi(z). With m(x) = Phi(-x) / phi(x) (the Mills ratio) and x = |z|,

    q(x) = e^(-x^2/2) (R(t) - x / sqrt(2 pi)),   t = 1 / (1 + x/4),

is gelu'(z) for z <= 0 and 1 - gelu'(z) for z > 0. R(t) stands for m(x) / sqrt(2 pi), which
falls like 1 / x, so that a short polynomial in t holds it for all x, and its
coefficients do not cancel in fp32. The fit is of q's relative error (absolute where
|R - x / sqrt(2 pi)| < 0.05, about the zero at x = 0.75), by weighted least squares
whose weights are raised where the error is largest (Lawson's method) until the
weighted error is level: 4.2e-8, below fp32's own step. In fp32 steps the derivative of 16-bit
z is within 2e-7, and from z = -1 down within 1e-6 of itself to z = -5, 2e-6 to z = -8
(the rounding of the exponential's argument). A polynomial in x of the same
degree has a level absolute error of 4e-6, more than a step of fp16 below z = -3.

    python -m tiled_dense_gemm_bias_amd.gelu_slope_fit
"""
import numpy as np

DEGREE, SCALE, X_MAX, CLAMP = 7, 0.25, 14.0, 16.0
# Of R, lowest first.
COEFFS = (0.0001873002465777, 0.0963644464504781, 0.1251299008583134, -0.0111699049002808,
          0.3387267891725851, -0.3203441591740204, 0.3682747148994894, -0.0971691083497504)


def target(x):
    from scipy.special import erfcx
    return erfcx(x / np.sqrt(2)) / 2


def fit(degree=DEGREE, x_max=X_MAX, nodes=6000, rounds=400):
    """Coefficients, lowest first, and the largest weighted error."""
    x = (1 - np.cos(np.linspace(0, np.pi, nodes))) / 2 * x_max
    powers, want = np.vander(1 / (1 + SCALE * x), degree + 1, increasing=True), target(x)
    w = 1 / np.maximum(np.abs(want - x / np.sqrt(2 * np.pi)), 0.05)
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
    f, d = np.float32, np.float64
    z = np.asarray(z, f)
    a = np.minimum(np.abs(z), f(CLAMP))
    t = (f(1) / (a * f(SCALE) + f(1)).astype(f)).astype(f)
    r = np.full_like(z, f(coeffs[-1] / 8))
    for k in coeffs[-2::-1]:
        r = (d(r) * d(t) + d(f(k / 8))).astype(f)                          # fma
    p = (d(a) * d(f(-0.3989422804014327 / 8)) + d(r)).astype(f)
    with np.errstate(over="ignore"):                                       # z^2 past the largest fp32: e^-inf
        e = (d((z * z).astype(f)) * d(f(-0.7213475204444817)) + 3).astype(f)
    q = (p * np.exp2(e).astype(f)).astype(f)
    return np.where(z > 0, f(1) - q, q)


if __name__ == "__main__":
    c, e = fit()
    print("weighted error %.3g" % e)
    for v in c:
        print("%.17g" % v)
