"""Plain float64 reference of rope_append."""
import numpy as np


def rotate(x, weight, eps, positions, inv_freq, axes, interleaved):
    """x float64 [N][H][D] (bf16 values): (result, the size of what was summed
    for each element), both float64."""
    N, H, D = x.shape
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    half = len(inv_freq)
    out, size = y.copy(), np.abs(y)
    if half:
        angle = positions[np.asarray(axes)].astype(np.float64).T * np.asarray(inv_freq)  # [N][half]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ya, yb = y[..., a], y[..., b]
        out[..., a], out[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = size[..., b] = np.abs(ya) + np.abs(yb)
    return out, size


def fp32_error(size, positions, inv_freq):
    """Error before the last rounding.  The norm's factor, the weights, cos and
    sin and the sums take some ten fp32 roundings (2^-24 each) of what is summed;
    the kernel's angle is off by 2^-24 of half a turn (pi 2^-24) and its
    frequency by 2^-53 of itself, the reference's angle by 2^-53 of itself twice."""
    far = 0.0 if not len(inv_freq) else float(np.abs(positions.astype(np.float64)).max() * np.abs(inv_freq).max())
    return (16 * 2.0 ** -24 + 4 * far * 2.0 ** -53) * size
