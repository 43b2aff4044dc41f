"""Plain 64-bit implementations of the microscaled formats, block by block from
their definitions, for the tests: value grids searched for the nearest point."""
import math

import numpy as np

FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # by code; even codes win ties


def power(top: float, limit: float, lowest: int, highest: int) -> int:
    """The least e in [lowest, highest] with top <= limit * 2^e (highest if none)."""
    for e in range(max(lowest, math.frexp(top)[1] - 12 if top else lowest), highest + 1):
        if top <= math.ldexp(limit, e):
            return e
    return highest


def fp4(v: float) -> float:
    a = abs(v)
    code = min(range(8), key=lambda c: (abs(a - FP4[c]), c & 1))
    return math.copysign(FP4[code], v)


def nearest_row(x, fmt: str):
    """The values a row of numbers stands for in MXFP4 or MXINT8."""
    out = []
    for k in range(0, len(x), 32):
        b = [float(v) for v in x[k:k + 32]]
        if not all(map(math.isfinite, b)):
            out += [math.nan] * len(b)
            continue
        top = max(abs(v) for v in b)
        if fmt == "mxfp4":
            e = power(top, 6.0, -127, 127)
            out += [math.ldexp(fp4(math.ldexp(v, -e)), e) for v in b]
        else:
            e = power(top, 127.0 / 64.0, -126, 127)
            q = [max(-127, min(127, round(math.ldexp(v, 6 - e)))) for v in b]  # round: ties to even
            out += [math.ldexp(float(t), e - 6) for t in q]
    return out


def nearest(x, fmt: str) -> np.ndarray:
    """nearest_row of every row of x [..., K], as float64."""
    x = np.asarray(x, np.float64)
    flat = x.reshape(-1, x.shape[-1])
    return np.array([nearest_row(r, fmt) for r in flat], np.float64).reshape(x.shape)
