"""64-bit definitions of the decoder-layer operators for the tests, in numpy."""
import math

import numpy as np

U = 2.0 ** -24                                             # half a step of fp32, relative
SMALL = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}  # half a step below the smallest normal number


def half_step(out):
    """Half a step of the output type relative to the value; an fp32 output's
    rounding is counted with the operation that forms it."""
    return {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}[out]


def product(x, xs, w, ws, bias=None):
    """(y, bound on |fp32 result - y|) of the 8-bit product: the conversion of
    the integer, the two scales and the bias are one rounding each."""
    y = (x.astype(np.int64) @ w.astype(np.int64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    err = 3.01 * U * np.abs(y)
    if bias is not None:
        y = y + bias.astype(np.float64)
        err = err + 1.01 * U * np.abs(y)
    return y, err


def rounded(y, err, out):
    """Bound on |output - y| once the fp32 value is rounded to `out`."""
    return err + (np.abs(y) + err) * half_step(out) + SMALL[out]


def _erfc(x):
    return np.vectorize(math.erfc, otypes=[np.float64])(x)


def activate(g, err, kind):
    """(act(g), bound on the fp32 result for a g that is off by err)."""
    if kind == "silu":
        # g / (1 + exp(-g)): one rounding each for the sum and the quotient, two
        # for exp; the slope of silu is at most 1.1
        e = np.exp(np.minimum(-g, 700.0))
        a = g / (1 + e)
        return a, 1.1 * err + 6 * U * np.abs(a)
    if kind == "gelu_tanh":
        # z carries six roundings, and exp(-2 z) makes them 2 |z| times as large relative to a
        z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        a = g / (1 + np.exp(np.minimum(-2 * z, 700.0)))
        return a, 1.2 * err + (6 + 2 * 8 * np.abs(z)) * U * np.abs(a)
    # 0.5 g erfc(-g / sqrt 2): the argument's two roundings are 2 x^2 + 1 times
    # as large relative to erfc for negative g; erfc itself within 16 units
    a = 0.5 * g * _erfc(-g / math.sqrt(2))
    return a, 1.2 * err + (40 + 4 * (g * g + 1)) * U * np.abs(a)


def gated(x, xs, wg, gs, wu, us, kind):
    g, ge = product(x, xs, wg, gs)
    u, ue = product(x, xs, wu, us)
    a, ae = activate(g, ge, kind)
    y = a * u
    return y, ae * np.abs(u) + ue * np.abs(a) + ae * ue + U * np.abs(y) + 2.0 ** -126 * (1 + np.abs(u))


def norm(r, y, weight, post, gate, alpha, eps):
    """(x, bound on x, h, bound on h) in 64 bits.  Bounds: a row's sum of
    squares is at most 32 + 6 + 16 fp32 additions deep, so its root is off by
    at most 28 U, and the quotient, the root, eps and the multiplications add 8."""
    r = r.astype(np.float64)
    if y is None:
        x, part = r, np.zeros_like(r)
    else:
        u = y.astype(np.float64)
        if post is not None:
            u = u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * post
        if gate is not None:
            u = u * gate
        part = alpha * u
        x = r + part
    ex = U * (1.01 * np.abs(x) + 42 * np.abs(part))
    rms = np.sqrt((x * x).mean(1, keepdims=True) + eps)
    w = 1.0 if weight is None else weight.astype(np.float64)
    h = x / rms * w
    # the error of x moves the root mean square by at most its own root mean square
    drift = np.sqrt((ex * ex).mean(1, keepdims=True)) / rms
    eh = np.abs(h) * (40 * U + drift) + np.abs(w) * ex / rms
    return x, ex, h, eh


def quant(x):
    """Codes and scales of fp32 rows, bit for bit."""
    x = x.astype(np.float32)
    bad = ~np.isfinite(x).all(1)
    top = np.where(bad, 0, np.abs(np.where(np.isfinite(x), x, 0)).max(1)).astype(np.float32)
    s = (top / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((x / s[:, None]).astype(np.float32))
    q = np.where((s > 0)[:, None] & ~bad[:, None], q, 0)
    q = np.clip(np.nan_to_num(q), -127, 127).astype(np.int8)
    return q, np.where(bad, np.float32(np.nan), s)


def positions(ctx, masks, n):
    ctx = np.maximum(np.asarray(ctx, dtype=np.int64), 0)
    p = np.zeros((len(ctx), n), dtype=np.int64)
    for b in range(len(ctx)):
        for i in range(n):
            p[b, i] = ctx[b] + (i if masks is None else bin(int(masks[b, i]) & ((1 << i) - 1)).count("1"))
    return p


def rotate(t, pos, freq, interleaved, scale):
    """(turned, bound): sine and cosine within 6 U (the reduced angle's rounding
    and two units of the functions), then scale, two products and a sum."""
    t = t.astype(np.float64)
    rot = 2 * len(freq)
    ang = pos[:, :, None, None].astype(np.float64) * freq.astype(np.float64)
    c, s = np.cos(ang), np.sin(ang)
    a, b = (t[..., 0:rot:2], t[..., 1:rot:2]) if interleaved else (t[..., :rot // 2], t[..., rot // 2:rot])
    out, err = t.copy(), np.zeros_like(t)
    y = scale * (a * c - b * s), scale * (b * c + a * s)
    e = abs(scale) * (np.abs(a) + np.abs(b)) * 10 * U
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2] = y
        err[..., 0:rot:2] = err[..., 1:rot:2] = e
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = y
        err[..., :rot // 2] = err[..., rot // 2:rot] = e
    return out, err
