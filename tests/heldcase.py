"""Plain 64-bit implementations of the head norms and of what caches of 16 and 8 bits hold, on the
CPU, and the inputs of their tests (test infrastructure; shares no code with the library)."""

import numpy as np
import torch

import cachecase as R

F64 = torch.float64
U = R.U_FP32
KINDS = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}
MOST = {"fp8": 448.0, "int8": 127.0}


# ---------------------------------------------------------------------------------- norms

def normed(x, w, eps):
    """w r x in 64 bits and how far fp32 may put it off: sums of hd squares in any order, a
    division, a root, two products."""
    x = x.detach().cpu().to(F64)
    if w is None:
        return x, torch.zeros_like(x)
    r = (x.square().mean(-1, keepdim=True) + float(np.float32(eps))) ** -0.5
    y = w.detach().cpu().to(F64) * r * x
    return y, y.abs() * (x.shape[-1] / 2 + 8) * U


def norm_rope(x, w, eps, pos, rot, layout, **kw):
    """The forward call on one tensor and its tolerance before the last rounding; rot 0: no
    rotation."""
    y, off = normed(x, w, eps)
    if not rot:
        return y, off
    out, size = R.rotate(y, pos, rot, layout, **kw)
    # the rotation takes the errors of both features of a pair; cos and sin are within 2^-20
    return out, size * 2.0 ** -20 + R.rotate(off, pos, rot, layout, **kw)[1] + off


def norm_rope_grad(x, w, eps, gy, pos, rot, layout, **kw):
    """Gradients of x and w (None without one), and how far fp32 may put them off."""
    gy = gy.detach().cpu().to(F64)
    g, eg = gy, torch.zeros_like(gy)
    if rot:
        g, size = R.rotate(gy, pos, rot, layout, True, **kw)
        eg = size * 2.0 ** -20
    if w is None:
        return g, None, eg, None
    x, w = x.detach().cpu().to(F64), w.detach().cpu().to(F64)
    hd = x.shape[-1]
    r = (x.square().mean(-1, keepdim=True) + float(np.float32(eps))) ** -0.5
    xh, wg = x * r, w * g
    dx = r * (wg - xh * (wg * xh).mean(-1, keepdim=True))
    dw = (g * xh).sum((0, 1))
    size = wg.abs() + xh.abs() * (wg * xh).abs().mean(-1, keepdim=True)
    dx_off = r * (w.abs() * eg + xh.abs() * (w.abs() * eg * xh.abs()).mean(-1, keepdim=True)) + r * size * (2 * hd + 32) * U
    dw_off = (eg * xh.abs()).sum((0, 1)) + (g * xh).abs().sum((0, 1)) * (hd / 2 + 8 + x.shape[0] * x.shape[1] + 64) * U
    return dx, dw, dx_off, dw_off


# ---------------------------------------------------------------------------------- caches

def exponents(top, kind):
    """The smallest exponents with top <= M 2^e, kept to the range (64-bit, any shape)."""
    mant, e = np.frexp(np.asarray(top, dtype=np.float64))
    lead, bits = np.frexp(MOST[kind])
    return np.clip(np.where(mant == 0, -1000, e - bits + (mant > lead)), -110, 118)


def held(x, kind):
    """The values that a cache holds of x, the scale bytes, and whether a block is NaN."""
    x = x.detach().cpu().to(F64)
    if kind == "bf16":
        return x.to(torch.bfloat16).to(F64), None
    b = x.unflatten(-1, (-1, 32)).numpy()
    bad = ~np.isfinite(b).all(-1)
    e = exponents(np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1)), kind)
    y = np.where(np.isfinite(b), b, 0.0) * 2.0 ** -e.astype(np.float64)[..., None]
    y = np.clip(y, -MOST[kind], MOST[kind])
    if kind == "int8":
        y = np.rint(y)
    else:
        _, p = np.frexp(y)
        step = 2.0 ** (np.maximum(np.where(y == 0, -100, p - 1), -6) - 3)
        y = np.rint(y / step) * step
    y = y * 2.0 ** e.astype(np.float64)[..., None]
    y[bad] = np.nan
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return torch.from_numpy(y).flatten(-2), torch.from_numpy(scale)


def values(codes, scales):
    """What codes of a pool (or rows of it) stand for, in 64 bits."""
    if scales is None:
        return codes.cpu().to(F64)
    c = codes.cpu().to(torch.float32).to(F64)
    s = scales.cpu().numpy().astype(np.int64)
    f = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    return (c.unflatten(-1, (-1, 32)) * torch.from_numpy(f)[..., None]).flatten(-2)


def pools(num_pages, page, n_kv, hd, kind, dev="cuda", fill=0):
    """Empty pools of one layer and their scales, every byte `fill`."""
    def make(*shape):
        return torch.full(shape, fill, dtype=torch.uint8).to(dev)
    if kind == "bf16":
        k, v = (make(num_pages, page, n_kv, 2 * hd).view(torch.bfloat16) for _ in range(2))
        return k, v, None, None
    k, v = (make(num_pages, page, n_kv, hd).view(KINDS[kind]) for _ in range(2))
    return k, v, make(num_pages, page, n_kv, hd // 32), make(num_pages, page, n_kv, hd // 32)


def hold(pool, kind):
    """A bf16 pool's rows as codes and scales (and the bf16 pool of the values they stand for)."""
    val, scale = held(pool, kind)
    if kind == "bf16":
        return pool, None, pool
    e = scale.to(torch.int64) - 127
    f = torch.where(scale == 255, 1.0, 2.0 ** e.to(F64))[..., None]
    code = torch.nan_to_num(val.unflatten(-1, (-1, 32)) / f).flatten(-2)
    dev = pool.device
    return code.to(torch.float32).to(KINDS[kind]).to(dev), scale.to(dev), val.to(torch.bfloat16).to(dev)
