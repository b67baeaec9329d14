"""Plain 64-bit forms of the operators around the cache: norm and rotation of
heads, the cache's row formats, and attention over a segment's rows.

Test infrastructure (numpy, float64), sharing nothing with the library: the
rotation multiplies complex numbers by phases reduced in integer-exact steps,
attention loops over tokens and rows' masks literally.
"""
from __future__ import annotations

import math

import numpy as np


# ----------------------------------------------------------------------------- rotation

def frequencies(head_dim, theta, nonrot_dim=0, scaling="none", factor=1.0, orig_ctx=0, low=0.0, high=0.0):
    """(w [rot/2], factor on the rotated dims) of a scaled rotation, one pair at a time."""
    rot = head_dim - nonrot_dim
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    out = []
    for f in range(rot // 2):
        w = theta ** (-2.0 * f / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "yarn":
            fast, slow = high or 32.0, low or 1.0

            def index(turns):
                return rot * math.log(orig_ctx / (turns * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
            r = min(max((f - a) / max(b - a, 0.001), 0.0), 1.0)
            w = r * (w / factor) + (1 - r) * w
        elif scaling == "bands":
            many, few = high or 4.0, low or 1.0
            turns = orig_ctx / (2 * math.pi / w)
            if turns < few:
                w = w / factor
            elif turns <= many:
                s = (turns - few) / (many - few)
                w = (1 - s) * w / factor + s * w
        out.append(w)
    m = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    return np.asarray(out), m


def turn(x, pos, omega, mscale=1.0, nonrot_dim=0, layout="half", norm=None, eps=1e-6):
    """Heads x [tokens][heads][hd] (any float type) normed and rotated at pos, float64."""
    x = np.asarray(x, np.float64)
    hd = x.shape[-1]
    rot = hd - nonrot_dim
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(norm, np.float64)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(omega)[None, None]
    z = mscale * np.exp(1j * ang)
    if layout == "half":
        c = (x[..., :rot // 2] + 1j * x[..., rot // 2:rot]) * z
    else:
        c = (x[..., 0:rot:2] + 1j * x[..., 1:rot:2]) * z
    y = x.copy()
    if layout == "interleaved":
        y[..., 0:rot:2], y[..., 1:rot:2] = c.real, c.imag
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = c.real, c.imag
    return y


# ----------------------------------------------------------------------------- row formats

def quantize_q4_0(x):
    """float32 rows [..., hd] as planar q4_0 (bytes [..., hd/2], fp16 scales [..., hd/32]), in the float32 steps that
    define it: d = m / -8 (m the first value of largest modulus), code = min(15, floor(x / d + 8.5))."""
    x = np.ascontiguousarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    at = np.abs(b).argmax(-1)[..., None]
    d = (np.take_along_axis(b, at, -1) * np.float32(-0.125)).astype(np.float32)
    safe = np.where(d == 0, np.float32(1), d)
    code = np.clip(np.floor((b / safe).astype(np.float32) + np.float32(8.5)), 0, 15)
    code = np.where(d == 0, 8, code).astype(np.uint8)
    data = code[..., :16] | (code[..., 16:] << 4)
    return data.reshape(*x.shape[:-1], x.shape[-1] // 2), (d[..., 0] + np.float32(0)).astype(np.float16)


def quantize_q8_0(x):
    """float32 rows [..., hd] as planar q8_0: d = amax / 127, code = x / d rounded half away from zero."""
    x = np.ascontiguousarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    d = (np.abs(b).max(-1, keepdims=True) / np.float32(127)).astype(np.float32)
    y = (b / np.where(d == 0, np.float32(1), d)).astype(np.float64)
    code = np.clip(np.sign(y) * np.floor(np.abs(y) + 0.5), -127, 127)
    return code.astype(np.int8).reshape(x.shape), d[..., 0].astype(np.float16)


def codes_q4_0(data):
    """q4_0 bytes [..., hd/2] as codes [..., hd] in 0 .. 15."""
    b = data.reshape(*data.shape[:-1], data.shape[-1] // 16, 16)
    return np.concatenate([b & 15, b >> 4], -1).reshape(*data.shape[:-1], data.shape[-1] * 2)


def values(data, scale, kind):
    """float64 values of a plane's rows."""
    if kind in ("f32", "f16"):
        return data.astype(np.float64)
    codes = codes_q4_0(data).astype(np.float64) - 8 if kind == "q4_0" else data.astype(np.float64)
    return codes * np.repeat(scale.astype(np.float64), 32, -1)


def hold(x, kind):
    """float32 rows in a plane's format: (data, scales or None)."""
    if kind == "f32":
        return np.ascontiguousarray(x, np.float32), None
    if kind == "f16":
        return np.ascontiguousarray(x).astype(np.float16), None
    return quantize_q8_0(x) if kind == "q8_0" else quantize_q4_0(x)


# ----------------------------------------------------------------------------- attention

def attend_rows(q, p, k, v, pos, window=0, sink=0, scale=None):
    """One token's heads q [G][hd] at position p over a segment's live rows k, v [n][hd] at pos [n]:
    (out [G][hd], lse [G], weights [G][n], logit magnitudes [G][n])."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    see = [r for r in range(len(pos)) if pos[r] <= p and (window == 0 or p - pos[r] < window or r < sink)]
    out, lse = np.zeros(q.shape), np.full(len(q), -np.inf)
    w, mag = np.zeros((len(q), len(pos))), np.zeros((len(q), len(pos)))
    if not see:
        return out, lse, w, mag
    logit = scale * (q @ k[see].T)
    top = logit.max(-1, keepdims=True)
    e = np.exp(logit - top)
    total = e.sum(-1, keepdims=True)
    w[:, see] = e / total
    mag[:, see] = scale * (np.abs(q) @ np.abs(k[see]).T)
    return (e / total) @ v[see], (top + np.log(total))[:, 0], w, mag
