"""Plain 64-bit restatement of the 8-bit operators, for their tests: e4m3
codes with power-of-two scales, rotary positions, masked attention and the
block-scaled product (numpy, no code shared with the library)."""
import math

import numpy as np

NAN_BYTE = 255


def e4m3_values():
    """The 256 code values; 0x7f and 0xff are NaN."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if c & 0x7f == 0x7f else (-x if c & 0x80 else x)
    return v


CODE_VALUES = e4m3_values()


def encode(y):
    """Round |y| <= 448 to the nearest code, ties to even."""
    a = np.abs(y)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6) - 3)
    q = np.rint(a / step) * step          # rint: ties to even, as the code's last bit is the step
    mag = np.arange(0x7f)
    lut = dict(zip(CODE_VALUES[mag].tolist(), mag.tolist()))
    code = np.array([lut[v] for v in q.ravel().tolist()], dtype=np.uint8).reshape(q.shape)
    return code | (np.signbit(y).astype(np.uint8) << 7)


def scale_byte(amax):
    if not math.isfinite(amax):
        return NAN_BYTE
    if amax == 0:
        return 127
    f, k = math.frexp(amax)                # amax = f * 2^k, f in [1/2, 1)
    return max(0, (k - 9 if f <= 0.875 else k - 8) + 127)


def quantise(x):
    """Blocks along the last axis: (codes, bytes)."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    codes = np.zeros(flat.shape, dtype=np.uint8)
    bytes_ = np.zeros(flat.shape[0], dtype=np.uint8)
    for i, row in enumerate(flat):
        b = scale_byte(np.abs(row).max() if np.isfinite(row).all() else math.nan)
        bytes_[i] = b
        if b != NAN_BYTE:
            codes[i] = encode(row * 2.0 ** (127 - b))
    return codes.reshape(x.shape), bytes_.reshape(x.shape[:-1])


def dequantise(codes, bytes_):
    s = np.where(bytes_ == NAN_BYTE, np.nan, 2.0 ** (bytes_.astype(np.float64) - 127))
    return CODE_VALUES[codes] * s[..., None]


def quantise_blocks(x):
    """[rows][K] -> codes [rows][K], bytes [ceil(K/128)][rows]."""
    rows, K = x.shape
    kb = -(-K // 128)
    codes = np.zeros((rows, K), dtype=np.uint8)
    bytes_ = np.zeros((kb, rows), dtype=np.uint8)
    for B in range(kb):
        codes[:, B * 128:(B + 1) * 128], bytes_[B] = quantise(x[:, B * 128:(B + 1) * 128])
    return codes, bytes_


def dequantise_blocks(codes, bytes_):
    out = np.zeros(codes.shape)
    for B in range(bytes_.shape[0]):
        out[:, B * 128:(B + 1) * 128] = dequantise(codes[:, B * 128:(B + 1) * 128], bytes_[B])
    return out


def rope_rates(rot, theta, scaling, factor, orig_len=4096.0, beta_fast=32.0, beta_slow=1.0):
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    rates, amp = [], 1.0
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        if scaling == "linear":
            f = f / factor
        if scaling == "by_parts":
            amp = 1 + 0.1 * math.log(factor)
            lo = rot * math.log(orig_len / (2 * math.pi * beta_fast)) / (2 * math.log(theta))
            hi = rot * math.log(orig_len / (2 * math.pi * beta_slow)) / (2 * math.log(theta))
            lo, hi = max(0, math.floor(lo)), min(rot // 2 - 1, math.ceil(hi))
            r = min(1, max(0, (i - lo) / max(hi - lo, 0.001)))
            f = r * f / factor + (1 - r) * f
        rates.append(f)
    return np.array(rates), amp


def rope(x, pos, rot, layout, rates, amp):
    """x [rows][heads][hd] float64."""
    out = x.copy()
    h = rot // 2
    i0 = np.arange(h) if layout == "half" else 2 * np.arange(h)
    i1 = i0 + h if layout == "half" else i0 + 1
    a = pos.astype(np.float64)[:, None] * rates
    c, s = (amp * np.cos(a))[:, None], (amp * np.sin(a))[:, None]
    out[..., i0] = x[..., i0] * c - x[..., i1] * s
    out[..., i1] = x[..., i1] * c + x[..., i0] * s
    return out


def attention(q, k, v, limits, scale):
    """q [R][H][hd], k/v [H_kv][T][hd], limits [R] -> (out, sum of p|v|, largest
    sum of |q||k| a row and head), the latter two for tolerances."""
    R, H, hd = q.shape
    g = H // k.shape[0]
    out, pv, sk = np.zeros((R, H, hd)), np.zeros((R, H, hd)), np.zeros((R, H, 1))
    for i in range(R):
        n = min(max(int(limits[i]), 0), k.shape[1])
        if n == 0:
            continue
        for h in range(H):
            kk, vv = k[h // g, :n], v[h // g, :n]
            z = scale * (kk @ q[i, h])
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h], pv[i, h] = p @ vv, p @ np.abs(vv)
            sk[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, pv, sk
