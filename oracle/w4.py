"""4-bit weights with group scales in float64 numpy: quantisation, packing, values.  Test infrastructure only.

"int4": value (c - 8) s, one scale per group of 32, 64 or 128 (stored bf16, plane by plane [K / group, rows]);
"fp4": E2M1 value times 2^(e - 127), one byte e per 32 (stored [ceil(K / 128), rows, 4])."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16(x):
    """The nearest bf16 values, ties to even (fp32 in between is exact for fp32 inputs)."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32) << np.uint32(16)
    return r.astype(np.uint32).view(np.float32).astype(np.float64)


def quantize(X, fmt, group):
    """Codes [rows, K] and scales [rows, K / group] (values for int4, bytes for fp4)."""
    X = np.asarray(X, np.float64)
    rows, K = X.shape
    g = X.reshape(rows, K // group, group)
    top = np.abs(g).max(axis=2)
    if fmt == "int4":
        s = bf16((top.astype(np.float32) / np.float32(7.0)))
        s = np.where(s == 0, 1.0, s)
        c = np.clip(np.rint(g / s[:, :, None]), -7, 7) + 8
        return c.reshape(rows, K).astype(np.uint8), s
    m, ex = np.frexp(top)
    k = np.where(top == 0, 0, np.clip(ex - 3 + (m > 0.75), -127, 127)).astype(np.int64)
    a = np.abs(g) / np.power(2.0, k)[:, :, None]
    d = np.abs(a[..., None] - E2M1)
    best = d.min(axis=-1, keepdims=True)
    near = d == best                       # two codes at a tie: the even one
    even = near & (np.arange(8) % 2 == 0)
    c = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    return (c + 8 * (g < 0)).reshape(rows, K).astype(np.uint8), (k + 127).astype(np.uint8)


def values(codes, scales, fmt):
    """Weights [rows, K] of codes [rows, K] and scales [rows, groups]."""
    c = np.asarray(codes, np.int64)
    rows, K = c.shape
    s = np.asarray(scales, np.float64) if fmt == "int4" else np.power(2.0, np.asarray(scales, np.float64) - 127.0)
    v = c - 8.0 if fmt == "int4" else np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    return v * np.repeat(s, K // s.shape[1], axis=1)


def pack(codes):
    c = np.asarray(codes, np.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def unpack(packed):
    p = np.asarray(packed, np.uint8)
    return np.stack([p & 15, p >> 4], axis=-1).reshape(p.shape[0], -1)


def store_scales(scales, fmt):
    """The layout in memory: int4 [groups, rows] (values), fp4 [ceil(groups / 4), rows, 4] (bytes, 127 as filling)."""
    s = np.asarray(scales)
    if fmt == "int4":
        return np.ascontiguousarray(s.T)
    rows, groups = s.shape
    out = np.full((rows, -(-groups // 4) * 4), 127, np.uint8)
    out[:, :groups] = s
    return np.ascontiguousarray(out.reshape(rows, -1, 4).transpose(1, 0, 2))
