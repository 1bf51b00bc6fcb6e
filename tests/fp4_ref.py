"""MXFP4 in 64 bits, from its definition: the reference of the 4-bit tests."""
import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(v):
    """v [R, C] float64 (values of f32, bf16 or f16) -> (codes [R, C], scale bytes [R, ceil(C/32)])."""
    r, c = v.shape
    nb = -(-c // 32)
    x = np.zeros((r, nb * 32))
    x[:, :c] = v
    x = x.reshape(r, nb, 32)
    bad = ~np.isfinite(x).all(-1)
    a = np.where(bad[..., None], 0.0, np.abs(x))
    top = a.max(-1)
    with np.errstate(divide="ignore"):
        s = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))) - 2, -127)
    # log2 may round up just below a power of two: the definition is 2^floor <= top
    s = np.where(np.ldexp(1.0, (s + 2).astype(int)) > top, s - 1, s)
    s = np.maximum(s, -127)
    q = a / np.ldexp(1.0, s.astype(int))[..., None]
    # nearest of VALUES, ties to the even code
    dist = np.abs(q[..., None] - VALUES)
    best = dist.min(-1, keepdims=True)
    cand = dist == best
    code = np.where(cand[..., ::2].any(-1), 2 * cand[..., ::2].argmax(-1), cand.argmax(-1))
    code = np.where(bad[..., None], 0, code | (np.signbit(x) << 3))
    return code.reshape(r, nb * 32)[:, :c].astype(np.uint8), np.where(bad, 255, s + 127).astype(np.uint8)


def values(codes, scales):
    """float64 values of codes [R, C] and scale bytes [R, ceil(C/32)]."""
    c = codes.shape[1]
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(s, 32, axis=1)[:, :c]


def rounded(v):
    """The values that v stands for in MXFP4."""
    return values(*quantize(v))


def unpack(q, s, rows, cols):
    """Codes and scale bytes out of the library's buffers (numpy u8), and whether all padding is zero."""
    cp = (cols + 255) // 256 * 256
    nb = -(-cols // 32)
    b = q.reshape(rows, cp // 2)
    codes = np.stack([b & 15, b >> 4], -1).reshape(rows, cp)
    rp = (rows + 127) // 128 * 128
    sc = np.zeros((rp, cp // 32), np.uint8)
    r, k = np.meshgrid(np.arange(rp), np.arange(cp // 32), indexing="ij")
    sc[r, k] = s.reshape(-1)[((r // 128) * (cp // 128) + k // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4]
    clean = not codes[:, cols:].any() and not sc[rows:].any() and not sc[:, nb:].any()
    return codes[:, :cols], sc[:rows, :nb], clean


def pack(codes, scales):
    """The library's buffers for codes [R, C] and scale bytes [R, ceil(C/32)]."""
    rows, cols = codes.shape
    cp = (cols + 255) // 256 * 256
    full = np.zeros((rows, cp), np.uint8)
    full[:, :cols] = codes
    s = np.zeros((rows + 127) // 128 * (cp // 128) * 512, np.uint8)
    r, k = np.meshgrid(np.arange(rows), np.arange(scales.shape[1]), indexing="ij")
    s[((r // 128) * (cp // 128) + k // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4] = scales
    return (full[:, ::2] | (full[:, 1::2] << 4)).reshape(-1), s
