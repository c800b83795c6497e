"""MXFP4 in plain numpy, in 64 bits, written from the format's definition: the
quantisation rule by search over the eight magnitudes, the decoder by table."""
import numpy as np

FP4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes, scale bytes) of a float64 matrix, blocks along rows: codes
    rows x 32 ceil(cols / 32) (padding 0), bytes rows x ceil(cols / 32)."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    v = np.zeros((rows, blocks * 32))
    v[:, :cols] = x
    v = v.reshape(rows, blocks, 32)
    codes = np.zeros(v.shape, np.uint8)
    byte = np.zeros((rows, blocks), np.uint8)
    for r in range(rows):
        for b in range(blocks):
            block = v[r, b]
            if not np.all(np.isfinite(block)):
                byte[r, b] = 255
                continue
            m = np.abs(block).max()
            # frexp: m = f 2^p, 0.5 <= f < 1
            e = max(int(np.frexp(m)[1]) - 1 - 2, -127) if m > 0 else -127
            byte[r, b] = e + 127
            a = np.abs(block) / 2.0 ** e
            for i, y in enumerate(a):
                d = np.abs(FP4 - y)
                near = np.flatnonzero(d == d.min())
                code = next((c for c in near if c % 2 == 0), near[0])
                codes[r, b, i] = code | (8 if np.signbit(block[i]) else 0)
    return codes.reshape(rows, -1), byte


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(data):
    rows = data.shape[0]
    return np.stack((data & 15, data >> 4), 2).reshape(rows, -1)


def decode(data, scales, cols):
    """float64 values of packed elements and scale bytes (NaN for byte 255)."""
    codes = unpack(data)[:, :cols]
    v = FP4[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    b = np.repeat(scales.astype(np.float64), 32, axis=1)[:, :cols]
    return v * np.where(b == 255, np.nan, 2.0 ** (b - 127))
