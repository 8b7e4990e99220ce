"""Plain 64-bit forms of the cache operators (numpy, written from the record
definitions): the source transform, the quantization of each format and the
values of a record. Test infrastructure; shares nothing with the library."""
import numpy as np

from swa_paged_decode_gb300 import workloads as W

EPS_E4M3, EPS_BF16, EPS_F16, EPS_F32 = 2.0 ** -4, 2.0 ** -8, 2.0 ** -11, 2.0 ** -24   # half steps


def transform(x, norm_weight=None, eps=0.0, positions=None, cos_sin=None, style=W.ROPE_NEOX):
    x = np.asarray(x, np.float64).copy()
    if norm_weight is not None:
        v = x[:, :512]
        x[:, :512] = v * np.asarray(norm_weight, np.float64) / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    if positions is not None:
        t = np.asarray(cos_sin, np.float64)[np.asarray(positions)]
        c, s = t[:, :32], t[:, 32:]
        r = x[:, -64:].copy()
        ia = np.arange(32) if style == W.ROPE_NEOX else 2 * np.arange(32)
        ib = ia + (32 if style == W.ROPE_NEOX else 1)
        out = np.empty_like(r)
        out[:, ia] = r[:, ia] * c - r[:, ib] * s
        out[:, ib] = r[:, ib] * c + r[:, ia] * s
        x[:, -64:] = out
    return x


def e4m3_values():
    c = np.arange(256)
    m, e = c & 7, (c >> 3) & 15
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


E4M3 = e4m3_values()
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])


def bf16_values(b):
    u = b.reshape(b.shape[0], -1, 2).astype(np.uint32)
    return ((u[..., 0] | (u[..., 1] << 8)) << 16).view(np.float32).astype(np.float64)


def record_values(fmt, rec):
    """[n, record] uint8 -> [n, dims] float64."""
    n = rec.shape[0]
    if fmt == W.FMT_NVFP4_288:
        nib = np.stack([rec[:, :256] & 15, rec[:, :256] >> 4], -1).reshape(n, 512)
        return E2M1[nib] * np.repeat(E4M3[rec[:, 256:]], 16, axis=1)

    def pow2(b, rep):
        v = np.exp2(b.astype(np.float64) - 127)
        v[b == 255] = np.nan
        return np.repeat(v, rep, axis=1)

    if fmt == W.FMT_MODEL1_584:
        return np.concatenate([E4M3[rec[:, :448]] * pow2(rec[:, 576:583], 64), bf16_values(rec[:, 448:576])], 1)
    if fmt == W.FMT_FP8_528_UE8M0:
        return E4M3[rec[:, :512]] * pow2(rec[:, 512:528], 32)
    with np.errstate(invalid="ignore"):
        v = E4M3[rec[:, :512]] * np.repeat(np.ascontiguousarray(rec[:, 512:528]).view(np.float32).astype(np.float64), 128, axis=1)
    return np.concatenate([v, bf16_values(rec[:, 528:])], 1) if fmt == W.FMT_V32_656 else v


def block_dims(fmt):
    return {W.FMT_FP8_528: 128, W.FMT_V32_656: 128, W.FMT_FP8_528_UE8M0: 32, W.FMT_MODEL1_584: 64,
            W.FMT_NVFP4_288: 16}[fmt]


def quant_bound(fmt, x):
    """Largest |value read back - x| the format allows, per element, for
    finite rows x [n, dims] (64 bits), from the format's definition.

    e4m3 codes: scale s, |x| / s <= 448 up to the scale's own rounding, the
    code off by half a step: |x| 2^-4, or s 2^-10 below the smallest normal.
    The power-of-two scales are at most 2 amax / 448; an fp32 scale is amax /
    448 within 2^-24 (so saturation costs at most that). NVFP4: the e4m3
    scale is amax / 6 off by 2^-4 of it (2^-10 absolute below 2^-6), half an
    e2m1 step is at most s (between 4 and 6) or |y| 2^-2 below, s/4 at least;
    a scale rounded down saturates: amax - 6 s. bf16 parts: 2^-8."""
    n, d = x.shape
    b = np.empty_like(x)
    codes = 448 if fmt == W.FMT_MODEL1_584 else 512
    size = block_dims(fmt)
    blk = np.abs(x[:, :codes]).reshape(n, -1, size)
    amax = blk.max(-1, keepdims=True)
    if fmt == W.FMT_NVFP4_288:
        s_hi = np.minimum(amax / 6 * (1 + EPS_E4M3) + 2.0 ** -10, 448.0)
        s_lo = np.minimum(np.maximum(amax / 6 * (1 - EPS_E4M3) - 2.0 ** -10, 0), 448.0)
        e = np.maximum(s_hi * np.where(blk > 3.9 * s_lo, 1.0, np.where(blk > 1.9 * s_lo, 0.5, 0.25)),
                       np.maximum(amax - 6 * s_lo, 0) * (blk > 5 * s_lo))
        # a scale that rounds to zero leaves zeros
        e = np.maximum(e, np.where(amax / 6 <= 2.0 ** -10, blk, 0))
    else:
        s = amax / 448 * (1 if size == 128 else 2)
        e = np.maximum(blk * EPS_E4M3, s * 2.0 ** -10) + amax * 2 * EPS_F32
    b[:, :codes] = e.reshape(n, codes)
    b[:, codes:] = np.abs(x[:, codes:]) * EPS_BF16 + 2.0 ** -133
    return b * (1 + 2.0 ** -20)
