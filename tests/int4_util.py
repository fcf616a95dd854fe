"""The 4-bit cache from its definition: blocks of bytes taken apart and put together (numpy), and the codes of a group."""
import numpy as np
import torch


def block_bytes(ps, D, group):
    return ps * (D + 8 * D // group)


def _order(ps, D):
    r, c = np.arange(ps)[:, None], np.arange(D // 32)[None]
    return c ^ (r * D // 256 % (D // 32))


def unpack(cache, ps, D, group):
    """uint8 [N, Hkv, bytes] -> for K and V: (codes [N, ps, Hkv, D] int, scale, zero [N, ps, Hkv, D / group] float64)."""
    cache = np.asarray(cache)
    N, H, _ = cache.shape
    half, m, order, got = ps * D // 2, ps * D // group * 4, _order(ps, D), []
    for i in (0, 1):
        c = cache[:, :, i * half:(i + 1) * half].reshape(N, H, ps, D // 32, 16)
        c = np.take_along_axis(c, np.broadcast_to(order[None, None, :, :, None], c.shape), 3).reshape(N, H, ps, D // 2)
        codes = np.stack((c & 15, c >> 4), -1).reshape(N, H, ps, D).astype(np.int64)
        meta = np.ascontiguousarray(cache[:, :, 2 * half + i * m:2 * half + (i + 1) * m]).view(np.float16).reshape(N, H, ps, D // group, 2)
        got.append(tuple(x.swapaxes(1, 2) for x in (codes, meta[..., 0].astype(np.float64), meta[..., 1].astype(np.float64))))
    return got


def pack(parts, ps, D, group):
    """The inverse of unpack: uint8 [N, Hkv, bytes]."""
    N, _, H, _ = parts[0][0].shape
    half, m, order = ps * D // 2, ps * D // group * 4, _order(ps, D)
    cache = np.zeros((N, H, block_bytes(ps, D, group)), np.uint8)
    for i, (codes, s, z) in enumerate(parts):
        c = codes.swapaxes(1, 2).astype(np.uint8)
        c = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(N, H, ps, D // 32, 16)
        lies = np.empty_like(c)
        np.put_along_axis(lies, np.broadcast_to(order[None, None, :, :, None], c.shape), c, 3)
        cache[:, :, i * half:(i + 1) * half] = lies.reshape(N, H, half)
        meta = np.ascontiguousarray(np.stack((s, z), -1).swapaxes(1, 2).astype(np.float16))
        cache[:, :, 2 * half + i * m:2 * half + (i + 1) * m] = meta.reshape(N, H, -1).view(np.uint8)
    return cache


def values(part, group):
    codes, s, z = part
    return codes * np.repeat(s, group, -1) + np.repeat(z, group, -1)


def toward(x, up):
    """float64 to the float16 grid (as float64), upwards or downwards."""
    h = x.astype(np.float16)
    with np.errstate(over="ignore"):
        other = np.nextafter(h, np.float16(np.inf if up else -np.inf))
    short = h.astype(np.float64) < x if up else h.astype(np.float64) > x
    return np.where(short, other, h).astype(np.float64)


def coded(x, group):
    """Codes, scale and zero of x [..., D] float64."""
    y = np.clip(x, -65504, 65504).reshape(*x.shape[:-1], -1, group)
    z = toward(y.min(-1), False)
    s = toward((y.max(-1) - z) / 15, True)
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.where(s[..., None] > 0, np.clip(np.round((y - z[..., None]) / s[..., None]), 0, 15), 0)
    return c.reshape(x.shape).astype(np.int64), s, z


def random_cache(rng, N, ps, H, D, group, spread=1.0):
    """A cache that holds the codes of N(0, spread^2) values, as a CUDA tensor and as its parts."""
    parts = [coded(spread * rng.standard_normal((N, ps, H, D)), group) for _ in "kv"]
    return torch.from_numpy(pack(parts, ps, D, group)).cuda(), parts
