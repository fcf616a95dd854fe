"""Helpers for the tests of the paged cache's operators: ragged batches over shuffled pages, and each
operator from its definition in 64 bits."""
import math

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8_e4m3": torch.float8_e4m3fn,
         "fp8_e5m2": torch.float8_e5m2, "int8": torch.int8}
MOST = {"fp8_e4m3": 448.0, "fp8_e5m2": 57344.0}
# half the smallest step of each type (its subnormals)
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150, "fp8_e4m3": 2.0 ** -10, "fp8_e5m2": 2.0 ** -17}


def half_step(dtype):
    """Largest error of one rounding, relative to the value."""
    return torch.finfo(TORCH[dtype]).eps / 2


def stored(x, dtype):
    """float64 numpy values as a tensor of `dtype` (CPU), saturated where the type is 8 bits wide."""
    t = torch.from_numpy(np.ascontiguousarray(x))
    if dtype == "int8":
        return t.round().clamp(-128, 127).to(torch.int8)
    if dtype in MOST:
        t = t.clamp(-MOST[dtype], MOST[dtype])
    return t.to(torch.float32).to(TORCH[dtype])


def f64(t):
    return t.detach().cpu().to(torch.float32 if t.dtype != torch.float64 else torch.float64).to(torch.float64).numpy()


class Batch:
    """q_lens / kv_lens of `num_seqs` sequences over shuffled pages, with room for more sequences, tokens before the
    first sequence (`lead`) and behind the last (`tail`)."""

    def __init__(self, rng, q_lens, kv_lens, ps, Hq, Hkv, D, kv="bf16", q="bf16", latent=False, lead=0, tail=0, spare_seqs=1,
                 spare_pages=2, k_scale=None, v_scale=None, **more):
        self.rng, self.q_lens, self.kv_lens_list, self.ps, self.Hq, self.Hkv, self.D = rng, list(q_lens), list(kv_lens), ps, Hq, Hkv, D
        self.kv, self.q, self.latent, self.S = kv, q, latent, len(q_lens)
        self.k_scale, self.v_scale, self.more = k_scale, v_scale, more
        pages = [-(-n // ps) for n in kv_lens]
        self.P = max([1] + pages) + 1
        self.N = sum(pages) + spare_pages + 1
        self.max_seqs = self.S + spare_seqs
        perm = rng.permutation(self.N)
        self.table = rng.integers(0, self.N, (self.max_seqs, self.P)).astype(np.int32)
        at = 0
        for s, n in enumerate(pages):
            self.table[s, :n] = perm[at:at + n]
            at += n
        self.free_pages = perm[at:].astype(np.int32)
        self.cu = np.full(self.max_seqs + 1, lead + sum(q_lens), np.int32)
        self.cu[:self.S + 1] = lead + np.concatenate(([0], np.cumsum(q_lens)))
        self.T = lead + sum(q_lens) + tail
        self.kv_lens = np.zeros(self.max_seqs, np.int32)
        self.kv_lens[:self.S] = kv_lens
        self.rows = Hkv if latent else 2 * Hkv

    def cfg(self):
        c = dict(num_q_tokens=self.T, num_q_heads=self.Hq, num_kv_heads=self.Hkv, head_dim=self.D, total_num_pages=self.N,
                 page_size=self.ps, max_num_seqs=self.max_seqs, pages_per_seq=self.P, kv_dtype=self.kv, q_dtype=self.q,
                 sm_scale=1 / math.sqrt(self.D), k_scale=self.k_scale, v_scale=self.v_scale)
        if self.latent:
            c.update(kv_layout="latent", v_head_dim=512)
        return dict(c, **self.more)

    def lens(self, dev="cuda:0"):
        return [torch.from_numpy(x.copy()).to(dev) for x in (self.kv_lens, self.table, self.cu)]

    def cache(self, dev="cuda:0"):
        x = self.rng.standard_normal((self.N, self.ps, self.rows, self.D))
        scale = self.k_scale or 1.0
        return stored(x / scale, self.kv).to(dev)

    def queries(self, dev="cuda:0"):
        return stored(self.rng.standard_normal((self.T, self.Hq, self.D)), self.q).to(dev)

    def slots(self, s, j):
        """Physical (page, place) of keys j of sequence s."""
        j = np.asarray(j)
        return self.table[s, j // self.ps], j % self.ps


def frequencies(rd, base=10000.0, scaling="none", factor=1.0, trained_len=0, low=1.0, high=4.0):
    w = [base ** (-2 * i / rd) for i in range(rd // 2)]
    if scaling == "linear":
        return [x / factor for x in w]
    if scaling == "base":
        return [(base * factor ** (rd / (rd - 2))) ** (-2 * i / rd) for i in range(rd // 2)]
    out = []
    for i, x in enumerate(w):
        if scaling == "rotations":
            t = min(max((trained_len * x / (2 * math.pi) - low) / (high - low), 0), 1)
        elif scaling == "index":
            a, b = (rd * math.log(trained_len / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (high, low))
            a, b = max(math.floor(a), 0), min(math.ceil(b), rd - 1)
            t = 1 - min(max((i - a) / max(b - a, 1e-3), 0), 1)
        else:
            t = 1
        out.append(t * x + (1 - t) * x / factor)
    return out


def rotate(x, pos, rope):
    """x [tokens, heads, D] float64 rotated at pos [tokens]; also the size |a| + |b| of each element's pair."""
    rd, off = rope["rotary_dim"], rope.get("rotary_offset", 0)
    w = np.array(frequencies(rd, **{k: v for k, v in rope.items() if k in ("base", "scaling", "factor", "trained_len", "low", "high")}))
    ang = pos.astype(np.float64)[:, None, None] * w
    c, s, m = np.cos(ang), np.sin(ang), rope.get("magnitude", 1.0)
    y, size = x.copy(), np.zeros_like(x)
    ia, ib = (np.arange(off, off + rd // 2), np.arange(off + rd // 2, off + rd)) if rope.get("pairing", "half") == "half" else \
             (np.arange(off, off + rd, 2), np.arange(off + 1, off + rd, 2))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = m * (a * c - b * s), m * (b * c + a * s)
    size[..., ia] = size[..., ib] = abs(m) * (np.abs(a) + np.abs(b))
    return y, size
