"""Codes, scales and zeros of the 4-bit append where 32 bits of a value do not decide them: behind a division by the cache's scale,
and far from zero for the group's range.  Positions are 0, so that a key's exact value is k times the magnitude."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as i4  # noqa: E402
import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch, f64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def append(b, k, v, group, **rope):
    cache = torch.full((b.N, b.Hkv, i4.block_bytes(b.ps, b.D, group)), 0x5a, dtype=torch.uint8, device="cuda")
    op = rpa.RopeAppend(**b.cfg(), **rope)
    op.append(torch.zeros((b.T, b.Hq, b.D), dtype=k.dtype, device="cuda"), k, v, cache, *b.lens(), b.S,
              positions=torch.zeros(b.T, dtype=torch.int32, device="cuda"))
    assert op.status() == rpa.RPA_OK
    page, at = b.slots(0, np.arange(b.kv_lens_list[0]))
    return [tuple(x[page, at] for x in p) for p in i4.unpack(cache.cpu().numpy(), b.ps, b.D, group)]


def same(got, want):
    for a, w, name in zip(got, want, ("codes", "scales", "zeros")):
        assert np.array_equal(a, w), (name, int((a != w).sum()), a.size)


def close(got, y, group):
    """A quotient as a pair of floats, q + (r + l) / s: |r| and |l| (what the quotient's and the product's rounding left) are at most
    2^-24 |q s| each; their sum, the reciprocal of s and the product are rounded (2^-24 each): off by 3 * 2^-24 * 2 * 2^-24 |q|, below
    2^-45 |q|.  A constant group far from zero shows it: 5 / fl(0.005) is 1000 + 375 * 2^-24 + 5e-13, whose scale is 26 * 2^-24, where
    the pair holds 1000 + 375 * 2^-24, whose scale is 25 * 2^-24.  So a group is coded as that of values off by as much or not at all."""
    ok = np.zeros(got[1].shape, bool)
    for d in (0.0, 2.0 ** -45, -2.0 ** -45):
        want = i4.coded(y * (1 + d), group)
        codes = (got[0] == want[0]).reshape(*got[1].shape, group).all(-1)
        ok |= codes & (got[1] == want[1]) & (got[2] == want[2])
    assert ok.all(), int((~ok).sum())


@pytest.mark.parametrize("D,group,q", [(128, 32, "f32"), (64, 64, "bf16"), (256, 128, "f16"), (128, 64, "f32")])
@pytest.mark.parametrize("offset,spread", [(0.0, 1.0), (1000.0, 0.1), (-30.0, 1e-3), (0.0, 3e4), (5.0, 2e-6)])
@pytest.mark.parametrize("k_scale,v_scale", [(None, None), (0.3, 1.7), (1.0, 1.0), (-0.7, 5e-3)])
def test_exact_codes(D, group, q, offset, spread, k_scale, v_scale):
    n = 1500
    b = Batch(np.random.default_rng([D, group, int(spread * 1e6)]), [n], [n], 16, 4, 4, D, kv="int4_g%d" % group, q=q, k_scale=k_scale,
              v_scale=v_scale)
    dtype = dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[q]
    k, v = (torch.from_numpy(offset + spread * b.rng.standard_normal((b.T, 4, D))).float().to(dtype).cuda() for _ in "kv")
    k, v = (x.clamp(-60000, 60000) for x in (k, v))
    # the magnitude is a float: products of it and of a value have up to 48 bits, which 64 and a pair of floats hold exactly
    magnitude = float(np.float32(1.3))
    got = append(b, k, v, group, magnitude=magnitude)
    for x, part, m, scale in ((k, got[0], magnitude, k_scale), (v, got[1], 1.0, v_scale)):
        y = f64(x)[:n] * m
        if scale is None:
            same(part, i4.coded(y, group))
        else:
            close(part, y / float(np.float32(scale)), group)


def test_values_at_the_ends_of_float16():
    """The product of a key and the magnitude next to 65504, beyond what 32 bits tell from it."""
    b = Batch(np.random.default_rng(1), [64], [64], 16, 1, 1, 64, kv="int4_g32", q="f32")
    m = np.float32(1.3)
    k = (np.float32(65504) / m) * (1 + b.rng.integers(-3, 4, (b.T, 1, 64)) * 2.0 ** -23)
    k[:, :, ::5] = b.rng.standard_normal(k[:, :, ::5].shape)
    k[b.T // 2:] *= -1
    x = torch.from_numpy(k).float().cuda()
    got = append(b, x, x, 32, magnitude=float(m))
    same(got[0], i4.coded(f64(x)[:64] * float(m), 32))
    same(got[1], i4.coded(f64(x)[:64], 32))
