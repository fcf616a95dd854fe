"""Values at the end of float16's range in a 4-bit cache.  A group's scale is rounded up, so its greatest code can stand for more
than the 65504 at which the append saturates (65520 over a zero of 0, 65536 over one of -65504): read and attended to as float16,
it is 65504 and no infinity."""
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


def saturated(b, group):
    """K and V rows of every key: groups from 0, from -65504, and between, up to 65504; infinities among them."""
    v = b.rng.uniform(-65504, 65504, (b.T, b.Hkv, b.D)).astype(np.float32)
    g = v.reshape(b.T, b.Hkv, -1, group)
    g[:, :, 0] = np.abs(g[:, :, 0])
    g[..., 0], g[..., 1] = 65504, np.inf
    g[:, :, 0, 2] = 0
    g[:, :, 1:, 3] = -65504
    return torch.from_numpy(v).half().cuda()


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 32)])
@pytest.mark.parametrize("q", ["f16", "bf16", "f32"])
def test_read(D, group, q):
    b = Batch(np.random.default_rng([1, D]), [40], [40], 16, 2, 2, D, kv="int4_g%d" % group, q="f16")
    v = saturated(b, group)
    cache = torch.zeros((b.N, 2, i4.block_bytes(16, D, group)), dtype=torch.uint8, device="cuda")
    lens, table, cu = b.lens()
    op = rpa.RopeAppend(**b.cfg(), rotary_dim=16)
    k = v.clamp(-65504, 65504)  # (not turned at position 0, but infinity times the sine is none)
    op.append(k, k, v, cache, lens, table, cu, 1, positions=torch.zeros(b.T, dtype=torch.int32, device="cuda"))
    assert op.status() == rpa.RPA_OK
    page, at = b.slots(0, np.arange(40))
    want = [i4.values(tuple(x[page, at] for x in p), group) for p in i4.unpack(cache.cpu().numpy(), 16, D, group)]
    assert max(w.max() for w in want) > 65519 and all(np.array_equal(want[0], w) for w in want)
    for scale in (None, 0.5, -1.0):
        got = rpa.RopeAppend(**dict(b.cfg(), q_dtype=q, k_scale=scale, v_scale=scale), rotary_dim=16).read(cache, lens, table, cu, 1)
        for x, w in zip(got, want):
            if q == "f16":
                w = np.minimum(w, 65504)  # as float16 has them
            assert torch.equal(x.cpu(), torch.from_numpy(w * (scale or 1.0)).float().to(x.dtype))


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("kv_lens", [[1, 1, 1], [20000, 3, 9000]])  # whole, and in pieces
@pytest.mark.parametrize("q", ["f16", "f32"])
def test_one_key_of_all_the_weight(D, group, kv_lens, q):
    """A decode whose last key draws all the weight gets that key's V, saturated as the read has it."""
    b = Batch(np.random.default_rng([2, D]), [1] * 3, kv_lens, 16, 2, 2, D, kv="int4_g%d" % group, q="f16")
    v = saturated(b, group)
    cache = torch.from_numpy(i4.pack([i4.coded(b.rng.standard_normal((b.N, 16, 2, D)), group) for _ in "kv"], 16, D, group)).cuda()
    lens, table, cu = b.lens()
    k = torch.full((b.T, 2, D), 40.0, dtype=torch.float16, device="cuda")  # logit of q = 40: 1600 sqrt(D), beside some +- 200 others
    op = rpa.RopeAppend(**b.cfg(), rotary_dim=16)
    op.append(k, k, v, cache, lens, table, cu, 3, positions=torch.zeros(b.T, dtype=torch.int32, device="cuda"))
    _, rows = op.read(cache, lens, table, cu, 3)
    assert op.status() == rpa.RPA_OK and torch.isfinite(rows[:3]).all()
    for scale in (None, 0.5, -1.0):
        att = rpa.RaggedPagedAttention(**dict(b.cfg(), q_dtype=q, v_scale=scale))
        out = att.forward(k.to(torch.float32 if q == "f32" else torch.float16), cache, lens, table, cu, 3)
        assert att.status() == rpa.RPA_OK
        # P = 1 times a scale is exact, its sums with codes and zeros are rounded in 32 bits (a few 2^-24 of 2^17), then o
        want = f64(rows[:3]) * (scale or 1.0)
        if q == "f32":
            page, at = (np.concatenate(x) for x in zip(*(b.slots(s, [n - 1]) for s, n in enumerate(kv_lens))))
            want = np.minimum(i4.values(tuple(x[page, at] for x in i4.unpack(cache.cpu().numpy(), 16, D, group)[1]), group), 65504) * (scale or 1.0)
        got = f64(out[:3])
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= (2.0 ** -10 if q == "f16" else 0) * np.abs(want) + 0.125).all()


@pytest.mark.parametrize("D,group,apart", [(64, 32, 256), (128, 64, 224), (256, 128, 160)])
def test_means_of_the_last_values(D, group, apart):
    """Channels that are 65504, or -65504, in every key: so is their mean, whatever P's rounding adds.  Two keys of a row draw its weight,
    the second up to 2^2 times the first, which holds the running maximum (`apart` keys on, where the same warp meets it): P is then
    up to 4 steps of 8736 and rounded by up to 8, and 8 times that over both weights can pass the 16 that are left to infinity."""
    S, H = 400, 8  # (as many that the two keys lie in one piece)
    b = Batch(np.random.default_rng([3, D]), [1] * S, [1000] * S, 16, H, 2, D, kv="int4_g%d" % group, q="f16")
    v = b.rng.uniform(-65504, 65504, (b.N, 16, 2, D))
    v[..., 0::4], v[..., 1::4] = 65504, -65504
    k = np.zeros((b.N, 16, 2, D))
    k[..., 0] = -1000
    for s in range(S):
        page, at = b.slots(s, [0, apart])
        k[page[0], at[0], :, 0], k[page[1], at[1], :, 0] = 0, 1
    parts = [i4.coded(x, group) for x in (k, v)]
    cache = torch.from_numpy(i4.pack(parts, 16, D, group)).cuda()
    q = torch.zeros(b.T, H, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = torch.from_numpy(b.rng.uniform(0.1, 1.38, (b.T, H)) * np.sqrt(D)).half().cuda()
    att = rpa.RaggedPagedAttention(**b.cfg())
    out = f64(att.forward(q, cache, *b.lens(), b.S))[:S]
    assert att.status() == rpa.RPA_OK and np.isfinite(out).all()
    # (P's rounding moves the mean by up to 8 * 8 / 2, o is rounded to a multiple of 32 there)
    assert (out[..., 0::4] >= 65504 - 64).all() and (out[..., 1::4] <= -65504 + 64).all()


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
def test_means_of_the_last_values_of_prompts(D, group):
    """The same in a prompt's f16 rows: P is rounded there by up to 2^-11 of it, the rows end at 65472, one step in front of 65504."""
    n = 600
    b = Batch(np.random.default_rng([4, D]), [n], [n], 64, 8, 2, D, kv="int4_g%d" % group, q="f16")
    v = b.rng.uniform(-65504, 65504, (b.N, 64, 2, D))
    v[..., 0::4], v[..., 1::4] = 65504, -65504
    parts = [i4.coded(x, group) for x in (b.rng.standard_normal((b.N, 64, 2, D)), v)]
    cache = torch.from_numpy(i4.pack(parts, 64, D, group)).cuda()
    att, q = rpa.RaggedPagedAttention(**b.cfg()), b.queries()
    for scale in (1, 4):  # some keys of the weight, and few
        out = f64(att.forward(q * scale, cache, *b.lens(), b.S))[:n]
        assert att.status() == rpa.RPA_OK and np.isfinite(out).all() and att.plan()[0][2] > 0
        # (a row of 65472, P's 2^-11 of it, and o's rounding)
        assert (out[..., 0::4] >= 65504 - 96).all() and (out[..., 1::4] <= -65504 + 96).all()
