"""Writing the 4-bit cache (rope append) and reading rows of every cache as values, against their definitions in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as i4  # noqa: E402
import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import TINY, Batch, f64, half_step, rotate, stored  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def new_rows(b, spread=1.0):
    """q, k, v as slices of one projection's output."""
    qkv = stored(spread * b.rng.standard_normal((b.T, b.Hq + 2 * b.Hkv, b.D)), b.q).cuda()
    return qkv[:, :b.Hq], qkv[:, b.Hq:b.Hq + b.Hkv], qkv[:, b.Hq + b.Hkv:]


def blank(b, group, fill=0x5a):
    return torch.full((b.N, b.Hkv, i4.block_bytes(b.ps, b.D, group)), fill, dtype=torch.uint8, device="cuda")


def slots_of(b):
    """token, page and place of every token of the batch's sequences, and its position."""
    t, page, at, pos = [], [], [], []
    for s, (a, n) in enumerate(zip(b.q_lens, b.kv_lens_list)):
        j = np.arange(n - a, n)
        p, x = b.slots(s, j)
        t.append(b.cu[s] + np.arange(a)), page.append(p), at.append(x), pos.append(j)
    return (np.concatenate(x) for x in (t, page, at, pos))


@pytest.mark.parametrize("D,group,ps,Hq,Hkv,q,rope", [
    (128, 128, 16, 8, 2, "bf16", {}),
    (128, 64, 20, 4, 4, "f16", dict(rotary_dim=64, rotary_offset=64, pairing="interleaved")),
    (64, 32, 64, 6, 3, "bf16", dict(rotary_dim=32, rotary_offset=8)),
    (256, 32, 4, 2, 1, "f32", dict(rotary_dim=48, rotary_offset=104)),
    (256, 128, 128, 16, 8, "bf16", dict(pairing="interleaved", scaling="linear", factor=4.0, magnitude=1.5)),
    (64, 64, 8, 1, 1, "f32", dict(rotary_dim=16)),
])
@pytest.mark.parametrize("scales", [{}, dict(k_scale=0.3, v_scale=2.5)])
def test_append(D, group, ps, Hq, Hkv, q, rope, scales):
    b = Batch(np.random.default_rng([D, group, ps]), [1, 1, 37, 0, 3, 90], [1, 300, 37, 20, 17, 200], ps, Hq, Hkv, D, kv="int4_g%d" % group, q=q,
              lead=2, tail=3, **scales)
    rope = dict(dict(rotary_dim=D), **rope)
    qs, k, v = new_rows(b)
    lens, table, cu = b.lens()
    op = rpa.RopeAppend(**b.cfg(), **rope)
    cache = blank(b, group)
    before = cache.clone()
    out = torch.full((b.T, Hq, D), 9.0, dtype=qs.dtype, device="cuda")
    op.append(qs, k, v, cache, lens, table, cu, b.S, q_out=out)
    assert op.status() == rpa.RPA_OK
    t, page, at, pos = slots_of(b)
    # q: as with every other cache
    want, size = rotate(f64(qs)[t], pos, rope)
    assert (np.abs(f64(out)[t] - want) <= half_step(q) * np.abs(want) + 2.0 ** -21 * size + TINY[q]).all()
    got = [tuple(x[page, at] for x in part) for part in i4.unpack(cache.cpu().numpy(), ps, D, group)]
    # V: divided by the scale in 32 bits, otherwise exact: the definition's very codes
    x = f64(v)[t]
    if b.v_scale:
        x = (x.astype(np.float32) / np.float32(b.v_scale)).astype(np.float64)
    for a, w in zip(got[1], i4.coded(x, group)):
        assert np.array_equal(a, w)
    # K: rotated (and divided) in 32 bits, off by e: a level half a step away, or off by what e moves the levels' ends
    x, size = rotate(f64(k)[t], pos, rope)
    e = 2.0 ** -21 * size.max() / (b.k_scale or 1.0)
    x /= b.k_scale or 1.0
    codes, s, z = got[0]
    lo, hi = (f(x.reshape(*x.shape[:-1], -1, group), -1) for f in (np.min, np.max))
    assert (z <= lo + e).all() and (z >= lo - 2.0 ** -10 * np.abs(lo) - 2.0 ** -24 - e).all()
    assert (z + 15 * s >= hi - e - 1e-12).all() and (15 * s <= (hi - z + 2 * e) * (1 + 2.0 ** -10) + 15 * 2.0 ** -24).all()
    assert (np.abs(i4.values(got[0], group) - x) <= np.repeat(s, group, -1) * 0.5 + 2 * e).all()
    # nothing else was written
    raw = [c.copy() for c in i4.unpack(before.cpu().numpy(), ps, D, group)[0]]
    keep = np.ones((b.N, ps), bool)
    keep[page, at] = False
    for i in (0, 1):
        a, w = i4.unpack(cache.cpu().numpy(), ps, D, group)[i], i4.unpack(before.cpu().numpy(), ps, D, group)[i]
        assert all(np.array_equal(x[keep], y[keep], equal_nan=True) for x, y in zip(a, w))
    assert raw and (out[:2] == 9).all() and (out[cu[b.S]:] == 9).all()


def test_positions_and_unaligned_fractions():
    """Positions far out, given apart from the slots: the codes are those of the exact angles (a rotation in 64 bits)."""
    b = Batch(np.random.default_rng(11), [1, 33], [40, 100], 16, 4, 2, 128, kv="int4_g64", q="bf16")
    qs, k, v = new_rows(b)
    pos = b.rng.integers(0, 2 ** 31, b.T).astype(np.int32)
    lens, table, cu = b.lens()
    cache = blank(b, 64)
    op = rpa.RopeAppend(**b.cfg(), base=500000.0)
    op.append(qs, k, v, cache, lens, table, cu, b.S, positions=torch.from_numpy(pos).cuda())
    assert op.status() == rpa.RPA_OK
    t, page, at, _ = slots_of(b)
    # 80-bit angles: 2^31 positions times a double frequency lose 2^-22 of a radian in 64 bits
    w = np.asarray(rpa.rope_frequencies(**b.cfg(), base=500000.0)).astype(np.longdouble)
    turn = (pos[t].astype(np.longdouble)[:, None] * w / (2 * np.longdouble("3.14159265358979323846264338327950288"))) % 1
    ang = (2 * np.pi * turn.astype(np.float64))[:, None]
    x = f64(k)[t]
    y = np.concatenate((x[..., :64] * np.cos(ang) - x[..., 64:] * np.sin(ang), x[..., 64:] * np.cos(ang) + x[..., :64] * np.sin(ang)), -1)
    codes, s, z = (c[page, at] for c in i4.unpack(cache.cpu().numpy(), 16, 128, 64)[0])
    # off by 2^-29 of a pair's size (the sines' 2^-30, their products'), beside the last bits of the 64-bit angle
    e = 2.0 ** -29 * 2 * np.abs(x).max() + 1e-9
    assert (np.abs(codes * np.repeat(s, 64, -1) + np.repeat(z, 64, -1) - y) <= np.repeat(s, 64, -1) * 0.5 + e).all()
    assert (z <= y.reshape(*y.shape[:-1], -1, 64).min(-1) + e).all()


def test_groups_without_a_range_and_odd_values():
    """Equal values, zeros, subnormals, values past float16, infinities and NaN, a group each."""
    b = Batch(np.random.default_rng(0), [6], [6], 16, 1, 1, 128, kv="int4_g32", q="f32")
    x = np.zeros((6, 128), np.float64)
    x[0] = 1.7
    x[1, :32], x[1, 32:64], x[1, 64:96] = 1e-9, -1e-9, np.linspace(-1e-7, 1e-7, 32)
    x[2] = np.linspace(-1e6, 1e6, 128)
    x[3, 5], x[3, 40], x[3, 70] = np.inf, -np.inf, np.nan
    x[4] = b.rng.standard_normal(128) * 60000
    x[5, ::2] = -0.0
    v = torch.from_numpy(x).float().cuda()[:, None]
    lens, table, cu = b.lens()
    cache = blank(b, 32)
    op = rpa.RopeAppend(**b.cfg(), rotary_dim=16)
    op.append(torch.zeros_like(v), torch.zeros_like(v), v, cache, lens, table, cu, 1)
    assert op.status() == rpa.RPA_OK
    page, at = b.slots(0, np.arange(6))
    part = tuple(c[page, at, 0] for c in i4.unpack(cache.cpu().numpy(), 16, 128, 32)[1])
    got = i4.values(part, 32)
    y = v[:, 0].double().cpu().numpy()
    bad = np.zeros((6, 128), bool)
    bad[3, 64:96] = True  # the group of the NaN
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
    y[bad] = 0
    want = i4.values(i4.coded(y, 32), 32)
    assert np.array_equal(got[~bad], want[~bad])
    k, vv = op.read(cache, lens, table, cu, 1)
    # (levels of the smallest scales are no multiples of float32's steps here, so 32 bits round them)
    w = torch.from_numpy(got).float()[:, None]
    assert torch.equal(torch.nan_to_num(vv.cpu(), 12345.0), torch.nan_to_num(w, 12345.0)) and (k == 0).all()


KV = [("bf16", 128), ("f16", 64), ("fp8_e4m3", 256), ("fp8_e5m2", 64), ("int8", 128), ("int4_g32", 64), ("int4_g64", 256), ("int4_g128", 128)]


@pytest.mark.parametrize("kv,D", KV)
@pytest.mark.parametrize("q,ps", [("bf16", 16), ("f16", 20), ("f32", 64)])
def test_read(kv, D, q, ps):
    scaled = kv not in ("bf16", "f16")
    b = Batch(np.random.default_rng(7), [1, 40, 0, 3, 64], [500, 40, 9, 77, 200], ps, 4, 2, D, kv=kv, q=q, lead=1, tail=2,
              **(dict(k_scale=0.05, v_scale=0.7) if scaled else {}))
    if kv.startswith("int4"):
        group = int(kv[6:])
        cache, parts = i4.random_cache(b.rng, b.N, ps, 2, D, group)
        K, V = (i4.values(p, group) for p in parts)
    else:
        cache = b.cache()
        K, V = f64(cache)[:, :, 0::2], f64(cache)[:, :, 1::2]
    lens, table, cu = b.lens()
    op = rpa.RopeAppend(**b.cfg())
    outs = [torch.full((b.T, 2, D), 5.0, dtype=f, device="cuda") for f in [torch.bfloat16 if q == "bf16" else torch.float16 if q == "f16" else torch.float32] * 2]
    got = op.read(cache, lens, table, cu, b.S, *outs)
    assert op.status() == rpa.RPA_OK and got[0] is outs[0]
    t, page, at, _ = slots_of(b)
    for o, x, sc in zip(outs, (K, V), (b.k_scale, b.v_scale)):
        want = x[page, at] * np.float64(np.float32(sc or 1.0))
        # at most two roundings in 32 bits (a 4-bit value: of the sum, and of the product with the cache's scale), then q's own;
        # a 4-bit sum of either sign is rounded relative to itself
        assert (np.abs(f64(o)[t] - want) <= (half_step(q) + 2.0 ** -23) * np.abs(want) + TINY[q]).all()
        rest = np.ones(b.T, bool)
        rest[t] = False
        assert (f64(o)[rest] == 5).all()


def test_read_latent():
    b = Batch(np.random.default_rng(2), [5, 1], [30, 64], 16, 16, 1, 576, latent=True)
    cache = b.cache()
    lens, table, cu = b.lens()
    k, v = rpa.RopeAppend(rotary_dim=64, rotary_offset=512, **b.cfg()).read(cache, lens, table, cu, b.S)
    t, page, at, _ = slots_of(b)
    assert v is None and np.array_equal(f64(k)[t], f64(cache)[page, at])


def test_bad_pages_and_lengths():
    b = Batch(np.random.default_rng(3), [3, 4, 2], [30, 40, 10], 16, 4, 2, 64, kv="int4_g32")
    cache, parts = i4.random_cache(b.rng, b.N, 16, 2, 64, 32)
    qs, k, v = new_rows(b)
    op = rpa.RopeAppend(**b.cfg())
    for kind in ("page", "length"):
        lens, table, cu = b.lens()
        if kind == "page":
            table[1, 2] = b.N  # of its keys 32 .. 39: its last four tokens
        else:
            lens[1] = b.P * 16 + 1
        a, w = op.read(cache, lens, table, cu, b.S, torch.full((b.T, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda"))
        assert op.status() == (rpa.RPA_ERR_BAD_PAGE_INDEX if kind == "page" else rpa.RPA_ERR_BAD_LENGTHS)
        assert (a[3:7] == 5).all() and not (a[:3] == 5).all() and not (a[7:] == 5).all()
        mine = cache.clone()
        op.append(qs, k, v, mine, lens, table, cu, b.S)
        assert op.status() == (rpa.RPA_ERR_BAD_PAGE_INDEX if kind == "page" else rpa.RPA_ERR_BAD_LENGTHS)
        page, at = b.slots(1, np.arange(30, 40))
        got, had = i4.unpack(mine.cpu().numpy(), 16, 64, 32), i4.unpack(cache.cpu().numpy(), 16, 64, 32)
        assert all(np.array_equal(x[page, at], y[page, at]) for p, r in zip(got, had) for x, y in zip(p, r))
    assert op.status() == rpa.RPA_OK


def test_key_rows_with_infinities_and_nan():
    """K's rows are rotated before they are coded: an infinity saturates its pair, a NaN takes its pair's groups."""
    b = Batch(np.random.default_rng(12), [3], [3], 16, 1, 1, 64, kv="int4_g32", q="f16")
    k = torch.zeros(3, 1, 64, dtype=torch.float16, device="cuda")
    k[0, 0, 40] = float("inf")    # not rotated
    k[1, 0, 50] = float("nan")
    k[2, 0, 3] = float("inf")     # rotated with channel 11
    lens, table, cu = b.lens()
    cache = blank(b, 32)
    op = rpa.RopeAppend(**b.cfg(), rotary_dim=16)
    op.append(torch.zeros_like(k), k, torch.zeros_like(k), cache, lens, table, cu, 1)
    assert op.status() == rpa.RPA_OK
    page, at = b.slots(0, np.arange(3))
    part = tuple(c[page, at, 0] for c in i4.unpack(cache.cpu().numpy(), 16, 64, 32)[0])
    got = i4.values(part, 32)
    assert got[0, 40] >= 65504 and np.isfinite(got[0]).all() and (got[0, :32] == 0).all()
    assert np.isnan(got[1, 32:]).all() and (got[1, :32] == 0).all()
    # position 2: cos(2 w) and sin(2 w) of pair 3 are positive, so both of its channels are infinite
    assert (got[2, [3, 11]] >= 65504).all() and np.isfinite(got[2]).all()


def test_many_sequences_and_refusals():
    b = Batch(np.random.default_rng(4), [1] * 700, [3 + i % 40 for i in range(700)], 16, 2, 1, 64, kv="int4_g64")
    qs, k, v = new_rows(b)
    lens, table, cu = b.lens()
    op = rpa.RopeAppend(**b.cfg())
    cache = blank(b, 64)
    op.append(qs, k, v, cache, lens, table, cu, b.S)
    a, w = op.read(cache, lens, table, cu, b.S)
    assert op.status() == rpa.RPA_OK
    codes = i4.coded(f64(v), 64)
    assert np.array_equal(f64(w), f64(torch.from_numpy(i4.values(codes, 64)).float().bfloat16()))
    with pytest.raises(ValueError):
        op.read(cache[:, :, :-4], lens, table, cu, b.S)
    with pytest.raises(ValueError):
        op.read(cache.view(torch.int16), lens, table, cu, b.S)
    with pytest.raises(ValueError):
        op.read(cache, lens, table, cu, b.S, k_out=torch.zeros(b.T, 1, 64, device="cuda"))
    with pytest.raises(rpa.RpaError):
        op.read(cache, lens, table, cu, b.max_seqs + 1)


def test_graph_and_streams():
    b = Batch(np.random.default_rng(5), [1, 20], [100, 60], 16, 4, 2, 128, kv="int4_g64")
    qs, k, v = new_rows(b)
    lens, table, cu = b.lens()
    op = rpa.RopeAppend(**b.cfg())
    cache = blank(b, 64)
    q0 = op.append(qs, k, v, cache, lens, table, cu, b.S).clone()
    k0, v0 = (x.clone() for x in op.read(cache, lens, table, cu, b.S))
    cache2, q1, k1, v1 = blank(b, 64), torch.zeros_like(q0), torch.zeros_like(k0), torch.zeros_like(v0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.append(qs, k, v, cache2, lens, table, cu, b.S, q_out=q1, stream=side)
    op.read(cache2, lens, table, cu, b.S, k1, v1, stream=side)
    side.synchronize()
    assert torch.equal(cache2, cache) and torch.equal(q1, q0) and torch.equal(k1, k0) and torch.equal(v1, v0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.append(qs, k, v, cache2, lens, table, cu, b.S, q_out=q1)
        op.read(cache2, lens, table, cu, b.S, k1, v1)
    for x in (cache2, q1, k1, v1):
        x.zero_()
    cache2.fill_(0x5a)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache2, cache) and torch.equal(q1, q0) and torch.equal(k1, k0) and torch.equal(v1, v0)
