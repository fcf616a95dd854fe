"""Rotary append on the GPU against its definition in 64 bits.

An output is off by its one rounding (half a step of its type, or half the smallest step of the type's
subnormals) and by the 32-bit arithmetic before it.  Of that: the sine and cosine are off by at most 2^-24
(the angle rounded to 32 bits, pi 2^-25 at most at half a turn) and 2 units of 2^-24 (sincospi), and again
by half a unit where the magnitude multiplies them; each of the two products and their sum rounds once:
(pi/2 + 2 + 1/2 + 1 + 1) 2^-24 of |a| + |b| at most, below 2^-21; the division by the scale 2^-24 more.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import MOST, TINY, TORCH, Batch, f64, half_step, rotate, stored  # noqa: E402

pytestmark = pytest.mark.gpu
ARITH = 2.0 ** -21


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def inputs(b, rng, fused=True):
    """q, k, v as slices of one projection, on the GPU."""
    heads = b.Hq + (1 if b.latent else 2) * b.Hkv
    qkv = stored(rng.standard_normal((b.T, heads, b.D)) * 3, b.q).cuda()
    parts = [qkv[:, :b.Hq], qkv[:, b.Hq:b.Hq + b.Hkv], None if b.latent else qkv[:, b.Hq + b.Hkv:]]
    return parts if fused else [None if x is None else x.contiguous() for x in parts]


def expected(b, q, k, v, rope, positions=None):
    """{sequence: (token rows, q values, their bounds, slots, cache rows, bounds)}"""
    out = {}
    for s in range(b.S):
        n, kl = b.q_lens[s], b.kv_lens_list[s]
        t = np.arange(b.cu[s], b.cu[s] + n)
        j = np.arange(kl - n, kl)
        pos = j if positions is None else positions[t]
        qy, qs = rotate(f64(q)[t], pos, rope)
        ky, ks = rotate(f64(k)[t], pos, rope)
        rows, size = [ky / (b.k_scale or 1)], [ks / (b.k_scale or 1)]
        if v is not None:
            rows.append(f64(v)[t] / (b.v_scale or 1))
            size.append(np.zeros_like(rows[1]))
        out[s] = (t, qy, qs, b.slots(s, j), np.stack(rows, 2).reshape(n, b.rows, b.D),
                  np.stack(size, 2).reshape(n, b.rows, b.D))
    return out


def near(got, want, size, dtype, what):
    if dtype == "int8":
        bound = 0.5 + ARITH * size + 2.0 ** -23 * np.abs(want)
        want = np.clip(want, -128, 127)
    else:
        want = np.clip(want, -MOST.get(dtype, np.inf), MOST.get(dtype, np.inf))
        bound = (half_step(dtype) + 2.0 ** -23) * (np.abs(want) + ARITH * size) + ARITH * size + TINY[dtype]
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - want)[bad].max():.3g}"


def check(b, q, k, v, q_out, before, after, rope, positions=None):
    want = expected(b, q, k, v, rope, positions)
    out = f64(q_out)
    kept = torch.ones(b.N, b.ps, dtype=torch.bool)
    for t, qy, qs, (page, at), rows, size in want.values():
        near(out[t], qy, qs, b.q, "q")
        near(f64(after.cpu()[page, at]) if after.element_size() > 1 or b.kv == "int8" else after.cpu().float()[page, at].double().numpy(),
             rows, size, b.kv, "cache")
        kept[page, at] = False
    # every other slot as it was
    assert torch.equal(before.cpu().view(torch.uint8)[kept], after.cpu().view(torch.uint8)[kept])


LATENT = dict(Hq=16, Hkv=1, D=576, latent=True)
CASES = [
    (0, dict(Hq=4, Hkv=2, D=64), dict(), [1], [1]),
    (1, dict(Hq=32, Hkv=8, D=128), dict(base=500000.0), [1] * 9, [1, 2, 16, 17, 300, 5, 31, 32, 33]),
    (2, dict(Hq=8, Hkv=8, D=256), dict(rotary_dim=64, pairing="interleaved"), [3, 1, 40, 0, 7], [3, 90, 41, 20, 7]),
    (3, dict(Hq=5, Hkv=1, D=64), dict(rotary_dim=16, rotary_offset=8), [9, 0, 33], [20, 0, 33]),
    (4, dict(Hq=6, Hkv=3, D=128), dict(rotary_dim=32, rotary_offset=96, pairing="interleaved"), [70], [131]),
    (5, dict(Hq=64, Hkv=1, D=128), dict(scaling="rotations", factor=8.0, trained_len=512), [5, 6], [700, 6]),
    (6, LATENT, dict(rotary_dim=64, rotary_offset=512), [4, 1], [4, 50]),
    (7, dict(LATENT, Hq=128), dict(rotary_dim=64, rotary_offset=512, pairing="interleaved", scaling="index", factor=40.0,
                                   trained_len=4096, high=32.0, magnitude=1.37), [2, 3, 1], [64, 3, 65]),
    (8, dict(Hq=16, Hkv=2, D=256), dict(rotary_dim=256, scaling="base", factor=4.0, magnitude=-0.5), [20, 11], [20, 1000]),
]


@pytest.mark.parametrize("seed,shape,rope,q_lens,kv_lens", CASES)
@pytest.mark.parametrize("q,kv", [("bf16", "bf16"), ("f32", "f16"), ("f16", "bf16")])
def test_append(seed, shape, rope, q_lens, kv_lens, q, kv):
    rng = np.random.default_rng(seed)
    b = Batch(rng, q_lens, kv_lens, 8 if seed % 2 else 16, kv=kv, q=q, lead=seed % 3, tail=seed % 2 * 3, **shape)
    rope = dict(dict(rotary_dim=b.D), **rope)
    x = inputs(b, rng, fused=seed % 2 == 0)
    cache = b.cache()
    before = cache.clone()
    op = rpa.RopeAppend(**rope, **b.cfg())
    out = torch.full((b.T, b.Hq, b.D), 7.0, dtype=TORCH[q], device="cuda")
    op.append(*x, cache, *b.lens(), b.S, q_out=out)
    assert op.status() == rpa.RPA_OK
    check(b, *x, out, before, cache, rope)
    # rows of tokens that no sequence covers are left as they were
    rest = np.ones(b.T, bool)
    rest[b.cu[0]:b.cu[b.S]] = False
    assert (f64(out)[rest] == 7.0).all()


@pytest.mark.parametrize("kv,k_scale,v_scale", [("fp8_e4m3", 0.05, 0.07), ("fp8_e5m2", None, 3.0), ("int8", 0.04, 0.02), ("bf16", 0.3, None),
                                                ("f16", 1e-3, 1.0)])
@pytest.mark.parametrize("q", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scaled_and_8_bit_caches(kv, k_scale, v_scale, q, D):
    rng = np.random.default_rng(11)
    b = Batch(rng, [7, 1, 12], [40, 23, 12], 4, 6, 2, D, kv=kv, q=q, k_scale=k_scale, v_scale=v_scale)
    rope = dict(rotary_dim=32, rotary_offset=16)
    x = inputs(b, rng)
    x[1][3, 1, 20], x[2][4, 0, 5] = 3e4, -3e4  # past the 8-bit types
    cache = b.cache()
    before = cache.clone()
    op = rpa.RopeAppend(**rope, **b.cfg())
    out = op.append(*x, cache, *b.lens(), b.S)
    assert op.status() == rpa.RPA_OK
    if kv == "f16":  # 3e4 / 1e-3 is past f16 too: infinite, as the type has it
        got = cache[tuple(torch.as_tensor(i).long() for i in b.slots(0, [36]))][0, 2]
        assert torch.isinf(got).any()
        return
    check(b, *x, out, before, cache, rope)


def test_nan_and_infinity_stay_in_their_pairs():
    rng = np.random.default_rng(12)
    for kv in ("bf16", "fp8_e4m3", "fp8_e5m2", "int8"):
        b = Batch(rng, [2], [2], 16, 2, 1, 64, kv=kv)
        x = inputs(b, rng)
        x[1][0, 0, 3] = float("nan")  # its pair is 3 + 32
        x[2][0, 0, 9], x[2][1, 0, 9] = float("inf"), float("nan")
        cache = torch.zeros_like(b.cache())
        op = rpa.RopeAppend(**b.cfg())
        op.append(*x, cache, *b.lens(), 1)
        page = int(b.table[0, 0])
        k, v = cache[page, 0, 0].float(), cache[page, :2, 1].float()
        if kv == "int8":
            assert k[3] == 0 and k[35] == 0 and v[0, 9] == 127 and v[1, 9] == 0
            continue
        assert torch.isnan(k).nonzero().flatten().tolist() == [3, 35]
        assert torch.isnan(v[1, 9]) and (torch.isinf(v[0, 9]) if kv == "bf16" else v[0, 9] == MOST[kv])


def test_far_positions():
    """Given positions: the angle is exact at 2^31 - 1 as at 0, and below 0."""
    rng = np.random.default_rng(13)
    b = Batch(rng, [6, 3], [6, 40], 16, 4, 2, 128, q="f32")
    rope = dict(rotary_dim=128, base=10000.0)
    pos = np.array([0, 1, 2 ** 31 - 1, 1000003, 2 ** 24 + 1, -5, -2 ** 31, 7, 123456789], np.int32)
    x = inputs(b, rng)
    cache = b.cache()
    before = cache.clone()
    op = rpa.RopeAppend(**rope, **b.cfg())
    out = op.append(*x, cache, *b.lens(), b.S, positions=torch.from_numpy(pos).cuda())
    assert op.status() == rpa.RPA_OK
    # numpy's own angle: pos * w rounded to 53 bits, at most 2^31 * 2^-53 = 2^-22 of |a| + |b| on top
    want = expected(b, *x, rope, pos)
    for t, qy, qs, slots, rows, size in want.values():
        far = 2.0 ** -21
        assert (np.abs(f64(out)[t] - qy) <= (half_step("f32") + ARITH + far) * (np.abs(qy) + qs)).all()
        got = f64(cache[tuple(torch.as_tensor(i).long() for i in slots)])
        assert (np.abs(got - rows) <= half_step("bf16") * np.abs(rows) * 1.001 + (ARITH + far) * size).all()
    kept = torch.ones(b.N, b.ps, dtype=torch.bool)
    for _, _, _, (page, at), _, _ in want.values():
        kept[page, at] = False
    assert torch.equal(before.cpu()[kept], cache.cpu()[kept])


def test_in_place_q_other_stream_and_graph():
    rng = np.random.default_rng(14)
    b = Batch(rng, [5, 1, 30], [5, 77, 31], 16, 8, 2, 128, tail=2)
    x = inputs(b, rng, fused=False)
    lens = b.lens()
    op = rpa.RopeAppend(**b.cfg())
    cache = b.cache()
    ref_cache = cache.clone()
    ref = op.append(*x, ref_cache, *lens, b.S)
    # in place, on a stream of its own
    q = x[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c1 = cache.clone()
    torch.cuda.synchronize()
    op.append(q, x[1], x[2], c1, *lens, b.S, q_out=q, stream=side)
    assert op.status(side) == rpa.RPA_OK
    assert torch.equal(q[:36], ref[:36]) and torch.equal(q[36:], x[0][36:]) and torch.equal(c1, ref_cache)
    # captured, replayed with other inputs in the same buffers
    q, k, v = (t.clone() for t in x)
    c2, out = cache.clone(), torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.append(q, k, v, c2, *lens, b.S, q_out=out)
    y = inputs(b, rng, fused=False)
    for d, s in zip((q, k, v), y):
        d.copy_(s)
    g.replay()
    c3 = cache.clone()
    want = op.append(*y, c3, *lens, b.S)
    assert torch.equal(out, want) and torch.equal(c2, c3) and op.status() == rpa.RPA_OK


def test_bad_lengths_and_pages_are_reported_and_skipped():
    rng = np.random.default_rng(15)
    b = Batch(rng, [3, 2, 4], [20, 2, 9], 8, 4, 2, 64)
    x = inputs(b, rng)
    op = rpa.RopeAppend(**b.cfg())
    kvl, table, cu = b.lens()
    for place, value in ((0, b.N), (0, -1), (1, 2 ** 30)):
        t = table.clone()
        t[2, place] = value  # tokens 5 .. 8 of sequence 2 sit in logical pages 0 and 1
        cache = b.cache()
        before = cache.clone()
        out = op.append(*x, cache, kvl, t, cu, b.S)
        assert op.status() == rpa.RPA_ERR_BAD_PAGE_INDEX
        assert op.status() == rpa.RPA_OK  # read once
        good = cache.clone()
        ref = op.append(*x, good, kvl, table, cu, b.S)
        assert op.status() == rpa.RPA_OK and torch.equal(out, ref)
        lost = table[2, place].item()  # the page that the bad id stood for: not written
        others = [i for i in range(b.N) if i != lost]
        assert torch.equal(cache[others], good[others]) and torch.equal(cache[lost], before[lost])
    for bad in ("kv", "short", "cu", "past"):
        k2, c2 = kvl.clone(), cu.clone()
        if bad == "kv":
            k2[1] = b.P * b.ps + 1
        elif bad == "short":
            k2[1] = 1  # fewer keys than query tokens
        elif bad == "cu":
            c2[2] = 1  # decreasing
        else:
            c2[3] = b.T + 1
        cache = b.cache()
        op.append(*x, cache, k2, table, c2, b.S)
        assert op.status() == rpa.RPA_ERR_BAD_LENGTHS, bad
    cache = b.cache()
    before = cache.clone()
    op.append(*x, cache, kvl, table, cu, 0)  # no sequences: nothing is written
    assert op.status() == rpa.RPA_OK and torch.equal(cache, before)


def test_refusals():
    rng = np.random.default_rng(16)
    b = Batch(rng, [2], [2], 16, 2, 1, 64)
    x = inputs(b, rng)
    cache, lens = b.cache(), b.lens()
    op = rpa.RopeAppend(**b.cfg())
    with pytest.raises(rpa.RpaError):
        op.append(*x, cache, *lens, b.max_seqs + 1)
    with pytest.raises(ValueError):
        op.append(x[0].cpu(), x[1], x[2], cache, *lens, 1, q_out=torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda"))
    odd = torch.zeros(2, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")  # tokens 520 bytes apart
    with pytest.raises(rpa.RpaError):
        op.append(odd[:, :128].unflatten(1, (2, 64)), x[1], x[2], cache, *lens, 1)
    op.close()
    with pytest.raises(ValueError):
        op.append(*x, cache, *lens, 1)


def test_no_tokens():
    rng = np.random.default_rng(17)
    b = Batch(rng, [0, 0], [3, 0], 16, 2, 1, 64)
    x = inputs(b, rng)
    cache = b.cache()
    op = rpa.RopeAppend(**b.cfg())
    op.append(*x, cache, *b.lens(), b.S)
    assert op.status() == rpa.RPA_OK
    kvl, table, cu = b.lens()
    cu[2] = 1
    op.append(*x, cache, kvl, table, cu, b.S)
    assert op.status() == rpa.RPA_ERR_BAD_LENGTHS


def test_append_then_attend():
    """A prompt chunk written by the operator and read by the library's attention on the same stream."""
    import oracle
    import rpa_inputs as ri

    rng = np.random.default_rng(18)
    b = Batch(rng, [40, 1, 9], [40, 90, 60], 16, 8, 2, 128)
    rope = dict(rotary_dim=128)
    x = inputs(b, rng)
    x[0].mul_(1 / 3), x[1].mul_(1 / 3)
    cache = b.cache()
    op, att = rpa.RopeAppend(**rope, **b.cfg()), rpa.RaggedPagedAttention(**b.cfg())
    lens = b.lens()
    q = op.append(*x, cache, *lens, b.S)
    o = att.forward(q, cache, *lens, b.S)
    assert op.status() == rpa.RPA_OK and att.status() == rpa.RPA_OK
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    p = ri.Problem(**b.cfg(), num_seqs=b.S, q=bits(q), kv_pages=bits(cache), kv_lens=b.kv_lens, page_indices=b.table, cu_q_lens=b.cu)
    ref = oracle.forward(p)
    assert (np.abs(f64(o) - ref) <= 2e-2 + 2e-2 * np.abs(ref)).all()


def test_many_sequences():
    """More sequences than two rounds of the lookup tell apart, some of them empty; tokens in every part of a CTA's run."""
    rng = np.random.default_rng(19)
    q_lens = [int(x) for x in rng.integers(0, 4, 2500)]
    b = Batch(rng, q_lens, [n + int(x) for n, x in zip(q_lens, rng.integers(0, 9, 2500))], 4, 2, 1, 64, lead=1, tail=1)
    rope = dict(rotary_dim=64)
    x = inputs(b, rng)
    cache = b.cache()
    before = cache.clone()
    op = rpa.RopeAppend(**b.cfg())
    out = op.append(*x, cache, *b.lens(), b.S)
    assert op.status() == rpa.RPA_OK
    check(b, *x, out, before, cache, rope)


@pytest.mark.parametrize("S", [1, 512, 513])
def test_several_rounds_of_tokens(S):
    """More tokens than all CTAs take at once, of as many sequences as their shared memory holds lengths for, and of one more."""
    rng = np.random.default_rng(22)
    q_lens = [int(x) for x in rng.integers(0, 2 * 13300 // S, S)] if S > 1 else [13300]
    b = Batch(rng, q_lens, [n + int(x) for n, x in zip(q_lens, rng.integers(0, 9, S))], 16, 2, 1, 64, lead=3, tail=5)
    assert b.T > 152 * 5 * 16
    x = inputs(b, rng)
    cache = b.cache()
    before = cache.clone()
    op = rpa.RopeAppend(**b.cfg())
    out = op.append(*x, cache, *b.lens(), b.S)
    assert op.status() == rpa.RPA_OK
    check(b, *x, out, before, cache, dict(rotary_dim=64))


def test_one_call_after_another():
    """Calls that follow each other on a stream without a wait, each writing the cache that the next rotates into."""
    rng = np.random.default_rng(20)
    b = Batch(rng, [7, 1, 30], [7, 20, 90], 16, 8, 2, 128)
    lens = b.lens()
    op = rpa.RopeAppend(**b.cfg())
    xs = [inputs(b, rng) for _ in range(8)]
    cache = b.cache()
    torch.cuda.synchronize()
    outs = [op.append(*x, cache, *lens, b.S) for x in xs]
    assert op.status() == rpa.RPA_OK
    for x, o in zip(xs, outs):
        again = b.cache()
        assert torch.equal(o, op.append(*x, again, *lens, b.S))
    last = cache.clone()
    op.append(*xs[-1], last, *lens, b.S)
    assert torch.equal(last, cache)
