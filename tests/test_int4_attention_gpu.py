"""Paged attention over a cache of 4-bit codes, against its definition in 64 bits."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as i4  # noqa: E402
import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch, f64, half_step  # noqa: E402
from long_cache_util import attend64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


class Case:
    """A batch over a 4-bit cache of N(0, 1) values, and what attention gives."""

    def __init__(self, seed, q_lens, kv_lens, ps, Hq, Hkv, D, group, q="bf16", **more):
        lead, tail = more.pop("lead", 2), more.pop("tail", 1)
        self.b = b = Batch(np.random.default_rng(seed), q_lens, kv_lens, ps, Hq, Hkv, D, kv="int4_g%d" % group, q=q, lead=lead, tail=tail, **more)
        self.group = group
        self.cache, self.parts = i4.random_cache(b.rng, b.N, ps, Hkv, D, group)
        self.q, self.lens = b.queries(), b.lens()

    def reference(self, **knobs):
        b, group = self.b, self.group
        K, V = (i4.values(p, group) for p in self.parts)
        S = np.repeat(self.parts[1][1], group, -1)

        def at(x):
            def rows(s):
                page, place = b.slots(s, np.arange(b.kv_lens_list[s]))
                return x[page, place]

            return rows

        ks, vs = (np.float64(np.float32(x or 1.0)) for x in (b.k_scale, b.v_scale))
        k, v, st = at(K), at(V), at(S)
        return attend64(f64(self.q), b.q_lens, b.kv_lens_list, b.cu, lambda s: (k(s) * ks, v(s) * vs), step=lambda s: st(s) * vs, **knobs)

    def make(self, **knobs):
        names = dict(window="sliding_window", first="first_keys", cap="soft_cap", causal="is_causal", sinks="sinks")
        return rpa.RaggedPagedAttention(**dict(self.b.cfg(), **{names[k]: v for k, v in knobs.items()}))

    def check(self, call=None, **knobs):
        b = self.b
        att = self.make(**knobs)
        out = torch.full((b.T, b.Hq, b.D), 7.0, dtype=self.q.dtype, device="cuda")
        if call:
            call(att, out)
        else:
            att.forward(self.q, self.cache, *self.lens, b.S, out=out)
            assert att.status() == rpa.RPA_OK
        ref, size, steps = self.reference(**knobs)
        # P = f16(p s) meets codes at most 8 from the middle; o is rounded once; logits in 32 bits (sums of at most 2^6 in units of
        # the logit, a few roundings each: 2^-14).  Prompts' rows are rounded to f16 (K: the sum of |q k| / sqrt(D) stays below
        # 16 half steps, V and P a half step of |p v| each) and, at D 256 with a cap, take tanh's approximation (2^-11 of the cap).
        # q of 32 bits is rounded to f16 (16 half steps of a logit again).
        h = half_step("f16")
        e = 2.0 ** -14 + 16 * h + (16 * h if b.q == "f32" else 0) + (knobs.get("cap") or 0) * 2.0 ** -11
        long_rows = np.zeros(b.T, bool)
        for s, n in enumerate(b.q_lens):
            long_rows[b.cu[s]:b.cu[s] + n] = n * b.Hq // b.Hkv > 8
        e_direct = 2.0 ** -14 + (16 * h if b.q == "f32" else 0)
        tol = half_step(b.q) * np.abs(ref) + 1e-6 + np.where(long_rows[:, None, None], 8 * h * steps + 2 * h * size + 2 * e * size,
                                                             8 * h * steps + 2 * e_direct * size)
        got = f64(out)
        assert np.isfinite(got).all()
        err = np.abs(got - ref) - tol
        assert err.max() <= 0, (err.max(), np.unravel_index(err.argmax(), err.shape))
        inside = np.zeros(b.T, bool)
        inside[b.cu[0]:b.cu[b.S]] = True
        assert (got[~inside] == 0).all()
        return out


SHAPES = [  # Hq, Hkv, D, group, ps, q
    (8, 2, 128, 128, 16, "bf16"),
    (32, 8, 128, 64, 64, "f16"),
    (4, 4, 128, 32, 20, "bf16"),   # pages that do not divide a stage: runs of 4
    (12, 1, 128, 128, 8, "bf16"),  # 16-row tiles
    (32, 2, 128, 64, 32, "f32"),
    (16, 1, 128, 32, 48, "f16"),
    (6, 2, 64, 64, 4, "f16"),
    (4, 1, 64, 32, 256, "bf16"),   # a page is two stages
    (40, 2, 64, 64, 12, "f16"),    # 20 heads a kv head: two blocks of 10
    (64, 1, 64, 32, 16, "bf16"),
    (8, 2, 256, 128, 16, "bf16"),
    (16, 1, 256, 64, 128, "f16"),
    (2, 2, 256, 32, 24, "f32"),
    (13, 1, 64, 64, 16, "f16"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_decode(shape):
    Hq, Hkv, D, group, ps, q = shape
    Case([1, D, Hq], [1] * 9, [1, 2, 31, 32, 33, 127, 129, 700, 300], ps, Hq, Hkv, D, group, q).check()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_few_tokens_and_prompts(shape):
    Hq, Hkv, D, group, ps, q = shape
    Case([2, D, Hq], [1, 3, 200, 0, 5, 17, 64], [300, 3, 500, 40, 200, 17, 140], ps, Hq, Hkv, D, group, q).check()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("window,first", [(100, 0), (100, 4), (3, 70), (1, 1), (333, 64), (70, 200)])
def test_window(shape, window, first):
    Hq, Hkv, D, group, ps, q = shape
    Case([3, D, Hq, window], [1, 90, 1, 4, 1, 33], [900, 700, 40, 600, window + first, 33], ps, Hq, Hkv, D, group, q).check(window=window, first=first)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
def test_knobs(D, group):
    c = Case([4, D], [1, 60, 3], [700, 400, 90], 16, 8, 2, D, group, k_scale=0.7, v_scale=1.3)
    c.check(cap=20.0)
    c.check(sinks=c.b.rng.standard_normal(8).astype(np.float32))
    c.check(causal=False)
    c.check(causal=False, window=50, first=3)
    c.check(window=50, first=3, cap=10.0, sinks=c.b.rng.standard_normal(8).astype(np.float32))


@pytest.mark.parametrize("Hq,Hkv,D,group,q_lens", [
    (4, 1, 128, 128, [1, 1, 2]), (16, 1, 64, 32, [1, 3, 1]), (4, 2, 256, 64, [1, 9, 1]), (8, 1, 128, 64, [5, 1, 8]),
])
@pytest.mark.parametrize("knobs", [{}, dict(window=20000, first=0), dict(window=9000, first=700)], ids=str)
def test_split_over_keys(Hq, Hkv, D, group, q_lens, knobs):
    """Few sequences of many keys: pieces, of several tiles too, and pieces that no row of a tile sees."""
    Case([5, D], q_lens, [30000, 12000, 7000], 16, Hq, Hkv, D, group).check(**knobs)


def test_prompts_without_room():
    """Sequences past the f16 room run in tiles of the direct kernel, prompts of many tiles and pieces among them."""
    c = Case(6, [300, 200, 100], [5000, 2000, 300], 16, 4, 1, 128, 128)
    want = c.check()

    def no_alloc(att, out):  # has no room at all
        r = rpa.lib().rpa_forward_noalloc(ctypes.byref(att._c), c.q.data_ptr(), c.cache.data_ptr(), *[x.data_ptr() for x in c.lens], c.b.S,
                                          out.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert r == rpa.RPA_OK

    got = c.check(call=no_alloc)
    assert not torch.equal(want, got)  # (the two paths round differently)


def test_large_and_small_values():
    """Scales and zeros of all sizes: V up to f16's range, K small enough for its logits."""
    c = Case(7, [1, 40, 2], [400, 300, 100], 16, 8, 2, 128, 64)
    b = c.b
    size = 10.0 ** b.rng.uniform(-4, 4.5, (b.N, 1, 2, 1))
    K = b.rng.standard_normal((b.N, 16, 2, 128)) * 10.0 ** b.rng.uniform(-3, -1, (b.N, 1, 2, 1))
    V = b.rng.standard_normal((b.N, 16, 2, 128)) * size
    c.parts = [i4.coded(x, 64) for x in (K, V)]
    c.cache = torch.from_numpy(i4.pack(c.parts, 16, 128, 64)).cuda()
    c.check()


@pytest.mark.parametrize("D,group,ps", [(128, 64, 16), (64, 32, 20), (256, 128, 64)])
def test_slots_behind_the_keys_may_hold_anything(D, group, ps):
    """All bits set (NaN scales and zeros) in unused pages, behind the last key, and in front of a window."""
    c = Case([8, D], [1, 50, 3], [77, 90, 250], ps, 8, 2, D, group)
    b = c.b
    for knobs in ({}, dict(window=30, first=5)):
        used = np.zeros((b.N, ps), bool)
        for s, (a, n) in enumerate(zip(b.q_lens, b.kv_lens_list)):
            j = np.arange(n)
            if knobs:
                j = j[(j < 5) | (j > n - a - 30)]
            page, place = b.slots(s, j)
            used[page, place] = True
        parts = [tuple(x.copy() for x in p) for p in c.parts]
        for codes, sc, z in parts:
            codes[~used] = 15
            sc[~used] = z[~used] = np.nan
        clean, c.cache = c.cache, torch.from_numpy(i4.pack(parts, ps, D, group)).cuda()
        got = c.check(**knobs)
        c.cache = clean
        assert torch.equal(got, c.check(**knobs))


def test_nan_in_a_visible_group_shows():
    c = Case(9, [1, 1], [50, 60], 16, 4, 2, 64, 32)
    page, place = c.b.slots(0, 10)
    for i in (0, 1):
        parts = [tuple(x.copy() for x in p) for p in c.parts]
        parts[i][2][page, place, 1, 0] = np.nan  # kv head 1's
        out = c.make().forward(c.q, torch.from_numpy(i4.pack(parts, 16, 64, 32)).cuda(), *c.lens, 2)
        got = torch.isnan(out[2])
        assert got[2:].any(-1).all() and not got[:2].any() and not torch.isnan(out[3]).any()


def test_host_graph_and_streams():
    c = Case(10, [1, 100, 2], [900, 300, 1200], 16, 8, 2, 128, 64)
    b = c.b

    def host(att, out):
        o = torch.empty(out.shape, dtype=out.dtype).pin_memory()
        att.forward_host(c.q.cpu().pin_memory(), c.cache, *[x.cpu() for x in c.lens], b.S, o)
        torch.cuda.synchronize()
        out.copy_(o)

    def graph(att, out):
        att.forward(c.q, c.cache, *c.lens, b.S, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            att.forward(c.q, c.cache, *c.lens, b.S, out=out)
        for _ in range(3):
            out.fill_(3.0)
            g.replay()
        torch.cuda.synchronize()

    def many(att, out):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        att.set_option(rpa.RPA_OPT_PLAN_EARLY, 1)
        outs = [torch.empty_like(out) for _ in range(6)]
        for o in outs:
            att.forward(c.q, c.cache, *c.lens, b.S, out=o, stream=side)
        side.synchronize()
        assert all(torch.equal(o, outs[0]) for o in outs)
        out.copy_(outs[0])

    outs = [c.check(call=f) for f in (None, host, graph, many)]
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_alternating_batches_of_one_handle():
    """The room and its tables serve one call after the other, without synchronisation."""
    b = Batch(np.random.default_rng(11), [1, 200, 30, 1], [1000, 900, 700, 50], 16, 8, 2, 128, kv="int4_g64")
    cache, _ = i4.random_cache(b.rng, b.N, 16, 2, 128, 64)
    att = rpa.RaggedPagedAttention(**b.cfg())
    q = b.queries()
    lens = []
    for kl in ([1000, 900, 700, 50], [1000, 300, 800, 40], [20, 700, 31, 300]):
        x = b.kv_lens.copy()
        x[:4] = np.minimum(kl, [b.P * 16] * 4)
        table = b.rng.integers(0, b.N, b.table.shape).astype(np.int32)
        lens.append([torch.from_numpy(x).cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(b.cu.copy()).cuda()])
    want = []
    for l in lens:
        want.append(att.forward(q, cache, *l, b.S))
        assert att.status() == rpa.RPA_OK
    order = b.rng.integers(0, 3, 30)
    outs = [att.forward(q, cache, *lens[i], b.S) for i in order]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for o, i in zip(outs, order))


def test_bad_pages_and_lengths():
    c = Case(12, [1, 40, 1], [300, 200, 90], 16, 4, 2, 128, 64)
    b = c.b
    want = c.check()
    for s, at in ((0, 3), (1, 5)):  # of the direct kernel, of a prompt's rows
        for bad in (-1, b.N, 1 << 30):
            table = c.lens[1].clone()
            table[s, at] = bad
            att = c.make()
            out = att.forward(c.q, c.cache, c.lens[0], table, c.lens[2], b.S)
            assert att.status() == rpa.RPA_ERR_BAD_PAGE_INDEX
            for k in range(3):
                if k != s:
                    assert torch.equal(out[b.cu[k]:b.cu[k + 1]], want[b.cu[k]:b.cu[k + 1]])
    for kl in (-1, b.P * 16 + 1, 0):
        lens = c.lens[0].clone()
        lens[1] = kl
        att = c.make()
        out = att.forward(c.q, c.cache, lens, c.lens[1], c.lens[2], b.S)
        assert att.status() == rpa.RPA_ERR_BAD_LENGTHS and (out == 0).all()


def test_no_sequences_and_no_tokens():
    c = Case(13, [1, 4], [30, 50], 16, 4, 2, 64, 64)
    att = c.make()
    out = att.forward(c.q, c.cache, *c.lens, 0)
    assert att.status() == rpa.RPA_OK and (out == 0).all()
    att = rpa.RaggedPagedAttention(**dict(c.b.cfg(), num_q_tokens=0))
    cu = torch.zeros_like(c.lens[2])
    out = att.forward(c.q[:0], c.cache, c.lens[0], c.lens[1], cu, 2)
    assert att.status() == rpa.RPA_OK and out.shape[0] == 0


def test_stalled_copies_give_up():
    """The producer issues nothing: the bounded waits run out and the context stays usable."""
    c = Case(14, [1, 1], [300, 200], 16, 8, 2, 128, 64)
    att = c.make()
    att.set_option(rpa.RPA_OPT_WAIT_TIMEOUT_MS, 20)
    att.set_option(rpa.RPA_OPT_TEST_STALL_PRODUCER, 1)
    att.forward(c.q, c.cache, *c.lens, c.b.S)
    assert att.status() == rpa.RPA_ERR_TIMEOUT
    att.set_option(rpa.RPA_OPT_TEST_STALL_PRODUCER, 0)
    c.check()


def test_append_then_attend():
    """A serving step: append to the cache, attend, append again."""
    rng = np.random.default_rng(15)
    b = Batch(rng, [1, 70, 2], [200, 70, 50], 16, 8, 2, 128, kv="int4_g64")
    cache, _ = i4.random_cache(rng, b.N, 16, 2, 128, 64)
    lens, table, cu = b.lens()
    rope, att = rpa.RopeAppend(**b.cfg()), rpa.RaggedPagedAttention(**b.cfg())
    q = b.queries()
    k, v = (b.queries()[:, :2].contiguous() for _ in "kv")
    qr = rope.append(q, k, v, cache, lens, table, cu, b.S)
    out = att.forward(qr, cache, lens, table, cu, b.S)
    assert att.status() == rpa.RPA_OK and rope.status() == rpa.RPA_OK
    K, V = (i4.values(p, 64) for p in i4.unpack(cache.cpu().numpy(), 16, 128, 64))

    def rows(s):
        page, place = b.slots(s, np.arange(b.kv_lens_list[s]))
        return K[page, place], V[page, place]

    ref, size = attend64(f64(qr), b.q_lens, b.kv_lens_list, b.cu, rows)
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 0.05 * size + 1e-6).all()
    kr, vr = rope.read(cache, lens, table, cu, b.S)
    page, place = b.slots(2, np.arange(48, 50))
    assert np.allclose(f64(kr)[b.cu[2]:b.cu[3]], K[page, place], rtol=2.0 ** -8, atol=0)


def test_refusals():
    c = Case(16, [1], [30], 16, 4, 2, 64, 64)
    att = c.make()
    with pytest.raises(ValueError):
        att.forward(c.q, c.cache[:, :1], *c.lens, 1)
    with pytest.raises(ValueError):
        att.forward(c.q, c.cache.view(torch.float16), *c.lens, 1)
    with pytest.raises(rpa.RpaError):
        rpa.RaggedPagedAttention(**dict(c.b.cfg(), kv_dtype="int4_g128"))
    with pytest.raises(rpa.RpaError):
        rpa.CacheEviction(budget=8, **c.b.cfg())
