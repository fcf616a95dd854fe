"""Calls of the long caches' operators as a serving engine makes them: steps in a graph, two handles at once, two graphs of one
handle, a room that only some prompts fit into, unused page ids, slices of a fused projection."""
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


def int4_cache(b, group):
    return i4.random_cache(b.rng, b.N, b.ps, b.Hkv, b.D, group)[0]


@pytest.mark.parametrize("D,group,ps", [(128, 64, 16), (64, 32, 20), (256, 128, 64)])
def test_page_ids_between_are_not_used(D, group, ps):
    """Of the direct kernel and of a prompt's f16 rows, whose 64-key pages reach in front of the window."""
    b = Batch(np.random.default_rng(D), [1, 80, 6], [2000, 1500, 900], ps, 16, 2, D, kv="int4_g%d" % group)
    q, cache = b.queries(), int4_cache(b, group)
    att = rpa.RaggedPagedAttention(**b.cfg(), sliding_window=200, first_keys=20)
    want = att.forward(q, cache, *b.lens(), b.S)
    for s, (a, n) in enumerate(zip(b.q_lens, b.kv_lens_list)):
        lo, hi = -(-20 // ps), (n - a - 200 + 1) // ps  # whole pages that no token sees
        assert hi > lo
        b.table[s, lo:hi] = b.rng.choice([-5, b.N, 1 << 30], hi - lo)
        b.table[s, -(-n // ps):] = -1
    got = att.forward(q, cache, *b.lens(), b.S)
    assert att.status() == rpa.RPA_OK
    assert torch.equal(got, want)


def test_the_widest_window_is_none():
    b = Batch(np.random.default_rng(1), [1, 100, 3], [300, 200, 40], 16, 8, 2, 128, kv="int4_g64")
    q, cache = b.queries(), int4_cache(b, 64)
    want = rpa.RaggedPagedAttention(**b.cfg()).forward(q, cache, *b.lens(), b.S)
    for window in (2 ** 31 - 1, 2 ** 40):
        for first in (0, 5, 2 ** 31 - 1):
            att = rpa.RaggedPagedAttention(**b.cfg(), sliding_window=window, first_keys=first)
            assert torch.equal(att.forward(q, cache, *b.lens(), b.S), want) and att.status() == rpa.RPA_OK


def test_a_room_for_some_prompts():
    """Three prompts of 6000 keys of 64 heads at D 256, two of which fit into 1 GiB of f16 rows: each as in a call of its own, but
    for the third, whose rows the direct kernel takes."""
    H, D, ps, n, a = 64, 256, 64, 6000, 500
    P = -(-n // ps)
    table = torch.from_numpy(np.random.default_rng(2).permutation(3 * P).reshape(3, P).astype(np.int32)).cuda()
    cfg = dict(num_q_heads=H, num_kv_heads=H, head_dim=D, total_num_pages=3 * P, page_size=ps, max_num_seqs=3, pages_per_seq=P,
               kv_dtype="int4_g128", sm_scale=D ** -0.5)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    gen = torch.Generator("cuda").manual_seed(3)
    rope = rpa.RopeAppend(**cfg, num_q_tokens=n)
    cache = torch.zeros((3 * P, H, ps * (D + 16)), dtype=torch.uint8, device="cuda")
    for s in range(3):
        k, v = (torch.randn(n, H, D, device="cuda", generator=gen).bfloat16() for _ in "kv")
        rope.append(k, k, v, cache, i32(n, 0, 0), table[[s, 0, 1]].contiguous(), i32(0, n, n, n), 1)
        assert rope.status() == rpa.RPA_OK
    att = rpa.RaggedPagedAttention(**cfg, num_q_tokens=3 * a)
    q = torch.randn(3 * a, H, D, device="cuda", generator=gen).bfloat16()
    out = att.forward(q, cache, i32(n, n, n), table, i32(0, a, 2 * a, 3 * a), 3)
    assert att.status() == rpa.RPA_OK
    alone = []
    for s in range(3):
        one = att.forward(q, cache, i32(*[n if i == s else 0 for i in range(3)]), table, i32(*[a * min(1, max(0, i - s)) + s * a for i in range(4)]), 3)
        alone.append(one[s * a:(s + 1) * a])
    alone = torch.cat(alone)
    assert torch.equal(out[:2 * a], alone[:2 * a])
    assert not torch.equal(out[2 * a:], alone[2 * a:])
    # both round P (2^-11 of |v| <= 6 at most each) and o (2^-8 of it): over thousands of keys a value is below 1
    assert (out.float() - alone.float()).abs().max() < 2.0 ** -7


def test_handles_on_two_streams():
    """A decoding and a prefilling handle over one 4-bit cache, and one with first keys over a 16-bit cache, at the same time."""
    rng = np.random.default_rng(4)
    dec = Batch(rng, [1] * 8, [3000 + 100 * i for i in range(8)], 16, 16, 4, 128, kv="int4_g64")
    pre = Batch(rng, [300, 200], [3000, 2000], 16, 16, 4, 128, kv="int4_g64")
    win = Batch(rng, [1, 200], [5000, 900], 16, 16, 4, 128)
    cache, wide = int4_cache(dec, 64), win.cache()
    pre.table %= dec.N
    calls = []
    for b, x, more in ((dec, cache, {}), (pre, cache, {}), (win, wide, dict(sliding_window=300, first_keys=7))):
        att = rpa.RaggedPagedAttention(**dict(b.cfg(), total_num_pages=x.shape[0]), **more)
        q, lens = b.queries(), b.lens()
        calls.append((att, q, x, lens, b.S, att.forward(q, x, *lens, b.S)))
        assert att.status() == rpa.RPA_OK
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.empty_like(c[-1]) for _ in range(10)] for c in calls]
    for i in range(10):
        for st, (att, q, x, lens, S, _), o in zip(streams, calls, outs):
            att.forward(q, x, *lens, S, out=o[i], stream=st)
    torch.cuda.synchronize()
    for (att, *_, want), o in zip(calls, outs):
        assert att.status() == rpa.RPA_OK and all(torch.equal(x, want) for x in o)


def test_two_graphs_of_one_handle():
    """Graphs of other lengths share the workspace and its room; replayed in turn they give what eager calls give."""
    b = Batch(np.random.default_rng(5), [1, 150, 20, 1], [900, 700, 600, 2000], 16, 8, 2, 128, kv="int4_g64")
    q, cache = b.queries(), int4_cache(b, 64)
    att = rpa.RaggedPagedAttention(**b.cfg())
    lens = [b.lens(), b.lens()]
    lens[1][0][:4] = torch.tensor([30, 150, 400, 1999], dtype=torch.int32, device="cuda")
    lens[1][1] = lens[1][1].flip(0).contiguous()
    want = [att.forward(q, cache, *x, b.S) for x in lens]
    outs, graphs = [torch.empty_like(w) for w in want], [torch.cuda.CUDAGraph() for _ in want]
    for g, x, o in zip(graphs, lens, outs):
        with torch.cuda.graph(g):
            att.forward(q, cache, *x, b.S, out=o)
    for i in (0, 1, 1, 0, 1, 0, 0):
        outs[i].fill_(3.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])
    assert att.status() == rpa.RPA_OK


def test_slices_of_a_fused_projection():
    b = Batch(np.random.default_rng(6), [70, 1, 3], [70, 300, 50], 16, 8, 2, 128, kv="int4_g64")
    op = rpa.RopeAppend(**b.cfg())
    fused = torch.from_numpy(b.rng.standard_normal((b.T, 12, 128))).cuda().bfloat16()
    parts = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    caches = [torch.full((b.N, 2, 16 * (128 + 16)), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [op.append(*x, c, *b.lens(), b.S) for x, c in zip((parts, [p.contiguous() for p in parts]), caches)]
    assert op.status() == rpa.RPA_OK
    assert torch.equal(*caches) and torch.equal(*outs)


@pytest.mark.parametrize("D,group", [(64, 64), (128, 128), (256, 32)])
def test_steps_of_a_server(D, group):
    """A prompt in two chunks and decode steps, the last ones replays of a graph, with a window and first keys: every step's
    attention against its definition over the rows that the cache holds."""
    H, Hq, ps, n0 = 2, 8, 16, 150
    rng = np.random.default_rng(D)
    gen = torch.Generator("cuda").manual_seed(D)
    cfg = dict(num_q_heads=Hq, num_kv_heads=H, head_dim=D, total_num_pages=40, page_size=ps, max_num_seqs=2, pages_per_seq=16, kv_dtype="int4_g%d" % group,
               q_dtype="f16", sm_scale=D ** -0.5)
    mask = dict(sliding_window=60, first_keys=4)
    table = torch.from_numpy(rng.permutation(40)[:32].reshape(2, 16).astype(np.int32)).cuda()
    cache = torch.full((40, H, ps * (D + 8 * D // group)), 0xff, dtype=torch.uint8, device="cuda")
    new = lambda t, h: torch.randn(t, h, D, device="cuda", generator=gen).half()  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    whole = rpa.RopeAppend(**dict(cfg, num_q_tokens=400, q_dtype="f32"))

    def check(qr, out, kl, ql):
        total = [0, kl[0], kl[0] + kl[1]]
        rows = [f64(x) for x in whole.read(cache, i32(*kl), table, i32(*total), 2)]
        assert whole.status() == rpa.RPA_OK
        cu = [0, ql[0], ql[0] + ql[1]]
        ref, size = attend64(f64(qr), ql, kl, cu, lambda s: [x[total[s]:total[s + 1]] for x in rows], window=60, first=4)
        # logits: q, K are f16 here, K of a prompt rounded to it (16 half steps: |q k| / sqrt(D) summed is below 16); P, V and o
        # a half step each (P's meets codes up to 8 from the middle, below 2 |v|'s size with the others)
        h = half_step("f16")
        err = np.abs(f64(out) - ref) - (h * np.abs(ref) + (2 * 16 * h + 8 * h + 2.0 ** -13) * (size + 1.0))
        assert err.max() <= 0, err.max()

    kl = [0, 0]
    for ql in ([n0, 20], [1, 90], [30, 1]):
        kl = [x + y for x, y in zip(kl, ql)]
        T = sum(ql)
        rope, att = rpa.RopeAppend(**cfg, num_q_tokens=T), rpa.RaggedPagedAttention(**cfg, **mask, num_q_tokens=T)
        lens, cu = i32(*kl), i32(0, ql[0], T)
        qr = rope.append(new(T, Hq), new(T, H), new(T, H), cache, lens, table, cu, 2)
        out = att.forward(qr, cache, lens, table, cu, 2)
        assert rope.status() == rpa.RPA_OK and att.status() == rpa.RPA_OK
        check(qr, out, kl, ql)
    # decode steps; the lengths are device tensors that the graph's replays read
    rope, att = rpa.RopeAppend(**cfg, num_q_tokens=2), rpa.RaggedPagedAttention(**cfg, **mask, num_q_tokens=2)
    q, k, v, qr, out = new(2, Hq), new(2, H), new(2, H), new(2, Hq), new(2, Hq)
    lens, cu, g = i32(*kl), i32(0, 1, 2), None

    def step():
        rope.append(q, k, v, cache, lens, table, cu, 2, q_out=qr)
        att.forward(qr, cache, lens, table, cu, 2, out=out)

    for i in range(6):
        kl = [x + 1 for x in kl]
        for dst, h in ((q, Hq), (k, H), (v, H)):
            dst.copy_(new(2, h))
        lens.copy_(i32(*kl))
        if i < 2:
            step()
        else:
            if g is None:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step()
            g.replay()
        assert rope.status() == rpa.RPA_OK and att.status() == rpa.RPA_OK
        check(qr, out, kl, [1, 1])


@pytest.mark.parametrize("q_lens,unfolded", [([113], 1), ([112], 0), ([79, 17, 17], 1), ([78, 17, 17], 0), ([62, 17, 17, 17], 0)])
def test_tokens_that_make_room(q_lens, unfolded):
    """The fewest tokens of which a sequence is computed from f16 rows (4 kv heads of 4 query heads: 113), and calls of fewer, for
    which a handle has no room: each against the definition."""
    from test_int4_attention_gpu import Case

    c = Case(len(q_lens), q_lens, [300 + 10 * n for n in q_lens], 16, 16, 4, 64, 32, "f16", lead=0, tail=0, spare_seqs=0)
    kept = []
    c.check(call=lambda att, out: kept.append((att, att.forward(c.q, c.cache, *c.lens, c.b.S, out=out))))
    att = kept[0][0]
    assert att.status() == rpa.RPA_OK
    info, items = att.plan()
    assert len({int(i[0]) for i in items[info[1]:]}) == unfolded


def test_pages_past_four_gigabytes():
    """The same calls over pages at the start and at the end of a cache of 5 GB, where byte offsets need more than 32 bits."""
    b = Batch(np.random.default_rng(7), [1, 150, 3], [900, 600, 70], 64, 16, 8, 128, kv="int4_g128")
    N = 72000
    q, k, v = b.queries(), *(b.queries()[:, :8].contiguous() for _ in "kv")
    big = torch.full((N, 8, 64 * (128 + 8)), 0x35, dtype=torch.uint8, device="cuda")
    assert big.numel() > 2 ** 32 + 2 ** 29
    cfg = dict(b.cfg(), total_num_pages=N)
    rope, att = rpa.RopeAppend(**cfg), rpa.RaggedPagedAttention(**cfg, sliding_window=300, first_keys=10)
    lens, table, cu = b.lens()
    got = []
    for at in (0, N - b.N):
        t = table + at
        big[at:at + b.N] = 0x35
        qr = rope.append(q, k, v, big, lens, t, cu, b.S)
        got.append((qr, att.forward(qr, big, lens, t, cu, b.S), *rope.read(big, lens, t, cu, b.S), big[at:at + b.N].clone()))
        assert rope.status() == rpa.RPA_OK and att.status() == rpa.RPA_OK
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("kv,q_lens", [("int4_g64", [1, 120, 1, 7]), ("int4_g64", [1, 1, 1, 1]), ("fp8_e4m3", [1, 120, 1, 7])])
def test_options_and_profile(kv, q_lens):
    """Fewer CTAs than the chip has, one after the other, and with the kernels timed: the same results, but for where keys are cut."""
    eight = dict(k_scale=0.05, v_scale=0.05) if kv == "fp8_e4m3" else {}
    b = Batch(np.random.default_rng(8), q_lens, [2000, 900, 3, 1500], 16, 16, 4, 128, kv=kv, **eight)
    cache = b.cache() if eight else int4_cache(b, 64)
    q, lens = b.queries(), b.lens()
    make = lambda: rpa.RaggedPagedAttention(**b.cfg(), sliding_window=800, first_keys=9)  # noqa: E731
    want = make().forward(q, cache, *lens, b.S)
    for options in ({rpa.RPA_OPT_DECODE_SMS: 3}, {rpa.RPA_OPT_PREFILL_SMS: 5, rpa.RPA_OPT_DECODE_SMS: 1}, {rpa.RPA_OPT_SERIAL: 1}, {rpa.RPA_OPT_PLAN_EARLY: 1}):
        att = make()
        for o, x in options.items():
            att.set_option(o, x)
        for _ in range(3):
            got = att.forward(q, cache, *lens, b.S)
            # P and o are rounded (2^-11 and 2^-8 of values below 4), at other running maxima where the cuts are others
            assert att.status() == rpa.RPA_OK and (got.float() - want.float()).abs().max() <= 2.0 ** -5
    att = make()
    att.profile_begin(4)
    for _ in range(4):
        got = att.forward(q, cache, *lens, b.S)
    ms = att.profile_read(4)
    assert att.status() == rpa.RPA_OK and torch.equal(got, want)
    assert np.isfinite(ms).all() and (np.asarray(ms) >= 0).all()
