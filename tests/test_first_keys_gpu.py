"""A sliding window in front of which the first keys stay visible, against its definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch, f64, half_step  # noqa: E402
from long_cache_util import attend64, cached_rows  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def tolerance(b, ref, size, cap):
    """P is rounded to the products' type, o to its own.  A logit is off by the rounding of q where its type is not the
    products' (|q k| / sqrt(D) summed is below 16 for these inputs: 16 half steps), by 32-bit sums (2^-18 at that size), and with
    a cap by tanh's approximation (2^-11 of at most the cap); an error e of the logits moves o by at most 2 e size."""
    prod = "bf16" if b.kv == "bf16" else "f16"
    e = 2.0 ** -18 + (0 if b.q == prod or (b.q == "bf16" and prod == "f16") else 16 * half_step(prod)) + (cap or 0) * 2.0 ** -11
    return half_step(b.q) * np.abs(ref) + (half_step(prod) + 2 * e) * size + 1e-6


def check(b, window, first, cap=None, sinks=None, causal=True, q=None, cache=None, call=None):
    q = b.queries() if q is None else q
    cache = b.cache() if cache is None else cache
    lens, table, cu = b.lens()
    cfg = dict(b.cfg(), sliding_window=window, first_keys=first, soft_cap=cap, is_causal=causal, sinks=sinks)
    att = rpa.RaggedPagedAttention(**cfg)
    out = torch.full((b.T, b.Hq, att.out_dim), 7.0, dtype=q.dtype, device="cuda")
    if call is None:
        att.forward(q, cache, lens, table, cu, b.S, out=out)
        assert att.status() == rpa.RPA_OK
    else:
        call(att, q, cache, lens, table, cu, out)
    vals = cache if b.kv not in ("fp8_e4m3", "fp8_e5m2") else cache
    ref, size = attend64(f64(q), b.q_lens, b.kv_lens_list, b.cu, cached_rows(b, f64(vals), b.k_scale or 1.0, b.latent), window=window,
                         first=first, cap=cap, causal=causal, sinks=sinks, Dv=att.out_dim)
    got = f64(out)
    assert np.isfinite(got).all()
    err = np.abs(got - ref) - tolerance(b, ref, size, cap)
    assert err.max() <= 0, (err.max(), np.unravel_index(err.argmax(), err.shape))
    return out


EIGHT = dict(k_scale=0.05, v_scale=0.05)


@pytest.mark.parametrize("Hq,Hkv,D,ps,kv,q", [
    (8, 2, 128, 16, "bf16", "bf16"),    # 8-row decode tiles, 128-key prefill tiles
    (16, 1, 64, 4, "f16", "f16"),       # 16-row tiles, short page runs
    (6, 2, 128, 20, "bf16", "f32"),     # page size not a power of two
    (8, 2, 256, 64, "bf16", "bf16"),    # 64-key tiles copied whole
    (4, 1, 256, 16, "f16", "f16"),      # ... by page runs
    (8, 2, 128, 16, "fp8_e4m3", "bf16"),
    (16, 4, 64, 32, "int8", "f16"),
])
@pytest.mark.parametrize("window,first", [(100, 4), (7, 70), (1, 1), (333, 64), (50, 200), (1000, 16), (64, 129)])
def test_decode_and_prompt(Hq, Hkv, D, ps, kv, q, window, first):
    rng = np.random.default_rng([Hq, D, window, first])
    b = Batch(rng, [1, 1, 150, 1, 33, 2, 1, 70], [900, 1, 700, window + first, 33, 5, window + 1, 600], ps, Hq, Hkv, D, kv=kv, q=q, lead=2, tail=3,
              **(EIGHT if kv in ("fp8_e4m3", "int8") else {}))
    check(b, window, first)


def test_latent():
    b = Batch(np.random.default_rng(5), [1, 20, 1, 3], [800, 500, 64, 900], 16, 16, 1, 576, latent=True)
    check(b, 90, 33)
    b = Batch(np.random.default_rng(6), [1, 9], [5000, 300], 64, 32, 1, 576, latent=True, kv="f16", q="f16")
    check(b, 2000, 4)


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("fp8_e4m3", 128), ("bf16", 256)])
def test_knobs(kv, D):
    """Soft cap, sinks, and a window without causality."""
    rng = np.random.default_rng(9)
    b = Batch(rng, [1, 60, 3], [700, 400, 90], 16, 8, 2, D, kv=kv, **(EIGHT if kv == "fp8_e4m3" else {}))
    check(b, 80, 10, cap=20.0)
    sinks = rng.standard_normal(8).astype(np.float32)
    check(b, 80, 10, sinks=sinks)
    check(b, 80, 10, causal=False)


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("fp8_e4m3", 128), ("bf16", 256)])
@pytest.mark.parametrize("first", [4, 600, 1500])
def test_split_decodes(kv, D, first):
    """Long bands cut into pieces, whose first has the first keys too (also where they outnumber a piece's keys)."""
    b = Batch(np.random.default_rng(first), [1, 1, 2], [9000, 30000, 12000], 16, 4, 2, D, kv=kv, **(EIGHT if kv == "fp8_e4m3" else {}))
    check(b, 7000, first)


def test_pages_between_are_not_used():
    """Page ids and rows behind the first keys and in front of the window may be anything."""
    b = Batch(np.random.default_rng(3), [1, 40], [2000, 1500], 16, 8, 2, 128)
    q, cache = b.queries(), b.cache()
    want = check(b, 200, 20, q=q, cache=cache).clone()
    for s, (n, a) in enumerate(((2000, 1), (1500, 40))):
        lo, hi = 2, (n - a - 200 + 1) // 16  # whole pages that no token sees
        cache[torch.from_numpy(b.table[s, lo:hi].astype(np.int64)).cuda()] = float("nan")
        b.table[s, lo:hi] = -5
    lens, table, cu = b.lens()
    att = rpa.RaggedPagedAttention(**dict(b.cfg(), sliding_window=200, first_keys=20))
    got = att.forward(q, cache, lens, table, cu, b.S)
    assert att.status() == rpa.RPA_OK
    assert torch.equal(got[:41], want[:41])


def test_more_first_keys_than_keys_is_no_window():
    b = Batch(np.random.default_rng(4), [1, 50, 1], [300, 200, 40], 16, 8, 2, 128)
    q, cache = b.queries(), b.cache()
    lens, table, cu = b.lens()
    a = rpa.RaggedPagedAttention(**dict(b.cfg(), sliding_window=10, first_keys=2 ** 31 - 1)).forward(q, cache, lens, table, cu, b.S)
    c = rpa.RaggedPagedAttention(**b.cfg()).forward(q, cache, lens, table, cu, b.S)
    assert torch.equal(a, c)


def test_host_no_alloc_and_graph():
    import ctypes

    b = Batch(np.random.default_rng(8), [1, 30, 2], [900, 300, 1200], 16, 8, 2, 128)

    def host(att, q, cache, lens, table, cu, out):
        o = torch.empty(out.shape, dtype=out.dtype).pin_memory()
        att.forward_host(q.cpu().pin_memory(), cache, lens.cpu(), table.cpu(), cu.cpu(), b.S, o)
        torch.cuda.synchronize()
        out.copy_(o)

    def no_alloc(att, q, cache, lens, table, cu, out):
        r = rpa.lib().rpa_forward_noalloc(ctypes.byref(att._c), q.data_ptr(), cache.data_ptr(), lens.data_ptr(), table.data_ptr(), cu.data_ptr(),
                                          b.S, out.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert r == rpa.RPA_OK

    def graph(att, q, cache, lens, table, cu, out):
        att.forward(q, cache, lens, table, cu, b.S, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            att.forward(q, cache, lens, table, cu, b.S, out=out)
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()

    q, cache = b.queries(), b.cache()
    outs = [check(b, 100, 20, q=q, cache=cache, call=c) for c in (None, host, no_alloc, graph)]
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("fp8_e4m3", 64), ("bf16", 256), ("int4_g64", 128), ("int4_g128", 256)])
@pytest.mark.parametrize("window,first", [(700, 4), (3000, 900), (5000, 64), (64, 0)])
def test_the_plan_covers_what_is_seen(kv, D, window, first):
    """Every (sequence, kv head, token, key) that is seen lies in one item, and items keep to the band and the first keys."""
    eight = EIGHT if kv == "fp8_e4m3" else {}
    b = Batch(np.random.default_rng(window + first), [1, 1, 120, 3, 700], [9000, 100, 2000, 6000, 900], 16, 8, 2, D, kv=kv, **eight)
    q = torch.zeros((b.T, 8, D), dtype=torch.bfloat16, device="cuda")
    cfg = dict(b.cfg(), sliding_window=window, first_keys=first)
    att = rpa.RaggedPagedAttention(**cfg)
    from ragged_paged_attention_02_gb300.binding import cache_shape

    cache = torch.zeros(cache_shape(att._c), dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    att.forward(q, cache, *b.lens(), b.S)
    assert att.status() == rpa.RPA_OK
    info, items = att.plan()
    count = [[np.zeros((a, n), int) for a, n in zip(b.q_lens, b.kv_lens_list)] for _ in range(2)]
    for s, head, t0, nt, lo, hi, part, piece in items:
        n, a = b.kv_lens_list[s], b.q_lens[s]
        p_lo = n - a + t0
        assert 0 <= lo <= hi <= n
        count[head][s][t0:t0 + nt, lo:hi] += 1
        if first and piece == 0 and lo > first:
            count[head][s][t0:t0 + nt, :first] += 1
            assert p_lo - window + 1 > first or lo > first
    for head in range(2):
        for s, (a, n) in enumerate(zip(b.q_lens, b.kv_lens_list)):
            pos, j = np.arange(n - a, n)[:, None], np.arange(n)[None]
            sees = (j <= pos) & ((j > pos - window) | (j < first))
            assert (count[head][s][sees] == 1).all()
