"""Eviction on the GPU against its definition in 64 bits.

Weights.  A weight is 2^(x - M) / L with x in 32 bits.  Its relative error is at most the absolute error of
x - M times ln 2 plus that of the exponential (2^-22), of L (as the weights) and of the sums.  x itself is a
32-bit sum of D exact products: the tensor core adds them in its own order and cuts instead of rounding, so
that each of the D / 16 steps loses up to 2^-22 of the largest partial sum, at most |q| |k|; the scale rounds
twice more.  With |q||k| sm_scale <= B this is 2 ln 2 log2(e) B (D / 16 + 2) 2^-22 for x - M, doubled for L:
4 B (D / 16 + 2) 2^-22, and 2^-20 for the rest.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch, f64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


# ---------------------------------------------------------------- weights
def weights(b, q, cache, s, h):
    """(weights [keys] of kv head h of sequence s summed over its rows, the largest |q| |k| sm_scale)"""
    c = b.cfg()
    n, kl = b.q_lens[s], b.kv_lens_list[s]
    G = b.Hq // b.Hkv
    j = np.arange(kl)
    page, at = b.slots(s, j)
    K = cache[page, at, 2 * h] * (b.k_scale or 1.0)  # [keys, D]
    Q = q[b.cu[s]:b.cu[s] + n, h * G:(h + 1) * G]
    x = np.einsum("igd,kd->igk", Q, K) * c["sm_scale"]
    B = np.linalg.norm(Q, axis=-1).max(initial=0) * np.linalg.norm(K, axis=-1).max(initial=0) * c["sm_scale"]
    if c.get("soft_cap"):
        x = c["soft_cap"] * np.tanh(x / c["soft_cap"])
    pos = np.arange(kl - n, kl)[:, None, None]
    sees = np.ones_like(x, bool)
    if c.get("is_causal", True):
        sees &= j <= pos
    if c.get("sliding_window"):
        sees &= j > pos - c["sliding_window"]
    x = np.where(sees, x, -np.inf)
    m = x.max(-1, keepdims=True)
    if c.get("sinks") is not None:
        m = np.maximum(m, c["sinks"][h * G:(h + 1) * G][None, :, None])
    p = np.exp(x - m)
    L = p.sum(-1, keepdims=True)
    if c.get("sinks") is not None:
        L = L + np.exp(c["sinks"][h * G:(h + 1) * G][None, :, None] - m)
    return (p / L).sum((0, 1)), B


def run_and_check(b, scores=None):
    q, cache = b.queries(), b.cache()
    c = b.cfg()
    op = rpa.CacheEviction(budget=1, **c)
    if scores is None:
        scores = torch.from_numpy(b.rng.random((b.N, b.Hkv, b.ps), np.float32) * 0.1).cuda()
    before = f64(scores)
    op.accumulate(q, cache, *b.lens(), b.S, scores)
    assert op.status() == rpa.RPA_OK
    got, qd = f64(scores), f64(q)
    kd = f64(cache) if cache.element_size() > 1 or b.kv == "int8" else cache.float().cpu().double().numpy()
    untouched = np.ones(got.shape, bool)
    for s in range(b.S):
        if b.q_lens[s] == 0:
            continue
        j = np.arange(b.kv_lens_list[s])
        page, at = b.slots(s, j)
        for h in range(b.Hkv):
            w, B = weights(b, qd, kd, s, h)
            old = np.where(j < b.kv_lens_list[s] - b.q_lens[s], before[page, h, at], 0.0)
            rel = 4 * B * (b.D / 16 + 2) * 2.0 ** -22 + 2.0 ** -20
            if c.get("soft_cap"):
                rel += 4 * c["soft_cap"] * 2.0 ** -22  # tanh and the cap's product
            err = np.abs(got[page, h, at] - (old + w))
            assert (err <= rel * w + 2.0 ** -23 * (old + w)).all(), (s, h, (err / (w + 1e-30)).max(), rel)
            untouched[page, h, at] = False
    assert (got[untouched] == before[untouched]).all()
    return op, q, cache, scores


WEIGH = [
    (0, dict(Hq=4, Hkv=4, D=64), [1], [1]),                                    # one token, one key
    (1, dict(Hq=32, Hkv=8, D=128), [1] * 7, [1, 15, 16, 17, 400, 2000, 129]),  # decode
    (2, dict(Hq=2, Hkv=2, D=256), [1, 1, 0, 2], [90, 1500, 30, 7]),            # one head a group: 8-byte padded logits
    (3, dict(Hq=6, Hkv=2, D=64), [5, 1, 0, 3], [5, 200, 0, 800]),              # 15, 3 and 9 rows
    (4, dict(Hq=16, Hkv=1, D=128), [1, 1], [3000, 33]),                        # 16 rows
    (5, dict(Hq=10, Hkv=2, D=128), [40, 70, 4, 3], [40, 300, 1000, 3]),        # several blocks beside one
    (6, dict(Hq=64, Hkv=1, D=64), [9, 1], [700, 64]),
    (7, dict(Hq=8, Hkv=2, D=256, sliding_window=100), [1, 37, 3], [1000, 400, 50]),
    (8, dict(Hq=8, Hkv=2, D=128, sliding_window=1), [1, 20, 5], [300, 60, 5]),
    (9, dict(Hq=8, Hkv=2, D=128, soft_cap=3.0, is_causal=False), [2, 30], [500, 90]),
    (10, dict(Hq=4, Hkv=1, D=64, is_causal=False, sliding_window=64), [4, 50], [500, 300]),
]


@pytest.mark.parametrize("seed,shape,q_lens,kv_lens", WEIGH)
@pytest.mark.parametrize("q,kv,ps", [("bf16", "bf16", 16), ("f16", "f16", 4), ("bf16", "fp8_e4m3", 12), ("f16", "int8", 64), ("f16", "fp8_e5m2", 20)])
def test_accumulate(seed, shape, q_lens, kv_lens, q, kv, ps):
    scale = {"fp8_e4m3": 0.05, "fp8_e5m2": 0.05, "int8": 0.04}.get(kv)
    b = Batch(np.random.default_rng(seed), q_lens, kv_lens, ps, kv=kv, q=q, k_scale=scale, v_scale=scale, lead=seed % 2 * 2, tail=seed % 3, **shape)
    run_and_check(b)


def test_rounded_queries():
    """q of another type is rounded to the operands' type, as the attention does: the same scores as from that q."""
    rng = np.random.default_rng(20)
    for q, kv in (("f32", "bf16"), ("f32", "f16"), ("f16", "bf16"), ("bf16", "f16"), ("f32", "fp8_e4m3")):
        b = Batch(rng, [1, 20], [90, 40], 16, 8, 2, 64, kv=kv, q=q)
        x, cache, lens = b.queries(), b.cache(), b.lens()
        to = torch.bfloat16 if kv == "bf16" else torch.float16
        b2 = dict(b.cfg(), q_dtype="bf16" if kv == "bf16" else "f16")
        scores = [torch.zeros(b.N, b.Hkv, b.ps, device="cuda") for _ in range(2)]
        rpa.CacheEviction(budget=1, **b.cfg()).accumulate(x, cache, *lens, b.S, scores[0])
        rpa.CacheEviction(budget=1, **b2).accumulate(x.to(to), cache, *lens, b.S, scores[1])
        assert torch.equal(*scores), (q, kv)


def test_sinks():
    rng = np.random.default_rng(21)
    b = Batch(rng, [1, 12], [200, 60], 16, 8, 2, 64, sinks=(rng.standard_normal(8) * 2).astype(np.float32))
    run_and_check(b)


def test_garbage_behind_the_keys_is_not_seen():
    rng = np.random.default_rng(22)
    b = Batch(rng, [1, 20], [37, 45], 16, 8, 2, 64)
    q, cache, lens = b.queries(), b.cache(), b.lens()
    op = rpa.CacheEviction(budget=1, **b.cfg())
    a = op.accumulate(q, cache, *lens, b.S, torch.zeros(b.N, 2, 16, device="cuda"))
    dirty = torch.full_like(cache, float("nan"))
    for s in range(b.S):
        page, at = (torch.as_tensor(x).long().cuda() for x in b.slots(s, np.arange(b.kv_lens_list[s])))
        dirty[page, at] = cache[page, at]
        dirty[page, at, 1::2] = float("inf")  # V is not read
    c = op.accumulate(q, dirty, *lens, b.S, torch.zeros(b.N, 2, 16, device="cuda"))
    assert torch.equal(a, c) and op.status() == rpa.RPA_OK


def test_infinite_and_hidden_logits():
    """Keys whose logit is minus infinity weigh nothing; a row that sees only such keys gives nothing."""
    b = Batch(np.random.default_rng(23), [1], [40], 16, 2, 2, 64)
    q, cache = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(b.N, 16, 4, 64, dtype=torch.bfloat16, device="cuda")
    page, at = (torch.as_tensor(x).long().cuda() for x in b.slots(0, np.arange(40)))
    cache[page[:39], at[:39], 0, 5] = -float("inf")
    cache[page, at, 2, 5] = -float("inf")
    scores = torch.full((b.N, 2, 16), 0.25, device="cuda")
    op = rpa.CacheEviction(budget=1, **b.cfg())
    op.accumulate(q, cache, *b.lens(), 1, scores)
    got = scores[page, :, at]
    assert (got[:39, 0] == 0.25).all() and abs(got[39, 0].item() - 1) < 1e-6
    assert (got[:39, 1] == 0.25).all() and got[39, 1] == 0


def test_bad_lengths_and_pages():
    rng = np.random.default_rng(24)
    b = Batch(rng, [1, 2], [50, 30], 8, 4, 2, 64)
    q, cache = b.queries(), b.cache()
    kvl, table, cu = b.lens()
    op = rpa.CacheEviction(budget=1, **b.cfg())
    for bad in range(3):
        k2, c2 = kvl.clone(), cu.clone()
        if bad == 0:
            k2[0] = b.P * b.ps + 1
        elif bad == 1:
            k2[1] = 1
        else:
            c2[1] = -1
        scores = torch.rand(b.N, 2, 8, device="cuda")
        was = scores.clone()
        op.accumulate(q, cache, k2, table, c2, b.S, scores)
        assert op.status() == rpa.RPA_ERR_BAD_LENGTHS and torch.equal(scores, was)
    # a bad page: its keys are not in the softmax, the others' weights add up to the rows
    for value in (-1, b.N):
        t = table.clone()
        t[0, 2] = value
        scores = torch.zeros(b.N, 2, 8, device="cuda")
        op.accumulate(q, cache, kvl, t, cu, b.S, scores)
        assert op.status() == rpa.RPA_ERR_BAD_PAGE_INDEX and op.status() == rpa.RPA_OK
        page = torch.as_tensor(b.table[0, :7]).long().cuda()
        assert scores[page[2]].abs().sum() == 0
        assert abs(scores[page].sum().item() - 4) < 1e-4 and torch.isfinite(scores).all()
    with pytest.raises(rpa.RpaError):
        op.accumulate(q, cache, kvl, table, cu, b.max_seqs + 1, torch.zeros(b.N, 2, 8, device="cuda"))
    scores = torch.rand(b.N, 2, 8, device="cuda")
    was = scores.clone()
    op.accumulate(q, cache, kvl, table, cu, 0, scores)
    assert op.status() == rpa.RPA_OK and torch.equal(scores, was)


def test_shared_pages_and_repeats():
    """Sequences that share their first pages both add to them; the same call twice gives the same bits."""
    rng = np.random.default_rng(25)
    b = Batch(rng, [1] * 6, [70, 80, 64, 65, 100, 77], 16, 8, 2, 128)
    b.table[:6, :4] = b.table[0, :4]
    q, cache, lens = b.queries(), b.cache(), b.lens()
    op = rpa.CacheEviction(budget=1, **b.cfg())
    z = lambda: torch.zeros(b.N, 2, 16, device="cuda")  # noqa: E731
    got, kd = f64(op.accumulate(q, cache, *lens, b.S, z())), f64(cache)
    want = np.zeros_like(got)
    for s in range(6):
        page, at = b.slots(s, np.arange(b.kv_lens_list[s]))
        for h in range(2):
            want[page, h, at] += weights(b, f64(q), kd, s, h)[0]
    # the last key of the third sequence (64 keys) is its own token: on a shared page, which a caller does not do
    page, at = b.slots(2, [63])
    got[page, :, at] = want[page, :, at] = 0
    assert (np.abs(got - want) <= 1e-4 * want).all()
    b = Batch(rng, [1, 40, 3], [700, 80, 640], 16, 8, 2, 128)
    q, cache, lens = b.queries(), b.cache(), b.lens()
    op = rpa.CacheEviction(budget=1, **b.cfg())
    one = op.accumulate(q, cache, *lens, b.S, torch.zeros(b.N, 2, 16, device="cuda"))
    for _ in range(5):
        assert torch.equal(one, op.accumulate(q, cache, *lens, b.S, torch.zeros(b.N, 2, 16, device="cuda")))


def test_logits_past_the_workspace_are_computed_again():
    """Long sequences over few pages: 64 x 8 heads x 16 rows x 40 k keys are more logits than the workspace keeps."""
    rng = np.random.default_rng(26)
    S, n, ps, N = 64, 40000, 64, 640
    b = Batch(rng, [1], [n], ps, 128, 8, 64, spare_pages=15, spare_seqs=S - 1)
    b.S, b.q_lens, b.kv_lens_list, b.T = S, [1] * S, [n - 3 * s for s in range(S)], S
    b.cu = np.arange(S + 1, dtype=np.int32)
    b.kv_lens = np.array(b.kv_lens_list, np.int32)
    b.table[:] = b.table[0]
    q, cache = b.queries(), b.cache()
    # one sequence's call alone keeps its logits; the sum of such calls is the whole call's
    op = rpa.CacheEviction(budget=1, **b.cfg())
    kvl, table, cu = b.lens()
    got = op.accumulate(q, cache, kvl, table, cu, S, torch.zeros(b.N, 8, ps, device="cuda")).double()
    assert op.status() == rpa.RPA_OK
    page, at = (torch.as_tensor(x).long().cuda() for x in b.slots(0, np.arange(n)))
    K = cache[page, at, 0::2].double()  # [keys, 8, 64]
    want = torch.zeros(n, 8, dtype=torch.float64, device="cuda")
    for s in range(S):
        m = b.kv_lens_list[s]
        x = torch.einsum("hgd,khd->hgk", q[s].double().view(8, 16, 64), K[:m]) / 8.0
        want[:m] += torch.softmax(x, -1).sum(1).t()
    # a sequence's own last key overwrites what the others gave it: left out
    own = sorted({b.kv_lens_list[s] - 1 for s in range(S)})
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[own] = False
    err = (got[page, :, at] - want)[keep].abs()
    # |q| |k| / 8 <= 18 and D = 64: as above, plus the sum of 64 additions in any order
    assert (err <= (4 * 18 * 6 * 2.0 ** -22 + 2.0 ** -20 + 64 * 2.0 ** -24) * want[keep]).all()


def test_accumulate_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(27)
    b = Batch(rng, [1, 30, 2], [400, 64, 90], 16, 8, 2, 128)
    q, cache, lens = b.queries(), b.cache(), b.lens()
    op = rpa.CacheEviction(budget=1, **b.cfg())
    want = op.accumulate(q, cache, *lens, b.S, torch.zeros(b.N, 2, 16, device="cuda"))
    side, scores = torch.cuda.Stream(), torch.zeros(b.N, 2, 16, device="cuda")
    torch.cuda.synchronize()
    op.accumulate(q, cache, *lens, b.S, scores, stream=side)
    side.synchronize()
    assert torch.equal(scores, want)
    g = torch.cuda.CUDAGraph()
    scores.zero_()
    with torch.cuda.graph(g):
        op.accumulate(q, cache, *lens, b.S, scores)
    for lens2 in ([400, 64, 90], [300, 50, 9]):
        lens[0][:3] = torch.tensor(lens2, dtype=torch.int32)
        scores.zero_()
        g.replay()
        other = op.accumulate(q, cache, *lens, b.S, torch.zeros(b.N, 2, 16, device="cuda"))
        assert torch.equal(scores, other)


def test_many_sequences():
    rng = np.random.default_rng(28)
    q_lens = [int(x) for x in rng.choice([0, 1, 1, 2, 9], 1100)]
    b = Batch(rng, q_lens, [n + int(x) for n, x in zip(q_lens, rng.integers(0, 60, 1100))], 8, 4, 2, 64)
    run_and_check(b)


def test_long_rows_beside_short_ones():
    """Hundreds of rows of a prompt, whose logits are computed again, beside decodes, whose logits are kept, windowed
    or not; two sequences of different kinds in every order."""
    for seed, q_lens, kv_lens, more in ((29, [1, 150, 1], [3000, 150, 20], {}), (30, [150, 1], [1500, 2500], {}),
                                        (31, [130, 1, 16], [400, 1900, 16], dict(sliding_window=200))):
        run_and_check(Batch(np.random.default_rng(seed), q_lens, kv_lens, 16, 8, 2, 64, **more))


@pytest.mark.parametrize("keys", [1300, 2700, 5300])
def test_many_heads(keys):
    """Enough keys and heads that a warp adds the weights of 2, 4 or 8 heads of 61, for whole and partial quads of keys."""
    for seed, shape in ((47, dict(Hq=61, Hkv=61)), (48, dict(Hq=122, Hkv=61, sliding_window=keys - 70))):
        rng = np.random.default_rng(seed)
        run_and_check(Batch(rng, [1, 3, 1, 2, 0], [keys, keys + 1, keys - 3, keys + 130, keys], 16, D=64, **shape))


def test_unaligned_scores_are_refused():
    b = Batch(np.random.default_rng(32), [1], [20], 16, 2, 2, 64)
    op = rpa.CacheEviction(budget=4, **b.cfg())
    scores = torch.zeros(b.N * 2 * 16 + 1, device="cuda")[1:].view(b.N, 2, 16)
    with pytest.raises(rpa.RpaError):
        op.accumulate(b.queries(), b.cache(), *b.lens(), 1, scores)
    with pytest.raises(rpa.RpaError):
        op.compact(b.cache(), scores, *b.lens()[:2], 1)


# ---------------------------------------------------------------- compaction
def kept_slots(x, n, budget, protect, recent):
    """The definition: x [n] scores -> kept slots in order."""
    if n <= budget:
        return np.arange(n)
    middle = np.arange(protect, n - recent)
    key = np.where(np.isnan(x[middle]), -np.inf, x[middle].astype(np.float64))
    rank = np.lexsort((middle, -key, np.isnan(x[middle])))  # numbers before NaN, then the score, then the slot
    best = np.sort(middle[rank[:budget - protect - recent]])
    return np.concatenate((np.arange(protect), best, np.arange(n - recent, n)))


def check_compact(b, budget, protect=0, recent=0, scores=None, mode="fresh", stream=None, bad_free=0):
    """mode: "fresh" pages, "place" (the same table), "equal" (a copy of it), "mixed" (the protected whole pages stay)."""
    rng = b.rng
    cache, lens = b.cache(), b.lens()
    if scores is None:
        scores = np.exp(rng.standard_normal((b.N, b.Hkv, b.ps)) * 2).astype(np.float32)
    sc = torch.from_numpy(scores.copy()).cuda()
    raw = (lambda t: t.view(torch.uint8).cpu().numpy() if t.element_size() == 1 else t.view(torch.int16).cpu().numpy())  # noqa: E731
    before = raw(cache).copy()
    new = b.table.copy()
    if mode in ("fresh", "mixed"):
        at = 0
        for s in range(b.S):
            pages = -(-min(budget, b.kv_lens_list[s]) // b.ps)
            first = protect // b.ps if mode == "mixed" else 0
            for i in range(first, pages):
                new[s, i] = b.free_pages[at]
                at += 1
    table2 = lens[1] if mode == "place" else torch.from_numpy(new).cuda()
    kept = torch.full((b.max_seqs, b.Hkv, budget), 77, dtype=torch.int32, device="cuda")
    out_lens = torch.full((b.max_seqs,), 55, dtype=torch.int32, device="cuda")
    op = rpa.CacheEviction(budget=budget, protect=protect, recent=recent, **b.cfg())
    torch.cuda.synchronize()
    op.compact(cache, sc, lens[0], lens[1], b.S, table2, out_lens, kept=kept, stream=stream)
    assert op.status(stream) == rpa.RPA_OK
    torch.cuda.synchronize()
    want, want_sc = before.copy(), scores.copy()
    # in place the kept rows land on slots that are read by none after them: the definition reads all, then writes
    for s in range(b.S):
        n = b.kv_lens_list[s]
        for h in range(b.Hkv):
            p0, a0 = b.slots(s, np.arange(n))
            idx = kept_slots(scores[p0, h, a0], n, budget, protect, recent)
            got = kept[s, h].cpu().numpy()
            assert (got[:len(idx)] == idx).all() and (got[len(idx):] == -1).all(), (s, h)
            i = np.arange(len(idx))
            pa, aa = b.slots(s, idx)
            pb, ab = new[s, i // b.ps], i % b.ps
            want[pb, ab, 2 * h:2 * h + 2] = before[pa, aa, 2 * h:2 * h + 2]
            want_sc[pb, h, ab] = scores[pa, h, aa]
    assert (out_lens[:b.S].cpu().numpy() == np.minimum(b.kv_lens_list, budget)).all() and (out_lens[b.S:] == 55).all()
    assert (kept[b.S:] == 77).all()
    assert (raw(cache) == want).all()
    np.testing.assert_array_equal(sc.cpu().numpy(), want_sc)


COMPACT = [
    (30, dict(Hkv=2, D=64), 16, [100, 40, 7, 0, 41], 40, 4, 8),
    (31, dict(Hkv=8, D=128), 16, [1500, 300, 2100], 301, 0, 0),
    (32, dict(Hkv=1, D=256), 64, [5000, 4999], 2500, 64, 700),
    (33, dict(Hkv=3, D=64), 4, [33, 34, 35, 1], 33, 33, 0),     # all protected
    (34, dict(Hkv=2, D=128), 20, [90, 200], 50, 0, 50),         # all recent
    (35, dict(Hkv=2, D=64), 12, [64, 65, 200], 1, 0, 0),        # one key
    (36, dict(Hkv=4, D=256), 8, [700], 699, 2, 1),              # one key goes
    (37, dict(Hkv=2, D=128), 16, [2, 1], 1, 1, 0),
    (38, dict(Hkv=1, D=64), 64, [43000, 41050, 90000], 20000, 100, 3000),  # more competing keys than a CTA keeps
]


@pytest.mark.parametrize("seed,shape,ps,kv_lens,budget,protect,recent", COMPACT)
@pytest.mark.parametrize("mode", ["fresh", "place", "equal", "mixed"])
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_compact(seed, shape, ps, kv_lens, budget, protect, recent, mode, kv):
    b = Batch(np.random.default_rng(seed), [0] * len(kv_lens), kv_lens, ps, Hq=shape["Hkv"], kv=kv,
              spare_pages=sum(-(-min(n, budget) // ps) for n in kv_lens) + 1, **shape)
    check_compact(b, budget, protect, recent, mode=mode)


@pytest.mark.parametrize("mode", ["place", "equal"])
def test_more_heads_than_ctas(mode):
    """Every (sequence, kv head) of a large batch moves in order."""
    rng = np.random.default_rng(46)
    b = Batch(rng, [0] * 90, [int(n) for n in rng.integers(20, 400, 90)], 16, Hq=8, Hkv=8, D=64)
    check_compact(b, 100, 5, 9, mode=mode)


@pytest.mark.parametrize("kind", ["equal", "few", "special", "negative", "tiny"])
def test_ties_and_special_scores(kind):
    rng = np.random.default_rng(40)
    b = Batch(rng, [0] * 3, [700, 90, 2049], 16, Hq=2, Hkv=2, D=64, spare_pages=80)
    shape = (b.N, b.Hkv, b.ps)
    sc = {"equal": np.full(shape, 0.5), "few": rng.integers(0, 3, shape) * 0.25,
          "special": rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, 1e-45], shape),
          "negative": -rng.random(shape), "tiny": rng.integers(0, 50, shape) * 1e-45}[kind].astype(np.float32)
    for mode in ("fresh", "place"):
        check_compact(b, 89, 3, 5, scores=sc, mode=mode)


def test_compact_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(41)
    b = Batch(rng, [0] * 3, [700, 90, 300], 16, Hq=2, Hkv=2, D=64, spare_pages=40)
    check_compact(b, 100, 3, 5, stream=torch.cuda.Stream())
    cache, lens = b.cache(), b.lens()
    sc = torch.rand(b.N, 2, 16, device="cuda")
    op = rpa.CacheEviction(budget=100, **b.cfg())
    c1, s1 = cache.clone(), sc.clone()
    l1 = op.compact(c1, s1, lens[0], lens[1], b.S)  # in place, new lengths in a tensor of their own
    assert l1.tolist() == [100, 90, 100, 0]
    c2, s2 = cache.clone(), sc.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.compact(c2, s2, lens[0], lens[1], b.S, new_kv_lens=lens[0])  # the lengths in place too
    g.replay()
    assert torch.equal(c1, c2) and torch.equal(s1, s2) and torch.equal(lens[0], l1)
    g.replay()  # nothing is over the budget now
    assert torch.equal(c1, c2) and torch.equal(s1, s2) and op.status() == rpa.RPA_OK


def test_compact_clusters_in_a_graph():
    """Long sequences, whose scores several CTAs share, captured and replayed with other lengths and scores."""
    rng = np.random.default_rng(44)
    b = Batch(rng, [0] * 2, [20000, 17000], 64, Hq=2, Hkv=2, D=64, spare_pages=330)
    new = b.table.copy()
    new[:2, :157] = b.free_pages[:314].reshape(2, 157)
    new = torch.from_numpy(new).cuda()
    cache, lens = b.cache(), b.lens()
    op = rpa.CacheEviction(budget=10000, protect=7, recent=130, **b.cfg())
    sc, out = torch.rand(b.N, 2, 64, device="cuda"), torch.zeros(b.max_seqs, dtype=torch.int32, device="cuda")
    kept = torch.zeros(b.max_seqs, 2, 10000, dtype=torch.int32, device="cuda")
    c2, s2 = cache.clone(), sc.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.compact(c2, s2, lens[0], lens[1], 2, new, out, kept=kept)
    for n in ([20000, 17000], [9000, 16999]):
        lens[0][:2] = torch.tensor(n, dtype=torch.int32)
        sc = torch.rand(b.N, 2, 64, device="cuda")
        s2.copy_(sc)
        c2.copy_(cache)
        g.replay()
        c1, s1, k1 = cache.clone(), sc.clone(), torch.zeros_like(kept)
        l1 = op.compact(c1, s1, lens[0], lens[1], 2, new, kept=k1)
        assert torch.equal(c1, c2) and torch.equal(s1, s2) and torch.equal(out[:2], l1[:2]) and torch.equal(kept[:2], k1[:2])
        x = f64(sc)
        for s in range(2):
            p0, a0 = b.slots(s, np.arange(n[s]))
            for h in range(2):
                want = kept_slots(x[p0, h, a0], n[s], 10000, 7, 130)
                assert (kept[s, h].cpu().numpy()[:len(want)] == want).all()
    assert op.status() == rpa.RPA_OK


def test_compact_bad_lengths_and_pages():
    rng = np.random.default_rng(42)
    b = Batch(rng, [0] * 3, [60, 50, 70], 8, Hq=2, Hkv=2, D=64, spare_pages=20)
    kvl, table, _ = b.lens()
    op = rpa.CacheEviction(budget=40, **b.cfg())
    for bad in (-1, b.P * b.ps + 1):
        k2 = kvl.clone()
        k2[1] = bad
        cache, sc = b.cache(), torch.rand(b.N, 2, 8, device="cuda")
        was, page = cache.clone(), torch.as_tensor(b.table[1, :7]).long().cuda()
        out = op.compact(cache, sc, k2, table, b.S)
        assert op.status() == rpa.RPA_ERR_BAD_LENGTHS
        assert out.tolist()[:3] == [40, bad, 40] and torch.equal(cache[page], was[page])
    for where in ("old", "new"):
        t, t2 = table.clone(), table.clone()
        (t if where == "old" else t2)[0, 1] = b.N + 5
        cache, sc = b.cache(), torch.rand(b.N, 2, 8, device="cuda")
        op.compact(cache, sc, kvl, t, b.S, new_page_indices=t2)
        assert op.status() == rpa.RPA_ERR_BAD_PAGE_INDEX and op.status() == rpa.RPA_OK
    with pytest.raises(rpa.RpaError):
        op.compact(b.cache(), torch.rand(b.N, 2, 8, device="cuda"), kvl, table, b.max_seqs + 1)
    op.compact(b.cache(), torch.rand(b.N, 2, 8, device="cuda"), kvl, table, 0)
    assert op.status() == rpa.RPA_OK


def test_decode_with_eviction():
    """Tokens appended with their positions, weighed, evicted in place and attended: the attention over the compacted
    cache is that over the kept keys."""
    rng = np.random.default_rng(43)
    Hq, Hkv, D, ps, S = 8, 2, 64, 16, 2
    lens = [60, 41]
    b = Batch(rng, lens, lens, ps, Hq, Hkv, D, spare_pages=8)
    rope = dict(rotary_dim=D)
    mk = lambda n, heads: torch.from_numpy(rng.standard_normal((n, heads, D)).astype(np.float32)).cuda().bfloat16()  # noqa: E731
    q, k, v = mk(b.T, Hq), mk(b.T, Hkv), mk(b.T, Hkv)
    cache = torch.zeros(b.N, ps, 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    scores = torch.full((b.N, Hkv, ps), 9.0, device="cuda")  # what earlier users of the pages left
    kvl, table, cu = b.lens()
    budget = 32
    cfg = b.cfg()
    op, ev = rpa.RopeAppend(**rope, **cfg), rpa.CacheEviction(budget=budget, protect=2, recent=8, **cfg)
    q1 = op.append(q, k, v, cache, kvl, table, cu, S)
    ev.accumulate(q1, cache, kvl, table, cu, S, scores)
    kept = torch.zeros(b.max_seqs, Hkv, budget, dtype=torch.int32, device="cuda")
    ev.compact(cache, scores, kvl, table, S, new_kv_lens=kvl, kept=kept)
    # one more token each: slot 32, position 60 and 41
    step = dict(cfg, num_q_tokens=S)
    op1, at1, ev1 = rpa.RopeAppend(**rope, **step), rpa.RaggedPagedAttention(**step), rpa.CacheEviction(budget=budget, protect=2, recent=8, **step)
    kvl[:S] += 1
    cu1 = torch.tensor([0, 1, 2, 2], dtype=torch.int32, device="cuda")
    nq, nk, nv = mk(S, Hq), mk(S, Hkv), mk(S, Hkv)
    q2 = op1.append(nq, nk, nv, cache, kvl, table, cu1, S, positions=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    o = at1.forward(q2, cache, kvl, table, cu1, S)
    ev1.accumulate(q2, cache, kvl, table, cu1, S, scores)
    assert all(x.status() == rpa.RPA_OK for x in (op, ev, op1, at1, ev1))
    from cache_util import rotate
    for s in range(S):
        t = np.arange(b.cu[s], b.cu[s] + lens[s])
        K = rotate(f64(k)[t], np.arange(lens[s]), rope)[0]
        K = f64(torch.from_numpy(K).float().bfloat16())
        V = f64(v)[t]
        Q = f64(torch.from_numpy(rotate(f64(nq)[s:s + 1], np.array([lens[s]]), rope)[0]).float().bfloat16())[0]
        KN = f64(torch.from_numpy(rotate(f64(nk)[s:s + 1], np.array([lens[s]]), rope)[0]).float().bfloat16())[0]
        page, at = b.slots(s, np.arange(budget + 1))
        for h in range(Hkv):
            idx = kept[s, h].cpu().numpy()
            assert (np.diff(idx) > 0).all() and idx[0] == 0 and idx[1] == 1 and idx[-1] == lens[s] - 1
            keys, vals = np.vstack((K[idx, h], KN[h])), np.vstack((V[idx, h], f64(nv)[s, h]))
            x = Q[h * 4:h * 4 + 4] @ keys.T / math.sqrt(D)
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            ref = p @ vals
            assert (np.abs(f64(o)[s, h * 4:h * 4 + 4] - ref) <= 2e-2 + 2e-2 * np.abs(ref)).all()
            # the new key starts from its own weight, whatever the page held before
            assert abs(scores[page[budget], h, at[budget]].item() - p[:, -1].sum()) <= 2e-2
