"""Compaction with page ids outside the cache, against its definition: the keys of such a page are neither read nor written
and their scores count as NaN; everything else of the call is as if the page were there."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def kept_slots(x, n, budget, protect, recent):
    if n <= budget:
        return np.arange(n)
    middle = np.arange(protect, n - recent)
    order = sorted(middle, key=lambda j: (np.isnan(x[j]), 0.0 if np.isnan(x[j]) else -float(x[j]), j))
    return np.concatenate((np.arange(protect), np.sort(order[:budget - protect - recent]), np.arange(n - recent, n))).astype(int)


def define(b, old, new, cache, scores, budget, protect, recent):
    """(cache, scores, kept, lengths) of the definition; cache [N, ps, rows, bytes], numpy."""
    out, out_sc = cache.copy(), scores.copy()
    kept, lens, used = np.full((b.max_seqs, b.Hkv, budget), 77), np.full(b.max_seqs, 55), False
    good = lambda page: (page >= 0) & (page < b.N)  # noqa: E731
    for s in range(b.S):
        n = b.kv_lens_list[s]
        j = np.arange(n)
        page, at = old[s, j // b.ps].astype(np.int64), j % b.ps
        ok = good(page)
        lens[s] = min(n, budget)
        for h in range(b.Hkv):
            x = np.where(ok, scores[np.where(ok, page, 0), h, at], np.nan)
            idx = kept_slots(x, n, budget, protect, recent)
            kept[s, h] = -1
            kept[s, h, :len(idx)] = idx
            to = np.arange(len(idx))
            p2 = new[s, to // b.ps].astype(np.int64)
            move = ok[idx] & good(p2)
            a, c = idx[move], to[move]
            out[p2[move], c % b.ps, 2 * h:2 * h + 2] = cache[page[a], at[a], 2 * h:2 * h + 2]
            out_sc[p2[move], h, c % b.ps] = scores[page[a], h, at[a]]
    return out, out_sc, kept, lens


SHAPES = [
    # (q lengths are none) kv lengths, budget, protect, recent; sequence 1 is below the budget
    (0, dict(Hkv=2, D=64), 8, [60, 33, 70], 40, 5, 9, "bf16"),
    (1, dict(Hkv=3, D=128), 16, [500, 100, 333, 160], 160, 32, 40, "fp8_e4m3"),
    (2, dict(Hkv=1, D=256), 64, [20000, 4000], 9000, 100, 700, "bf16"),  # several CTAs a head
]


@pytest.mark.parametrize("seed,shape,ps,kv_lens,budget,protect,recent,kv", SHAPES)
@pytest.mark.parametrize("mode,where", [("place", "both")] + [(m, w) for m in ("fresh", "mixed", "equal") for w in ("old", "new", "both")])
def test_bad_pages(seed, shape, ps, kv_lens, budget, protect, recent, kv, mode, where):
    rng = np.random.default_rng(seed)
    b = Batch(rng, [0] * len(kv_lens), kv_lens, ps, Hq=shape["Hkv"], kv=kv,
              spare_pages=sum(-(-min(n, budget) // ps) for n in kv_lens) + 1, **shape)
    old, new = b.table.copy(), b.table.copy()
    if mode in ("fresh", "mixed"):
        at = 0
        for s in range(b.S):
            for i in range(protect // ps if mode == "mixed" else 0, -(-min(budget, kv_lens[s]) // ps)):
                new[s, i] = b.free_pages[at]
                at += 1
    # of sequence 0 the first page (protected, of which a part may compete), one between and that of the last keys; of
    # sequence 1 one page
    last, middle = (kv_lens[0] - 1) // ps, -(-min(budget, kv_lens[0]) // ps) - 1
    for t, name in ((old, "old"), (new, "new")):
        if where in (name, "both"):
            t[0, [0, middle, last]] = [-1, b.N, 2 ** 31 - 1]
            t[1, 1] = -2 ** 31
    scores = np.exp(rng.standard_normal((b.N, b.Hkv, ps)) * 2).astype(np.float32)
    scores[rng.random(scores.shape) < 0.05] = np.nan
    cache = b.cache()
    raw = cache.view(torch.uint8).cpu().numpy().reshape(b.N, ps, b.rows, -1)
    sc, kvl = torch.from_numpy(scores.copy()).cuda(), b.lens()[0]
    told = torch.from_numpy(old).cuda()
    tnew = told if mode == "place" else torch.from_numpy(new).cuda()
    kept = torch.full((b.max_seqs, b.Hkv, budget), 77, dtype=torch.int32, device="cuda")
    out = torch.full((b.max_seqs,), 55, dtype=torch.int32, device="cuda")
    op = rpa.CacheEviction(budget=budget, protect=protect, recent=recent, **b.cfg())
    want = define(b, old, old if mode == "place" else new, raw.copy(), scores, budget, protect, recent)
    torch.cuda.synchronize()
    op.compact(cache, sc, kvl, told, b.S, tnew, out, kept=kept)
    assert op.status() == rpa.RPA_ERR_BAD_PAGE_INDEX and op.status() == rpa.RPA_OK
    np.testing.assert_array_equal(kept.cpu().numpy(), want[2])
    np.testing.assert_array_equal(out.cpu().numpy(), want[3])
    np.testing.assert_array_equal(sc.cpu().numpy(), want[1])
    assert (cache.view(torch.uint8).cpu().numpy().reshape(raw.shape) == want[0]).all()
