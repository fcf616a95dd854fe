"""Key ranges of the plan's items under a window with visible first keys: the band that the unit's tokens see and nothing else."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch  # noqa: E402
from ragged_paged_attention_02_gb300.binding import cache_shape  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def band(p_lo, p_hi, n, window, first):
    """Keys that tokens at p_lo .. p_hi see, without the first ones where a gap follows those."""
    lo = max(0, p_lo - window + 1)
    return (0 if lo <= first else lo), min(n, p_hi + 1)


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("f16", 64), ("fp8_e4m3", 64), ("bf16", 256), ("int4_g64", 128), ("int4_g128", 256)])
@pytest.mark.parametrize("window,first", [(700, 4), (3000, 900), (5000, 64), (64, 0), (1, 1), (9000, 3)])
def test_items_keep_to_the_band(kv, D, window, first):
    G = 4
    scales = dict(k_scale=0.05, v_scale=0.05) if kv == "fp8_e4m3" else {}
    b = Batch(np.random.default_rng(window + first), [1, 1, 120, 3, 700, 0], [9000, 100, 2000, 6000, 900, 50], 16, 2 * G, 2, D, kv=kv, q="f16" if kv == "f16" else "bf16",
              **scales)
    q = torch.zeros((b.T, 2 * G, D), dtype=torch.float16 if kv == "f16" else torch.bfloat16, device="cuda")
    att = rpa.RaggedPagedAttention(**b.cfg(), sliding_window=window, first_keys=first)
    dtype = torch.bfloat16 if kv == "bf16" else torch.float16 if kv == "f16" else torch.uint8
    att.forward(q, torch.zeros(cache_shape(att._c), dtype=dtype, device="cuda"), *b.lens(), b.S)
    assert att.status() == rpa.RPA_OK
    info, items = att.plan()
    count = [[np.zeros((a, n), int) for a, n in zip(b.q_lens, b.kv_lens_list)] for _ in range(2)]
    ranges = {}  # of split or whole units: their pieces
    for i, (s, head, t0, nt, lo, hi, part, piece) in enumerate(items.tolist()):
        n, a = b.kv_lens_list[s], b.q_lens[s]
        assert 0 <= lo < hi <= n and 0 <= t0 and 0 < nt <= a - t0
        # units of few tokens (and a 4-bit cache's tiles) have the band of their whole sequence, prompts' tiles their own
        whole = i < info[1] or (info[15] >> 1 & 1 and a * G <= info[5])
        p0 = n - a + (0 if whole else t0)
        p1 = n - 1 if whole else n - a + t0 + nt - 1
        ranges.setdefault((s, head, t0, nt, band(p0, p1, n, window, first)), []).append((piece, lo, hi))
        count[head][s][t0:t0 + nt, lo:hi] += 1
        if first and piece == 0 and lo > first:
            assert n - a + t0 - window + 1 >= lo  # no token of the unit sees a key of the gap
            count[head][s][t0:t0 + nt, :first] += 1
    for (*_, (lo, hi)), pieces in ranges.items():
        pieces.sort()
        assert [p[0] for p in pieces] == list(range(len(pieces)))
        assert pieces[0][1] == lo and pieces[-1][2] == hi and all(x[2] == y[1] for x, y in zip(pieces, pieces[1:]))
    for head in range(2):
        for s, (a, n) in enumerate(zip(b.q_lens, b.kv_lens_list)):
            pos, j = np.arange(n - a, n)[:, None], np.arange(n)[None]
            sees = (j <= pos) & ((j > pos - window) | (j < first))
            assert (count[head][s][sees] == 1).all() and (count[head][s] <= 1).all()
