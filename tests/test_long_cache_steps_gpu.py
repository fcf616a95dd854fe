"""A prompt in chunks and decode steps over a 4-bit cache, each step's attention against its definition over what the cache holds,
within the attention's own bounds."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as i4  # noqa: E402
import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import f64, half_step  # noqa: E402
from long_cache_util import attend64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("D,group", [(64, 64), (128, 128), (128, 32), (256, 64)])
@pytest.mark.parametrize("mask", [{}, dict(sliding_window=60, first_keys=4)], ids=["all", "window"])
def test_steps(D, group, mask):
    H, Hq, ps = 2, 8, 16
    gen = torch.Generator("cuda").manual_seed(D + group)
    cfg = dict(num_q_heads=Hq, num_kv_heads=H, head_dim=D, total_num_pages=60, page_size=ps, max_num_seqs=2, pages_per_seq=24, kv_dtype="int4_g%d" % group,
               q_dtype="f16", sm_scale=D ** -0.5, k_scale=0.7, v_scale=1.5)
    table = np.random.default_rng(D).permutation(60)[:48].reshape(2, 24).astype(np.int32)
    tab = torch.from_numpy(table).cuda()
    cache = torch.full((60, H, i4.block_bytes(ps, D, group)), 0xff, dtype=torch.uint8, device="cuda")
    new = lambda t, h: torch.randn(t, h, D, device="cuda", generator=gen).half()  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kl = [0, 0]
    for ql in ([150, 20], [1, 200], [30, 1], [1, 1], [1, 1], [2, 5]):
        kl = [x + y for x, y in zip(kl, ql)]
        T = sum(ql)
        rope, att = rpa.RopeAppend(**cfg, num_q_tokens=T), rpa.RaggedPagedAttention(**cfg, **mask, num_q_tokens=T)
        lens, cu = i32(*kl), i32(0, ql[0], T)
        qr = rope.append(new(T, Hq), new(T, H), new(T, H), cache, lens, tab, cu, 2)
        out = att.forward(qr, cache, lens, tab, cu, 2)
        assert rope.status() == rpa.RPA_OK and att.status() == rpa.RPA_OK
        parts = i4.unpack(cache.cpu().numpy(), ps, D, group)
        ks, vs = float(np.float32(0.7)), float(np.float32(1.5))
        K, V, S = ks * i4.values(parts[0], group), vs * i4.values(parts[1], group), vs * np.repeat(parts[1][1], group, -1)
        at = lambda x: lambda s: x[table[s, np.arange(kl[s]) // ps], np.arange(kl[s]) % ps]  # noqa: E731
        ref, size, steps = attend64(f64(qr), ql, kl, [0, ql[0], T], lambda s: (at(K)(s), at(V)(s)), step=at(S),
                                    window=mask.get("sliding_window"), first=mask.get("first_keys", 0))
        # the larger of the two kernels' bounds.  P = f16(p s) meets codes at most 8 from the middle, o is rounded, logits are 32-bit
        # sums; a prompt's rows are rounded to f16 (K: 16 half steps of a logit, whose |q k| / sqrt(D) add up to less than 16 here; V, P)
        h = half_step("f16")
        tol = h * np.abs(ref) + 1e-6 + 8 * h * steps + 2 * h * size + 2 * (2.0 ** -14 + 16 * h) * size
        assert (np.abs(f64(out) - ref) <= tol).all(), (ql, np.abs(f64(out) - ref).max())
