"""A handle over a 4-bit cache on a GPU that has little memory left: the room for prompts' f16 rows is as large as can be had, or
none, and its calls give what they gave."""
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


GIB = 1 << 30


@pytest.mark.parametrize("left", [6 * GIB, GIB // 5])
def test_a_room_that_cannot_be_had(left):
    """Pages for one sequence of 8 GiB of f16 rows; `left` bytes of the GPU are free when the handle is made."""
    b = Batch(np.random.default_rng(1), [300, 1, 200], [700, 400, 200], 64, 16, 8, 128, kv="int4_g64")
    P = 8 * GIB // (64 * 2 * 8 * 128 * 2) + 64  # pages of 64 keys
    table = np.zeros((b.max_seqs, P), np.int32)
    table[:, :b.P] = b.table
    cfg = dict(b.cfg(), pages_per_seq=P, total_num_pages=P)
    small = i4.random_cache(b.rng, b.N, 64, 8, 128, 64)
    cache = torch.zeros((P, *small[0].shape[1:]), dtype=torch.uint8, device="cuda")
    cache[:b.N] = small[0]
    lens, _, cu = b.lens()
    table, q = torch.from_numpy(table).cuda(), b.queries()
    warm, out = rpa.RaggedPagedAttention(**dict(b.cfg(), total_num_pages=P)), torch.empty_like(q)
    warm.forward(q, cache, lens, table[:, :b.P].contiguous(), cu, b.S, out=out)  # (loads the kernels)
    assert warm.status() == rpa.RPA_OK
    warm.close()
    out.fill_(7.0)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    hold = torch.empty(free - left, dtype=torch.uint8, device="cuda")
    try:
        assert torch.cuda.mem_get_info()[0] < 8 * GIB
        att = rpa.RaggedPagedAttention(**cfg)
        att.forward(q, cache, lens, table, cu, b.S, out=out)
        assert att.status() == rpa.RPA_OK
        info, _ = att.plan()
        assert info[2] > 0  # (a part of the 8 GiB fits, and the prompts into it: they still become rows)
        att.close()
    finally:
        del hold
        torch.cuda.empty_cache()
    K, V = (i4.values(p, 64) for p in small[1])
    step = np.repeat(small[1][1][1], 64, -1)
    at = lambda x: lambda s: x[b.slots(s, np.arange(b.kv_lens_list[s]))]  # noqa: E731
    ref, size, steps = attend64(f64(q), b.q_lens, b.kv_lens_list, b.cu, lambda s: (at(K)(s), at(V)(s)), step=at(step))
    h = half_step("f16")  # the larger of the two kernels' bounds: K, V and P of f16 rows, 16 half steps of a logit
    tol = 2.0 ** -8 * np.abs(ref) + 1e-6 + 8 * h * steps + 2 * h * size + 2 * (2.0 ** -14 + 16 * h) * size
    assert (np.abs(f64(out) - ref) <= tol).all()
