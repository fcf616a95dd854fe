"""How small the values of a 4-bit cache may be.  The direct kernel rounds a probability times a scale to float16, whose steps stop at
2^-24: small values keep their digits where v_scale brings them up, and lose 2^-25 a key, in units of a code, where it does not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as i4  # noqa: E402
import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import f64, half_step  # noqa: E402
from test_int4_attention_gpu import Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("size", [1e-2, 1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("up", [False, True])
def test_size_of_v(size, D, group, up):
    by = 2.0 ** 13 if up else 1.0
    c = Case([40, D], [1, 1, 2], [3000, 200, 700], 16, 8, 2, D, group, "f32", v_scale=1 / by)
    b = c.b
    c.parts[1] = i4.coded(by * size * b.rng.standard_normal((b.N, 16, 2, D)), group)
    c.cache = torch.from_numpy(i4.pack(c.parts, 16, D, group)).cuda()
    att = c.make()
    got = f64(att.forward(c.q, c.cache, *c.lens, b.S))
    assert att.status() == rpa.RPA_OK
    ref, total, steps = c.reference()
    # P = f16(p s), p = 2^(x - m) with m at most the row's maximum: half a step of it, or 2^-25 where that is less, meets codes up to
    # 8 from the middle.  Relative to the sum of p, which is at least that of exp(x - max), for each of the keys.  Logits: q is rounded
    # to f16 (16 half steps), sums in 32 bits.  The sums of P and of p (z + 8 s), and o, in 32 bits: a few 2^-24 of 8 steps and |v|.
    h = half_step("f16")
    K = i4.values(c.parts[0], group)
    lost = np.zeros((b.T, b.Hq, 1))
    for s, (a, n) in enumerate(zip(b.q_lens, b.kv_lens_list)):
        page, place = b.slots(s, np.arange(n))
        for i in range(a):
            for head in range(b.Hq):
                x = f64(c.q)[b.cu[s] + i, head] @ K[page, place, head // 4].T / np.sqrt(D)
                x = x[:n - a + i + 1]
                lost[b.cu[s] + i, head] = 8 * 2.0 ** -25 * len(x) / np.exp(x - x.max()).sum() / by
    tol = 8 * h * steps + 2 * (2.0 ** -14 + 16 * h) * total + lost + 2.0 ** -20 * (8 * steps + total)
    assert (np.abs(got - ref) <= tol).all()
    if up:  # no more than an eighth of the bound is lost, at any of these sizes but the smallest
        assert size < 5e-5 or (lost <= tol / 8)[b.cu[0]:b.cu[b.S]].all()
