"""First keys that draw most of the weight, which is what they are kept visible for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as i4  # noqa: E402
from cache_util import Batch, stored  # noqa: E402
from test_first_keys_gpu import EIGHT, check  # noqa: E402
from test_int4_attention_gpu import Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


Q_LENS, KV_LENS = [1, 1, 150, 2, 1], [900, 3000, 700, 500, 12000]


def drawn(rng, T, H, D):
    """Queries with a part along one direction u of +-1, and the key along it: a logit of some 6 beside others of N(0, 1.2^2).
    Both sums of |q k| / sqrt(D) stay below 16, as the tolerances of the functions called here want (the 576 channels of latent rows
    with the products' own type need no such bound)."""
    u = rng.choice([-1.0, 1.0], D)
    return rng.standard_normal((T, H, D)) + 0.5 * u, 12 / np.sqrt(D) * u


def first_rows(b, first):
    page, at = zip(*(b.slots(s, np.arange(min(first, n))) for s, n in enumerate(b.kv_lens_list)))
    return np.concatenate(page), np.concatenate(at)


@pytest.mark.parametrize("Hq,Hkv,D,kv,q", [(8, 2, 128, "bf16", "bf16"), (16, 1, 64, "f16", "f16"), (8, 2, 256, "bf16", "bf16"), (8, 2, 128, "fp8_e4m3", "bf16"),
                                           (16, 4, 64, "int8", "f16"), (16, 1, 576, "bf16", "bf16")])
@pytest.mark.parametrize("window,first", [(400, 4), (100, 1), (2000, 70)])
def test_16_and_8_bits(Hq, Hkv, D, kv, q, window, first):
    rng = np.random.default_rng([D, window])
    b = Batch(rng, Q_LENS, KV_LENS, 16, Hq, Hkv, D, kv=kv, q=q, latent=D == 576, **(EIGHT if kv in ("fp8_e4m3", "int8") else {}))
    x, k = drawn(rng, b.T, Hq, D)
    cache = b.cache().cpu()
    page, at = first_rows(b, first)
    rows = slice(None) if b.latent else slice(0, None, 2)
    cache[page, at, rows] = stored(np.broadcast_to(k / (b.k_scale or 1.0), (len(page), Hkv, D)), kv)
    check(b, window, first, q=stored(x, q).cuda(), cache=cache.cuda())


@pytest.mark.parametrize("Hq,Hkv,D,group", [(8, 2, 128, 64), (16, 1, 64, 32), (8, 2, 256, 128)])
@pytest.mark.parametrize("window,first", [(400, 4), (100, 1), (2000, 70)])
def test_4_bits(Hq, Hkv, D, group, window, first):
    c = Case([30, D, window], Q_LENS, KV_LENS, 16, Hq, Hkv, D, group, "f16")
    x, k = drawn(c.b.rng, c.b.T, Hq, D)
    page, at = first_rows(c.b, first)
    for dst, new in zip(c.parts[0], i4.coded(np.broadcast_to(k, (len(page), Hkv, D)), group)):
        dst[page, at] = new
    c.cache = torch.from_numpy(i4.pack(c.parts, 16, D, group)).cuda()
    c.q = stored(x, "f16").cuda()
    c.check(window=window, first=first)
    # (they do draw weight: without them the outputs are others)
    with_them, without = c.reference(window=window, first=first)[0], c.reference(window=window)[0]
    t = c.b.cu[1]
    assert np.abs(with_them[t] - without[t]).mean() > 2.0 ** -6
