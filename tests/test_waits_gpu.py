"""Copy warps that give up in the middle of their work: they wait for the copies that they have issued and for no others, the kernel
returns its status, and the handle works on."""
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as i4  # noqa: E402
import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("kv,Hq,D", [("int4_g64", 8, 64), ("int4_g64", 8, 128), ("int4_g128", 8, 256), ("bf16", 8, 128), ("bf16", 32, 128), ("f16", 8, 64)])
def test_giving_up_midway(kv, Hq, D):
    """Before the n-th stage of a CTA, in the first to third round of its ring.  The consumers' waits run out once; a wait of the copy
    warp for a stage that it did not fill would run out behind that, and take as long again."""
    b = Batch(np.random.default_rng(D), [1] * 24, [4000] * 24, 16, Hq, 2, D, kv=kv)
    cache = i4.random_cache(b.rng, b.N, 16, 2, D, int(kv[6:]))[0] if kv.startswith("int4") else b.cache()
    q, lens = b.queries(), b.lens()
    att = rpa.RaggedPagedAttention(**b.cfg())
    want = att.forward(q, cache, *lens, b.S)
    assert att.status() == rpa.RPA_OK
    att.set_option(rpa.RPA_OPT_WAIT_TIMEOUT_MS, 200)
    for n in range(2, 9):
        att.set_option(rpa.RPA_OPT_TEST_STALL_PRODUCER, n)
        t0 = time.perf_counter()
        att.forward(q, cache, *lens, b.S)
        status = att.status()
        took = time.perf_counter() - t0
        # (a CTA may have fewer stages than n)
        if status == rpa.RPA_OK:
            assert n > 3 and took < 0.19, (n, took)
        else:
            assert status == rpa.RPA_ERR_TIMEOUT and 0.19 < took < 0.39, (n, status, took)
    att.set_option(rpa.RPA_OPT_TEST_STALL_PRODUCER, 0)
    got = att.forward(q, cache, *lens, b.S)
    assert att.status() == rpa.RPA_OK and torch.equal(got, want)


def test_the_hook_takes_counts():
    b = Batch(np.random.default_rng(1), [1], [30], 16, 4, 2, 64)
    att = rpa.RaggedPagedAttention(**b.cfg())
    for n in (-1, 1 << 40):
        with pytest.raises(rpa.RpaError):
            att.set_option(rpa.RPA_OPT_TEST_STALL_PRODUCER, n)
