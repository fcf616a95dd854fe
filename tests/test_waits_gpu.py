"""Copy warps that give up: they wait for the copies that they have issued and for no others, the kernel
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
@pytest.mark.parametrize("kv_lens", [[1, 200, 300], [500 + 37 * i for i in range(40)], [4000] * 200], ids=["a stage or two", "some", "many"])
def test_giving_up(kv, Hq, D, kv_lens):
    """Behind the last copy that a CTA issues, wherever its ring then is.  The consumers' waits run out once; a wait of the copy warp for
    a stage that it did not fill would run out as well, and take as long again for each."""
    b = Batch(np.random.default_rng(D), [1] * len(kv_lens), kv_lens, 16, Hq, 2, D, kv=kv)
    cache = i4.random_cache(b.rng, b.N, 16, 2, D, int(kv[6:]))[0] if kv.startswith("int4") else b.cache()
    q, lens = b.queries(), b.lens()
    att = rpa.RaggedPagedAttention(**b.cfg())
    want = att.forward(q, cache, *lens, b.S)
    assert att.status() == rpa.RPA_OK
    att.set_option(rpa.RPA_OPT_WAIT_TIMEOUT_MS, 300)
    for stall in (2, 0, 2):
        att.set_option(rpa.RPA_OPT_TEST_STALL_PRODUCER, stall)
        t0 = time.perf_counter()
        got = att.forward(q, cache, *lens, b.S)
        status = att.status()
        took = time.perf_counter() - t0
        assert torch.equal(got, want)  # every stage was there
        if stall:
            assert status == rpa.RPA_ERR_TIMEOUT and 0.29 < took < 0.55, (status, took)
        else:
            assert status == rpa.RPA_OK and took < 0.29


def test_the_hook_takes_two_values():
    b = Batch(np.random.default_rng(1), [1], [30], 16, 4, 2, 64)
    att = rpa.RaggedPagedAttention(**b.cfg())
    for n in (-1, 3):
        with pytest.raises(rpa.RpaError):
            att.set_option(rpa.RPA_OPT_TEST_STALL_PRODUCER, n)
