"""Calls of the paged cache's operators that their documentation allows or has to refuse, as far as no GPU is needed."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from ragged_paged_attention_02_gb300.cache import RopeAppend, make_rope_cfg  # noqa: E402

CFG = dict(num_q_tokens=22, num_q_heads=4, num_kv_heads=2, head_dim=64, total_num_pages=16, page_size=16, max_num_seqs=3,
           pages_per_seq=4, sm_scale=0.125)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("factor", [0.0, -1.0, 0.5, math.nan, math.inf])
def test_the_factor_of_plain_frequencies_does_not_count(factor):
    """Without scaling the factor is neither checked nor used."""
    want = rpa.rope_frequencies(**CFG)
    assert rpa.validate_rope_cfg(factor=factor, **CFG) == rpa.RPA_OK
    got = rpa.rope_frequencies(factor=factor, **CFG)
    assert np.isfinite(want).all() and (got == want).all()


def test_sinks_of_the_attention_do_not_hinder_an_append():
    """RopeAppend takes RaggedPagedAttention's keywords, with sinks in host memory too, as that takes them."""
    sinks = np.linspace(-1, 1, 4).astype(np.float32)
    assert rpa.validate_cfg(sinks=sinks, **CFG) == rpa.RPA_OK
    assert rpa.validate_rope_cfg(sinks=sinks, **CFG) == rpa.RPA_OK
    assert (rpa.rope_frequencies(sinks=sinks, **CFG) == rpa.rope_frequencies(**CFG)).all()
    c = make_rope_cfg(sinks=sinks, **CFG)
    assert not c.cache.has_sinks and not c.cache.sinks  # a host address stays out of the handle


class FakeStream:
    def __init__(self, device, pointer):
        self.device, self.cuda_stream = torch.device("cuda", device), pointer


class FakeTensor:
    def __init__(self):
        self.on = []

    def record_stream(self, stream):
        self.on.append(stream)


def test_streams_of_other_devices_are_refused():
    """Also their default streams, whose pointer is the one of this device's."""
    op = object.__new__(RopeAppend)
    op._h, op._device, op._current = None, 0, lambda device: 0
    assert op._stream(None) == 0 and op._stream(FakeStream(0, 0)) == 0
    for pointer in (0, 77):
        with pytest.raises(ValueError, match="cuda:0"):
            op._stream(FakeStream(1, pointer))
    t, side = FakeTensor(), FakeStream(0, 77)
    assert op._stream(side, (t, None)) == 77 and t.on == [side]


def test_one_head_may_have_any_stride():
    """Keys and values of a single kv head kept as [head, token, D], or taken out of a wider tensor: the heads of a token
    are contiguous whatever the stride of a dimension of one."""
    cfg = dict(CFG, num_kv_heads=1)
    op = object.__new__(RopeAppend)
    op._h, op._c = None, make_rope_cfg(**cfg)
    op._checks(op._c.cache)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    args = dict(q=torch.zeros(22, 4, 64, dtype=torch.bfloat16), kv_pages=torch.zeros(16, 16, 2, 64, dtype=torch.bfloat16), kv_lens=i(3),
                page_indices=i(3, 4), cu_q_lens=i(4), positions=None, q_out=torch.zeros(22, 4, 64, dtype=torch.bfloat16))
    k = torch.zeros(1, 22, 64, dtype=torch.bfloat16).transpose(0, 1)
    assert k.stride() == (64, 22 * 64, 1)
    v = torch.zeros(22, 3, 192, dtype=torch.bfloat16)[:, 1:2, 64:128]
    op._check(k=k, v=v, **args)
    for bad in (torch.zeros(22, 1, 128, dtype=torch.bfloat16)[..., ::2], torch.zeros(1, 22, 64, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            op._check(k=bad, v=v, **args)
