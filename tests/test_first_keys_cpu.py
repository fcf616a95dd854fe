"""first_keys on the host: what the configuration takes and refuses."""
import ctypes

import pytest

import ragged_paged_attention_02_gb300 as rpa
from ragged_paged_attention_02_gb300.binding import RpaCfg

BASE = dict(num_q_tokens=22, num_q_heads=4, num_kv_heads=2, head_dim=64, total_num_pages=16, page_size=16, max_num_seqs=3,
            pages_per_seq=4, sm_scale=0.125)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("change,code", [
    (dict(sliding_window=8, first_keys=4), rpa.RPA_OK),
    (dict(sliding_window=8, first_keys=0), rpa.RPA_OK),
    (dict(sliding_window=1, first_keys=2 ** 31 - 1), rpa.RPA_OK),
    (dict(sliding_window=8, first_keys=-1), rpa.RPA_ERR_INVALID_ARG),
    (dict(first_keys=4), rpa.RPA_ERR_INVALID_ARG),  # nothing hides them
])
def test_validate(change, code):
    assert rpa.validate_cfg(**dict(BASE, **change)) == code


def test_the_field_shares_the_reserved_word():
    assert RpaCfg.first_keys.offset == RpaCfg.reserved.offset
    c = rpa.make_cfg(**dict(BASE, sliding_window=8, first_keys=5))
    assert c.reserved == 5
    rpa.lib().rpa_cfg_init(ctypes.byref(c))
    assert c.first_keys == 0


def test_operators_without_a_window_refuse_it():
    cfg = dict(BASE, sliding_window=8, first_keys=4)
    assert rpa.validate_prefix_cfg(**cfg) == rpa.RPA_ERR_UNSUPPORTED
    assert rpa.validate_evict_cfg(budget=32, **cfg) == rpa.RPA_ERR_UNSUPPORTED
    assert rpa.validate_evict_cfg(budget=32, **dict(BASE, sliding_window=8)) == rpa.RPA_OK
    assert rpa.validate_rope_cfg(**cfg) == rpa.RPA_OK  # writes rows: no attention


def test_numbers_past_32_bits_do_not_wrap():
    assert rpa.make_cfg(**dict(BASE, sliding_window=8, first_keys=2 ** 32 + 5)).first_keys == 2 ** 31 - 1
    assert rpa.validate_cfg(**dict(BASE, sliding_window=8, first_keys=-2 ** 32)) == rpa.RPA_ERR_INVALID_ARG
