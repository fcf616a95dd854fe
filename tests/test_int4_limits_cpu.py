"""What the configurations of a 4-bit cache refuse at the end of 32-bit key numbers."""
import pytest

import ragged_paged_attention_02_gb300 as rpa

BASE = dict(num_q_tokens=22, num_q_heads=4, num_kv_heads=2, head_dim=64, total_num_pages=16, page_size=1024, max_num_seqs=3, sm_scale=0.125)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("kv,pages,ps,code", [
    ("int4_g64", 2 ** 21 - 1, 1024, rpa.RPA_OK),
    ("int4_g64", 2 ** 29 - 1, 4, rpa.RPA_ERR_UNSUPPORTED),  # a stage behind the last key has no 32-bit number
    ("int4_g64", 2 ** 29 - 256, 4, rpa.RPA_OK),
    ("int4_g64", 2 ** 29 - 255, 4, rpa.RPA_ERR_UNSUPPORTED),
    ("int4_g64", 2 ** 21, 1024, rpa.RPA_ERR_INVALID_ARG),
    ("fp8_e4m3", 2 ** 29 - 1, 4, rpa.RPA_OK),  # as before
])
def test_the_longest_sequences(kv, pages, ps, code):
    cfg = dict(BASE, kv_dtype=kv, pages_per_seq=pages, page_size=ps)
    assert rpa.validate_cfg(**cfg) == code and rpa.validate_rope_cfg(**cfg) == code
