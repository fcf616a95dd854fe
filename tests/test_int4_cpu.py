"""The 4-bit cache on the host: what the configurations take and refuse, and the layout's definition."""
import numpy as np
import pytest

import int4_util as i4
import ragged_paged_attention_02_gb300 as rpa

BASE = dict(num_q_tokens=22, num_q_heads=4, num_kv_heads=2, head_dim=64, total_num_pages=16, page_size=16, max_num_seqs=3,
            pages_per_seq=4, sm_scale=0.125)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("change,code", [
    (dict(kv_dtype="int4_g32"), rpa.RPA_OK),
    (dict(kv_dtype="int4_g64", page_size=20), rpa.RPA_OK),
    (dict(kv_dtype="int4_g64", page_size=6), rpa.RPA_ERR_UNSUPPORTED),
    (dict(kv_dtype="int4_g64", page_size=65536), rpa.RPA_OK),
    (dict(kv_dtype="int4_g64", page_size=65540), rpa.RPA_ERR_UNSUPPORTED),
    (dict(kv_dtype="int4_g64", num_q_heads=130, num_kv_heads=2), rpa.RPA_ERR_UNSUPPORTED),
    (dict(kv_dtype="int4_g64", sliding_window=4, first_keys=3), rpa.RPA_OK),
    (dict(kv_dtype="int4_g128"), rpa.RPA_ERR_UNSUPPORTED),  # wider than the head
    (dict(kv_dtype="int4_g128", head_dim=128), rpa.RPA_OK),
    (dict(kv_dtype="int4_g128", head_dim=256, q_dtype="f16"), rpa.RPA_OK),
    (dict(kv_dtype="int4_g32", kv_layout="latent", head_dim=576, v_head_dim=512, num_q_heads=16, num_kv_heads=1, page_size=64),
     rpa.RPA_ERR_UNSUPPORTED),
])
def test_validate(change, code):
    assert rpa.validate_cfg(**dict(BASE, **change)) == code


def test_operators_that_do_not_take_it():
    cfg = dict(BASE, kv_dtype="int4_g32")
    assert rpa.validate_prefix_cfg(**cfg) == rpa.RPA_ERR_UNSUPPORTED
    assert rpa.validate_evict_cfg(budget=32, **cfg) == rpa.RPA_ERR_UNSUPPORTED
    assert rpa.validate_rope_cfg(**cfg) == rpa.RPA_OK


def test_null_and_misaligned_read():
    assert rpa.lib().rpa_rope_read(None, None, None, None, None, 0, None, None, None) == rpa.RPA_ERR_INVALID_ARG


@pytest.mark.parametrize("ps,D,group", [(16, 64, 32), (20, 128, 128), (4, 256, 64)])
def test_pack_and_unpack_are_inverse(ps, D, group):
    rng = np.random.default_rng(1)
    parts = [i4.coded(rng.standard_normal((3, ps, 2, D)), group) for _ in "kv"]
    cache = i4.pack(parts, ps, D, group)
    assert cache.shape[2] == i4.block_bytes(ps, D, group)
    for a, b in zip(i4.unpack(cache, ps, D, group), parts):
        for x, y in zip(a, b):
            assert np.array_equal(x, y)


def test_chunks_of_eight_slots_lie_in_eight_columns():
    for D in (64, 128, 256):
        order = i4._order(64, D)
        for c in range(D // 32):
            for r in range(0, 64, 8):
                columns = {((r + i) * D // 2 + 16 * order[r + i, c]) // 16 % 8 for i in range(8)}
                assert len(columns) == 8


@pytest.mark.parametrize("group", [32, 64, 128])
def test_codes_cover_the_group(group):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((50, 256)) * 10.0 ** rng.uniform(-3, 3, (50, 1))
    codes, s, z = i4.coded(x, group)
    y = i4.values((codes, s, z), group)
    assert (np.abs(x - y) <= np.repeat(s, group, -1) * 0.5 * (1 + 1e-12)).all()
