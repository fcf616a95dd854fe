"""Eviction on the CPU: configurations and the binding's refusals."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from ragged_paged_attention_02_gb300.cache import CacheEviction, make_evict_cfg  # noqa: E402

CFG = dict(num_q_tokens=22, num_q_heads=4, num_kv_heads=2, head_dim=64, total_num_pages=16, page_size=16, max_num_seqs=3,
           pages_per_seq=4, sm_scale=0.125, budget=32)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("change,code", [
    ({}, rpa.RPA_OK),
    (dict(budget=64), rpa.RPA_OK),
    (dict(budget=65), rpa.RPA_ERR_INVALID_ARG),  # more than a sequence can have
    (dict(budget=0), rpa.RPA_ERR_INVALID_ARG),
    (dict(protect=16, recent=16), rpa.RPA_OK),
    (dict(protect=16, recent=17), rpa.RPA_ERR_INVALID_ARG),
    (dict(protect=-1), rpa.RPA_ERR_INVALID_ARG),
    (dict(recent=-1), rpa.RPA_ERR_INVALID_ARG),
    (dict(kv_dtype="int8", k_scale=0.04), rpa.RPA_OK),
    (dict(soft_cap=30.0, sliding_window=100, is_causal=False), rpa.RPA_OK),
    (dict(head_dim=96), rpa.RPA_ERR_UNSUPPORTED),
    (dict(head_dim=576, v_head_dim=512, kv_layout="latent", num_q_heads=16, num_kv_heads=1), rpa.RPA_ERR_UNSUPPORTED),
    (dict(num_q_tokens=1 << 30), rpa.RPA_ERR_UNSUPPORTED),  # 2^31 rows of a kv head
    (dict(page_size=1 << 20, pages_per_seq=1 << 10), rpa.RPA_OK),
    (dict(page_size=1 << 20, pages_per_seq=(1 << 10) + 1), rpa.RPA_ERR_UNSUPPORTED),  # keys of a piece behind 2^30 others
])
def test_validate(change, code):
    assert rpa.validate_evict_cfg(**dict(CFG, **change)) == code


def test_null_arguments():
    L = rpa.lib()
    bad = rpa.RPA_ERR_INVALID_ARG
    assert L.rpa_evict_validate_cfg(None) == bad
    assert L.rpa_evict_accumulate(None, None, None, None, None, None, 0, None, None) == bad
    assert L.rpa_evict_compact(None, None, None, None, None, 0, None, None, None, None) == bad
    assert L.rpa_evict_get_status(None, None) == bad
    assert L.rpa_evict_create(ctypes.byref(make_evict_cfg(**CFG)), None) == bad
    c = make_evict_cfg(**CFG)
    c.reserved = 1
    assert L.rpa_evict_validate_cfg(ctypes.byref(c)) == bad
    L.rpa_evict_destroy(None)


def _op(**over):
    a = object.__new__(CacheEviction)  # argument checks only: no handle
    a._h = None
    a._c = make_evict_cfg(**dict(CFG, **over))
    a._checks(a._c.cache)
    return a


def _i(*n):
    return torch.zeros(*n, dtype=torch.int32)


def _accumulate():
    return dict(q=torch.zeros(22, 4, 64, dtype=torch.bfloat16), kv_pages=torch.zeros(16, 16, 4, 64, dtype=torch.bfloat16), kv_lens=_i(3),
                page_indices=_i(3, 4), cu_q_lens=_i(4), scores=torch.zeros(16, 2, 16))


def _compact():
    return dict(kv_pages=torch.zeros(16, 16, 4, 64, dtype=torch.bfloat16), scores=torch.zeros(16, 2, 16), kv_lens=_i(3),
                page_indices=_i(3, 4), new_page_indices=_i(3, 4), new_kv_lens=_i(3), kept=_i(3, 2, 32))


def test_well_formed_arguments_pass():
    _op()._check_accumulate(**_accumulate())
    _op()._check_compact(**_compact())
    _op()._check_compact(**dict(_compact(), kept=None))


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(22, 4, 64)), ("kv_pages", torch.zeros(16, 16, 4, 64)), ("kv_lens", _i(4)), ("page_indices", _i(4, 3)),
    ("cu_q_lens", _i(3)), ("scores", torch.zeros(16, 16, 2)), ("scores", torch.zeros(16, 2, 16, dtype=torch.bfloat16)),
    ("scores", torch.zeros(16, 16, 2).transpose(1, 2)),
])
def test_malformed_accumulate_is_refused(name, bad):
    with pytest.raises(ValueError):
        _op()._check_accumulate(**dict(_accumulate(), **{name: bad}))


@pytest.mark.parametrize("name,bad", [
    ("kv_pages", torch.zeros(16, 16, 4, 64)), ("scores", torch.zeros(16, 2, 15)), ("kv_lens", torch.zeros(3)),
    ("new_page_indices", _i(3, 5)), ("new_kv_lens", _i(2)), ("kept", _i(3, 2, 31)), ("kept", _i(2, 2, 32)),
])
def test_malformed_compact_is_refused(name, bad):
    with pytest.raises(ValueError):
        _op()._check_compact(**dict(_compact(), **{name: bad}))


def test_division_by_a_product():
    """The kernels' j / d by one high product, for every divisor a page size or group can be near and far."""
    import random

    rng = random.Random(5)
    divisors = list(range(1, 300)) + [2 ** k for k in range(31)] + [2 ** k - 1 for k in range(2, 31)] + [rng.randrange(1, 2 ** 31) for _ in range(300)]
    for d in divisors:
        shift = max(0, (d - 1).bit_length())
        m = ((2 ** 32 * (2 ** shift - d)) // d + 1) % 2 ** 32
        for j in {0, 1, d - 1, d, d + 1, 2 * d - 1, 2 ** 31 - 1, 2 ** 31 - d, *[rng.randrange(2 ** 31) for _ in range(20)]}:
            if 0 <= j < 2 ** 31:
                t = (m * j >> 32) + j
                assert t < 2 ** 32 and t >> shift == j // d, (d, j)
