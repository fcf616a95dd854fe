"""Shared-prefix attention on the CPU: configurations and the binding's refusals."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from ragged_paged_attention_02_gb300.cache import SharedPrefixAttention  # noqa: E402

CFG = dict(num_q_tokens=22, num_q_heads=4, num_kv_heads=2, head_dim=64, total_num_pages=16, page_size=16, max_num_seqs=3,
           pages_per_seq=4, sm_scale=0.125)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("change,code", [
    ({}, rpa.RPA_OK),
    (dict(max_groups=3), rpa.RPA_OK),
    (dict(max_groups=4), rpa.RPA_ERR_INVALID_ARG),
    (dict(max_groups=0), rpa.RPA_ERR_INVALID_ARG),
    (dict(sliding_window=100), rpa.RPA_ERR_UNSUPPORTED),  # rows of a group would see different parts of the prefix
    (dict(is_causal=False), rpa.RPA_ERR_UNSUPPORTED),
    (dict(soft_cap=30.0, kv_dtype="fp8_e4m3", k_scale=0.1), rpa.RPA_OK),
    (dict(head_dim=576, v_head_dim=512, kv_layout="latent", num_q_heads=16, num_kv_heads=1), rpa.RPA_ERR_UNSUPPORTED),
    (dict(num_q_tokens=(1 << 31) - 60), rpa.RPA_ERR_UNSUPPORTED),
    (dict(head_dim=80), rpa.RPA_ERR_UNSUPPORTED),
    (dict(page_size=1 << 20, pages_per_seq=1 << 10), rpa.RPA_OK),
    (dict(page_size=1 << 20, pages_per_seq=(1 << 10) + 1), rpa.RPA_ERR_UNSUPPORTED),  # keys of a piece behind 2^30 others
])
def test_validate(change, code):
    assert rpa.validate_prefix_cfg(**dict(CFG, **change)) == code


def test_null_arguments():
    L = rpa.lib()
    assert L.rpa_prefix_validate_cfg(None, 1) == rpa.RPA_ERR_INVALID_ARG
    assert L.rpa_prefix_forward(None, None, None, None, None, None, 0, None, None, 0, None, None) == rpa.RPA_ERR_INVALID_ARG
    assert L.rpa_prefix_get_status(None, None) == rpa.RPA_ERR_INVALID_ARG
    assert L.rpa_prefix_create(ctypes.byref(rpa.make_cfg(**CFG)), 1, None) == rpa.RPA_ERR_INVALID_ARG
    L.rpa_prefix_destroy(None)


def _op(**over):
    a = object.__new__(SharedPrefixAttention)  # argument checks only: no handle
    a._h = None
    a._c = rpa.make_cfg(**dict(CFG, **over))
    a._checks(a._c)
    return a


def _i(*n):
    return torch.zeros(*n, dtype=torch.int32)


def _args():
    q = torch.zeros(22, 4, 64, dtype=torch.bfloat16)
    return dict(q=q, kv_pages=torch.zeros(16, 16, 4, 64, dtype=torch.bfloat16), kv_lens=_i(3), page_indices=_i(3, 4), cu_q_lens=_i(4),
                cu_groups=_i(3), prefix_lens=_i(2), num_groups=2, out=torch.zeros_like(q))


def test_well_formed_arguments_pass():
    _op()._check(**_args())
    _op()._check(**dict(_args(), cu_groups=_i(9), prefix_lens=_i(9)))


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(22, 4, 64)), ("out", torch.zeros(22, 4, 64)), ("kv_pages", torch.zeros(16, 16, 4, 64)), ("kv_lens", _i(2)),
    ("page_indices", _i(3, 3)), ("cu_q_lens", _i(3)), ("cu_groups", _i(2)), ("prefix_lens", _i(1)),
    ("prefix_lens", torch.zeros(2, dtype=torch.int64)), ("cu_groups", _i(3, 1)),
])
def test_malformed_arguments_are_refused(name, bad):
    with pytest.raises(ValueError):
        _op()._check(**dict(_args(), **{name: bad}))
