"""Rotary append on the CPU: configurations, frequencies and the binding's refusals."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import frequencies  # noqa: E402
from ragged_paged_attention_02_gb300.cache import RopeAppend, make_rope_cfg  # noqa: E402

CFG = dict(num_q_tokens=22, num_q_heads=4, num_kv_heads=2, head_dim=64, total_num_pages=16, page_size=16, max_num_seqs=3,
           pages_per_seq=4, sm_scale=0.125)
LATENT = dict(CFG, head_dim=576, v_head_dim=512, kv_layout="latent", num_q_heads=16, num_kv_heads=1)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("cfg,code", [
    (dict(CFG), rpa.RPA_OK),
    (dict(CFG, rotary_dim=16, rotary_offset=48), rpa.RPA_OK),
    (dict(CFG, rotary_dim=16, rotary_offset=8), rpa.RPA_OK),
    (dict(LATENT, rotary_dim=64, rotary_offset=512), rpa.RPA_OK),
    (dict(CFG, rotary_dim=24), rpa.RPA_ERR_UNSUPPORTED),
    (dict(CFG, rotary_dim=32, rotary_offset=4), rpa.RPA_ERR_UNSUPPORTED),
    (dict(CFG, rotary_dim=64, rotary_offset=8), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, rotary_dim=0), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, rotary_dim=128), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, rotary_offset=-8), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, base=1.0), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, base=float("nan")), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, magnitude=float("inf")), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, scaling="linear", factor=0.5), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, scaling="linear", factor=4.0), rpa.RPA_OK),
    (dict(CFG, scaling="rotations", factor=4.0), rpa.RPA_ERR_INVALID_ARG),  # no trained_len
    (dict(CFG, scaling="index", factor=4.0, trained_len=4096, low=4.0, high=4.0), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, scaling="index", factor=4.0, trained_len=4096, low=1.0, high=32.0), rpa.RPA_OK),
    (dict(CFG, kv_dtype="fp8_e4m3", k_scale=0.0), rpa.RPA_ERR_INVALID_ARG),
    (dict(CFG, head_dim=96), rpa.RPA_ERR_UNSUPPORTED),  # the cache's own checks come first
])
def test_validate(cfg, code):
    assert rpa.validate_rope_cfg(**cfg) == code


def test_validate_rejects_unknown_codes_and_reserved():
    c = make_rope_cfg(**CFG)
    ok = rpa.lib().rpa_rope_validate_cfg
    for field, bad in (("pairing", 2), ("scaling", 5), ("scaling", -1), ("reserved", 1)):
        c = make_rope_cfg(**CFG)
        setattr(c, field, bad)
        assert ok(ctypes.byref(c)) == rpa.RPA_ERR_INVALID_ARG, field
    assert ok(None) == rpa.RPA_ERR_INVALID_ARG


@pytest.mark.parametrize("rope", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0, base=1e6),
    dict(scaling="rotations", factor=8.0, trained_len=8192, low=1.0, high=4.0),
    dict(scaling="index", factor=16.0, trained_len=4096, low=1.0, high=32.0),
    dict(scaling="index", factor=2.0, trained_len=30, low=1.0, high=32.0),  # the ramp starts at 0
])
@pytest.mark.parametrize("rd", [16, 64])
def test_frequencies(rope, rd):
    got = rpa.rope_frequencies(rotary_dim=rd, **rope, **CFG)
    # pow, log and a blend in 64 bits on both sides: a few units of 2^-53
    np.testing.assert_allclose(got, frequencies(rd, **rope), rtol=2e-14)
    assert got[0] <= 1.0


def test_cfg_init_defaults():
    from ragged_paged_attention_02_gb300.binding import RpaRopeCfg

    c = RpaRopeCfg()
    c.cache.num_q_tokens, c.cache.num_q_heads, c.cache.num_kv_heads, c.cache.head_dim = 22, 4, 2, 64
    c.cache.total_num_pages, c.cache.page_size, c.cache.max_num_seqs, c.cache.pages_per_seq = 16, 16, 3, 4
    c.reserved = 7
    rpa.lib().rpa_rope_cfg_init(ctypes.byref(c))
    assert (c.rotary_dim, c.rotary_offset, c.base, c.magnitude, c.reserved) == (64, 0, 10000.0, 1.0, 0)
    assert rpa.lib().rpa_rope_validate_cfg(ctypes.byref(c)) == rpa.RPA_OK


def test_null_arguments():
    L = rpa.lib()
    assert L.rpa_rope_append(None, None, 0, None, 0, None, 0, None, None, None, None, None, 0, None, None) == rpa.RPA_ERR_INVALID_ARG
    assert L.rpa_rope_get_status(None, None) == rpa.RPA_ERR_INVALID_ARG
    assert L.rpa_rope_create(ctypes.byref(make_rope_cfg(**CFG)), None) == rpa.RPA_ERR_INVALID_ARG
    h = ctypes.c_void_p(1)
    assert L.rpa_rope_create(ctypes.byref(make_rope_cfg(**dict(CFG, rotary_dim=24))), ctypes.byref(h)) == rpa.RPA_ERR_UNSUPPORTED
    assert not h.value
    assert L.rpa_rope_frequencies(ctypes.byref(make_rope_cfg(**CFG)), None) == rpa.RPA_ERR_INVALID_ARG
    L.rpa_rope_destroy(None)


def _op(**over):
    a = object.__new__(RopeAppend)  # argument checks only: no handle
    a._h = None
    a._c = make_rope_cfg(**dict(CFG, **over))
    a._checks(a._c.cache)
    return a


def _args():
    qkv = torch.zeros(22, 8, 64, dtype=torch.bfloat16)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    return dict(q=qkv[:, :4], k=qkv[:, 4:6], v=qkv[:, 6:], kv_pages=torch.zeros(16, 16, 4, 64, dtype=torch.bfloat16), kv_lens=i(3),
                page_indices=i(3, 4), cu_q_lens=i(4), positions=i(22), q_out=torch.zeros(22, 4, 64, dtype=torch.bfloat16))


def test_well_formed_arguments_pass():
    _op()._check(**_args())
    _op()._check(**dict(_args(), positions=None))
    _op(kv_dtype="int8")._check(**dict(_args(), kv_pages=torch.zeros(16, 16, 4, 64, dtype=torch.int8)))


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(22, 4, 64)), ("q", torch.zeros(22, 5, 64, dtype=torch.bfloat16)),
    ("q", torch.zeros(22, 4, 128, dtype=torch.bfloat16)[..., ::2]),
    ("q", torch.zeros(4, 22, 64, dtype=torch.bfloat16).transpose(0, 1)),  # heads are not contiguous
    ("k", torch.zeros(22, 4, 64, dtype=torch.bfloat16)), ("v", None),
    ("kv_pages", torch.zeros(16, 16, 4, 64, dtype=torch.uint8)), ("kv_pages", torch.zeros(16, 16, 2, 64, dtype=torch.bfloat16)),
    ("kv_lens", torch.zeros(3, dtype=torch.int64)), ("page_indices", torch.zeros(3, 5, dtype=torch.int32)),
    ("cu_q_lens", torch.zeros(3, dtype=torch.int32)), ("positions", torch.zeros(22, dtype=torch.int64)),
    ("q_out", torch.zeros(22, 4, 64)),
])
def test_malformed_arguments_are_refused(name, bad):
    with pytest.raises(ValueError):
        _op()._check(**dict(_args(), **{name: bad}))


def test_closed_handle_is_refused():
    a = _op()
    with pytest.raises(ValueError, match="closed"):
        a.status()
