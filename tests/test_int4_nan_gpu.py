"""Rows whose every visible logit is a NaN come out as NaN over a 4-bit cache, whole or cut into pieces."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as i4  # noqa: E402
import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch, f64, half_step  # noqa: E402
from test_int4_attention_gpu import Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def holds(c, got, nan, knobs):
    """`nan` [T, Hq, D] are NaN, everything else is the definition's (the direct kernel's tolerance, as in Case.check)."""
    ref, size, steps = c.reference(**knobs)
    e = 2.0 ** -14 + (16 * half_step("f16") if c.b.q == "f32" else 0)
    tol = half_step(c.b.q) * np.abs(ref) + 1e-6 + 8 * half_step("f16") * steps + 2 * e * size
    assert np.isnan(got[nan]).all()
    assert (np.abs(got - ref) <= tol)[~nan].all()


SHAPES = [  # Hq, Hkv, D, group, q, q_lens, kv_lens; the last two in pieces
    (8, 2, 128, 64, "bf16", [1, 1, 1, 1], [1, 5, 33, 700]),
    (13, 1, 64, 32, "f16", [1, 1, 1], [1, 64, 300]),
    (4, 2, 256, 128, "f32", [1, 2, 1], [1, 50, 300]),
    (8, 2, 128, 128, "bf16", [1, 2], [30000, 12000]),
    (16, 1, 256, 64, "f16", [1], [20000]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("sinks", [False, True])
def test_nan_in_a_query(shape, sinks):
    Hq, Hkv, D, group, q, q_lens, kv_lens = shape
    c = Case([20, D, Hq], q_lens, kv_lens, 16, Hq, Hkv, D, group, q)
    knobs = dict(sinks=c.b.rng.standard_normal(Hq).astype(np.float32)) if sinks else {}
    clean, c.q = c.q, c.q.clone()
    nan = np.zeros((c.b.T, Hq, D), bool)
    for i, t in enumerate(range(c.b.cu[0], c.b.cu[c.b.S])):
        h = (5 * i + 1) % Hq
        c.q[t, h, 7 * i % D] = float("nan")
        nan[t, h] = True
    att = c.make(**knobs)
    got = f64(att.forward(c.q, c.cache, *c.lens, c.b.S))
    assert att.status() == rpa.RPA_OK
    c.q = clean
    holds(c, got, nan, knobs)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("part", ["K", "V"])
def test_nan_in_every_key(shape, part):
    """Of kv head 0 of sequence 0: K's make whole rows NaN, a group of V's its own channels."""
    Hq, Hkv, D, group, q, q_lens, kv_lens = shape
    c = Case([21, D, Hq], q_lens, kv_lens, 16, Hq, Hkv, D, group, q)
    page, place = c.b.slots(0, np.arange(kv_lens[0]))
    parts = [tuple(x.copy() for x in p) for p in c.parts]
    parts[part == "V"][2][page, place, 0, 0] = np.nan
    cache = torch.from_numpy(i4.pack(parts, 16, D, group)).cuda()
    att = c.make()
    got = f64(att.forward(c.q, cache, *c.lens, c.b.S))
    assert att.status() == rpa.RPA_OK
    nan = np.zeros((c.b.T, Hq, D), bool)
    nan[c.b.cu[0]:c.b.cu[1], :Hq // Hkv, :D if part == "K" else group] = True
    holds(c, got, nan, {})


def test_pieces_of_an_8bit_cache():
    """The merge of pieces is shared with the 8-bit caches' kernel, whose unsplit rows show a NaN as well."""
    b = Batch(np.random.default_rng(22), [1, 1], [30000, 200], 16, 8, 2, 128, kv="fp8_e4m3", k_scale=0.05, v_scale=0.05)
    q, cache = b.queries(), b.cache()
    q[0, 3, 5] = q[1, 6, 0] = float("nan")
    att = rpa.RaggedPagedAttention(**b.cfg())
    got = torch.isnan(att.forward(q, cache, *b.lens(), b.S))
    assert att.status() == rpa.RPA_OK
    assert got[0, 3].all() and got[1, 6].all() and got.sum() == 2 * 128
