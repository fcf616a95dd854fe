"""Calls of the paged cache's operators that their documentation allows and that the tests of each operator's values do
not make: a fresh handle's first call on a stream of its own, and more."""
import math
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
from cache_util import Batch  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def same(a, b):
    raw = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t  # noqa: E731
    return torch.equal(raw(a), raw(b))


class Calls:
    """One batch, and a call of each handle kind on it: make(kind) a handle, call(kind, handle, stream) its output."""

    KINDS = ("forward", "rope", "prefix", "accumulate", "compact")

    def __init__(self, seed, kv="bf16"):
        scale = None if kv == "bf16" else 0.05
        b = self.b = Batch(np.random.default_rng(seed), [1, 30, 2, 1], [300, 64, 90, 700], 16, 8, 2, 128, kv=kv, k_scale=scale, v_scale=scale)
        self.cache, self.q, self.lens = b.cache(), b.queries(), b.lens()
        self.kv = [b.queries()[:, :2].contiguous() for _ in range(2)]
        self.groups = torch.tensor([0, 1, b.S], dtype=torch.int32, device="cuda")
        self.prefix_lens = torch.tensor([200, 0], dtype=torch.int32, device="cuda")
        self.scores = torch.rand(b.N, 2, 16, device="cuda")

    def make(self, kind):
        cfg = self.b.cfg()
        return {"forward": lambda: rpa.RaggedPagedAttention(**cfg), "rope": lambda: rpa.RopeAppend(**cfg),
                "prefix": lambda: rpa.SharedPrefixAttention(max_groups=2, **cfg),
                "accumulate": lambda: rpa.CacheEviction(budget=60, **cfg), "compact": lambda: rpa.CacheEviction(budget=60, **cfg)}[kind]()

    def buffers(self):
        """What a call writes, in buffers of its own."""
        return [torch.zeros_like(self.q), self.cache.clone(), self.scores.clone(), torch.zeros_like(self.lens[0])]

    def call(self, kind, op, out, stream=None):
        q, cache, scores, kvl = out
        lens, table, cu = self.lens
        S = self.b.S
        if kind == "forward":
            op.forward(self.q, cache, lens, table, cu, S, out=q, stream=stream)
        elif kind == "rope":
            op.append(self.q, *self.kv, cache, lens, table, cu, S, q_out=q, stream=stream)
        elif kind == "prefix":
            op.forward(self.q, cache, lens, table, cu, S, self.groups, self.prefix_lens, 2, out=q, stream=stream)
        elif kind == "accumulate":
            op.accumulate(self.q, cache, lens, table, cu, S, scores, stream=stream)
        else:
            op.compact(cache, scores, lens, table, S, new_kv_lens=kvl, stream=stream)


@pytest.mark.parametrize("kind", Calls.KINDS)
def test_first_call_of_a_fresh_handle_on_a_stream_of_its_own(kind):
    """A side stream does not wait for the default one, which is still busy when the handle is made: what the handle's
    memory starts with is there all the same."""
    x = Calls(0)
    old = x.make(kind)
    want = x.buffers()
    x.call(kind, old, want)
    out, side = x.buffers(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    fresh = x.make(kind)
    x.call(kind, fresh, out, side)
    assert fresh.status(side) == rpa.RPA_OK
    torch.cuda.synchronize()
    assert fresh.status(side) == rpa.RPA_OK
    assert all(same(a, b) for a, b in zip(out, want))
    # the handle's memory was not set after its first call either
    again = x.buffers()
    x.call(kind, fresh, again, side)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(again, want)) and fresh.status(side) == rpa.RPA_OK


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_prefix_calls_of_different_groupings_in_turn(kv):
    """Calls on one handle that follow each other without a wait, each with other groups, so that the row of the page
    table of every virtual sequence changes from call to call: a row of the call before would give other keys."""
    from gpu_util import TOL

    scale = dict(k_scale=0.05, v_scale=0.05) if kv != "bf16" else {}
    rng = np.random.default_rng(1)
    S, pre = 24, 160
    q_lens = [int(n) for n in rng.choice([1, 1, 1, 3, 20], S)]
    b = Batch(rng, q_lens, [pre + n + int(x) for n, x in zip(q_lens, rng.integers(0, 150, S))], 16, 8, 2, 128, kv=kv, **scale)
    for s in range(S):  # pairs of neighbours share 160 keys: any grouping of whole pairs' halves is a valid one
        b.table[s, :10] = b.table[s - s % 2, :10]
    cache, q = b.cache(), b.queries()
    kvl, table, cu = b.lens()
    args = (q, cache, kvl, table, cu, S)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    groupings = []
    for n in range(8):
        # pair p is one group with a prefix, or two groups of one, or a part of a group without a prefix
        cu_groups, lens = [0], []
        for p in range(S // 2):
            kind = int(rng.integers(0, 3))
            if kind == 0:
                cu_groups.append(2 * p + 2)
                lens.append(int(rng.integers(1, pre + 1)))
            elif kind == 1:
                cu_groups += [2 * p + 1, 2 * p + 2]
                lens += [int(rng.integers(0, pre + 1)), 0]
            elif lens and lens[-1] == 0:
                cu_groups[-1] = 2 * p + 2
            else:
                cu_groups.append(2 * p + 2)
                lens.append(0)
        groupings.append((i32(cu_groups), i32(lens), len(lens)))
    op, plain = rpa.SharedPrefixAttention(max_groups=S, **b.cfg()), rpa.RaggedPagedAttention(**b.cfg())
    ref = plain.forward(*args).double().cpu().numpy()
    want = []
    for g in groupings:
        want.append(op.forward(*args, *g))
        torch.cuda.synchronize()
        # the prefix's definition is plain attention's: both are within a + r |exact| of the exact result
        a, r = TOL[kv]
        assert (np.abs(want[-1].double().cpu().numpy() - ref) <= 2 * (a + r * (np.abs(ref) + a) / (1 - r))).all()
    order = [int(n) for n in rng.integers(0, 8, 60)]
    outs = [op.forward(*args, *groupings[n]) for n in order]
    assert op.status() == rpa.RPA_OK
    for n, got in zip(order, outs):
        assert torch.equal(got, want[n])


class Chain:
    """Appends of other values to the same slots, each read by an operator right behind it: nothing of the append before
    may be seen."""

    def __init__(self, seed, q_lens, kv_lens, kv="bf16", D=128):
        scale = dict(k_scale=0.05, v_scale=0.05) if kv != "bf16" else {}
        b = self.b = Batch(np.random.default_rng(seed), q_lens, kv_lens, 16, 8, 2, D, kv=kv, **scale)
        self.inputs = [[b.queries(), b.queries()[:, :2].contiguous(), b.queries()[:, :2].contiguous()] for _ in range(4)]
        self.cache, self.lens = b.cache(), b.lens()
        self.rope = rpa.RopeAppend(**b.cfg())
        self.order = [int(n) for n in b.rng.integers(0, 4, 40)]

    def check(self, read):
        """read(q) -> a fresh output tensor."""
        step = lambda n: read(self.rope.append(*self.inputs[n], self.cache, *self.lens, self.b.S))  # noqa: E731
        want = []
        for n in range(4):
            torch.cuda.synchronize()
            want.append(step(n))
        torch.cuda.synchronize()
        assert not torch.equal(want[0], want[1])
        outs = [step(n) for n in self.order]
        assert self.rope.status() == rpa.RPA_OK
        for n, got in zip(self.order, outs):
            assert torch.equal(got, want[n])


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 64), ("fp8_e4m3", 256)])
def test_weights_of_keys_that_the_call_before_wrote(kv, D):
    """Prompts of many rows, whose logits are computed twice, from K rows that an append in front of the call wrote."""
    x = Chain(2, [40, 200, 1], [40, 260, 90], kv=kv, D=D)
    op = rpa.CacheEviction(budget=1, **x.b.cfg())
    x.check(lambda q: op.accumulate(q, x.cache, *x.lens, x.b.S, torch.zeros(x.b.N, 2, 16, device="cuda")))
    assert op.status() == rpa.RPA_OK


@pytest.mark.parametrize("kind", ["forward", "prefix"])
@pytest.mark.parametrize("kv,D", [("bf16", 128), ("f16", 64), ("fp8_e4m3", 128)])
def test_attention_of_keys_that_the_call_before_wrote(kind, kv, D):
    """Decodes beside prompts, whose kernels run at once, over K/V rows and queries that an append in front wrote."""
    x = Chain(3, [1, 200, 1, 60, 1], [700, 260, 90, 60, 300], kv=kv, D=D)
    b = x.b
    if kind == "forward":
        op = rpa.RaggedPagedAttention(**b.cfg())
        read = lambda q: op.forward(q, x.cache, *x.lens, b.S)  # noqa: E731
    else:
        op = rpa.SharedPrefixAttention(max_groups=3, **b.cfg())
        groups, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1, 4, 5], [600, 0, 250]))
        read = lambda q: op.forward(q, x.cache, *x.lens, b.S, groups, lens, 3)  # noqa: E731
    x.check(read)
    assert op.status() == rpa.RPA_OK


def test_no_sequences_and_no_groups():
    """A step without work: the tensor of the groups' prefixes is empty, its address NULL."""
    b = Batch(np.random.default_rng(4), [3], [20], 16, 4, 2, 64)
    op = rpa.SharedPrefixAttention(max_groups=1, **b.cfg())
    kvl, table, cu = b.lens()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert none[:0].data_ptr() == 0
    out = torch.full((b.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    op.forward(b.queries(), b.cache(), kvl, table, cu, 0, none, none[:0], 0, out=out)
    assert op.status() == rpa.RPA_OK and (out == 0).all()
    with pytest.raises(rpa.RpaError):  # sequences have groups
        op.forward(b.queries(), b.cache(), kvl, table, cu, 1, none, none[:0], 0, out=out)
    op.forward(b.queries(), b.cache(), kvl, table, cu, 1, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), none, 1, out=out)
    assert op.status() == rpa.RPA_OK and not (out == 0).all()


def test_rotation_in_place_of_a_slice_is_refused():
    """q_out is contiguous: with q a slice of wider rows from the same address on, the rows of one token would land on
    those of others that are still to be read."""
    b = Batch(np.random.default_rng(5), [9], [20], 16, 4, 2, 64)
    wide = torch.zeros(b.T * 8 * 64, dtype=torch.bfloat16, device="cuda")
    q, q_out = wide.view(b.T, 8, 64)[:, :4], wide[:b.T * 4 * 64].view(b.T, 4, 64)
    k, v = b.queries()[:, :2].contiguous(), b.queries()[:, :2].contiguous()
    cache, lens = b.cache(), b.lens()
    before = cache.clone()
    op = rpa.RopeAppend(**b.cfg())
    with pytest.raises(rpa.RpaError) as e:
        op.append(q, k, v, cache, *lens, 1, q_out=q_out)
    assert e.value.code == rpa.RPA_ERR_INVALID_ARG and torch.equal(cache, before)
    # contiguous in place, and one token of a wider row in place, are fine
    x = b.queries()
    want = op.append(x.clone(), k, v, cache, *lens, 1)
    assert same(op.append(x, k, v, cache, *lens, 1, q_out=x), want)
    one = Batch(np.random.default_rng(6), [1], [20], 16, 4, 2, 64, tail=0)
    op1 = rpa.RopeAppend(**one.cfg())
    row = torch.randn(1, 8, 64, device="cuda").bfloat16()
    want = op1.append(row[:, :4].clone(), row[:, 4:6], row[:, 6:], one.cache(), *one.lens(), 1)
    op1.append(row[:, :4], row[:, 4:6], row[:, 6:], one.cache(), *one.lens(), 1, q_out=row[:, :4])
    assert same(row[:, :4], want) and op1.status() == op.status() == rpa.RPA_OK


def test_one_head_of_any_stride():
    """Keys kept as [head, token, D] and values out of a wider tensor give what contiguous ones give."""
    b = Batch(np.random.default_rng(7), [5, 2], [20, 70], 16, 4, 1, 64)
    q, op = b.queries(), rpa.RopeAppend(**b.cfg())
    k, v = b.queries()[:, :1], b.queries()[:, 1:2]
    cache = b.cache()
    c1, c2 = cache.clone(), cache.clone()
    op.append(q, k.contiguous(), v.contiguous(), c1, *b.lens(), b.S)
    op.append(q, k.transpose(0, 1).contiguous().transpose(0, 1), v, c2, *b.lens(), b.S)
    assert same(c1, c2) and not same(c1, cache) and op.status() == rpa.RPA_OK


def test_more_keys_than_the_weights_can_count():
    """Sequences that share one page as often as their tables allow: 17 x 2^30 keys of 8 heads are 17 x 2^27 blocks of 64,
    past 31 bits.  Refused, and the scores are left as they were; 2^10 keys of the same sequences are weighed."""
    S, ps = 17, 1 << 16
    cfg = dict(num_q_tokens=S, num_q_heads=8, num_kv_heads=8, head_dim=64, total_num_pages=1, page_size=ps, max_num_seqs=S,
               pages_per_seq=(1 << 30) // ps, sm_scale=0.125, kv_dtype="int8", k_scale=0.02)
    op = rpa.CacheEviction(budget=1, **cfg)
    q = torch.randn(S, 8, 64, device="cuda").bfloat16()
    cache = torch.randint(-100, 100, (1, ps, 16, 64), dtype=torch.int8, device="cuda")
    table = torch.zeros(S, cfg["pages_per_seq"], dtype=torch.int32, device="cuda")
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    scores = torch.full((1, 8, ps), 3.0, device="cuda")
    lens = torch.full((S,), 1 << 30, dtype=torch.int32, device="cuda")
    op.accumulate(q, cache, lens, table, cu, S, scores)
    assert op.status() == rpa.RPA_ERR_BAD_LENGTHS and (scores == 3.0).all()
    lens.fill_(1 << 10)
    op.accumulate(q, cache, lens, table, cu, S, scores)
    assert op.status() == rpa.RPA_OK and (scores[0, :, 1 << 10:] == 3.0).all() and (scores[0, :, :1 << 10] != 3.0).all()


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def turns(w, p):
    """The angle p w as a fraction of a turn in [-1/2, 1/2), exact but for the 80 digits of pi."""
    x = Fraction(w) * int(p) / (2 * PI)
    return x - math.floor(x + Fraction(1, 2))


@pytest.mark.parametrize("rope", [dict(base=10000.0), dict(base=500000.0, scaling="rotations", factor=8.0, trained_len=8192)])
def test_angles_of_far_positions(rope):
    """Pair i turned at positions p where p w_i is just beside a whole turn: there the sine shows the angle itself.  The
    fraction of a turn is off by 2^-34 (p times the rounding of w_i / 2 pi, 2^-65) and 2^-33 (its upper 32 bits), the sine
    relative to its size by 2^-24 (its argument as a float) and 2 units of 2^-23 (sincospi): of angles below 2^-9 of a
    turn 2 pi (2^-34 + 2^-33 + 2.5 2^-23 2^-9) at most."""
    b = Batch(np.random.default_rng(8), [128], [128], 16, 1, 1, 128, q="f32")
    w = rpa.rope_frequencies(**rope, **b.cfg())
    pos = np.zeros(128, np.int32)
    for i in range(64):
        f = int(Fraction(w[i]) * (1 << 300) / (2 * PI))  # turns a position, of 300 bits
        at, n = ((1 << 31) - 1) * f >> 300, 0  # whole turns
        while n < 2:
            p = (at * (1 << 300) + (1 << 289)) // f  # about 2^-11 of a turn past them
            if p < 1 << 31 and 1 << 286 < abs((p * f + (1 << 299)) % (1 << 300) - (1 << 299)) < 1 << 291:  # 2^-14 .. 2^-9
                pos[2 * i + n] = -p if n else p
                n += 1
            at -= 1
    q = torch.zeros(128, 1, 128, device="cuda")
    q[:, 0, :64] = 1.0  # the sine of each pair lands in its second element
    out = torch.zeros_like(q)
    op = rpa.RopeAppend(**rope, **b.cfg())
    kv = torch.zeros(128, 1, 128, device="cuda")
    op.append(q, kv, kv, b.cache(), *b.lens(), 1, positions=torch.from_numpy(pos).cuda(), q_out=out)
    assert op.status() == rpa.RPA_OK
    out = out.double().cpu().numpy()
    for k in range(128):
        want = math.sin(2 * math.pi * float(turns(w[k // 2], pos[k])))
        assert abs(out[k, 0, 64 + k // 2] - want) <= 2 * math.pi * (2.0 ** -34 + 2.0 ** -33 + 2.5 * 2.0 ** -32), (k, pos[k])


def test_memory_of_a_shared_prefix_handle():
    """256 tokens and sequences of 32 / 8 heads, D 128, one group: partial rows of 130 floats for (2 x 4 + 113 + 1 + 3) tiles
    of 256 rows a kv head (113 sequences can have more than 8 rows; 3 of rounding up), (257 + 1) pieces of 16 rows a kv head,
    and for each of the GPU's CTAs 4 tiles (one an SM) and 4 pieces (three an SM); a MB for the rest."""
    cfg = dict(num_q_tokens=256, num_q_heads=32, num_kv_heads=8, head_dim=128, total_num_pages=64, page_size=16, max_num_seqs=256,
               pages_per_seq=64, sm_scale=0.1)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 8 * 256 * (2 * 4 + 113 + 1 + 3) + 8 * 16 * 258 + sms * (4 * 256 + 4 * 3 * 16)
    torch.cuda.synchronize()
    ops = [rpa.SharedPrefixAttention(**cfg)]  # what the first handle of a process loads is no handle's
    before = torch.cuda.mem_get_info()[0]
    ops += [rpa.SharedPrefixAttention(**cfg) for _ in range(4)]
    each = (before - torch.cuda.mem_get_info()[0]) / 4
    assert each <= rows * 130 * 4 + (4 << 20), (each, rows * 130 * 4)
