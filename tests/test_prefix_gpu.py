"""Shared-prefix attention on the GPU: rpa_forward's definition, so the oracle and the stated tolerances of rpa_forward
(2e-2 + 2e-2 |o| for 2-byte K/V, 6e-2 for 8-bit K/V).  The merge adds partials in 32 bits to kernels that meet them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import ragged_paged_attention_02_gb300 as rpa  # noqa: E402
import rpa_inputs as ri  # noqa: E402
from cache_util import Batch, f64  # noqa: E402
from gpu_util import assert_close  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


class Shared:
    """groups: [(prefix length, [(q_len, keys behind the prefix)])].  Whole prefix pages are the first sequence's in
    the plain table, and no pages at all (an id past the cache) in the table that the operator gets; the page in which
    a prefix ends holds the same keys in every sequence."""

    def __init__(self, seed, groups, ps, Hq, Hkv, D, **more):
        rng = np.random.default_rng(seed)
        self.groups = groups
        seqs = [(n, pre + max(own, n)) for pre, g in groups for n, own in g]
        b = self.b = Batch(rng, [n for n, _ in seqs], [kl for _, kl in seqs], ps, Hq, Hkv, D, **more)
        self.cu_groups = np.cumsum([0] + [len(g) for _, g in groups]).astype(np.int32)
        self.prefix_lens = np.array([pre for pre, _ in groups], np.int32)
        self.cache, self.q = b.cache(), b.queries()
        self.table = b.table.copy()
        raw = self.cache.view(torch.uint8) if self.cache.element_size() == 1 else self.cache
        for g, (pre, members) in enumerate(groups):
            lo, hi = self.cu_groups[g], self.cu_groups[g + 1]
            if hi == lo:
                continue
            n = pre // ps
            b.table[lo:hi, :n] = b.table[lo, :n]
            self.table[lo:hi, :n] = b.table[lo, :n]
            self.table[lo + 1:hi, :n] = b.N + 7
            if pre % ps:
                for s in range(lo + 1, hi):
                    raw[b.table[s, n], :pre % ps] = raw[b.table[lo, n], :pre % ps]

    def args(self):
        kvl, _, cu = self.b.lens()
        d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        return (self.q, self.cache, kvl, d(self.table), cu, self.b.S, d(self.cu_groups), d(self.prefix_lens), len(self.groups))

    def op(self, **more):
        return rpa.SharedPrefixAttention(max_groups=len(self.groups), **dict(self.b.cfg(), **more))

    def reference(self):
        b = self.b
        q = self.q.cpu()
        kv = self.cache.cpu()
        bits = {2: torch.int16, 1: torch.uint8}
        kvn = kv.numpy() if b.kv == "int8" else kv.view(bits[kv.element_size()]).numpy()
        kvn = kvn.view(ri.KV_STORAGE[b.kv])
        qn = q.numpy() if b.q == "f32" else q.view(torch.int16).numpy().view(np.uint16)
        p = ri.Problem(**b.cfg(), num_seqs=b.S, q=qn, kv_pages=kvn, kv_lens=b.kv_lens, page_indices=b.table, cu_q_lens=b.cu)
        return oracle.forward(p)

    def check(self):
        op = self.op()
        o = op.forward(*self.args())
        assert op.status() == rpa.RPA_OK
        got, ref = f64(o), self.reference()
        assert_close(got, ref, self.b.kv, "shared prefix")
        rest = np.ones(self.b.T, bool)
        rest[self.b.cu[0]:self.b.cu[self.b.S]] = False
        assert (got[rest] == 0).all()
        return op, o


one = lambda *own: [(1, n) for n in own]  # noqa: E731
GROUPS = [
    (0, [(64, one(1))]),                                                     # one sequence, one key of its own
    (1, [(100, one(5, 30, 1, 200))]),                                        # the prefix ends inside a page
    (2, [(1, one(7, 9)), (0, one(40, 3)), (3, one(1))]),                     # hardly any prefix, none
    (3, [(1500, one(*range(1, 40)))]),
    (4, [(300, [(1, 10), (0, 5), (4, 4), (2, 90)]), (130, [(3, 8)])]),       # several tokens, a sequence without any
    (5, [(640, [(30, 50), (1, 10), (70, 70), (1, 1)])]),                     # prompt chunks beside decodes
    (6, [(500, one(3, 600)), (0, []), (700, one(*[20] * 9)), (64, one(1, 1))]),  # an empty group
    (7, [(2000, [(2, 20)] * 20), (999, [(150, 300)]), (128, one(2000, 900))]),
]
SHAPES = [
    dict(Hq=8, Hkv=2, D=128, ps=16), dict(Hq=4, Hkv=4, D=64, ps=8), dict(Hq=12, Hkv=4, D=64, ps=64), dict(Hq=16, Hkv=1, D=128, ps=32),
    dict(Hq=10, Hkv=2, D=256, ps=16), dict(Hq=64, Hkv=1, D=64, ps=16), dict(Hq=4, Hkv=2, D=128, ps=4),
]


@pytest.mark.parametrize("seed,groups", GROUPS)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_against_the_oracle(seed, groups, shape, kv):
    scale = dict(k_scale=0.05, v_scale=0.07) if kv == "fp8_e4m3" else {}
    Shared(seed, groups, kv=kv, lead=seed % 2, tail=seed % 3, **scale, **shape).check()


@pytest.mark.parametrize("more", [
    dict(soft_cap=5.0), dict(sinks=True), dict(q="f32"), dict(q="f16", kv="f16"), dict(q="f16"), dict(kv="f16"), dict(kv="int8", k_scale=0.04, v_scale=0.04),
    dict(kv="fp8_e5m2", k_scale=0.1, v_scale=0.1, q="f32", soft_cap=20.0, sinks=True),
])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_knobs_and_types(more, D):
    more = dict(more)
    if more.get("sinks"):
        more["sinks"] = np.linspace(-3, 3, 8).astype(np.float32)
    Shared(20, [(777, one(5, 30, 1, 200, 17, 60)), (65, [(40, 70), (2, 2)])], ps=16, Hq=8, Hkv=2, D=D, **more).check()


def test_long_prefix_many_pieces():
    Shared(21, [(20011, one(*[50] * 70))], ps=64, Hq=8, Hkv=2, D=128).check()
    Shared(22, [(30000, one(9))], ps=64, Hq=2, Hkv=2, D=64).check()  # decode pieces of a prefix


def test_many_sequences():
    """More virtual sequences than the planner keeps in shared memory, and many groups."""
    rng = np.random.default_rng(29)
    groups = [(int(pre), [(1, int(n)) for n in rng.integers(1, 20, int(k))]) for pre, k in ((200, 900), (0, 300), (17, 400))]
    Shared(29, groups, ps=16, Hq=4, Hkv=2, D=64, lead=2, tail=1).check()
    groups = [(int(rng.integers(0, 300)), [(int(rng.integers(0, 3)), int(n)) for n in rng.integers(1, 40, int(k))]) for k in rng.integers(0, 6, 70)]
    groups.append((64, one(5)))
    Shared(30, groups, ps=16, Hq=8, Hkv=2, D=128).check()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_garbage_in_front_of_a_suffix(kv):
    """The other sequences' copies of the keys before the prefix's end, and everything behind the keys, may hold any bits."""
    scale = dict(k_scale=0.05, v_scale=0.07) if kv == "fp8_e4m3" else {}
    x = Shared(31, [(100, one(5, 30, 1, 200)), (1000, [(2, 9), (40, 50)])], ps=16, Hq=8, Hkv=2, D=128, kv=kv, **scale)
    ref = x.reference()
    b, raw = x.b, x.cache.view(torch.uint8)
    used = torch.zeros(b.N, 16, dtype=torch.bool)
    for g, (pre, members) in enumerate(x.groups):
        for s in range(x.cu_groups[g], x.cu_groups[g + 1]):
            first = 0 if s == x.cu_groups[g] else pre
            page, at = b.slots(s, np.arange(first, b.kv_lens_list[s]))
            used[page, at] = True
    raw[~used.cuda()] = 0x7F if kv == "fp8_e4m3" else 0xFF  # NaN
    op = x.op()
    o = op.forward(*x.args())
    assert op.status() == rpa.RPA_OK
    assert_close(f64(o), ref, kv, "garbage around the keys")


def test_large_scores_meet_across_the_parts():
    """Logits of very different sizes before and behind the prefix's end: either side may hold all the weight."""
    for where in (0, 1):
        x = Shared(23, [(200, one(64, 64, 64))], ps=16, Hq=8, Hkv=2, D=64)
        page, at = x.b.slots(0, np.arange(200))
        if where == 0:
            x.cache[torch.as_tensor(page).long().cuda(), torch.as_tensor(at).long().cuda(), 0::2] *= 30
            for s in (1, 2):  # the shared end of the last prefix page
                x.cache[int(x.b.table[s, 12]), :8] = x.cache[int(x.b.table[0, 12]), :8]
        else:
            for s in range(3):
                page, at = x.b.slots(s, np.arange(208, 264))
                x.cache[torch.as_tensor(page).long().cuda(), torch.as_tensor(at).long().cuda(), 0::2] *= 30
        x.check()


def test_equal_to_itself_alone_and_repeated():
    x = Shared(24, GROUPS[7][1], ps=16, Hq=8, Hkv=2, D=128)
    op, o = x.check()
    for _ in range(5):
        assert torch.equal(o, op.forward(*x.args()))
    # forty calls over two batches without a wait
    y = Shared(25, GROUPS[7][1], ps=16, Hq=8, Hkv=2, D=128)
    xa, ya = x.args(), y.args()
    op2 = y.op(total_num_pages=x.b.N)
    want = op.forward(*ya).clone()
    outs = [op.forward(*(ya if i % 2 else xa)) for i in range(40)]
    for i, got in enumerate(outs):
        assert torch.equal(got, want if i % 2 else o)
    op2.close()


@pytest.mark.parametrize("D", [128, 256])
def test_graph_and_streams(D):
    x = Shared(26, GROUPS[5][1], ps=16, Hq=8, Hkv=2, D=D)
    op, want = x.check()
    args = x.args()
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(*args, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    # other lengths in the captured buffers
    args[2][1] -= 5
    g.replay()
    got = out.clone()
    assert torch.equal(got, op.forward(*args))
    args[2][1] += 5
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = op.forward(*args, stream=side)
    assert op.status(side) == rpa.RPA_OK and torch.equal(a, want)
    # two handles on two streams at once
    op2, s2 = x.op(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [(o.forward(*args, stream=st)) for _ in range(10) for o, st in ((op, side), (op2, s2))]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in outs)


def test_bad_lengths_groups_and_pages():
    x = Shared(27, [(100, one(5, 30, 20)), (40, one(6, 7))], ps=16, Hq=8, Hkv=2, D=64)
    op, want = x.check()
    names = ["q", "kv", "kv_lens", "table", "cu", "S", "cu_groups", "prefix_lens", "groups"]

    def bad(name, at, value):
        args = list(x.args())
        i = names.index(name)
        args[i] = args[i].clone()
        args[i].view(-1)[at] = value
        return op.forward(*args)

    for name, at, value in (("kv_lens", 0, x.b.P * 16 + 1), ("kv_lens", 1, 100), ("cu", 2, 0), ("cu", 5, x.b.T + 1), ("cu_groups", 0, 1),
                            ("cu_groups", 1, 6), ("cu_groups", 1, -1), ("cu_groups", 2, 4), ("prefix_lens", 0, -1), ("prefix_lens", 1, 46),
                            ("prefix_lens", 0, x.b.P * 16 + 1)):
        o = bad(name, at, value)
        assert op.status() == rpa.RPA_ERR_BAD_LENGTHS and (o == 0).all(), (name, at)
    o = bad("table", 2, x.b.N)  # a prefix page of the first sequence
    assert op.status() == rpa.RPA_ERR_BAD_PAGE_INDEX and op.status() == rpa.RPA_OK
    assert torch.equal(o[3:], want[3:])  # the other group's rows
    assert torch.equal(op.forward(*x.args()), want) and op.status() == rpa.RPA_OK
    args = list(x.args())
    for i, v in ((5, x.b.max_seqs + 1), (8, 0)):
        a = list(args)
        a[i] = v
        with pytest.raises(rpa.RpaError):
            op.forward(*a)
    with pytest.raises(ValueError):
        op.forward(*args[:8], 3)
    # no sequences at all
    args[5], args[8] = 0, 0
    assert (op.forward(*args) == 0).all() and op.status() == rpa.RPA_OK


def test_append_share_weigh_and_attend():
    """A shared prompt written once, three questions behind it: the operators in a row, as a server calls them."""
    rng = np.random.default_rng(28)
    ps, Hq, Hkv, D = 16, 8, 2, 64
    pre, own = 48, [5, 9, 3]
    b = Batch(rng, own, [pre + n for n in own], ps, Hq, Hkv, D)
    b.table[1:3, :3] = b.table[0, :3]
    cfg = b.cfg()
    kvl, table, cu = b.lens()
    cache = torch.zeros(b.N, ps, 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros(b.N, Hkv, ps, device="cuda")
    mk = lambda n, h: torch.from_numpy(rng.standard_normal((n, h, D)).astype(np.float32)).cuda().bfloat16()  # noqa: E731
    # the prompt, by the first sequence alone
    p_cfg = dict(cfg, num_q_tokens=pre)
    lens0 = torch.tensor([pre, 0, 0, 0], dtype=torch.int32, device="cuda")
    cu0 = torch.tensor([0, pre, pre, pre, pre], dtype=torch.int32, device="cuda")
    prompt = rpa.RopeAppend(**p_cfg)
    prompt.append(mk(pre, Hq), mk(pre, Hkv), mk(pre, Hkv), cache, lens0, table, cu0, 1)
    # the questions
    ask = rpa.RopeAppend(**cfg)
    q = ask.append(mk(b.T, Hq), mk(b.T, Hkv), mk(b.T, Hkv), cache, kvl, table, cu, 3)
    groups, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [pre]))
    shared, plain = rpa.SharedPrefixAttention(max_groups=1, **cfg), rpa.RaggedPagedAttention(**cfg)
    o = shared.forward(q, cache, kvl, table, cu, 3, groups, lens, 1)
    ref = plain.forward(q, cache, kvl, table, cu, 3)
    weigh = rpa.CacheEviction(budget=32, protect=0, recent=4, **cfg)
    weigh.accumulate(q, cache, kvl, table, cu, 3, scores)
    assert all(x.status() == rpa.RPA_OK for x in (prompt, ask, shared, plain, weigh))
    # both round once to bf16 and round P to bf16 in parts of their own: 2 (2^-8 + 2^-8) of at most |v| <= 5
    assert ((o.float() - ref.float()).abs() <= 4 * 2.0 ** -8 * (1 + ref.float().abs())).all()
    # every row's weights add up to 1: heads x tokens in all
    assert abs(scores.sum().item() - Hq * b.T) <= 1e-3
