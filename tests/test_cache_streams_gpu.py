"""The paged cache's operators at once: handles of their own on two streams from two host threads, two graphs of one
handle in turn, and a serving step of all of them in one graph."""
import threading

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


class Step:
    """Append, attend (the first two sequences share their first page), weigh and evict onto fresh pages or in place."""

    def __init__(self, seed, kv, q_lens, kv_lens, in_place, D=128):
        rng = np.random.default_rng(seed)
        b = self.b = Batch(rng, q_lens, kv_lens, 16, 8, 2, D, kv=kv, spare_pages=64, k_scale=0.05 if kv != "bf16" else None,
                           v_scale=0.05 if kv != "bf16" else None)
        b.table[1, 0] = b.table[0, 0]
        cfg = b.cfg()
        self.rope, self.prefix = rpa.RopeAppend(**cfg), rpa.SharedPrefixAttention(max_groups=2, **cfg)
        self.evict = rpa.CacheEviction(budget=90, protect=16, recent=20, **cfg)
        self.cache, self.lens = b.cache(), b.lens()
        self.q, self.k, self.v = b.queries(), b.queries()[:, :2].contiguous(), b.queries()[:, :2].contiguous()
        self.groups = torch.tensor([0, 2, b.S], dtype=torch.int32, device="cuda")
        self.prefix_lens = torch.tensor([16, 0], dtype=torch.int32, device="cuda")
        new = b.table.copy()
        for s in range(b.S):
            new[s, :6] = b.free_pages[6 * s:6 * s + 6]
        self.new = self.lens[1] if in_place else torch.from_numpy(new).cuda()
        self.state = [torch.empty_like(self.cache), torch.empty(b.N, 2, 16, device="cuda"), torch.empty_like(self.q), torch.empty_like(self.q),
                      torch.zeros_like(self.lens[0])]

    def run(self):
        """Everything from the same start: [cache, scores, rotated q, o, lengths]."""
        cache, scores, q, o, kvl = self.state
        cache.copy_(self.cache)
        scores.zero_()
        lens, table, cu = self.lens
        S = self.b.S
        self.rope.append(self.q, self.k, self.v, cache, lens, table, cu, S, q_out=q)
        self.prefix.forward(q, cache, lens, table, cu, S, self.groups, self.prefix_lens, 2, out=o)
        self.evict.accumulate(q, cache, lens, table, cu, S, scores)
        scores[self.b.table[0, 0]] = 1.0  # of the shared page, whose sums have no order (protected)
        self.evict.compact(cache, scores, lens, table, S, self.new, kvl)

    def result(self):
        assert self.rope.status() == self.prefix.status() == self.evict.status() == rpa.RPA_OK
        return [t.clone() for t in self.state]


def same(a, b):
    raw = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t  # noqa: E731
    return all(torch.equal(raw(x), raw(y)) for x, y in zip(a, b))


CASES = [("bf16", [1, 1, 5, 1, 40], [700, 150, 300, 80, 900]), ("fp8_e4m3", [2, 1, 90, 1], [200, 1500, 100, 60])]


def test_two_threads_on_two_streams():
    steps = [Step(0, *CASES[0], in_place=False), Step(1, *CASES[1], in_place=False)]
    want = []
    for x in steps:
        x.run()
        torch.cuda.synchronize()
        want.append(x.result())
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(25):
                    steps[i].run()
                    torch.cuda.current_stream().synchronize()
                    if not same(steps[i].result(), want[i]):
                        failed.append(i)
        except Exception as e:  # noqa: BLE001 -- reported by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed


@pytest.mark.parametrize("kv,q_lens,kv_lens", CASES)
def test_a_step_in_a_graph(kv, q_lens, kv_lens):
    x = Step(2, kv, q_lens, kv_lens, in_place=False)
    x.run()
    torch.cuda.synchronize()
    want = x.result()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.run()
    for _ in range(3):
        for t in x.state:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(x.result(), want)


def test_two_graphs_of_one_handle():
    """Graphs of one handle share its workspace: replayed one after another each gives its own results."""
    a = Step(3, *CASES[0], in_place=False)
    b = Step(4, *CASES[0], in_place=False)
    b.rope, b.prefix, b.evict = a.rope, a.prefix, a.evict  # (the same configuration)
    want, graphs = [], []
    for x in (a, b):
        x.run()
        torch.cuda.synchronize()
        want.append(x.result())
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for i in (0, 1, 0, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert same(a.result(), want[0]) and same(b.result(), want[1])


def test_a_step_in_place():
    """In place the sequences' own pages hold the kept rows; the same rows as on fresh pages."""
    for kv, q_lens, kv_lens in CASES:
        a, b = Step(5, kv, q_lens, kv_lens, in_place=False), Step(5, kv, q_lens, kv_lens, in_place=True)
        a.b.table[1, 0] = b.b.table[1, 0]
        for x in (a, b):
            # the shared page is protected: it stays where it is on fresh pages too
            if x is a:
                x.new[:, 0] = x.lens[1][:, 0]
            x.run()
        ra, rb = a.result(), b.result()
        assert torch.equal(ra[4], rb[4]) and torch.equal(ra[3], rb[3])
        for s in range(a.b.S):
            n = int(ra[4][s])
            j = torch.arange(n, device="cuda")
            pa, pb = (x.new[s].long()[j // 16] for x in (a, b))
            raw = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t  # noqa: E731
            assert torch.equal(raw(ra[0])[pa, j % 16], raw(rb[0])[pb, j % 16])
            assert torch.equal(ra[1][pa, :, j % 16], rb[1][pb, :, j % 16])
