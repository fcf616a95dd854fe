"""Cases and plain forms of the operators of long caches.

* ``window``  paged attention with a sliding window in front of which the first keys of a sequence stay visible;
* ``append``  rotary positions and the write of new keys and values to a cache of 4 bits, then the rows as it holds them;
* ``read``    rows of a 4-bit cache as values;
* ``attend``  paged attention over a 4-bit cache.

``run`` computes them in plain torch operations, or with ``own`` set through the package's entry points.

The 4-bit cache is uint8 [pages, Hkv, page_size (D + 8 D / group)]: of one page and kv head the K codes [page_size, D / 2],
the V codes, K's (scale, zero) float16 [page_size, D / group, 2], V's.  A channel is code * scale + zero of its group.  A byte
holds channel 2 i (low half) and 2 i + 1; the 16-byte chunks of slot r lie at chunk ^ (r D / 256 mod D / 32).
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8_e4m3": torch.float8_e4m3fn, "int8": torch.int8}
BYTES = {"bf16": 2, "f16": 2, "fp8_e4m3": 1, "int8": 1}
SCALE = {"fp8_e4m3": 0.05, "int8": 0.04}  # K/V scales of the 8-bit caches
MOST16 = 65504.0


def listed():
    return [
        # a decode batch of long conversations that look at the last 4 k keys and the first four
        dict(name="window decode 64", op="window", q="bf16", kv="bf16", Hq=32, Hkv=8, D=128, ps=16, S=64, q_min=1, q_max=1, kv_min=1000,
             kv_max=20000, window=4096, first=4, cap=0.0, mix=1),
        # prompt chunks far into long documents
        dict(name="window prompt 4 x 2k", op="window", q="bf16", kv="bf16", Hq=32, Hkv=8, D=128, ps=64, S=4, q_min=1500, q_max=2100, kv_min=9000,
             kv_max=16000, window=1024, first=100, cap=0.0, mix=2),
        # a mixed batch over an fp8 cache, soft cap
        dict(name="window fp8 mixed", op="window", q="bf16", kv="fp8_e4m3", Hq=16, Hkv=8, D=256, ps=16, S=32, q_min=1, q_max=64, kv_min=256,
             kv_max=16384, window=4096, first=64, cap=50.0, mix=3),
        # one decode step of a few users: 8 tokens, where latency counts
        dict(name="append decode 8", op="append", q="bf16", Hq=32, Hkv=8, D=128, group=64, ps=16, S=8, q_min=1, q_max=1, kv_max=8192, rd=128, off=0,
             pairing="half", mix=4),
        # a prompt chunk of 4 k tokens out of a fused qkv projection
        dict(name="append prompt 4k", op="append", q="bf16", Hq=32, Hkv=8, D=128, group=32, ps=64, S=3, q_min=1000, q_max=1700, kv_max=32768,
             rd=128, off=0, pairing="half", mix=5),
        # two short prompts taken to a cache of another type
        dict(name="read 2 x 700", op="read", q="f16", Hq=16, Hkv=4, D=64, group=64, ps=16, S=2, q_min=600, q_max=700, kv_max=700, mix=6),
        # eight whole sequences
        dict(name="read 8 x 8k", op="read", q="bf16", Hq=32, Hkv=8, D=128, group=128, ps=64, S=8, q_min=5000, q_max=8192, kv_max=8192, mix=7),
        # a few users' decode step
        dict(name="attend decode 4", op="attend", q="bf16", Hq=32, Hkv=8, D=128, group=128, ps=16, S=4, q_min=1, q_max=1, kv_min=500, kv_max=2000,
             window=0, first=0, cap=0.0, mix=8),
        # a full decode batch
        dict(name="attend decode 128", op="attend", q="bf16", Hq=32, Hkv=8, D=128, group=64, ps=16, S=128, q_min=1, q_max=1, kv_min=512,
             kv_max=16384, window=0, first=0, cap=0.0, mix=9),
        # one to five (drafted) tokens a sequence
        dict(name="attend drafts 32", op="attend", q="f16", Hq=16, Hkv=4, D=64, group=32, ps=32, S=32, q_min=1, q_max=5, kv_min=1000, kv_max=6000,
             window=0, first=0, cap=0.0, mix=10),
        # prompt chunks on top of what the cache holds
        dict(name="attend prompt 3 x 2k", op="attend", q="bf16", Hq=32, Hkv=8, D=128, group=64, ps=64, S=3, q_min=800, q_max=2048, kv_min=4000,
             kv_max=16000, window=0, first=0, cap=0.0, mix=11),
        # long decodes with a window and visible first keys, soft cap
        dict(name="attend window 16 x 30k", op="attend", q="bf16", Hq=16, Hkv=8, D=256, group=128, ps=16, S=16, q_min=1, q_max=1, kv_min=3000,
             kv_max=30000, window=4096, first=16, cap=50.0, mix=12),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = drawn(rng)
        w = work(case)
        padded = case["S"] * case["Hkv"] * case["D"] * most_keys(case)
        logits = case["S"] * case["Hq"] * case["q_max"] * most_keys(case) if case["op"] in ("window", "attend") else 0
        if max(w["bytes"], w["flops"] / 200) <= 1.2e9 and padded <= 2.2e9 and logits <= 1.1e9:  # no more than the largest listed
            return case


def drawn(rng):
    op = rng.choice(["window", "window", "append", "read", "attend", "attend", "attend"])
    ps = rng.choice([8, 16, 32, 64, 20, 128])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    group = rng.choice([g for g in (32, 64, 128) if g <= D])
    q = rng.choice(["bf16", "f16"])
    mix = rng.randrange(1 << 20)
    c = dict(op=op, q=q, Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps, q_min=1, mix=mix)
    if op == "window":
        c["q"], c["kv"] = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8_e4m3"), ("f16", "int8")])
    else:
        c["group"] = group
    if op in ("append", "read"):
        S = spread(rng, 1, 100)
        n = 1 if rng.random() < 0.3 else spread(rng, 2, max(2, 4000 // S))
        if op == "append":
            rd = rng.choice([r for r in (32, 64, 128, 256) if r <= D])
            c.update(rd=rd, off=rng.choice([0, D - rd]), pairing=rng.choice(["half", "interleaved"]))
        return dict(c, S=S, q_max=n, kv_max=n + spread(rng, 1, 8000))
    S = spread(rng, 1, 128)
    q_max = 1 if rng.random() < 0.5 else spread(rng, 2, 5) if rng.random() < 0.5 else spread(rng, 6, 2000)
    kv_max = q_max + spread(rng, 16, 16000)
    window, first = 0, 0
    if op == "window" or rng.random() < 0.3:
        window, first = spread(rng, 1, kv_max), rng.choice([1, 4, 4, 16, 64, 100, spread(rng, 1, 500)])
    return dict(c, S=S, q_max=q_max, kv_min=max(q_max, kv_max // 4), kv_max=kv_max, window=window, first=first, cap=rng.choice([0.0, 0.0, 30.0]))


def lengths(case):
    """The sequences' query tokens and keys."""
    r = random.Random("%s %s" % (case["op"], case["mix"]))
    ql = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["S"])]
    if case["op"] == "read" and case["kv_max"] == case["q_max"]:  # whole sequences
        return ql, list(ql)
    return ql, [r.randint(max(n, case.get("kv_min", n)), case["kv_max"]) for n in ql]


def band(case):
    """The keys that a sequence's queries see behind the first ones: where they begin, and how many there are at most."""
    ql, kl = lengths(case)
    if not case["window"]:
        return [0] * len(kl), max(kl)
    lo = [max(0, b - a + 1 - case["window"]) for a, b in zip(ql, kl)]
    return lo, max(b - x for b, x in zip(kl, lo))


def most_keys(case):
    return band(case)[1] + case["first"] if case["op"] in ("window", "attend") else 0


def frequencies(case):
    """Angle a position turns each pair by."""
    return 500000.0 ** (-2 * torch.arange(case["rd"] // 2, dtype=torch.float64) / case["rd"])


def block_bytes(case):
    return case["ps"] * (case["D"] + 8 * case["D"] // case["group"])


def chunk_order(case):
    """Where the 16-byte chunks of a page's slots lie [page_size, D / 32]."""
    r, c = torch.arange(case["ps"], device="cuda"), torch.arange(case["D"] // 32, device="cuda")
    return c[None] ^ ((r * case["D"] // 256) % (case["D"] // 32))[:, None]


def values(shape, dtype, gen, scale=None):
    """N(0, 1) values; in an 8-bit cache divided by its scale."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    if scale:
        x = x / scale
    if dtype == "int8":
        return x.round_().clamp_(-127, 127).to(torch.int8)
    return x.to(DT[dtype])


def small_cache(case, N, gen):
    """A 4-bit cache of N pages that holds the codes of N(0, 1) values."""
    Hkv, ps, D, g = case["Hkv"], case["ps"], case["D"], case["group"]
    cache = torch.empty((N, Hkv, block_bytes(case)), dtype=torch.uint8, device="cuda")
    order = chunk_order(case)
    half = ps * D // 2
    step = max(1, (1 << 26) // (Hkv * ps * D))  # pages at once
    for a in range(0, N, step):
        n = min(step, N - a)
        for i in (0, 1):
            x = torch.randn((n, Hkv, ps, D // g, g), generator=gen, device="cuda", dtype=torch.bfloat16)
            lo, hi = x.amin(-1).half(), x.amax(-1).half()
            s = ((hi.float() - lo.float()) / 15 * 1.001).half()
            codes = ((x - lo[..., None]) / s[..., None]).round_().clamp_(0, 15).to(torch.uint8).flatten(-2)
            packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).unflatten(-1, (-1, 16))  # [n, Hkv, ps, chunks, 16]
            lies = torch.empty_like(packed)
            lies.scatter_(3, order[None, None, :, :, None].expand(packed.shape), packed)
            cache[a:a + n, :, i * half:(i + 1) * half] = lies.flatten(2)
            meta = torch.stack((s, lo), -1).flatten(2).view(torch.uint8)
            m = ps * D // g * 4
            cache[a:a + n, :, 2 * half + i * m:2 * half + (i + 1) * m] = meta
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, S, ps, D, Hq, Hkv = case["op"], case["S"], case["ps"], case["D"], case["Hq"], case["Hkv"]
    ql, kl = lengths(case)
    T, P = sum(ql), -(-max(kl) // ps)
    pages = [-(-n // ps) for n in kl]
    N = sum(pages) + 3
    perm = torch.randperm(N, generator=gen, device="cuda").to(torch.int32)  # physical pages in a shuffled order
    start = torch.tensor([0] + pages).cumsum(0)[:-1].to(torch.int32).cuda()
    table = perm[(start[:, None] + torch.arange(P, device="cuda", dtype=torch.int32)[None]).clamp(max=N - 1).long()].contiguous()
    s = dict(case=case, S=S, T=T, table=table, kv_lens=torch.tensor(kl, dtype=torch.int32).cuda(), mq=max(ql),
             cu=torch.tensor([0] + ql).cumsum(0).to(torch.int32).cuda())
    scale = s["scale"] = SCALE.get(case.get("kv"))
    cfg = dict(num_q_tokens=T, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, total_num_pages=N, page_size=ps, max_num_seqs=S, pages_per_seq=P,
               kv_dtype=case.get("kv") or "int4_g%d" % case["group"], q_dtype=case["q"], sm_scale=1 / math.sqrt(D), k_scale=scale, v_scale=scale)
    if op in ("window", "attend"):
        lo, s["band"] = band(case)
        s["lo"] = torch.tensor(lo).cuda()
        cfg.update(soft_cap=case["cap"] or None)
        if case["window"]:
            cfg.update(sliding_window=case["window"], first_keys=case["first"])
        s["q"] = values((T, Hq, D), case["q"], gen)
        s["out"] = torch.empty_like(s["q"])
    if op == "window":
        s["kv_pages"] = values((N, ps, 2 * Hkv, D), case["kv"], gen, scale)
    elif op == "append":
        s["kv_pages"] = torch.zeros((N, Hkv, block_bytes(case)), dtype=torch.uint8, device="cuda")
        qkv = values((T, Hq + 2 * Hkv, D), case["q"], gen)  # slices of one fused projection's output, as a model has them
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["w"] = frequencies(case).cuda()
        s["out"] = torch.empty((T, Hq, D), dtype=DT[case["q"]], device="cuda")
    else:
        s["kv_pages"] = small_cache(case, N, gen)
    if op in ("append", "read"):
        s["k_out"], s["v_out"] = (torch.empty((T, Hkv, D), dtype=DT[case["q"]], device="cuda") for _ in "kv")
    if own:
        from ragged_paged_attention_02_gb300 import RaggedPagedAttention, RopeAppend

        if op == "append":
            s["op"] = RopeAppend(rotary_dim=case["rd"], rotary_offset=case["off"], pairing=case["pairing"], base=500000.0, **cfg)
        elif op == "read":
            s["op"] = RopeAppend(**cfg)
        else:
            s["op"] = RaggedPagedAttention(**cfg)
    return s


def run(state):
    s, op = state, state["case"]["op"]
    if op in ("window", "attend"):
        if own:
            return s["op"].forward(s["q"], s["kv_pages"], s["kv_lens"], s["table"], s["cu"], s["S"], out=s["out"])
        return plain_attention(s)
    if op == "append":
        if own:
            s["op"].append(s["q"], s["k"], s["v"], s["kv_pages"], s["kv_lens"], s["table"], s["cu"], s["S"], q_out=s["out"])
        else:
            plain_append(s)
    if own:
        s["op"].read(s["kv_pages"], s["kv_lens"], s["table"], s["cu"], s["S"], k_out=s["k_out"], v_out=s["v_out"])
    else:
        plain_read(s)
    return {"k": s["k_out"], "v": s["v_out"]} if op == "read" else {"q": s["out"], "k": s["k_out"], "v": s["v_out"]}


def tokens(s):
    """Sequence and slot of every query token."""
    cu, at = s["cu"].long(), torch.arange(s["T"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(s["S"], device="cuda"), cu[1:] - cu[:-1], output_size=s["T"])
    return seq, s["kv_lens"].long()[seq] - cu[seq + 1] + at


def rows_of(s, page, at):
    """K and V of slots (page, at) [...] in 32 bits [..., Hkv, D]."""
    case = s["case"]
    if case["op"] == "window":
        kv = s["kv_pages"]
        kv = (kv.view(torch.uint8) if kv.element_size() == 1 else kv)[page, at].view(kv.dtype).float()
        if s["scale"]:
            kv *= s["scale"]
        return kv[..., 0::2, :], kv[..., 1::2, :]
    N, Hkv, D, ps, g = s["kv_pages"].shape[0], case["Hkv"], case["D"], case["ps"], case["group"]
    half, m = ps * D // 2, ps * D // g * 4
    order = chunk_order(case)[at][..., None, :, None]

    def part(i):
        codes = s["kv_pages"][:, :, i * half:(i + 1) * half].unflatten(2, (ps, D // 32, 16))[page, :, at]  # [..., Hkv, chunks, 16]
        codes = codes.gather(-2, order.expand(codes.shape)).flatten(-2)
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, g)).float()
        meta = s["kv_pages"][:, :, 2 * half + i * m:2 * half + (i + 1) * m].unflatten(2, (ps, D // g * 4))[page, :, at]
        meta = meta.contiguous().view(torch.float16).unflatten(-1, (-1, 2)).float()
        return (codes * meta[..., :1] + meta[..., 1:]).flatten(-2)

    return part(0), part(1)


def plain_attention(s):
    case, S, first = s["case"], s["S"], s["case"]["first"]
    cu, kl = s["cu"].long(), s["kv_lens"].long()
    i, c = torch.arange(s["mq"], device="cuda"), torch.arange(first + s["band"], device="cuda")
    # the keys that any query of a sequence can see: the first ones, then the band behind them
    lo = torch.maximum(s["lo"], torch.full_like(s["lo"], first))
    j = torch.where(c[None] < first, c[None], lo[:, None] + c[None] - first)  # [S, keys]
    inside = j < kl[:, None]
    j = j.clamp(max=case["ps"] * s["table"].shape[1] - 1)
    k, v = rows_of(s, s["table"].long().gather(1, j // case["ps"]), j % case["ps"])
    n = cu[1:] - cu[:-1]
    q = s["q"][(cu[:-1, None] + i[None]).clamp(max=s["T"] - 1)].float()
    pos = kl[:, None] - n[:, None] + i[None]
    sees = (j[:, None] <= pos[..., None]) & inside[:, None] & (i[None] < n[:, None])[..., None]
    if case["window"]:
        sees &= (j[:, None] > pos[..., None] - case["window"]) | (j[:, None] < first)
    M, K = s["mq"], len(c)
    q = q.view(S, M, case["Hkv"], -1, case["D"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).view(S, case["Hkv"], -1, M, K) / math.sqrt(case["D"])
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    x = x.masked_fill_(~sees[:, None, None], -torch.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).view(S, case["Hkv"], -1, M, case["D"])
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [S, tokens, Hq, D]
    seq, slot = tokens(s)
    s["out"].copy_(o[seq, torch.arange(s["T"], device="cuda") - cu[seq]])
    return s["out"]


def toward(x, up):
    """float64 values rounded to float16 upwards or downwards."""
    h = x.clamp(-MOST16, MOST16).half()
    short = (h.double() < x) if up else (h.double() > x)
    bits = h.view(torch.int16).int()
    away = (h > 0) if up else (h < 0)  # the next value lies further from 0
    nearest = torch.full_like(bits, 1 if up else -0x7fff)  # of 0, the smallest value on that side
    next_ = torch.where(h == 0, nearest, torch.where(away, bits + 1, bits - 1))
    return torch.where(short, next_, bits).to(torch.int16).view(torch.float16)


def plain_append(s):
    # in 64 bits: positions' angles, and values that may lie next to the border of two codes
    case = s["case"]
    rd, off, ps, D, g, Hkv = case["rd"], case["off"], case["ps"], case["D"], case["group"], case["Hkv"]
    seq, slot = tokens(s)
    angle = slot.double()[:, None] * s["w"][None]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def turn(x):
        x = x.double()
        y = x.clone()
        a, b = (x[..., off:off + rd // 2], x[..., off + rd // 2:off + rd]) if case["pairing"] == "half" else \
               (x[..., off:off + rd:2], x[..., off + 1:off + rd:2])
        c, d = a * cos - b * sin, b * cos + a * sin
        y[..., off:off + rd] = torch.cat((c, d), -1) if case["pairing"] == "half" else torch.stack((c, d), -1).flatten(-2)
        return y

    s["out"].copy_(turn(s["q"]))
    page, at = s["table"][seq, slot // ps].long(), slot % ps
    half, m = ps * D // 2, ps * D // g * 4
    order = chunk_order(case)[at][:, None, :, None]
    for i, x in enumerate((turn(s["k"]), s["v"].double())):
        x = x.clamp(-MOST16, MOST16).unflatten(-1, (-1, g))  # [T, Hkv, groups, g]
        zero = toward(x.amin(-1), False)
        step = toward((x.amax(-1) - zero.double()) / 15, True)
        codes = torch.round((x - zero.double()[..., None]) / step.double()[..., None].clamp(min=1e-30)).clamp_(0, 15).to(torch.uint8).flatten(-2)
        packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).unflatten(-1, (-1, 16))
        lies = torch.empty_like(packed)
        lies.scatter_(2, order.expand(packed.shape), packed)
        s["kv_pages"][:, :, i * half:(i + 1) * half].unflatten(2, (ps, D // 2))[page, :, at] = lies.flatten(2)
        meta = torch.stack((step, zero), -1).flatten(2).view(torch.uint8)
        s["kv_pages"][:, :, 2 * half + i * m:2 * half + (i + 1) * m].unflatten(2, (ps, D // g * 4))[page, :, at] = meta


def plain_read(s):
    seq, slot = tokens(s)
    k, v = rows_of(s, s["table"][seq, slot // s["case"]["ps"]].long(), slot % s["case"]["ps"])
    s["k_out"].copy_(k)
    s["v_out"].copy_(v)


def work(case):
    ql, kl = lengths(case)
    T, D, Hkv, Hq = sum(ql), case["D"], case["Hkv"], case["Hq"]
    qb = BYTES[case["q"]]
    small = D + 8 * D // case["group"] if "group" in case else 0  # bytes of a key's rows of one kv head
    if case["op"] == "read":
        return {"bytes": T * Hkv * (small + 2 * D * qb), "flops": 4 * T * Hkv * D}
    if case["op"] == "append":  # and the rows read back
        return {"bytes": T * (D * qb * (2 * Hq + 2 * Hkv) + 2 * Hkv * small + 2 * Hkv * D * qb), "flops": 3 * T * case["rd"] * (Hq + Hkv) + 20 * T * Hkv * D}
    key = small or 2 * D * BYTES[case["kv"]]
    F, W = case["first"], case["window"]

    def seen(a, b):
        """Keys that any of the last a of b tokens sees, and pairs of tokens and keys they see."""
        if not W:
            return b, a * (b - a) + a * (a + 1) // 2
        keys = min(b, F) + max(0, b - max(F, b - a + 1 - W))
        return keys, sum(min(p + 1, F) + max(0, p + 1 - max(F, p + 1 - W)) for p in range(b - a, b))

    both = [seen(a, b) for a, b in zip(ql, kl)]
    return {"bytes": sum(k for k, _ in both) * Hkv * key + 2 * T * Hq * D * qb, "flops": 4 * sum(p for _, p in both) * Hq * D}


def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence at a time."""
    s = prepare_plainly(case, seed)
    ql, kl = lengths(case)
    ps, D, Hkv, S, op = case["ps"], case["D"], case["Hkv"], case["S"], case["op"]
    starts = [sum(ql[:i]) for i in range(S)]

    def held(b, j):
        """K and V rows [Hkv, keys, D] of keys j of sequence b."""
        page, at = s["table"][b].long()[j // ps], j % ps
        if op == "window":
            raw = s["kv_pages"].view(torch.uint8) if s["kv_pages"].element_size() == 1 else s["kv_pages"]
            rows = raw[page, at].view(DT[case["kv"]]).double().transpose(0, 1) * (s["scale"] or 1.0)
            return rows[0::2], rows[1::2]
        g, n = case["group"], len(j)
        blocks = s["kv_pages"][page].transpose(0, 1)  # [Hkv, keys, bytes]
        line = torch.arange(D // 2, device="cuda")
        got = []
        for kind in (0, 1):
            # byte x of a row is byte x % 16 of chunk x // 16
            where = kind * ps * D // 2 + at[:, None] * (D // 2) + 16 * ((line // 16)[None] ^ (at * D // 256 % (D // 32))[:, None]) + line % 16
            bytes_ = blocks.gather(2, where[None].expand(Hkv, n, D // 2)).int()
            code = torch.empty((Hkv, n, D), dtype=torch.float64, device="cuda")
            code[..., 0::2], code[..., 1::2] = (bytes_ % 16).double(), (bytes_ // 16).double()
            x = 4 * (D // g)
            where = ps * D + kind * ps * x + at[:, None] * x + torch.arange(x, device="cuda")[None]
            pair = blocks.gather(2, where[None].expand(Hkv, n, x)).contiguous().view(torch.float16).double().view(Hkv, n, D // g, 2)
            got.append(code * pair[..., 0].repeat_interleave(g, -1) + pair[..., 1].repeat_interleave(g, -1))
        return got

    if op in ("window", "attend"):
        G = case["Hq"] // Hkv
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b in range(S):
            p0 = kl[b] - ql[b]
            j = torch.arange(kl[b], device="cuda")
            if case["window"]:
                j = torch.cat((j[:case["first"]], j[max(case["first"], p0 + 1 - case["window"], 0):]))
            k, v = held(b, j)
            pos = torch.arange(p0, kl[b], device="cuda")[:, None]
            hidden = j[None] > pos
            if case["window"]:
                hidden |= (j[None] + case["window"] <= pos) & (j[None] >= case["first"])
            for h in range(Hkv):
                x = torch.einsum("tgd,kd->gtk", s["q"][starts[b]:starts[b] + ql[b], h * G:(h + 1) * G].double(), k[h]) / math.sqrt(D)
                if case["cap"]:
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                p = torch.softmax(x.masked_fill(hidden[None], -math.inf), -1)
                out[starts[b]:starts[b] + ql[b], h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", p, v[h])
        return out
    k_out = torch.zeros((s["T"], Hkv, D), dtype=torch.float64, device="cuda")
    v_out, q_out = torch.zeros_like(k_out), None
    if op == "read":
        for b in range(S):
            k, v = held(b, torch.arange(kl[b] - ql[b], kl[b], device="cuda"))
            t = slice(starts[b], starts[b] + ql[b])
            k_out[t], v_out[t] = k.transpose(0, 1), v.transpose(0, 1)
        return {"k": k_out, "v": v_out}
    rd, off, g = case["rd"], case["off"], case["group"]
    w = frequencies(case).cuda()

    def rotated(x, pos):
        x = x.double().clone()
        turn = torch.polar(torch.ones((len(pos), rd // 2), dtype=torch.float64, device="cuda"), pos.double()[:, None] * w[None])[:, None]
        part = x[..., off:off + rd]
        if case["pairing"] == "half":
            z = torch.complex(part[..., :rd // 2].contiguous(), part[..., rd // 2:].contiguous()) * turn
            part[..., :rd // 2], part[..., rd // 2:] = z.real, z.imag
        else:
            part.copy_(torch.view_as_real(torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2))
        return x

    def kept(x):
        """What a group's 16 levels make of its values."""
        y = x.clamp(-MOST16, MOST16).view(*x.shape[:-1], D // g, g)
        low, high = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        # the levels' ends on the 16-bit grid, whose step is 2^-10 of the power of two below
        grid = lambda a: torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -14))) - 10)  # noqa: E731
        z = torch.floor(low / grid(low)) * grid(low)
        a = (high - z) / 15
        st = torch.ceil(a / grid(a)) * grid(a)
        level = torch.where(st > 0, torch.round((y - z) / torch.where(st > 0, st, 1.0)).clamp(0, 15), 0.0)
        return (level * st + z).view(x.shape)

    q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(S):
        t = slice(starts[b], starts[b] + ql[b])
        pos = torch.arange(kl[b] - ql[b], kl[b], device="cuda")
        q_out[t] = rotated(s["q"][t], pos)
        k_out[t] = kept(rotated(s["k"][t], pos))
        v_out[t] = kept(s["v"][t].double())
    return {"q": q_out, "k": k_out, "v": v_out}


def prepare_plainly(case, seed):
    """The inputs alone, whatever `own` says."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was
