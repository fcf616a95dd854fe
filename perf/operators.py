"""Cases and plain forms of the paged cache's operators.

Four operators around the paged K/V cache of a serving engine:

* ``append``  rotary positions on q and the new keys, and the write of the new K/V rows to their page slots;
* ``prefix``  attention of a batch whose sequences share a long prefix (the result of the ordinary paged attention);
* ``weigh``   accumulation of the softmax weight every cached key receives;
* ``evict``   choice of the keys to keep by that weight, and the compaction of the cache.

``run`` computes them in plain torch operations, or with ``own`` set through the package's entry points.
Layouts are the package's: kv_pages [pages, page_size, 2 Hkv, D] (row 2h = K of kv head h, 2h + 1 its V) or, for the
latent layout, [pages, page_size, Hkv, D]; scores [pages, Hkv, page_size].
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8_e4m3": torch.float8_e4m3fn,
      "fp8_e5m2": torch.float8_e5m2, "int8": torch.int8}
MOST = {"fp8_e4m3": 448.0, "fp8_e5m2": 57344.0}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "fp8_e4m3": 1, "fp8_e5m2": 1, "int8": 1}
SCALE = {"fp8_e4m3": 0.05, "fp8_e5m2": 0.05, "int8": 0.04}  # K/V scales of the 8-bit caches


def listed():
    return [
        # one decode step of a few users: 8 tokens, where latency counts
        dict(name="append decode 8", op="append", q="bf16", kv="bf16", Hq=32, Hkv=8, D=128, ps=16, S=8, q_min=1, q_max=1, kv_max=8192,
             rd=128, off=0, pairing="half", scaling="none", given=False, mix=1),
        # a prompt chunk of 8 k tokens out of a fused qkv projection, frequencies scaled for a long context
        dict(name="append prompt 8k", op="append", q="bf16", kv="bf16", Hq=64, Hkv=8, D=128, ps=64, S=5, q_min=1000, q_max=2600, kv_max=32768,
             rd=128, off=0, pairing="half", scaling="rotations", given=False, mix=2),
        # a mixed batch over an fp8 cache, rotary pairs side by side on a quarter of the head, positions kept apart from slots (an evicted cache)
        dict(name="append fp8 mixed", op="append", q="bf16", kv="fp8_e4m3", Hq=16, Hkv=8, D=256, ps=16, S=65, q_min=1, q_max=64, kv_max=16384,
             rd=64, off=0, pairing="interleaved", scaling="index", given=True, mix=3),
        # a few requests behind one system prompt, one token each
        dict(name="prefix 4 x 1k", op="prefix", q="bf16", kv="bf16", Hq=32, Hkv=8, D=128, ps=16, S=4, groups=1, q_min=1, q_max=1,
             pre_min=1024, pre_max=1024, suf_min=17, suf_max=200, cap=0.0, mix=4),
        # 61 answers to questions about one document
        dict(name="prefix 61 x 8k", op="prefix", q="bf16", kv="bf16", Hq=32, Hkv=8, D=128, ps=16, S=61, groups=1, q_min=1, q_max=1,
             pre_min=8007, pre_max=8007, suf_min=1, suf_max=700, cap=0.0, mix=5),
        # a full decode batch behind a long shared context
        dict(name="prefix 256 x 16k", op="prefix", q="bf16", kv="bf16", Hq=32, Hkv=8, D=128, ps=64, S=256, groups=1, q_min=1, q_max=1,
             pre_min=16384, pre_max=16384, suf_min=16, suf_max=1024, cap=0.0, mix=6),
        # three system prompts over an fp8 cache, one to four (drafted) tokens a sequence, soft cap
        dict(name="prefix fp8 3 groups", op="prefix", q="bf16", kv="fp8_e4m3", Hq=16, Hkv=8, D=256, ps=16, S=48, groups=3, q_min=1, q_max=4,
             pre_min=2000, pre_max=6000, suf_min=30, suf_max=500, cap=50.0, mix=7),
        # the decode batch's weights, every step
        dict(name="weigh decode 64", op="weigh", q="bf16", kv="bf16", Hq=32, Hkv=8, D=128, ps=16, S=64, q_min=1, q_max=1, kv_min=512, kv_max=8192,
             mix=8),
        # the weights that the end of a prompt gives its keys
        dict(name="weigh prompt end", op="weigh", q="f16", kv="f16", Hq=16, Hkv=8, D=64, ps=32, S=6, q_min=20, q_max=64, kv_min=1000, kv_max=6000,
             mix=9),
        # two short conversations cut to 512 keys
        dict(name="evict 2 x 1.5k", op="evict", kv="bf16", Hkv=8, D=128, ps=16, S=2, kv_min=1400, kv_max=1600, budget=512, protect=4, recent=64,
             mix=10),
        # a batch cut to 2 k keys, some of it below the budget already
        dict(name="evict 64 x 8k", op="evict", kv="bf16", Hkv=8, D=128, ps=16, S=64, kv_min=1500, kv_max=8192, budget=2048, protect=4,
             recent=256, mix=11),
        # two long documents over an fp8 cache
        dict(name="evict 2 x 100k", op="evict", kv="fp8_e4m3", Hkv=8, D=128, ps=64, S=2, kv_min=90000, kv_max=100000, budget=16001, protect=64,
             recent=1000, mix=12),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = drawn(rng)
        w = work(case)
        padded = case["S"] * max(lengths(case)[1]) * case["Hkv"] * case["D"]
        if max(w["bytes"], w["flops"] / 50) <= 1.3e9 and (case["op"] in ("append", "evict") or padded <= 4.5e9):  # the largest listed one's
            return case


def drawn(rng):
    op = rng.choice(["append", "append", "prefix", "prefix", "weigh", "evict"])
    ps = rng.choice([8, 16, 32, 64])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    mix = rng.randrange(1 << 20)
    if op == "append":
        q = rng.choice(["bf16", "bf16", "f16", "f32"])
        kv = rng.choice(["bf16", "bf16", "f16", "fp8_e4m3", "fp8_e5m2"])
        S = spread(rng, 1, 200)
        q_max = 1 if rng.random() < 0.4 else spread(rng, 2, max(2, 6000 // S))
        latent = rng.random() < 0.15 and kv in ("bf16", "f16")
        if latent:
            D, Hkv, G, rd, off = 576, 1, 16, 64, 512
        else:
            rd = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= D])
            off = rng.choice([0, 0, D - rd])
        return dict(op=op, q=q, kv=kv, Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps, S=S, q_min=1, q_max=q_max, kv_max=q_max + spread(rng, 1, 8000), rd=rd,
                    off=off, pairing=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "base", "index", "rotations"]),
                    given=rng.random() < 0.3, mix=mix)
    if op == "prefix":
        q, kv = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8_e4m3"), ("f16", "int8"), ("f16", "fp8_e5m2")])
        S = spread(rng, 1, 200)
        groups = rng.randint(1, min(S, 4))
        pre = spread(rng, 64, 12000)
        suf = spread(rng, 8, 600)
        return dict(op=op, q=q, kv=kv, Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps, S=S, groups=groups, q_min=1, q_max=rng.choice([1, 1, 1, 4]), pre_min=pre // 2,
                    pre_max=pre, suf_min=5, suf_max=suf, cap=rng.choice([0.0, 0.0, 30.0]), mix=mix)
    if op == "weigh":
        q, kv = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8_e4m3"), ("f16", "int8")])
        S = spread(rng, 1, 64)
        q_max = 1 if rng.random() < 0.6 else spread(rng, 2, 70)
        kv_max = q_max + spread(rng, 16, 8000)
        return dict(op=op, q=q, kv=kv, Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps, S=S, q_min=1, q_max=q_max, kv_min=q_max, kv_max=kv_max, mix=mix)
    kv = rng.choice(["bf16", "f16", "fp8_e4m3", "int8"])
    S = spread(rng, 1, 64)
    kv_max = spread(rng, 100, min(100000, 300000 // S))
    budget = spread(rng, 40, max(41, kv_max * 3 // 4))
    recent = rng.randint(0, budget // 3)
    return dict(op=op, kv=kv, Hkv=Hkv, D=D, ps=ps, S=S, kv_min=kv_max // 2, kv_max=kv_max, budget=budget, protect=rng.randint(0, budget // 4),
                recent=recent, mix=mix)


def lengths(case):
    """The sequences' lengths: (query tokens, keys) each, and for shared prefixes (first sequence of each group, prefix of each group)."""
    r = random.Random("%s %s" % (case["op"], case["mix"]))
    S = case["S"]
    if case["op"] == "append":
        ql = [r.randint(case["q_min"], case["q_max"]) for _ in range(S)]
        return ql, [r.randint(n, max(n, case["kv_max"])) for n in ql], None, None
    if case["op"] == "prefix":
        first = [0] + sorted(r.sample(range(1, S), case["groups"] - 1)) + [S]
        pre = [r.randint(case["pre_min"], case["pre_max"]) for _ in range(case["groups"])]
        ql = [r.randint(case["q_min"], case["q_max"]) for _ in range(S)]
        kl = [pre[g] + max(ql[s], r.randint(case["suf_min"], case["suf_max"])) for g in range(case["groups"]) for s in range(first[g], first[g + 1])]
        return ql, kl, first, pre
    if case["op"] == "weigh":
        ql = [r.randint(case["q_min"], case["q_max"]) for _ in range(S)]
        return ql, [r.randint(max(n, case["kv_min"]), case["kv_max"]) for n in ql], None, None
    return [0] * S, [r.randint(case["kv_min"], case["kv_max"]) for _ in range(S)], None, None


def is_latent(case):
    return case["D"] == 576


def kv_rows(case):
    """Rows of a slot."""
    return case["Hkv"] if is_latent(case) else 2 * case["Hkv"]


def frequencies(case):
    """Angle a position turns each pair by (float64) and the factor of the rotated values."""
    rd, base, factor, trained = case["rd"], 500000.0, 8.0, 8192.0
    i = torch.arange(rd // 2, dtype=torch.float64)
    w = base ** (-2 * i / rd)
    if case["scaling"] == "linear":
        return w / factor, 1.0
    if case["scaling"] == "base":
        return (base * factor ** (rd / (rd - 2))) ** (-2 * i / rd), 1.0
    if case["scaling"] == "rotations":  # by the turns within the trained length: few are stretched, many are not
        keep = ((trained * w / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return w * keep + w / factor * (1 - keep), 1.0
    if case["scaling"] == "index":  # a ramp over the pairs between those of 32 turns and of one turn
        at = [rd * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
        keep = 1 - ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return w * keep + w / factor * (1 - keep), 0.1 * math.log(factor) + 1
    return w, 1.0


def cache_cfg(case, T, N, P):
    scale = SCALE.get(case["kv"])
    cfg = dict(num_q_tokens=T, num_q_heads=case.get("Hq", case["Hkv"]), num_kv_heads=case["Hkv"], head_dim=case["D"], total_num_pages=N,
               page_size=case["ps"], max_num_seqs=case["S"], pages_per_seq=P, kv_dtype=case["kv"], q_dtype=case.get("q", "bf16"),
               sm_scale=1 / math.sqrt(case["D"]), k_scale=scale, v_scale=scale, soft_cap=case.get("cap") or None)
    if is_latent(case):
        cfg.update(kv_layout="latent", v_head_dim=512)
    return cfg


def values(shape, dtype, gen, scale):
    """N(0, 1) values; in an 8-bit cache divided by its scale."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16 if dtype != "f32" else torch.float32)
    if scale:
        x = x / scale
    if dtype == "int8":
        return x.round_().clamp_(-127, 127).to(torch.int8)
    return x.to(DT[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    S, ps, D, Hkv = case["S"], case["ps"], case["D"], case["Hkv"]
    ql, kl, first, pre = lengths(case)
    T = sum(ql)
    P = -(-max(kl) // ps)
    scale = SCALE.get(case["kv"])
    # physical pages in a shuffled order; sequences of a group share the pages of their prefix
    own_pages = [-(-n // ps) for n in kl]
    budget_pages = -(-case["budget"] // ps) if case["op"] == "evict" else 0
    N = sum(own_pages) + S * budget_pages + 3
    perm = torch.randperm(N, generator=gen, device="cuda").to(torch.int32)
    start = torch.tensor([0] + own_pages).cumsum(0)[:-1].to(torch.int32).cuda()
    table = perm[(start[:, None] + torch.arange(P, device="cuda", dtype=torch.int32)[None]).clamp(max=N - 1).long()]
    if first:
        for g in range(len(pre)):
            n = pre[g] // ps  # whole pages
            table[first[g]:first[g + 1], :n] = table[first[g], :n].clone()
    s = dict(case=case, S=S, kv_lens=torch.tensor(kl, dtype=torch.int32).cuda(), table=table.contiguous(), T=T, scale=scale,
             cu=torch.tensor([0] + ql).cumsum(0).to(torch.int32).cuda(), P=P)
    if case["op"] == "append":
        s["kv_pages"] = torch.zeros((N, ps, kv_rows(case), D), dtype=torch.uint8 if BYTES[case["kv"]] == 1 else DT[case["kv"]],
                                    device="cuda").view(DT[case["kv"]])
    else:
        s["kv_pages"] = values((N, ps, kv_rows(case), D), case["kv"], gen, scale)
    cfg = cache_cfg(case, T, N, P)
    if case["op"] == "append":
        # slices of one fused projection's output, as a model has them
        Hq = case["Hq"]
        rows = Hq + (1 if is_latent(case) else 2) * Hkv
        qkv = values((T, rows, D), case["q"], gen, None)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        s["v"] = None if is_latent(case) else qkv[:, Hq + Hkv:]
        w, s["factor"] = frequencies(case)
        s["w"] = w.cuda()
        s["positions"] = None
        if case["given"]:
            s["positions"] = torch.randint(0, 1 << 20, (T,), generator=gen, device="cuda").to(torch.int32)
        s["q_out"] = torch.empty((T, Hq, D), dtype=DT[case["q"]], device="cuda")
        if own:
            from ragged_paged_attention_02_gb300 import RopeAppend

            kinds = {"none": {}, "linear": dict(scaling="linear", factor=8.0), "base": dict(scaling="base", factor=8.0),
                     "rotations": dict(scaling="rotations", factor=8.0, trained_len=8192, low=1.0, high=4.0),
                     "index": dict(scaling="index", factor=8.0, trained_len=8192, low=1.0, high=32.0,
                                   magnitude=0.1 * math.log(8.0) + 1)}
            s["op"] = RopeAppend(rotary_dim=case["rd"], rotary_offset=case["off"], pairing=case["pairing"], base=500000.0,
                                 **kinds[case["scaling"]], **cfg)
    elif case["op"] == "prefix":
        if any(p % ps for p in pre):
            raw = s["kv_pages"].view(torch.uint8) if BYTES[case["kv"]] == 1 else s["kv_pages"]
            for g, p in enumerate(pre):  # the shared part of the page in which the prefix ends
                n = p // ps
                if p % ps:
                    at = table[first[g]:first[g + 1], n].long()
                    raw[at, :p % ps] = raw[at[:1], :p % ps].clone()
        s["q"] = values((T, case["Hq"], D), case["q"], gen, None)
        s["groups"] = torch.tensor(first, dtype=torch.int32).cuda()
        s["prefix_lens"] = torch.tensor(pre, dtype=torch.int32).cuda()
        s["out"] = torch.empty_like(s["q"])
        s["mq"] = max(ql)
        if own:
            from ragged_paged_attention_02_gb300 import SharedPrefixAttention

            s["op"] = SharedPrefixAttention(max_groups=len(pre), **cfg)
    elif case["op"] == "weigh":
        s["q"] = values((T, case["Hq"], D), case["q"], gen, None)
        s["scores"] = torch.rand((N, Hkv, ps), generator=gen, device="cuda") * (2.0 * T * case["Hq"] / Hkv / sum(kl))  # of the weights' size
        s["mq"] = max(ql)
        if own:
            from ragged_paged_attention_02_gb300 import CacheEviction

            s["op"] = CacheEviction(budget=max(kl), **cfg)
    else:
        # what steps of decoding leave: a few keys with most of the weight, many with little, some with none at all
        x = torch.randn((N, Hkv, ps), generator=gen, device="cuda").mul_(2.0).exp_()
        s["scores"] = x * (torch.rand((N, Hkv, ps), generator=gen, device="cuda") > 0.05)
        fresh = perm[sum(own_pages):sum(own_pages) + S * budget_pages]
        s["new_table"] = table.clone()
        s["new_table"][:, :min(P, budget_pages)] = fresh.view(S, budget_pages)[:, :P]
        s["new_kv_lens"] = torch.empty_like(s["kv_lens"])
        s["kept"] = torch.empty((S, Hkv, case["budget"]), dtype=torch.int32, device="cuda")
        if own:
            from ragged_paged_attention_02_gb300 import CacheEviction

            s["op"] = CacheEviction(budget=case["budget"], protect=case["protect"], recent=case["recent"], **cfg)
    return s


def run(state):
    s, op = state, state["case"]["op"]
    if op == "append":
        if own:
            s["op"].append(s["q"], s["k"], s["v"], s["kv_pages"], s["kv_lens"], s["table"], s["cu"], s["S"], positions=s["positions"],
                           q_out=s["q_out"])
        else:
            plain_append(s)
        return {"q": s["q_out"], "kv_pages": s["kv_pages"]}
    if op == "prefix":
        if own:
            return s["op"].forward(s["q"], s["kv_pages"], s["kv_lens"], s["table"], s["cu"], s["S"], s["groups"], s["prefix_lens"],
                                   len(s["prefix_lens"]), out=s["out"])
        return plain_attention(s)
    if op == "weigh":
        if own:
            s["op"].accumulate(s["q"], s["kv_pages"], s["kv_lens"], s["table"], s["cu"], s["S"], s["scores"])
        else:
            plain_weigh(s)
        return s["scores"]
    if own:
        s["op"].compact(s["kv_pages"], s["scores"], s["kv_lens"], s["table"], s["S"], s["new_table"], s["new_kv_lens"], kept=s["kept"])
    else:
        plain_evict(s)
    return {"kv_pages": s["kv_pages"], "scores": s["scores"], "kv_lens": s["new_kv_lens"], "kept": s["kept"]}


def raw(pages):
    """A cache as a type that indexing takes."""
    return pages.view(torch.uint8) if pages.element_size() == 1 else pages


def tokens(s):
    """Sequence and slot of every query token."""
    cu, at = s["cu"].long(), torch.arange(s["T"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(s["S"], device="cuda"), cu[1:] - cu[:-1], output_size=s["T"])
    return seq, s["kv_lens"].long()[seq] - cu[seq + 1] + at


def plain_append(s):
    case = s["case"]
    rd, off, ps, D = case["rd"], case["off"], case["ps"], case["D"]
    seq, slot = tokens(s)
    pos = slot if s["positions"] is None else s["positions"]
    angle = pos.double()[:, None] * s["w"][None]
    cos, sin = (angle.cos() * s["factor"]).float()[:, None], (angle.sin() * s["factor"]).float()[:, None]

    def turn(x):
        x = x.float()
        y = x.clone()
        a, b = (x[..., off:off + rd // 2], x[..., off + rd // 2:off + rd]) if case["pairing"] == "half" else \
               (x[..., off:off + rd:2], x[..., off + 1:off + rd:2])
        c, d = a * cos - b * sin, b * cos + a * sin
        y[..., off:off + rd] = torch.cat((c, d), -1) if case["pairing"] == "half" else torch.stack((c, d), -1).flatten(-2)
        return y

    def stored(x):
        if s["scale"]:
            x = x / s["scale"]
        if case["kv"] in MOST:
            x = x.clamp(-MOST[case["kv"]], MOST[case["kv"]])
        return x.to(DT[case["kv"]])

    s["q_out"].copy_(turn(s["q"]))
    k = stored(turn(s["k"]))
    row = k if s["v"] is None else torch.stack((k, stored(s["v"].float())), 2).flatten(1, 2)
    flat = s["table"][seq, slot // ps].long() * ps + slot % ps
    raw(s["kv_pages"]).view(-1, kv_rows(case), D)[flat] = raw(row)


def gathered(s):
    """The sequences' cached rows [S, keys, rows, D] in 32 bits, their queries [S, most tokens, Hq, D], and where each query sees each key."""
    case = s["case"]
    kv = raw(s["kv_pages"])[s["table"].long()].view(DT[case["kv"]]).float().flatten(1, 2)
    if s["scale"]:
        kv *= s["scale"]
    cu, i = s["cu"].long(), torch.arange(s["mq"], device="cuda")
    n = cu[1:] - cu[:-1]
    q = s["q"][(cu[:-1, None] + i[None]).clamp(max=s["T"] - 1)].float()
    pos = s["kv_lens"].long()[:, None] - n[:, None] + i[None]
    sees = (torch.arange(kv.shape[1], device="cuda")[None, None] <= pos[..., None]) & (i[None] < n[:, None])[..., None]
    return kv, q, sees


def weights(s, k, q, sees):
    """Softmax weights [S, Hkv, G, tokens, keys]; rows that are no query's are 0."""
    case = s["case"]
    S, M = q.shape[:2]
    q = q.view(S, M, case["Hkv"], -1, case["D"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).view(S, case["Hkv"], -1, M, k.shape[1]) / math.sqrt(case["D"])
    if case.get("cap"):
        x = case["cap"] * torch.tanh(x / case["cap"])
    x = x.masked_fill(~sees[:, None, None], -torch.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def plain_attention(s):
    case = s["case"]
    kv, q, sees = gathered(s)
    p = weights(s, kv[:, :, 0::2], q, sees)
    o = torch.matmul(p.flatten(2, 3), kv[:, :, 1::2].transpose(1, 2)).view(*p.shape[:4], case["D"])
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [S, tokens, Hq, D]
    seq, slot = tokens(s)
    at = torch.arange(s["T"], device="cuda") - s["cu"].long()[seq]
    s["out"].copy_(o[seq, at])
    return s["out"]


def plain_weigh(s):
    ps = s["case"]["ps"]
    kv, q, sees = gathered(s)
    got = weights(s, kv[:, :, 0::2], q, sees).sum((2, 3))  # [S, Hkv, keys]
    slot = torch.arange(kv.shape[1], device="cuda")[None]
    kl, cu = s["kv_lens"].long()[:, None], s["cu"].long()
    seq, j = torch.nonzero(slot < kl, as_tuple=True)
    page, at = s["table"].long()[seq, j // ps], j % ps
    old = s["scores"][page, :, at]
    new = j >= (s["kv_lens"].long() - cu[1:] + cu[:-1])[seq]  # keys of this call's tokens start at nothing
    s["scores"][page, :, at] = torch.where(new[:, None], 0.0, old) + got[seq, :, j]


def plain_evict(s):
    case = s["case"]
    S, ps, Hkv, B = s["S"], case["ps"], case["Hkv"], case["budget"]
    table, kl = s["table"].long(), s["kv_lens"].long()
    L = table.shape[1] * ps
    j = torch.arange(L, device="cuda")
    x = s["scores"][table].transpose(1, 2).reshape(S, Hkv, L)
    keep = (j[None] < case["protect"]) | (j[None] >= kl[:, None] - case["recent"])
    x = x.masked_fill(keep[:, None], torch.inf).masked_fill((j[None] >= kl[:, None])[:, None], -torch.inf)
    order = torch.sort(x, stable=True, dim=-1, descending=True).indices[..., :B]  # ties: the lowest first
    n = kl.clamp(max=B)
    rank = torch.arange(order.shape[-1], device="cuda")
    order = order.masked_fill(rank[None, None] >= n[:, None, None], L).sort(-1).values
    s["kept"].fill_(-1)
    s["kept"][..., :order.shape[-1]] = torch.where(order < L, order, -1).to(torch.int32)
    seq, head, to = torch.nonzero(order < L, as_tuple=True)
    src = order[seq, head, to]
    new = s["new_table"].long()
    a, b = table[seq, src // ps], src % ps
    c, d = new[seq, to // ps], to % ps
    pages = raw(s["kv_pages"]).view(-1, ps, Hkv, 2, case["D"])
    pages[c, d, head] = pages[a, b, head]
    s["scores"][c, head, d] = s["scores"][a, head, b]
    s["new_kv_lens"].copy_(n)


def work(case):
    ql, kl, first, pre = lengths(case)
    T, D, Hkv = sum(ql), case["D"], case["Hkv"]
    kvb = BYTES[case["kv"]]
    if case["op"] == "append":
        rows = (1 if is_latent(case) else 2) * Hkv
        return {"bytes": T * D * (2 * case["Hq"] * BYTES[case["q"]] + rows * (BYTES[case["q"]] + kvb)), "flops": 3 * T * case["rd"] * (case["Hq"] + Hkv)}
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(ql, kl))
    if case["op"] == "prefix":
        keys = sum(kl) - sum(pre[g] * (first[g + 1] - first[g] - 1) for g in range(len(pre)))
        return {"bytes": keys * 2 * Hkv * D * kvb + 2 * T * case["Hq"] * D * BYTES[case["q"]], "flops": 4 * pairs * case["Hq"] * D}
    if case["op"] == "weigh":
        return {"bytes": sum(kl) * Hkv * (D * kvb + 8) + T * case["Hq"] * D * BYTES[case["q"]], "flops": 2 * pairs * case["Hq"] * D}
    kept = sum(min(n, case["budget"]) for n in kl)
    return {"bytes": sum(kl) * Hkv * 4 + kept * Hkv * (4 * D * kvb + 8), "flops": 0}


def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence at a time."""
    s = prepare_plainly(case, seed)
    ql, kl, first, pre = lengths(case)
    ps, D, Hkv, S = case["ps"], case["D"], case["Hkv"], case["S"]
    starts = [sum(ql[:i]) for i in range(S)]
    scale = SCALE.get(case["kv"]) or 1.0
    if case["op"] == "append":
        rd, off = case["rd"], case["off"]
        w, factor = frequencies(case)
        q, cache = s["q"].double(), s["kv_pages"].double()
        for b in range(S):
            t = slice(starts[b], starts[b] + ql[b])
            slot = torch.arange(kl[b] - ql[b], kl[b], device="cuda")
            pos = slot if s["positions"] is None else s["positions"][t].long()
            turn = torch.polar(torch.full((ql[b], rd // 2), float(factor), dtype=torch.float64, device="cuda"), pos.double()[:, None] * w.cuda()[None])

            def rotated(x):
                x = x.double().clone()
                part = x[..., off:off + rd]
                if case["pairing"] == "half":
                    z = torch.complex(part[..., :rd // 2].contiguous(), part[..., rd // 2:].contiguous()) * turn[:, None]
                    part[..., :rd // 2], part[..., rd // 2:] = z.real, z.imag
                else:
                    part.copy_(torch.view_as_real(torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn[:, None]).flatten(-2))
                return x

            q[t] = rotated(s["q"][t])
            page, at = s["table"][b, slot // ps].long(), slot % ps
            most = MOST.get(case["kv"], math.inf)
            k = (rotated(s["k"][t]) / scale).clamp(-most, most)
            if is_latent(case):
                cache[page, at] = k
            else:
                cache[page, at, 0::2] = k
                cache[page, at, 1::2] = (s["v"][t].double() / scale).clamp(-most, most)
        return {"q": q, "kv_pages": cache}
    if case["op"] in ("prefix", "weigh"):
        G = case["Hq"] // Hkv
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        scores = s["scores"].double() if case["op"] == "weigh" else None
        for b in range(S):
            kv = raw(s["kv_pages"])[s["table"][b].long()].view(DT[case["kv"]]).flatten(0, 1)[:kl[b]].double() * scale
            q = s["q"][starts[b]:starts[b] + ql[b]].double()
            hidden = torch.arange(kl[b], device="cuda")[None] > torch.arange(kl[b] - ql[b], kl[b], device="cuda")[:, None]
            for h in range(Hkv):
                x = torch.einsum("tgd,kd->gtk", q[:, h * G:(h + 1) * G], kv[:, 2 * h]) / math.sqrt(D)
                if case.get("cap"):
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                p = torch.softmax(x.masked_fill(hidden[None], -math.inf), -1)
                if scores is None:
                    out[starts[b]:starts[b] + ql[b], h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", p, kv[:, 2 * h + 1])
                    continue
                j = torch.arange(kl[b], device="cuda")
                page, at = s["table"][b].long()[j // ps], j % ps
                before = scores[page, h, at].masked_fill(j >= kl[b] - ql[b], 0.0)
                scores[page, h, at] = before + p.sum((0, 1))
        return out if scores is None else scores
    cache, scores = s["kv_pages"].double() if case["kv"] != "int8" else s["kv_pages"].clone(), s["scores"].double()
    kept = torch.full((S, Hkv, case["budget"]), -1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([min(n, case["budget"]) for n in kl], dtype=torch.int32, device="cuda")
    for b in range(S):
        j = torch.arange(kl[b], device="cuda")
        for h in range(Hkv):
            idx = j
            if kl[b] > case["budget"]:
                middle = j[case["protect"]:kl[b] - case["recent"]]
                x = s["scores"][s["table"][b].long()[middle // ps], h, middle % ps]
                best = torch.argsort(-x.double(), stable=True)[:case["budget"] - case["protect"] - case["recent"]]
                idx = torch.cat((j[:case["protect"]], middle[best].sort().values, j[kl[b] - case["recent"]:]))
            to = torch.arange(len(idx), device="cuda")
            a, at = s["table"][b].long()[idx // ps], idx % ps
            c, ct = s["new_table"][b].long()[to // ps], to % ps
            cache[c, ct, 2 * h:2 * h + 2] = cache[a, at, 2 * h:2 * h + 2]
            scores[c, h, ct] = s["scores"][a, h, at].double()
            kept[b, h, :len(idx)] = idx.to(torch.int32)
    return {"kv_pages": cache if case["kv"] != "int8" else None, "scores": scores, "kv_lens": lens, "kept": kept}


def prepare_plainly(case, seed):
    """The inputs alone, whatever `own` says."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was
