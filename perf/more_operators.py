"""Cases, plain forms and 64-bit definitions of three more operators of the paged prefix cache: the append with normalised
query and key heads, attention with a sliding window and first tokens that stay visible, and attention of forks whose
common prefix is read once for all of them."""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one new token of each of eight candidate plans enters the 16-bit cache: the smallest call, latency
        dict(name="norm_append_step", op="append", n=8, q=1, lo=789, hi=838, H=8, Hkv=1, Dh=128, page=16, fp8=False,
             rot=128, half=True, scaling=0, heads_first=True),
        # one new token of every sequence of a serving batch enters the 8-bit cache, long-context frequencies
        dict(name="norm_append_batch_fp8", op="append", n=96, q=1, lo=40, hi=9000, H=16, Hkv=2, Dh=128, page=64,
             fp8=True, rot=128, half=True, scaling=1, heads_first=True),
        # the tokens of a large ragged prefill enter the 16-bit cache, half of each head rotated
        dict(name="norm_append_prefill", op="append", n=12, q=1024, lo=1500, hi=4000, H=16, Hkv=4, Dh=128, page=32,
             fp8=False, rot=64, half=False, scaling=0, heads_first=False),
        # odd chunks of narrow heads into the 8-bit cache
        dict(name="norm_append_odd", op="append", n=9, q=333, lo=400, hi=5000, H=10, Hkv=2, Dh=64, page=32, fp8=True,
             rot=48, half=True, scaling=0, heads_first=False),
        # a local layer of one robot's long episode: one token, its window and the first four tokens
        dict(name="sink_one_token", op="sink", n=1, q=1, lo=5000, hi=5000, H=8, Hkv=1, Dh=128, page=16, fp8=False,
             causal=True, window=512, sinks=4, heads_first=True),
        # the same layer of a serving batch over long ragged histories, 8-bit cache
        dict(name="sink_batch_fp8", op="sink", n=48, q=1, lo=700, hi=12000, H=16, Hkv=2, Dh=128, page=64, fp8=True,
             causal=True, window=2048, sinks=64, heads_first=True),
        # a long episode's history prefilled in a large chunk; the first view's tokens stay visible
        dict(name="sink_long_chunk", op="sink", n=1, q=4096, lo=12288, hi=12288, H=16, Hkv=2, Dh=128, page=64,
             fp8=False, causal=True, window=2000, sinks=256, heads_first=True),
        # odd ragged chunks, 64-wide heads in groups of five, 8-bit cache
        dict(name="sink_odd_chunks", op="sink", n=9, q=333, lo=400, hi=5000, H=10, Hkv=2, Dh=64, page=32, fp8=True,
             causal=True, window=300, sinks=37, heads_first=False),
        # eight candidate plans forked from one 788-token observation, one token each
        dict(name="shared_few_plans", op="shared", groups=1, each=8, q=1, prefix=788, own=50, H=8, Hkv=1, Dh=128,
             page=16, fp8=False, causal=True, heads_first=True),
        # a serving batch that shares a long episode's history, one token of every sequence
        dict(name="shared_batch", op="shared", groups=1, each=128, q=1, prefix=8192, own=400, H=16, Hkv=2, Dh=128,
             page=64, fp8=False, causal=True, heads_first=True),
        # three scenes with their candidates, a few tokens each (drafts to be verified), narrow heads, 8-bit cache
        dict(name="shared_scenes_fp8", op="shared", groups=3, each=24, q=5, prefix=3001, own=130, H=10, Hkv=2, Dh=64,
             page=32, fp8=True, causal=True, heads_first=False),
        # sixteen candidates that each add a 50-token chunk which sees all of itself
        dict(name="shared_chunks", op="shared", groups=1, each=16, q=50, prefix=4100, own=50, H=16, Hkv=2, Dh=128,
             page=16, fp8=False, causal=False, heads_first=True),
    ]


HEADS = [(8, 1, 128), (16, 2, 128), (10, 2, 64), (6, 6, 64), (12, 4, 128), (14, 2, 64)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "sink", "sink", "shared", "shared"])
    heads = rng.choice(HEADS)
    base = dict(op=op, H=heads[0], Hkv=heads[1], Dh=heads[2], page=rng.choice([16, 32, 64, 128, 256]),
                fp8=rng.random() < 0.5, heads_first=rng.random() < 0.5)
    if op == "append":
        n = _log(rng, 1, 96)
        q = _log(rng, 1, max(1, 12000 // n))
        hi = q + _log(rng, 1, 6000)
        dh = rng.choice([heads[2], heads[2], 80, 96, 256])
        if dh == 256:
            base["H"], base["Hkv"] = 4, 1
        base["Dh"] = dh
        return dict(base, n=n, q=q, lo=max(1, hi // 2), hi=hi, rot=rng.choice([0, 16, 48, 64, dh]),
                    half=rng.random() < 0.5, scaling=rng.randint(0, 1))
    if op == "sink":
        if rng.random() < 0.4:
            n, q, hi = _log(rng, 1, 48), _log(rng, 1, 12), _log(rng, 20, 9000)
        else:
            n, q = rng.randint(1, 6), _log(rng, 20, 1400)
            hi = q + _log(rng, 1, 6000)
        return dict(base, n=n, q=q, lo=max(1, hi // rng.choice([1, 3, 10])), hi=hi, causal=rng.random() < 0.8,
                    window=_log(rng, 1, 3000), sinks=_log(rng, 1, 300))
    groups, q = rng.choice([1, 1, 2, 3, 5]), rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 8, 64)])
    each = _log(rng, 2, min(96, max(2, 1200 // (groups * q))))
    prefix = _log(rng, 16, max(100, min(8000, 500000 // (groups * each))))
    return dict(base, groups=groups, each=each, q=q, prefix=prefix, own=q + _log(rng, 1, 400), causal=rng.random() < 0.7)


def _spread(lo, hi, n, salt=0):
    """n whole numbers of lo..hi, the same for every seed; the first is hi."""
    r = random.Random(salt * 1000003 + lo * 31 + hi * 17 + n)
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _groups(c):
    """(shared tokens, entries) of each group of a batch of forks."""
    shared = _spread(max(1, c["prefix"] // 2), c["prefix"], c["groups"], 3)
    each = _spread(max(1, c["each"] // 2), c["each"], c["groups"], 4)
    return shared, each


def _shape(c):
    """(lengths after the chunk, new tokens) of each entry of a batch."""
    if c["op"] == "shared":
        shared, each = _groups(c)
        n, q = sum(each), c["q"]
        new = [max(1, x) for x in _spread(max(1, q // 2), q, n, 1)]
        mine = [max(a, b) for a, b in zip(new, _spread(max(1, c["own"] // 3), c["own"], n, 2))]
        of = [s for s, e in zip(shared, each) for _ in range(e)]
        return [a + b for a, b in zip(of, mine)], new
    n, q = c["n"], c["q"]
    lens = _spread(c["lo"], c["hi"], n)
    new = [max(1, x) for x in _spread(max(1, q // 2), q, n, 1)]
    return lens, [min(a, b) for a, b in zip(new, lens)]


def _up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------------------------- inputs


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _batch(case, seed):
    """A cache whose sequences lie on scattered pages, and the packed new tokens of a batch of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    page, hkv, dh = case["page"], case["Hkv"], case["Dh"]
    lens, new = _shape(case)
    n = len(lens)
    shared, each = _groups(case) if case["op"] == "shared" else ([0] * n, [1] * n)
    lead, first = [], [0]   # of every entry, the first of its group and the tokens they share
    for s, e in zip(shared, each):
        lead += [(first[-1], s)] * e
        first.append(first[-1] + e)
    total = sum(_up(x, page) - (s // page if i != j else 0) for i, (x, (j, s)) in enumerate(zip(lens, lead)))
    pages, seqs = total + 5, n + 3
    stride = max(_up(x, page) for x in lens) + 2
    order, rows = r.sample(range(pages), total), r.sample(range(seqs), n)
    table, ln, books, begun = [[-1] * stride for _ in range(seqs)], [0] * seqs, [], []
    for i, (x, (j, s)) in enumerate(zip(lens, lead)):
        book = [] if i == j else books[j][:s // page]
        book = book + [order.pop() for _ in range(_up(x, page) - len(book))]
        if i != j and s % page:   # a begun page that was copied when the fork wrote to it
            begun.append((books[j][s // page], book[s // page], s % page))
        books.append(book)
        table[rows[i]][:len(book)], ln[rows[i]] = book, x
    shape = (1, pages, hkv, page, dh) if case["heads_first"] else (1, pages, page, hkv, dh)
    pools = []
    for _ in range(2):
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        t = t.transpose(2, 3) if case["heads_first"] else t
        if begun:
            src, dst, part = (torch.tensor(x, device="cuda") for x in zip(*begun))
            keep = (torch.arange(page, device="cuda")[None] < part[:, None])[None, :, :, None, None]
            t[:, dst] = torch.where(keep, t[:, src], t[:, dst])
        pools.append(t.mul_(16.0).clamp_(-448, 448).to(torch.float8_e4m3fn) if case["fp8"] else t)
    start = [0]
    for x in new:
        start.append(start[-1] + x)
    s = dict(case=case, lens_host=lens, new_host=new, shared_host=shared, first_host=first, tokens=start[-1])
    s["k"], s["v"] = pools
    s["table"], s["lens"], s["seq"], s["start"] = _dev(table), _dev(ln), _dev(rows), _dev(start)
    s["first"], s["shared"] = _dev(first), _dev(shared)
    s["refs"] = torch.bincount(s["table"][s["table"] >= 0].long(), minlength=pages).int()
    s["k_scale"] = torch.full((1,), 0.0625 * 1.1, device="cuda") if case["fp8"] else None
    s["v_scale"] = torch.full((1,), 0.0625 * 0.9, device="cuda") if case["fp8"] else None
    # token -> entry and place among the entry's new tokens, as every form of the operators needs them
    s["entry"] = torch.repeat_interleave(torch.arange(n, device="cuda"), _dev(new).long())
    s["within"] = torch.arange(s["tokens"], device="cuda") - s["start"][s["entry"]]
    return g, s


def _frequencies(case):
    """(angle per position of each rotated pair, in radians; factor on cos and sin)."""
    rot, theta, factor, original = case["rot"], 10000.0, 8.0, 4096.0
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == 0 or rot == 0:
        return f, 1.0
    # fast pairs kept, slow pairs squeezed, a ramp between 32 turns and one turn within the first length
    where = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    a, b = max(math.floor(where(32.0)), 0), min(math.ceil(where(1.0)), rot - 1)
    ramp = [min(1.0, max(0.0, (i - a) / max(b - a, 0.001))) for i in range(rot // 2)]
    return [x / factor * t + x * (1 - t) for x, t in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    g, s = _batch(case, seed)
    H, hkv, dh = case["H"], case["Hkv"], case["Dh"]
    if case["op"] == "append":
        # a merged projection's output; heads differ in size, which the norm takes out
        x = torch.randn((s["tokens"], H + 2 * hkv, dh), generator=g, device="cuda")
        x *= torch.exp(torch.randn((1, H + 2 * hkv, 1), generator=g, device="cuda"))
        s["qkv"] = x.to(torch.bfloat16)
        s["q_out"] = torch.zeros((s["tokens"], H, dh), device="cuda", dtype=torch.bfloat16)
        s["q_gamma"], s["k_gamma"] = (1.0 + 0.2 * torch.randn(dh, generator=g, device="cuda") for _ in range(2))
        f, s["mag"] = _frequencies(case)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    else:
        s["q"] = torch.randn((s["tokens"], H, dh), generator=g, device="cuda", dtype=torch.bfloat16) * 1.5
        s["out"] = torch.zeros_like(s["q"])
    if own:  # the handles that a user's program keeps: pointers to the buffers above, a workspace
        import flow_matching_action_denoise_gb300 as fmad
        s["fmad"] = fmad
        s["cache"] = fmad.KvCache(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["k_scale"], s["v_scale"])
        s["batch"] = fmad.KvBatch(s["start"], s["tokens"], max(s["new_host"]), max(s["lens_host"]), s["seq"])
        if case["op"] == "append":
            s["rope"] = fmad.Rope(case["rot"], theta=10000.0, half=case["half"],
                                  scaling=(fmad.ROPE_PLAIN, fmad.ROPE_BY_PARTS)[case["scaling"]], factor=8.0,
                                  original_len=4096.0, beta_fast=32.0, beta_slow=1.0)
        elif case["op"] == "sink":
            need = fmad.paged_attention_workspace_size(s["cache"], s["batch"], H)
        else:
            most = max(b - a for a, b in zip(s["first_host"], s["first_host"][1:]))
            s["groups"] = fmad.KvGroups(s["first"], s["shared"], most, max(s["shared_host"]))
            need = fmad.shared_attention_workspace_size(s["cache"], s["batch"], s["groups"], H)
        if case["op"] != "append":
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------- passes


def run(s):
    return {"append": _append, "sink": _sink, "shared": _shared}[s["case"]["op"]](s)


def _positions(s):
    new = s["start"][1:] - s["start"][:-1]
    return (s["lens"][s["seq"].long()] - new).long()[s["entry"]] + s["within"]


def _append(s):
    c = s["case"]
    H, hkv = c["H"], c["Hkv"]
    q, k, v = s["qkv"][:, :H], s["qkv"][:, H:H + hkv], s["qkv"][:, H + hkv:]
    if own:
        s["fmad"].norm_rope_append(s["cache"], 0, s["batch"], s["rope"], q, k, v, s["q_out"], s["q_gamma"], s["k_gamma"],
                                   eps=1e-6)
        return s["q_out"], s["k"], s["v"]
    pos = _positions(s)
    x = s["qkv"][:, :H + hkv].float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    x = torch.cat((x[:, :H] * s["q_gamma"], x[:, H:] * s["k_gamma"]), 1)
    rot, pairs = c["rot"], c["rot"] // 2
    if rot:
        angle = pos[:, None].double() * s["freq"]
        cos, sin = ((f(angle) * s["mag"]).float()[:, None] for f in (torch.cos, torch.sin))  # [T, 1, rot / 2]
        if c["half"]:
            a, b = x[..., :pairs], x[..., pairs:rot]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        x = torch.cat((turned, x[..., rot:]), -1)
    s["q_out"].copy_(x[:, :H])
    at = s["table"][s["seq"].long()[s["entry"]], pos // c["page"]].long()
    for pool, y, scale in ((s["k"], x[:, H:], s["k_scale"]), (s["v"], v.float(), s["v_scale"])):
        if c["fp8"]:
            codes = (y / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            pool.view(torch.uint8)[0][at, pos % c["page"]] = codes.view(torch.uint8)
        else:
            pool[0][at, pos % c["page"]] = y.to(torch.bfloat16)
    return s["q_out"], s["k"], s["v"]


def _rows(pool, pages, within):
    """Rows of layer 0's pages; 8-bit values are gathered as bytes."""
    if pool.dtype == torch.float8_e4m3fn:
        return pool.view(torch.uint8)[0][pages, within].view(torch.float8_e4m3fn)
    return pool[0][pages, within]


def _attend(s, window, sinks):
    """Every entry's new tokens over its own table row, in 32 bits."""
    c = s["case"]
    n, page, hkv, dh = len(s["lens_host"]), c["page"], c["Hkv"], c["Dh"]
    group, longest, most = c["H"] // hkv, max(s["lens_host"]), max(s["new_host"])
    at = torch.arange(longest, device="cuda")
    idx = s["table"][s["seq"].long()][:, at // page].long().clamp(min=0)  # [n, longest]
    lens = s["lens"][s["seq"].long()]
    k, v = (_rows(s[x], idx, at % page).float() for x in ("k", "v"))  # [n, longest, Hkv, Dh]
    if c["fp8"]:
        k, v = k * s["k_scale"], v * s["v_scale"]
    q = torch.zeros((n, most, c["H"], dh), device="cuda")
    q[s["entry"], s["within"]] = s["q"].float()
    q = q.view(n, most, hkv, group, dh).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * most, dh)
    scores = (q @ k.permute(0, 2, 3, 1)).view(n, hkv, group, most, longest) / math.sqrt(dh)
    new = s["start"][1:] - s["start"][:-1]
    pos = ((lens - new)[:, None] + torch.arange(most, device="cuda"))[:, :, None]  # [n, most, 1]
    ok = (at < lens[:, None, None]) & (pos >= 0)
    if c["causal"]:
        ok = ok & (at <= pos)
    if window:
        ok = ok & ((at > pos - window) | (at < sinks))
    scores = scores.masked_fill_(~ok[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = scores.sum(-1, keepdim=True)
    o = scores.view(n, hkv, group * most, longest) @ v.permute(0, 2, 1, 3)
    o = o.view(n, hkv, group, most, dh) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(n, most, c["H"], dh)
    s["out"].copy_(o[s["entry"], s["within"]])
    return s["out"]


def _sink(s):
    c = s["case"]
    if own:
        s["fmad"].sink_attention(s["cache"], 0, s["batch"], s["q"], s["out"], s["ws"], causal=c["causal"],
                                 window=c["window"], sinks=c["sinks"])
        return s["out"]
    return _attend(s, c["window"], c["sinks"])


def _shared(s):
    if own:
        s["fmad"].shared_attention(s["cache"], 0, s["batch"], s["groups"], s["q"], s["out"], s["ws"],
                                   causal=s["case"]["causal"])
        return s["out"]
    return _attend(s, 0, 0)


# ---------------------------------------------------------------------------------------------------- work


def _visible(c, pos, ln):
    """Keys that a token at `pos` sees."""
    end = min(pos + 1, ln) if c["causal"] else ln
    if c["op"] == "shared":
        return end
    low = max(0, pos - c["window"] + 1)
    return max(0, end - low) + min(c["sinks"], low, end)


def work(case):
    c = case
    lens, new = _shape(c)
    tokens = sum(new)
    if c["op"] == "append":
        row = c["Dh"] * tokens
        return {"bytes": 2 * row * (2 * c["H"] + 2 * c["Hkv"]) + 2 * row * c["Hkv"] * (1 if c["fp8"] else 2) + 8 * c["Dh"],
                "flops": 4 * row * (c["H"] + c["Hkv"]) + 3 * tokens * (c["H"] + c["Hkv"]) * c["rot"]}
    pairs = sum(_visible(c, ln - q + i, ln) for ln, q in zip(lens, new) for i in range(q))
    if c["op"] == "sink":
        keys = 0   # of all tokens of an entry together
        for ln, q in zip(lens, new):
            low = max(0, ln - q - c["window"] + 1)
            keys += ln - low + min(c["sinks"], low)
    else:
        shared, each = _groups(c)
        keys = sum(lens) - sum(s * (e - 1) for s, e in zip(shared, each))
    row = 2 * c["Hkv"] * c["Dh"] * (1 if c["fp8"] else 2)
    return {"bytes": 2 * 2 * tokens * c["H"] * c["Dh"] + keys * row, "flops": 4 * c["Dh"] * c["H"] * pairs}


# ---------------------------------------------------------------------------------------------------- definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    H, hkv, dh = c["H"], c["Hkv"], c["Dh"]
    if c["op"] == "append":
        rot, pos = c["rot"], _positions(s)
        x = s["qkv"].double()
        size = (x.pow(2).sum(-1, keepdim=True) / dh + 1e-6).sqrt()
        gain = torch.cat((s["q_gamma"].expand(H, dh), s["k_gamma"].expand(hkv, dh))).double()
        x[:, :H + hkv] = x[:, :H + hkv] / size[:, :H + hkv] * gain
        if rot:
            z = torch.polar(torch.full((s["tokens"], rot // 2), s["mag"], dtype=torch.float64, device="cuda"),
                            pos[:, None] * s["freq"])
            part = x[:, :H + hkv, :rot]
            pair = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["half"] else part.unflatten(-1, (rot // 2, 2))
            pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[:, None])
            x[:, :H + hkv, :rot] = (pair.transpose(-1, -2) if c["half"] else pair).flatten(-2)
        k, v = s["k"].to(torch.float64), s["v"].to(torch.float64)
        where = s["table"][s["seq"].long()[s["entry"]], pos // c["page"]].long()
        ks, vs = (s[n].double() if c["fp8"] else 1.0 for n in ("k_scale", "v_scale"))
        k[0, where, pos % c["page"]] = x[:, H:H + hkv] / ks
        v[0, where, pos % c["page"]] = x[:, H + hkv:] / vs
        return x[:, :H], k, v
    out = torch.zeros((s["tokens"], H, dh), dtype=torch.float64, device="cuda")
    begin = 0
    for i, (ln, q) in enumerate(zip(s["lens_host"], s["new_host"])):
        at = torch.arange(ln, device="cuda")
        pages = s["table"][s["seq"][i].long()][at // c["page"]].long()
        k, v = (s[x].to(torch.float64)[0][pages, at % c["page"]] for x in ("k", "v"))
        if c["fp8"]:
            k, v = k * s["k_scale"].double(), v * s["v_scale"].double()
        pos = torch.arange(ln - q, ln, device="cuda")[:, None]
        hidden = torch.zeros((q, ln), dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden |= at > pos
        if c["op"] == "sink":
            hidden |= (at <= pos - c["window"]) & (at >= c["sinks"])
        for h in range(hkv):
            heads = slice(h * (H // hkv), (h + 1) * (H // hkv))
            w = torch.einsum("thd,kd->htk", s["q"][begin:begin + q, heads].double(), k[:, h]) * dh ** -0.5
            w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
            out[begin:begin + q, heads] = torch.einsum("htk,kd->thd", torch.nan_to_num(w), v[:, h])
        begin += q
    return out
