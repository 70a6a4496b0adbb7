"""Cases, plain forms and 64-bit definitions of the paged prefix-cache operators: attention of a chunk of new tokens
over a paged cache, rotary positions with the store into the cache, the pages' bookkeeping and copies, and the
residual RMS norm with an 8-bit output."""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one robot asks for one token after its 788-token prefix (8 heads on 1 KV head): the smallest call, latency
        dict(name="attn_one_token", op="attn", n=1, q=1, lo=789, hi=789, H=8, Hkv=1, Dh=128, page=16, fp8=False,
             causal=True, window=0, heads_first=True),
        # a serving batch of single tokens over long ragged histories, 8-bit cache: bound by reading the cache
        dict(name="attn_batch_fp8", op="attn", n=48, q=1, lo=700, hi=12000, H=16, Hkv=2, Dh=128, page=64, fp8=True,
             causal=True, window=0, heads_first=True),
        # one image view (256 tokens) of several cameras refreshed over 1024-token prefixes, every token sees all keys
        dict(name="attn_view_full", op="attn", n=6, q=256, lo=788, hi=1044, H=16, Hkv=2, Dh=128, page=16, fp8=False,
             causal=False, window=0, heads_first=False),
        # a long episode's history prefilled in a large chunk, causal: bound by the tensor cores
        dict(name="attn_long_chunk", op="attn", n=1, q=4096, lo=12288, hi=12288, H=16, Hkv=2, Dh=128, page=64,
             fp8=False, causal=True, window=0, heads_first=True),
        # odd ragged chunks with a sliding window, 64-wide heads in groups of five, 8-bit cache
        dict(name="attn_window_odd", op="attn", n=9, q=333, lo=400, hi=5000, H=10, Hkv=2, Dh=64, page=32, fp8=True,
             causal=True, window=1000, heads_first=False),
        # one new token of every sequence of a serving batch enters the 8-bit cache
        dict(name="append_tokens", op="append", n=32, q=1, lo=40, hi=9000, H=16, Hkv=2, Dh=128, page=64, fp8=True,
             rot=128, half=True, scaling=2, heads_first=True),
        # the tokens of a large ragged prefill enter the 16-bit cache; only half of each head is rotated
        dict(name="append_prefill", op="append", n=12, q=1024, lo=1500, hi=4000, H=16, Hkv=4, Dh=128, page=32,
             fp8=False, rot=64, half=False, scaling=0, heads_first=False),
        # rows of a small batch before a projection
        dict(name="norm_few_rows", op="norm", T=10, d=1024, block=0, f32=True, res=True),
        # a prefill's rows, one scale per 128 columns
        dict(name="norm_prefill", op="norm", T=12000, d=2048, block=128, f32=False, res=True),
        # one observation's prefix forked for a few candidate plans, each of which then adds a chunk
        dict(name="pages_fork_few", op="fork", n=8, lo=788, hi=788, add=50, L=18, Hkv=1, Dh=128, page=16, pages=160,
             one=True),
        # many sequences each forked once and extended by one token: every shared last page is copied
        dict(name="pages_fork_many", op="fork", n=64, lo=500, hi=3000, add=1, L=28, Hkv=2, Dh=128, page=64,
             pages=2200, one=False),
        # a fragmented pool drawn together before its tail is handed back
        dict(name="pages_compact", op="compact", live=1500, move=600, L=18, Hkv=1, Dh=128, page=16, pages=2500, seqs=24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "norm", "fork", "compact"])
    heads = rng.choice([(8, 1, 128), (16, 2, 128), (10, 2, 64), (6, 6, 64), (12, 4, 128), (14, 2, 64)])
    if op == "attn":
        if rng.random() < 0.4:
            n, q, hi = _log(rng, 1, 48), _log(rng, 1, 12), _log(rng, 20, 9000)
        else:
            n, q = rng.randint(1, 6), _log(rng, 20, 1400)
            hi = q + _log(rng, 1, 4000)
        return dict(op="attn", n=n, q=q, lo=max(1, hi // rng.choice([1, 3, 10])), hi=hi, H=heads[0], Hkv=heads[1],
                    Dh=heads[2], page=rng.choice([16, 32, 64, 128, 256]), fp8=rng.random() < 0.5,
                    causal=rng.random() < 0.7, window=rng.choice([0, 0, _log(rng, 1, 2000)]),
                    heads_first=rng.random() < 0.5)
    if op == "append":
        n = _log(rng, 1, 40)
        q = _log(rng, 1, max(1, 12000 // n))
        hi = q + _log(rng, 1, 6000)
        return dict(op="append", n=n, q=q, lo=max(1, hi // 2), hi=hi, H=heads[0], Hkv=heads[1], Dh=heads[2],
                    page=rng.choice([16, 32, 64, 128, 256]), fp8=rng.random() < 0.5,
                    rot=rng.choice([16, 32, 48, 64, heads[2]]), half=rng.random() < 0.5, scaling=rng.randint(0, 3),
                    heads_first=rng.random() < 0.5)
    if op == "norm":
        d = 16 * _log(rng, 4, 512)
        return dict(op="norm", T=_log(rng, 1, 12000 * 2048 // d), d=d, block=rng.choice([0, 128]),
                    f32=rng.random() < 0.5, res=rng.random() < 0.7)
    page = rng.choice([16, 32, 64, 128])
    layers = rng.randint(1, 28)
    if op == "fork":
        n, hi = _log(rng, 1, 64), _log(rng, 2, 3000)
        add = _log(rng, 1, 100)
        return dict(op="fork", n=n, lo=max(1, hi // 3), hi=hi, add=add, L=layers, Hkv=heads[1], Dh=heads[2], page=page,
                    pages=n * (hi // page + 1 + add // page + 3) + rng.randint(0, 40), one=rng.random() < 0.3)
    live = _log(rng, 10, 60000 // page)
    return dict(op="compact", live=live, move=rng.randint(1, max(1, live // 2)), L=layers, Hkv=heads[1], Dh=heads[2],
                page=page, pages=live + live // 2 + rng.randint(1, 40), seqs=rng.randint(1, 30))


def _spread(case, lo, hi, n, salt=0):
    """n whole numbers of lo..hi, the same for every seed; the first is hi."""
    r = random.Random(salt * 1000003 + lo * 31 + hi * 17 + n)
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _shape(case):
    """(lengths after the chunk, new tokens) of each entry of a batch."""
    n, q = case["n"], case["q"]
    lens = _spread(case, case["lo"], case["hi"], n)
    new = [max(1, x) for x in _spread(case, max(1, q // 2), q, n, 1)]
    return lens, [min(a, b) for a, b in zip(new, lens)]


def _up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------------------------- inputs


def _pool(g, case, layers, pages):
    """K and V pools [layers, pages, page, Hkv, Dh], heads outside or inside of the tokens in memory."""
    page, hkv, dh = case["page"], case["Hkv"], case["Dh"]
    first = case.get("heads_first", True)
    shape = (layers, pages, hkv, page, dh) if first else (layers, pages, page, hkv, dh)
    out = []
    for _ in range(2):
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if case.get("fp8"):
            t = t.mul_(16.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        out.append(t.transpose(2, 3) if first else t)
    return out


def _prepare_batch(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    lens, new = _shape(case)
    n, page = case["n"], case["page"]
    held = [_up(x, page) for x in lens]
    seqs, stride = n + 3, max(held) + 2
    pages = sum(held) + 5
    s = dict(case=case, lens_host=lens, new_host=new)
    s["k"], s["v"] = _pool(g, case, 1, pages)
    order = r.sample(range(pages), sum(held))
    rows = r.sample(range(seqs), n)
    table, ln = [[-1] * stride for _ in range(seqs)], [0] * seqs
    for i, row in enumerate(rows):
        ln[row] = lens[i]
        for j in range(held[i]):
            table[row][j] = order.pop()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s["table"], s["lens"], s["seq"] = dev(table), dev(ln), dev(rows)
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["refs"][s["table"][s["table"] >= 0].long()] = 1
    start = [0]
    for x in new:
        start.append(start[-1] + x)
    s["start"], s["tokens"] = dev(start), start[-1]
    s["k_scale"] = torch.full((1,), 0.0625 * 1.1, device="cuda") if case["fp8"] else None
    s["v_scale"] = torch.full((1,), 0.0625 * 0.9, device="cuda") if case["fp8"] else None
    # token -> entry and position, as every form of the operators needs them
    s["entry"] = torch.repeat_interleave(torch.arange(n, device="cuda"), dev(new).long())
    s["within"] = torch.arange(s["tokens"], device="cuda") - s["start"][s["entry"]]
    return g, s


def _rope_frequencies(case):
    """(angle per position of each rotated pair, in radians; factor on cos and sin)."""
    rot, theta, factor, original = case["rot"], 10000.0, 8.0, 4096.0
    if case["scaling"] == 2:  # the base grows so that the slowest pair turns `factor` times slower
        theta *= factor ** (rot / (rot - 2.0))
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == 1:  # positions squeezed
        return [x / factor for x in f], 1.0
    if case["scaling"] == 3:  # fast pairs kept, slow pairs squeezed, a ramp over the turns within the first length
        fast, slow = 32.0, 1.0
        where = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        a, b = max(math.floor(where(fast)), 0), min(math.ceil(where(slow)), rot - 1)
        ramp = [min(1.0, max(0.0, (i - a) / max(b - a, 0.001))) for i in range(rot // 2)]
        return [x / factor * t + x * (1 - t) for x, t in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    if case["op"] == "attn":
        g, s = _prepare_batch(case, seed)
        s["q"] = torch.randn((s["tokens"], case["H"], case["Dh"]), generator=g, device="cuda", dtype=torch.bfloat16)
        s["q"] *= 1.5
        s["out"] = torch.zeros_like(s["q"])
    elif case["op"] == "append":
        g, s = _prepare_batch(case, seed)
        heads = case["H"] + 2 * case["Hkv"]
        qkv = torch.randn((s["tokens"], heads, case["Dh"]), generator=g, device="cuda", dtype=torch.bfloat16)
        s["qkv"] = qkv
        s["q_out"] = torch.zeros((s["tokens"], case["H"], case["Dh"]), device="cuda", dtype=torch.bfloat16)
        f, s["mag"] = _rope_frequencies(case)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    elif case["op"] == "norm":
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = torch.float32 if case["f32"] else torch.bfloat16
        x = torch.randn((case["T"], case["d"]), generator=g, device="cuda")
        # a few loud columns, as residual streams have
        x[:, :: max(1, case["d"] // 7)] *= 12.0
        s = dict(case=case, x=x.to(t))
        s["r"] = torch.randn((case["T"], case["d"]), generator=g, device="cuda").to(torch.bfloat16) if case["res"] else None
        s["gamma"] = 1.0 + 0.2 * torch.randn(case["d"], generator=g, device="cuda")
        cols = _up(case["d"], case["block"]) if case["block"] else 1
        s["x_out"] = torch.empty_like(s["x"])
        s["codes"] = torch.empty((case["T"], case["d"]), dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty((case["T"], cols), device="cuda")
    else:
        s = _prepare_pages(case, seed)
    if own:  # the handles that a user's program keeps: pointers to the buffers above, a workspace
        import flow_matching_action_denoise_gb300 as fmad
        s["fmad"] = fmad
        if case["op"] != "norm":
            s["cache"] = fmad.KvCache(s["k"], s["v"], s["table"], s["lens"], s["refs"], s.get("k_scale"), s.get("v_scale"))
        if case["op"] in ("attn", "append"):
            s["batch"] = fmad.KvBatch(s["start"], s["tokens"], max(s["new_host"]), max(s["lens_host"]), s["seq"])
        if case["op"] == "attn":
            s["ws"] = torch.empty(fmad.paged_attention_workspace_size(s["cache"], s["batch"], case["H"]),
                                  dtype=torch.uint8, device="cuda")
        if case["op"] == "append":
            kinds = (fmad.ROPE_PLAIN, fmad.ROPE_LINEAR, fmad.ROPE_BASE, fmad.ROPE_BY_PARTS)
            s["rope"] = fmad.Rope(case["rot"], theta=10000.0, half=case["half"], scaling=kinds[case["scaling"]],
                                  factor=8.0, original_len=4096.0, beta_fast=32.0, beta_slow=1.0)
        if case["op"] in ("fork", "compact"):
            s["ws"] = torch.empty(fmad.kv_workspace_size(s["cache"], case.get("n", 0)), dtype=torch.uint8, device="cuda")
    return s


def _prepare_pages(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    page, pages = case["page"], case["pages"]
    s = dict(case=case)
    s["k"], s["v"] = _pool(g, case, case["L"], pages)
    if case["op"] == "fork":
        n = case["n"]
        lens = [case["hi"]] if case["one"] else _spread(case, case["lo"], case["hi"], n)
        held = [_up(x, page) for x in lens]
        seqs, stride = len(lens) + n + 1, max(held) + _up(case["add"], page) + 1
        rows = r.sample(range(seqs), len(lens) + n)
        order = r.sample(range(pages), sum(held))
        src = [rows[0] if case["one"] else rows[i] for i in range(n)]
        dst = rows[len(lens):]
    else:
        # `live` pages held, all but `move` of them among the lowest `live`
        live, move = case["live"], min(case["move"], case["live"], pages - case["live"])
        holes = set(r.sample(range(live), move))
        order = [i for i in range(live) if i not in holes] + r.sample(range(live, pages), move)
        r.shuffle(order)
        seqs = min(case["seqs"], live)
        held = [live // seqs + (i < live % seqs) for i in range(seqs)]
        lens = [x * page - r.randrange(page) for x in held]
        stride, rows = max(held) + 1, list(range(seqs))
        s["moves"], src, dst = move, [], []
    book = [[-1] * stride for _ in range(seqs)]
    ln, refs = [0] * seqs, [0] * pages
    for i, x in enumerate(lens):
        ln[rows[i]] = x
        for j in range(held[i]):
            book[rows[i]][j] = order.pop()
            refs[book[rows[i]][j]] = 1
    # one buffer holds the table, the lengths and the counts, so that a pass begins with one copy of it
    flat = [v for row in book for v in row] + ln + refs
    s["book0"] = torch.tensor(flat, dtype=torch.int32, device="cuda")
    s["book"] = s["book0"].clone()
    a, b = seqs * stride, seqs * stride + seqs
    s["table"], s["lens"], s["refs"] = s["book"][:a].view(seqs, stride), s["book"][a:b], s["book"][b:]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s["src"], s["dst"] = dev(src), dev(dst)
    s["add"] = torch.full((len(dst),), case.get("add", 0), dtype=torch.int32, device="cuda")
    s["status"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------- passes


def run(s):
    op = s["case"]["op"]
    return {"attn": _attn, "append": _append, "norm": _norm, "fork": _fork, "compact": _compact}[op](s)


def _attn(s):
    c = s["case"]
    if own:
        s["fmad"].paged_attention(s["cache"], 0, s["batch"], s["q"], s["out"], s["ws"], causal=c["causal"],
                                  window=c["window"])
        return s["out"]
    n, page, hkv, dh = c["n"], c["page"], c["Hkv"], c["Dh"]
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
    pos = (lens - new)[:, None] + torch.arange(most, device="cuda")  # [n, most]
    ok = at[None, None] < lens[:, None, None]
    if c["causal"]:
        ok = ok & (at[None, None] <= pos[:, :, None])
    else:
        ok = ok & (pos[:, :, None] >= 0)
    if c["window"]:
        ok = ok & (at[None, None] > pos[:, :, None] - c["window"])
    scores = scores.masked_fill_(~ok[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = scores.sum(-1, keepdim=True)
    o = scores.view(n, hkv, group * most, longest) @ v.permute(0, 2, 1, 3)
    o = o.view(n, hkv, group, most, dh) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(n, most, c["H"], dh)
    s["out"].copy_(o[s["entry"], s["within"]])
    return s["out"]


def _rows(pool, pages, within):
    """Rows of layer 0's pages; 8-bit values are gathered as bytes."""
    if pool.dtype == torch.float8_e4m3fn:
        return pool.view(torch.uint8)[0][pages, within].view(torch.float8_e4m3fn)
    return pool[0][pages, within]


def _positions(s):
    ln = s["lens"][s["seq"].long()]
    new = s["start"][1:] - s["start"][:-1]
    return (ln - new).long()[s["entry"]] + s["within"]


def _append(s):
    c = s["case"]
    H, hkv = c["H"], c["Hkv"]
    q, k, v = s["qkv"][:, :H], s["qkv"][:, H:H + hkv], s["qkv"][:, H + hkv:]
    if own:
        s["fmad"].rope_append(s["cache"], 0, s["batch"], s["rope"], q, k, v, s["q_out"])
        return s["q_out"], s["k"], s["v"]
    pos = _positions(s)
    angle = pos[:, None].double() * s["freq"]
    cos, sin = ((f(angle) * s["mag"]).float()[:, None] for f in (torch.cos, torch.sin))  # [T, 1, rot / 2]
    x = s["qkv"][:, :H + hkv].float()
    rot, pairs = c["rot"], c["rot"] // 2
    if c["half"]:
        a, b = x[..., :pairs], x[..., pairs:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    x = torch.cat((turned, x[..., rot:]), -1)
    s["q_out"].copy_(x[:, :H])
    at = s["table"][s["seq"].long()[s["entry"]], pos // c["page"]].long()
    kk, vv = x[:, H:], v.float()
    if c["fp8"]:
        kk = (kk / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        vv = (vv / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["k"].view(torch.uint8)[0][at, pos % c["page"]] = kk.view(torch.uint8)
        s["v"].view(torch.uint8)[0][at, pos % c["page"]] = vv.view(torch.uint8)
    else:
        s["k"][0][at, pos % c["page"]] = kk.to(torch.bfloat16)
        s["v"][0][at, pos % c["page"]] = vv.to(torch.bfloat16)
    return s["q_out"], s["k"], s["v"]


def _norm(s):
    c = s["case"]
    if own:
        s["fmad"].norm_quant(s["x"], s["r"], s["gamma"], 1e-6, s["x_out"], s["codes"], s["scales"], block=c["block"])
        return s["x_out"], s["codes"], s["scales"]
    x = s["x"].float()
    if s["r"] is not None:
        x = x + s["r"].float()
    s["x_out"].copy_(x)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["gamma"]
    block = c["block"] or c["d"]
    cols = _up(c["d"], block)
    y = torch.nn.functional.pad(y, (0, cols * block - c["d"])).view(c["T"], cols, block)
    scale = y.abs().amax(-1) / 448.0
    y = y / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    s["codes"].copy_(y.clamp(-448, 448).view(c["T"], cols * block)[:, :c["d"]])
    s["scales"].copy_(scale)
    return s["x_out"], s["codes"], s["scales"]


def _fork(s):
    c = s["case"]
    s["book"].copy_(s["book0"])
    if own:
        s["fmad"].kv_fork(s["cache"], s["src"], s["dst"], s["status"])
        s["fmad"].kv_reserve(s["cache"], s["dst"], s["add"], s["status"], s["ws"])
        return s["k"], s["v"], s["table"], s["lens"], s["refs"], s["status"]
    table, lens, refs, page = s["table"], s["lens"], s["refs"], c["page"]
    src, dst = s["src"].long(), s["dst"].long()
    # the fork: the rows and lengths copied, every page of them counted once more
    rows = table[src]
    refs.scatter_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).int().flatten())
    table[dst], lens[dst] = rows, lens[src]
    # the pages wanted: a copy of a shared last page that is begun, and pages for the new tokens
    ln = lens[dst].long()
    part, have, want = ln % page, (ln + page - 1) // page, (ln + s["add"] + page - 1) // page
    last = torch.where(part > 0, rows.gather(1, (ln // page).clamp(max=rows.shape[1] - 1)[:, None])[:, 0].long(),
                       -1 - torch.arange(len(dst), device="cuda"))
    earlier = ((last[:, None] == last[None]) & (torch.arange(len(dst), device="cuda")[:, None]
                                                 > torch.arange(len(dst), device="cuda"))).sum(1)
    copied = (part > 0) & (refs[last.clamp(min=0)] - earlier > 1)
    need = want - have + copied
    before = need.cumsum(0) - need
    free = torch.argsort((refs > 0).int(), stable=True)
    slot = torch.arange(table.shape[1], device="cuda")[None]
    mine = (copied[:, None] & (slot == (ln // page)[:, None]))
    fresh = (slot >= have[:, None]) & (slot < want[:, None])
    place = before[:, None] + torch.where(mine, torch.zeros_like(slot), copied[:, None] + slot - have[:, None])
    new = free[place.clamp(0, len(free) - 1)].int()
    table[dst] = torch.where(mine | fresh, new, table[dst])
    refs.scatter_add_(0, new.flatten().long(), (mine | fresh).int().flatten())
    refs.scatter_add_(0, last.clamp(min=0), -copied.int())
    lens[dst] += s["add"]
    target = torch.where(copied, free[before.clamp(max=len(free) - 1)], last.clamp(min=0))
    keep = (torch.arange(page, device="cuda")[None] < part[:, None])[None, :, :, None, None]
    last = last.clamp(min=0)
    for_one = copied[None, :, None, None, None] & keep
    s["k"][:, target] = torch.where(for_one, s["k"][:, last], s["k"][:, target])
    s["v"][:, target] = torch.where(for_one, s["v"][:, last], s["v"][:, target])
    s["status"].zero_()
    s["status"][1] = need.sum()
    return s["k"], s["v"], table, lens, refs, s["status"]


def _compact(s):
    s["book"].copy_(s["book0"])
    if own:
        s["fmad"].kv_compact(s["cache"], s["status"], s["ws"])
        return s["k"], s["v"], s["table"], s["lens"], s["refs"], s["status"]
    table, refs, moves = s["table"], s["refs"], s["moves"]
    at = torch.arange(len(refs), device="cuda")
    live = refs > 0
    count = live.sum()
    src = torch.argsort((live & (at >= count)).int(), descending=True, stable=True)[:moves]
    dst = torch.argsort((~live & (at < count)).int(), descending=True, stable=True)[:moves]
    s["k"][:, dst], s["v"][:, dst] = s["k"][:, src], s["v"][:, src]
    to = at.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    refs[dst] = refs[src]
    refs[src] = 0
    s["status"].zero_()
    s["status"][1] = len(src)
    return s["k"], s["v"], table, s["lens"], refs, s["status"]


# ---------------------------------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "attn":
        lens, new = _shape(c)
        pairs = keys = 0
        for ln, q in zip(lens, new):
            first = ln - q
            w = c["window"] or ln + 1
            if c["causal"]:
                a = [min(first + i + 1, w) for i in range(q)]
                keys += ln - max(0, first + 1 - w)
            else:
                a = [ln - max(0, first + i + 1 - w) for i in range(q)]
                keys += ln - max(0, first + 1 - w)
            pairs += sum(a)
        byte = 2 * 2 * sum(new) * c["H"] * c["Dh"] + 2 * keys * c["Hkv"] * c["Dh"] * (1 if c["fp8"] else 2)
        return {"bytes": byte, "flops": 4 * c["Dh"] * c["H"] * pairs}
    if c["op"] == "append":
        t = sum(_shape(c)[1])
        row = c["Dh"] * t
        return {"bytes": 2 * row * (2 * c["H"] + 2 * c["Hkv"]) + 2 * row * c["Hkv"] * (1 if c["fp8"] else 2),
                "flops": 3 * t * (c["H"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "norm":
        cols = _up(c["d"], c["block"]) if c["block"] else 1
        each = 2 * (4 if c["f32"] else 2) + (2 if c["res"] else 0) + 1
        return {"bytes": c["T"] * (c["d"] * each + 4 * cols) + 4 * c["d"], "flops": 8 * c["T"] * c["d"]}
    row = 2 * c["L"] * c["Hkv"] * c["Dh"] * 2
    if c["op"] == "fork":
        lens = [c["hi"]] * c["n"] if c["one"] else _spread(c, c["lo"], c["hi"], c["n"])
        rows = sum(x % c["page"] for x in lens)
        book = 4 * (c["pages"] + sum(2 * _up(x, c["page"]) for x in lens))
    else:
        move = min(c["move"], c["live"], c["pages"] - c["live"])
        rows, book = move * c["page"], 4 * (2 * c["pages"] + 2 * c["live"])
    return {"bytes": 2 * row * rows + book, "flops": 0}


# ---------------------------------------------------------------------------------------------------- definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "attn":
        out = torch.zeros((s["tokens"], c["H"], c["Dh"]), dtype=torch.float64, device="cuda")
        begin = 0
        for i, (ln, q) in enumerate(zip(s["lens_host"], s["new_host"])):
            at = torch.arange(ln, device="cuda")
            pages = s["table"][s["seq"][i].long()][at // c["page"]].long()
            k, v = (s[x].to(torch.float64)[0][pages, at % c["page"]] for x in ("k", "v"))
            if c["fp8"]:
                k, v = k * s["k_scale"].double(), v * s["v_scale"].double()
            pos = torch.arange(ln - q, ln, device="cuda")[:, None]
            key = torch.arange(ln, device="cuda")[None]
            ok = torch.ones((q, ln), dtype=torch.bool, device="cuda")
            if c["causal"]:
                ok &= key <= pos
            if c["window"]:
                ok &= key > pos - c["window"]
            for h in range(c["H"]):
                kv = h // (c["H"] // c["Hkv"])
                w = (s["q"][begin:begin + q, h].double() @ k[:, kv].T) * c["Dh"] ** -0.5
                w = torch.softmax(w.masked_fill(~ok, -math.inf), -1)
                out[begin:begin + q, h] = torch.nan_to_num(w) @ v[:, kv]
            begin += q
        return out
    if c["op"] == "append":
        T, H, hkv, rot = s["tokens"], c["H"], c["Hkv"], c["rot"]
        pos = _positions(s)
        z = torch.polar(torch.full((T, rot // 2), s["mag"], dtype=torch.float64, device="cuda"), pos[:, None] * s["freq"])
        x = s["qkv"].double().clone()
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
    if c["op"] == "norm":
        x = s["x"].double() + (s["r"].double() if c["res"] else 0.0)
        y = x / (x.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * s["gamma"].double()
        b = c["block"] or c["d"]
        parts = y.split(b, 1)
        scale = torch.stack([p.abs().max(1).values / 448.0 for p in parts], 1)
        return x, torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1), scale
    return None
