"""The operators at the two edges of a verification step, as a user's program
calls them, and their plain forms in elementary torch operations.

  reserve  sv_reserve_kv: blocks of a step's rows taken from the pool, their
           table entries, cache slots and positions
  stage    sv_stage_qkv: head norms and rotation of Q and K, K and V written
           into the paged cache
  shape    sv_shape_logits: penalties for repeated tokens, biases and grammar
           masks on the logits of every draft node
"""

import math

import torch

own = False

PAGE = 16  # tokens of a cache page


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one request of an interactive session, six draft rows behind a context of a few thousand tokens
        reserve("reserve one chain", 1, 4096, 4096, 6, 6),
        # a served batch whose requests all verify four drafts, as the budget step has it
        reserve("reserve 256 chains", 256, 1024, 8192, 5, 5),
        # sixty-four draft trees, and a pool that has too few blocks for the last of them
        reserve("reserve 64 trees, short pool", 64, 17, 32768, 33, 65, tree=True, short=True),
        # prompts of ragged lengths admitted at once, none of them in the cache yet
        reserve("reserve 48 prompts", 48, 0, 0, 1, 4001, prompts=True),
        # the draft rows of one request: launch and latency only
        stage("stage one chain", 6, 32, 8, 128),
        # the rows of a batch of 256 requests, heads normed, packed projection output, the last rows padding
        stage("stage 256 chains", 1280, 40, 8, 128, pad=37),
        # video positions on three axes, a rotation of half of a small head, pairs side by side, an odd number of rows
        stage("stage three axes", 4099, 14, 2, 64, rotary=32, axes=3, interleaved=True, far=1 << 20),
        # a long prompt's rows through the same call
        stage("stage a prompt", 20000, 64, 8, 128, far=131072),
        # the target logits of one chain, its history as long as its context
        shape("shape one chain", 1, 6, 6, 128256, 4096, 4096),
        # a served batch of ragged chains, histories of hundreds to tens of thousands of tokens, a few biased tokens each
        shape("shape 64 chains", 64, 2, 9, 128256, 512, 32768, bias=24),
        # structured output: every node of a few trees has a grammar's mask that lets few tokens through, 16-bit logits of an odd, padded vocabulary
        shape("shape 16 trees, grammar", 16, 33, 65, 50257, 100, 2000, tree=True, half=True, masks="few", padded=47),
        # the largest served batch, with masks that bar a few tokens
        shape("shape 256 chains", 256, 5, 5, 151936, 1024, 8192, bias=300, masks="most"),
    ]


def reserve(name, requests, ctx_lo, ctx_hi, rows_lo, rows_hi, tree=False, prompts=False, short=False):
    return {"name": name, "op": "reserve", "requests": requests, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "rows_lo": rows_lo, "rows_hi": rows_hi, "tree": tree, "prompts": prompts, "short": short}


def stage(name, rows, heads, kv_heads, dim, rotary=None, axes=1, interleaved=False, norm=True, far=8192, pad=0):
    return {"name": name, "op": "stage", "rows": rows, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": dim if rotary is None else rotary, "axes": axes, "interleaved": interleaved, "norm": norm,
            "far": far, "pad": pad}


def shape(name, requests, rows_lo, rows_hi, vocab, hist_lo, hist_hi, tree=False, half=False, bias=0, masks="none",
          padded=0, penalties=True):
    return {"name": name, "op": "shape", "requests": requests, "rows_lo": rows_lo, "rows_hi": rows_hi, "vocab": vocab,
            "hist_lo": hist_lo, "hist_hi": hist_hi, "tree": tree, "half": half, "bias": bias, "masks": masks,
            "padded": padded, "penalties": penalties}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["reserve", "stage", "shape", "shape"])
    if op == "reserve":
        kind = rng.choice(["chains", "trees", "prompts"])
        hi = {"chains": log(1, 128), "trees": log(2, 128), "prompts": log(16, 4000)}[kind]
        requests = min(log(1, 512), max(1, 100000 // hi))
        ctx = 0 if kind == "prompts" and rng.random() < 0.5 else log(1, 32768)
        c = reserve("", requests, min(ctx, log(1, 512)), ctx, rng.randint(1, hi), hi, tree=kind == "trees",
                    prompts=kind == "prompts", short=rng.random() < 0.3)
    elif op == "stage":
        dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.randint(1, 8)
        rows = min(log(1, 20000), 180_000_000 // ((heads + 2 * kv_heads) * dim))
        axes = rng.choice([1, 1, 2, 3])
        c = stage("", rows, heads, kv_heads, dim, rotary=rng.choice([dim, dim // 2, dim // 4, 16]), axes=axes,
                  interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, far=log(64, 1 << 20),
                  pad=rng.choice([0, 0, min(rows - 1, log(1, 64))]))
    else:
        vocab = log(1000, 151936)
        tree = rng.random() < 0.4
        hi = log(2, 100) if tree else log(1, 16)
        requests = min(log(1, 256), max(1, 150_000_000 // (hi * vocab)))
        hist = log(1, 32768)
        c = shape("", requests, rng.randint(1, hi), hi, vocab, min(hist, log(1, 1000)), hist, tree=tree,
                  half=rng.random() < 0.5, bias=rng.choice([0, 0, log(1, 400)]), masks=rng.choice(["none", "few", "most"]),
                  padded=rng.choice([0, 0, rng.randint(1, 127)]), penalties=rng.random() < 0.8)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"reserve": prepare_reserve, "stage": prepare_stage, "shape": prepare_shape}[case["op"]](case, g)
    s["op"] = case["op"]
    if own:
        s["call"] = bind(s)
    return s


def ints(g, lo, hi, *size):
    """Whole numbers lo .. hi, both among them."""
    return torch.randint(lo, hi + 1, size, generator=g, device="cuda", dtype=torch.int32)


def sizes(lo, hi, n, log=False):
    """n whole numbers that fill lo .. hi evenly (over their logarithm)."""
    u = [(i + 0.5) / n for i in range(n)]
    return [min(hi, max(lo, round(lo * (hi / lo) ** x if log and lo else lo + (hi - lo) * x))) for x in u]


def dealt(g, values):
    """The values in an order of the seed's."""
    v = torch.tensor(values, dtype=torch.int32, device="cuda")
    return v[torch.randperm(v.numel(), generator=g, device="cuda")]


def offsets(n):
    cu = torch.zeros(n.numel() + 1, dtype=torch.int32, device="cuda")
    cu[1:] = n.cumsum(0)
    return cu


def topology(g, cu, total, tree):
    """Parents of packed chains, or of trees whose nodes hang below any earlier one."""
    owner = torch.repeat_interleave(torch.arange(cu.numel() - 1, device="cuda"), (cu[1:] - cu[:-1]).long())
    j = torch.arange(total, device="cuda") - cu[owner].long()
    u = torch.rand(total, generator=g, device="cuda", dtype=torch.float64)
    up = (u * j).floor().long().clamp(max=(j - 1).clamp(min=0)) if tree else j - 1
    return owner, j, torch.where(j == 0, -torch.ones_like(j), up).int()


def prepare_reserve(c, g):
    R = c["requests"]
    ctx = dealt(g, sizes(c["ctx_lo"], c["ctx_hi"], R, log=True))
    rows = dealt(g, sizes(c["rows_lo"], c["rows_hi"], R, log=c["prompts"]))
    cu = offsets(rows)
    total = int(cu[-1])
    _, _, parent = topology(g, cu, total, c["tree"])
    have, need = (ctx + PAGE - 1) // PAGE, (ctx + rows + PAGE - 1) // PAGE
    used, new = int(have.sum()), int((need - have).sum())
    free = max(1, int(new * 0.6)) if c["short"] else new + new // 4 + 3
    ids = torch.randperm(used + free, generator=g, device="cuda").int()
    width = -(-(c["ctx_hi"] + c["rows_hi"]) // PAGE) + 4
    t = torch.arange(width, device="cuda")
    first = (have.cumsum(0) - have).long()
    tables = torch.where(t < have[:, None], ids[(first[:, None] + t).clamp(max=max(0, used + free - 1))], -1)
    start = torch.cat([tables.reshape(-1), torch.tensor([free], dtype=torch.int32, device="cuda")])
    live = start.clone()  # tables and free count, put back before each step
    free_list = torch.full((used + free + 1,), -1, dtype=torch.int32, device="cuda")
    free_list[:free] = ids[used:]
    out = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"cu": cu, "parent": None if c["prompts"] else parent, "tokens": torch.zeros_like(parent), "ctx": ctx,
            "max_rows": int(rows.max()), "start": start, "live": live, "tables": live[:-1].view(R, width),
            "count": live[-1:], "list": free_list, "blocks": used + free + 1, "slots": out(total),
            "positions": out(total), "taken": out(R), "shift": ints(g, 0, 50, R)}


def prepare_stage(c, g):
    N, H, K, D = c["rows"], c["heads"], c["kv_heads"], c["dim"]
    qkv = torch.randn(N, (H + 2 * K) * D, generator=g, device="cuda").mul_(1.5).bfloat16()
    blocks = -(-N // PAGE) + 5
    slots = torch.randperm(blocks * PAGE, generator=g, device="cuda")[:N].int()
    if c["pad"]:
        slots[-c["pad"]:] = -1
    positions = ints(g, 0, c["far"], c["axes"], N)
    half = c["rotary"] // 2
    inv_freq = (500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    w = lambda: 1 + 0.2 * torch.randn(D, generator=g, device="cuda")  # noqa: E731
    cache = lambda: torch.randn(blocks, K, PAGE, D, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = qkv.split([H * D, K * D, K * D], 1)
    return {"q": q.unflatten(1, (H, D)), "k": k.unflatten(1, (K, D)), "v": v.unflatten(1, (K, D)), "slots": slots,
            "positions": positions if c["axes"] > 1 else positions[0], "inv_freq": inv_freq,
            "axis": torch.arange(half, device="cuda").int() % c["axes"] if c["axes"] > 1 else None,
            "rotary": c["rotary"], "interleaved": c["interleaved"], "qw": w() if c["norm"] else None,
            "kw": w() if c["norm"] else None, "eps": 1e-6, "k_cache": cache(), "v_cache": cache(),
            "out": torch.zeros(N, H, D, dtype=torch.bfloat16, device="cuda")}


def prepare_shape(c, g):
    R, V = c["requests"], c["vocab"]
    rows = dealt(g, sizes(c["rows_lo"], c["rows_hi"], R))
    cu = offsets(rows)
    N = int(cu[-1])
    _, _, parent = topology(g, cu, N, c["tree"])
    words = lambda *n: (V * torch.rand(*n, generator=g, device="cuda", dtype=torch.float64) ** 4).int().clamp(max=V - 1)  # noqa: E731
    logits = torch.randn(N, V + c["padded"], generator=g, device="cuda").mul_(3)
    length = dealt(g, sizes(c["hist_lo"], c["hist_hi"], R, log=True))
    s = {"cu": cu, "parent": parent, "tokens": words(N), "max_rows": int(rows.max()), "vocab": V,
         "logits": (logits.bfloat16() if c["half"] else logits)[:, :V],
         "history": None, "length": None, "prompt": None, "rho": None, "freq": None, "pres": None,
         "bias_begin": None, "bias_token": None, "bias_value": None, "mask": None, "mask_row": None,
         "out": torch.empty(N, V, device="cuda")}
    if c["penalties"]:
        s["history"], s["length"] = words(R, int(length.max())), length
        s["prompt"] = (length * 0.7).int()
        s["rho"] = 1 + 0.3 * torch.rand(R, generator=g, device="cuda")
        s["freq"] = 0.5 * torch.rand(R, generator=g, device="cuda")
        s["pres"] = torch.rand(R, generator=g, device="cuda")
    if c["bias"]:
        n = ints(g, 0, 2 * c["bias"], R).clamp(max=V)
        s["bias_begin"] = offsets(n)
        stride = V // (2 * c["bias"] + 1) or 1  # every request's tokens differ
        at = torch.cat([torch.arange(int(k), device="cuda") for k in n.tolist()] or [n])
        s["bias_token"] = ((at * stride + ints(g, 0, stride - 1, at.numel())) % V).int()
        s["bias_value"] = 4 * torch.randn(at.numel(), generator=g, device="cuda")
    if c["masks"] != "none":
        n = max(1, N // 2)  # a mask for every second row, some rows sharing one, some without
        W = (V + 31) // 32
        if c["masks"] == "few":
            tok = ints(g, 0, V - 1, n, 48).long()
            bit = torch.ones_like(tok) << (tok % 32)
            m = torch.zeros(n, W, dtype=torch.int64, device="cuda").scatter_reduce_(1, tok // 32, bit, "amax")
        else:
            m = torch.zeros(n, W, dtype=torch.int64, device="cuda")
            for _ in range(4):  # one token in sixteen is barred
                m |= torch.randint(0, 1 << 32, (n, W), generator=g, device="cuda")
        s["mask"] = torch.where(m >= 1 << 31, m - (1 << 32), m).int()
        s["mask_row"] = (torch.arange(N, device="cuda").int() % (n + 1)) - 1
    return s


# ------------------------------------------------- the framework's own calls --

def bind(s):
    from speculative_decoding_verification_padding_gb300 import api
    if s["op"] == "reserve":
        batch = api.Batch(s["cu"], s["parent"], s["tokens"], s["max_rows"])
        page = torch.empty(s["blocks"], 1, PAGE, 64, dtype=torch.bfloat16, device="cuda")
        kv = api.PagedKV(page, page, s["tables"], s["ctx"])
        return api.bind_reserve_kv(kv, batch, api.BlockPool(s["list"], s["count"]), s["slots"], s["positions"],
                                   s["taken"], pos_offset=s["shift"])
    if s["op"] == "stage":
        nothing = torch.zeros(1, dtype=torch.int32, device="cuda")
        kv = api.PagedKV(s["k_cache"], s["v_cache"], nothing.view(1, 1), nothing)
        rotary = api.Rotary(s["inv_freq"], s["rotary"], freq_axis=s["axis"], interleaved=s["interleaved"])
        return api.bind_stage_qkv(kv, s["q"], s["k"], s["v"], s["slots"], s["positions"], rotary, s["out"],
                                  q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"])
    batch = api.Batch(s["cu"], s["parent"], s["tokens"], s["max_rows"])
    rules = api.LogitRules(history=s["history"], history_len=s["length"], prompt_len=s["prompt"], repetition=s["rho"],
                           frequency=s["freq"], presence=s["pres"], bias_begin=s["bias_begin"],
                           bias_token=s["bias_token"], bias_value=s["bias_value"], mask=s["mask"],
                           mask_row=s["mask_row"])
    return api.bind_shape_logits(batch, s["logits"], rules, s["out"])


# -------------------------------------------------------------------- run --

def run(s):
    if s["op"] == "reserve":
        s["live"].copy_(s["start"])
        s["call"]() if own else plain_reserve(s)
        return {"tables": s["tables"], "count": s["count"], "slots": s["slots"], "positions": s["positions"],
                "taken": s["taken"]}
    if s["op"] == "stage":
        s["call"]() if own else plain_stage(s)
        return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    s["call"]() if own else plain_shape(s)
    return {"logits": s["out"]}


def plain_reach(cu, parent, owner, j, m):
    """[requests, m, m]: 1 where the second node is the first or one of its ancestors."""
    R = cu.numel() - 1
    up = torch.eye(m, device="cuda").repeat(R, 1, 1)
    has = parent >= 0
    up[owner, j, parent.long().clamp(min=0)] = torch.where(has, 1.0, up[owner, j, parent.long().clamp(min=0)])
    for _ in range(max(1, (m - 1).bit_length())):
        up = (up @ up).clamp(max=1)
    return up


def plain_owner(cu, n):
    at = torch.arange(n, device="cuda")
    owner = torch.searchsorted(cu, at.int(), right=True) - 1
    return owner, at - cu[owner].long()


def plain_reserve(s):
    cu, ctx, tables = s["cu"].long(), s["ctx"].long(), s["tables"]
    R, N = ctx.numel(), s["slots"].numel()
    rows = cu[1:] - cu[:-1]
    t = torch.arange(tables.shape[1], device="cuda")
    ask = (t >= (ctx // PAGE)[:, None]) & (t < ((ctx + rows + PAGE - 1) // PAGE)[:, None]) & (tables < 0)
    n = ask.sum(1)
    upto = n.cumsum(0)
    free = s["count"].long()
    served = (upto <= free) | (n == 0)
    rank = (upto - n)[:, None] + ask.cumsum(1) - 1
    ids = s["list"][(free - 1 - rank).clamp(min=0)]
    tables.copy_(torch.where(ask & served[:, None], ids, tables))
    s["taken"].copy_(torch.where(served, n, -1))
    s["count"].sub_((n * served).sum().int())
    owner, j = plain_owner(s["cu"], N)
    at = ctx[owner] + j
    slot = tables[owner, at // PAGE].long() * PAGE + at % PAGE
    if s["parent"] is None:
        depth = j
    else:
        depth = plain_reach(s["cu"], s["parent"], owner, j, s["max_rows"])[owner, j].sum(1).long() - 1
    s["slots"].copy_(torch.where(served[owner], slot, -1))
    s["positions"].copy_(torch.where(served[owner], ctx[owner] + s["shift"][owner] + depth, -1))


def plain_stage(s):
    rd, half = s["rotary"], s["rotary"] // 2
    pos = s["positions"]
    pos = pos[:, None].double() if s["axis"] is None else pos.double()[s["axis"].long()].T
    angle = pos * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w
        a, b = (x[..., :rd:2], x[..., 1:rd:2]) if s["interleaved"] else (x[..., :half], x[..., half:rd])
        a, b = a * cos - b * sin, b * cos + a * sin
        both = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([both, x[..., rd:]], -1).bfloat16()

    keep = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"][keep].long()
    s["out"][keep] = turned(s["q"], s["qw"])[keep]
    s["k_cache"][at // PAGE, :, at % PAGE] = turned(s["k"], s["kw"])[keep]
    s["v_cache"][at // PAGE, :, at % PAGE] = s["v"][keep]


def plain_shape(s):
    V, N = s["vocab"], s["out"].shape[0]
    owner, j = plain_owner(s["cu"], N)
    y = s["logits"].float()
    if s["history"] is not None:
        R, L = s["history"].shape
        at = torch.arange(L, device="cuda")
        old, told = (at < s["prompt"][:, None]).float(), (at < s["length"][:, None]).float()
        token = s["history"].long()
        asked = torch.zeros(R, V, device="cuda").scatter_add_(1, token, old)
        count = torch.zeros(R, V, device="cuda").scatter_add_(1, token, told - old)[owner]
        m = s["max_rows"]
        reach = plain_reach(s["cu"], s["parent"], owner, j, m)[owner, j]
        reach[:, 0] = 0  # the root's token is in the history
        nodes = (s["cu"][owner].long()[:, None] + torch.arange(m, device="cuda")).clamp(max=N - 1)
        count.scatter_add_(1, s["tokens"].long()[nodes], reach)
        rho = s["rho"][owner, None]
        seen = (count > 0) | (asked > 0)[owner]
        y = torch.where(seen, torch.where(y > 0, y / rho, y * rho), y)
        y = y - (s["freq"][owner, None] * count + s["pres"][owner, None] * (count > 0))
    if s["bias_begin"] is not None:
        n = (s["bias_begin"][1:] - s["bias_begin"][:-1]).long()
        whose = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n)
        bias = torch.zeros(n.numel(), V, device="cuda")
        bias[whose, s["bias_token"].long()] = s["bias_value"]
        y = y + bias[owner]
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        row = s["mask_row"].long()
        bits = (s["mask"][row.clamp(min=0)][:, v // 32] >> (v % 32).int()) & 1
        y = torch.where((bits == 0) & (row >= 0)[:, None], -math.inf, y)
    s["out"].copy_(y)


# ------------------------------------------------------------------- work --

def work(c):
    if c["op"] == "reserve":
        R, N = c["requests"], sum(sizes(c["rows_lo"], c["rows_hi"], c["requests"], log=c["prompts"]))
        new = N / PAGE  # blocks, as many entries again end inside a page
        # offsets, lengths and shifts; parents; table entries and ids; slots and positions; the counts
        return {"bytes": 12 * R + (0 if c["prompts"] else 4 * N) + 4 * (new + R) + 8 * new + 8 * N + 4 * R + 12,
                "flops": 10 * N}
    if c["op"] == "stage":
        N = c["rows"] - c["pad"]
        width = (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
        turned = (c["heads"] + c["kv_heads"]) * (6 * c["rotary"] / 2 + 4 * c["dim"])
        return {"bytes": 4 * N * width + 4 * c["rows"] + 4 * N * c["axes"], "flops": N * turned}
    R, V = c["requests"], c["vocab"]
    N = sum(sizes(c["rows_lo"], c["rows_hi"], R))
    n = max(1, N // 2)
    masked = 0.0 if c["masks"] == "none" else N * n / (n + 1)
    let = {"none": 1.0, "few": min(1.0, 48 / V), "most": 1.0}[c["masks"]]  # barred logits need not be read
    read = (2 if c["half"] else 4) * V * (N - masked + masked * let)
    hist = sum(sizes(c["hist_lo"], c["hist_hi"], R, log=True)) if c["penalties"] else 0
    bits = 0 if c["masks"] == "none" else n * V / 8
    return {"bytes": read + 4 * N * V + bits + 4 * hist + 8 * R * c["bias"] + 8 * N, "flops": 6 * N * V}


# ------------------------------------------------------------------ exact --

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "reserve":
        return exact_reserve(s)
    return exact_stage(s) if c["op"] == "stage" else {"logits": exact_shape(s)}


def exact_reserve(s):
    """One request after the other, as a scheduler would serve them."""
    tables, free = s["start"][:-1].view_as(s["tables"]).tolist(), int(s["start"][-1])
    pool, cu, ctx, shift = (s[k].tolist() for k in ("list", "cu", "ctx", "shift"))
    parent = None if s["parent"] is None else s["parent"].tolist()
    slots, positions, taken, asked, left = [], [], [], 0, free
    for i, table in enumerate(tables):
        n = cu[i + 1] - cu[i]
        new = [t for t in range(ctx[i] // PAGE, (ctx[i] + n - 1) // PAGE + 1) if table[t] < 0]
        asked += len(new)
        if new and asked > free:
            slots += [-1] * n
            positions += [-1] * n
            taken.append(-1)
            continue
        for t in new:
            left -= 1
            table[t] = pool[left]
        taken.append(len(new))
        depth = []
        for j in range(n):
            depth.append(j if parent is None else depth[parent[cu[i] + j]] + 1 if j else 0)
            slots.append(table[(ctx[i] + j) // PAGE] * PAGE + (ctx[i] + j) % PAGE)
            positions.append(ctx[i] + shift[i] + depth[j])
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"tables": whole(tables), "count": whole([left]), "slots": whole(slots), "positions": whole(positions),
            "taken": whole(taken)}


def exact_stage(s):
    rd = s["rotary"]
    pos = s["positions"].double().reshape(-1, s["positions"].shape[-1])
    half = rd // 2
    q, k_cache, v_cache = s["out"].double(), s["k_cache"].double(), s["v_cache"].double()
    live = s["slots"] >= 0
    first = torch.arange(half, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else half)

    def rotated(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
        y = x.clone()
        for f in range(half):
            axis = 0 if s["axis"] is None else int(s["axis"][f])
            turn = torch.polar(torch.ones_like(pos[axis]), pos[axis] * float(s["inv_freq"][f]))
            z = torch.complex(x[..., first[f]], x[..., second[f]]) * turn[:, None]
            y[..., first[f]], y[..., second[f]] = z.real, z.imag
        return y

    q[live] = rotated(s["q"], s["qw"])[live]
    slot = s["slots"][live].long()
    k_cache[slot // PAGE, :, slot % PAGE] = rotated(s["k"], s["kw"])[live]
    v_cache[slot // PAGE, :, slot % PAGE] = s["v"].double()[live]
    return {"q": q, "k_cache": k_cache, "v_cache": v_cache}


def exact_shape(s):
    V = s["vocab"]
    out = s["logits"].double()
    cu, parent = s["cu"].tolist(), s["parent"].tolist()
    mask_row = None if s["mask"] is None else s["mask_row"].tolist()
    for i in range(len(cu) - 1):
        told = asked = None
        if s["history"] is not None:
            n, p = int(s["length"][i]), int(s["prompt"][i])
            told = torch.bincount(s["history"][i, p:n], minlength=V)
            asked = torch.bincount(s["history"][i, :p], minlength=V) > 0
            rho, f, a = (float(s[x][i]) for x in ("rho", "freq", "pres"))
        for r in range(cu[i], cu[i + 1]):
            x = out[r]
            if told is not None:
                path, node = [], r - cu[i]
                while node > 0:
                    path.append(cu[i] + node)
                    node = parent[cu[i] + node]
                n = told
                if path:
                    n = told + torch.bincount(s["tokens"][torch.tensor(path, device="cuda")], minlength=V)
                seen = asked | (n > 0)
                x[seen] = torch.maximum(x[seen], x[seen] * 0) / rho + torch.minimum(x[seen], x[seen] * 0) * rho
                x -= f * n.double() + a * (n > 0)
            if s["bias_begin"] is not None:
                b0, b1 = int(s["bias_begin"][i]), int(s["bias_begin"][i + 1])
                x[s["bias_token"][b0:b1].long()] += s["bias_value"][b0:b1].double()
            if mask_row is not None and mask_row[r] >= 0:
                word = s["mask"][mask_row[r]].long() & 0xFFFFFFFF
                let = ((word[:, None] >> torch.arange(32, device="cuda")) & 1).flatten()[:V]
                x[let == 0] = -math.inf
    return out
