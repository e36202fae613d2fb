"""Attention of draft rows that reads less of a long cache, as a user's program
calls it, and its plain forms in elementary torch operations.

  bounds  sv_bound_pages: least and greatest key of each complete cache page
  score   sv_score_pages: for each draft row and KV head, an upper bound of the
          products of its queries with the keys of each page
  select  sv_select_pages: the pages a row attends, by those scores
  sparse  sv_page_attend: attention of each row over its own selected pages
  prefix  sv_prefix_attend: attention of a batch whose requests share a prefix,
          the prefix's pages read once for all of them
"""

import math

import torch

own = False

PAGE = 16  # tokens of a cache page


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the pages that a served batch filled in its last step: a few here and there, launch and latency
        bounds("bounds after a step", 64, 4096, 32768, 8, 128, last=9),
        # prompts of ragged lengths that have just been admitted, every page of them
        bounds("bounds of prompts", 24, 500, 40000, 8, 128),
        # six draft rows of one long conversation
        score("score one chain", 1, 20001, 20001, 6, 6, 32, 8, 128),
        # a served batch of ragged chains over contexts of all lengths
        score("score 48 chains", 48, 2000, 60000, 2, 9, 40, 8, 128),
        # the same conversation's choice of pages
        select("select one chain", 1, 65537, 65537, 6, 6, 8, 128),
        # a served batch's, a few short requests among them that keep every page
        select("select 64 chains", 64, 1000, 100000, 2, 9, 8, 96),
        # one request decoded token by token, without drafts
        sparse("sparse one token", 1, 60001, 60001, 1, 1, 32, 8, 128, 64),
        # a served batch of ragged chains
        sparse("sparse 48 chains", 48, 4000, 60000, 2, 9, 40, 8, 128, 128),
        # draft trees of a model with small heads, an odd group of heads
        sparse("sparse 12 trees", 12, 3000, 30000, 20, 65, 14, 2, 64, 40, tree=True),
        # a few sessions behind one system prompt
        prefix("prefix 4 chains", 1, 4, 2048, 2048, 10, 300, 5, 5, 32, 8, 128),
        # a batch of agents behind one long document, every request with a short history of its own
        prefix("prefix 64 chains", 1, 64, 24576, 24576, 100, 2000, 5, 9, 64, 8, 128),
        # draft trees behind three prompts, small heads
        prefix("prefix 3 groups of trees", 3, 30, 512, 8000, 1, 500, 17, 65, 14, 2, 64, tree=True),
    ]


def common(name, op, requests, ctx_lo, ctx_hi, rows_lo, rows_hi, heads, kv_heads, dim, tree=False):
    return {"name": name, "op": op, "requests": requests, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "rows_lo": rows_lo,
            "rows_hi": rows_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "tree": tree}


def bounds(name, requests, ctx_lo, ctx_hi, kv_heads, dim, last=0):
    """last: at most so many tokens since the pages were bounded before (0: never)."""
    return {**common(name, "bounds", requests, ctx_lo, ctx_hi, 1, 1, kv_heads, kv_heads, dim), "last": last}


def score(name, requests, ctx_lo, ctx_hi, rows_lo, rows_hi, heads, kv_heads, dim, tree=False):
    return common(name, "score", requests, ctx_lo, ctx_hi, rows_lo, rows_hi, heads, kv_heads, dim, tree)


def select(name, requests, ctx_lo, ctx_hi, rows_lo, rows_hi, kv_heads, keep):
    return {**common(name, "select", requests, ctx_lo, ctx_hi, rows_lo, rows_hi, kv_heads, kv_heads, 64), "keep": keep}


def sparse(name, requests, ctx_lo, ctx_hi, rows_lo, rows_hi, heads, kv_heads, dim, keep, tree=False):
    return {**common(name, "sparse", requests, ctx_lo, ctx_hi, rows_lo, rows_hi, heads, kv_heads, dim, tree),
            "keep": keep}


def prefix(name, groups, requests, prefix_lo, prefix_hi, own_lo, own_hi, rows_lo, rows_hi, heads, kv_heads, dim,
           tree=False):
    return {**common(name, "prefix", requests, own_lo, own_hi, rows_lo, rows_hi, heads, kv_heads, dim, tree),
            "groups": groups, "prefix_lo": prefix_lo, "prefix_hi": prefix_hi}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["bounds", "score", "select", "sparse", "sparse", "prefix", "prefix"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16])
    tree = rng.random() < 0.35
    rows_hi = log(2, 100) if tree else log(1, 12)
    rows_lo = rng.randint(1, rows_hi)
    if op == "prefix":
        groups = log(1, 6)
        top = log(16, 24576)
        requests = max(1, min(log(1, 64), 3500 * 24576 // (top * rows_hi * (heads // kv_heads))))
        groups = min(groups, requests)
        c = prefix("", groups, requests, log(1, top), top, 1, log(1, 4000), rows_lo, rows_hi, heads, kv_heads, dim,
                   tree)
    else:
        hi = log(40, 60000)
        cache = kv_heads * dim * hi  # elements of a request's keys
        requests = max(1, min(log(1, 64), 400_000_000 // cache))
        lo = log(1 if op == "sparse" else PAGE, hi)
        if op == "bounds":
            c = bounds("", requests, lo, hi, kv_heads, dim, last=rng.choice([0, 0, log(1, 300)]))
        elif op == "score":
            requests = max(1, min(requests, 40_000_000 // (rows_hi * heads * hi // PAGE)))
            c = score("", requests, lo, hi, rows_lo, rows_hi, heads, kv_heads, dim, tree)
        elif op == "select":
            requests = max(1, min(requests, 8_000_000 // (rows_hi * kv_heads * (hi // PAGE + 1))))
            c = select("", requests, lo, hi, rows_lo, rows_hi, kv_heads, log(4, 512))
        else:
            keep = log(4, 300)
            requests = max(1, min(requests, 1_500_000 // (rows_hi * heads * keep)))
            c = sparse("", requests, lo, hi, rows_lo, rows_hi, heads, kv_heads, dim, keep, tree)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

def sizes(lo, hi, n, log=False):
    """n whole numbers that fill lo .. hi evenly (over their logarithm)."""
    u = [(i + 0.5) / n for i in range(n)]
    return [min(hi, max(lo, round(lo * (hi / lo) ** x if log else lo + (hi - lo) * x))) for x in u]


def dealt(g, values):
    """The values in an order of the seed's, as a list."""
    return [values[k] for k in torch.randperm(len(values), generator=g, device="cuda").tolist()]


def whole(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def offsets(n):
    cu = [0]
    for k in n:
        cu.append(cu[-1] + k)
    return cu


def parents(g, rows, tree):
    """Chains, or trees whose nodes hang below any earlier one."""
    u = torch.rand(sum(rows), generator=g, device="cuda", dtype=torch.float64).tolist()
    out = []
    for n in rows:
        out += [-1 if j == 0 else int(u[len(out)] * j) if tree else j - 1 for j in range(n)]
    return out


def keys(g, blocks, c):
    """Cached keys: every channel of a head has a mean of its own."""
    mean = torch.randn(1, c["kv_heads"], 1, c["dim"], generator=g, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(blocks, c["kv_heads"], PAGE, c["dim"], generator=g, device="cuda", dtype=torch.bfloat16)
    return k.add_(mean)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    c = case
    R, op, H, K, D = c["requests"], c["op"], c["heads"], c["kv_heads"], c["dim"]
    ctx = dealt(g, sizes(c["ctx_lo"], c["ctx_hi"], R, log=True))
    rows = dealt(g, sizes(c["rows_lo"], c["rows_hi"], R))
    cu, s = offsets(rows), {"op": op}
    if op == "prefix":
        s["groups"] = offsets(sizes(R // c["groups"], -(-R // c["groups"]), c["groups"]))
        s["groups"][-1] = R
        s["prefix"] = [-(-n // PAGE) * PAGE for n in sizes(c["prefix_lo"], c["prefix_hi"], c["groups"], log=True)]
        for p, a, b in zip(s["prefix"], s["groups"], s["groups"][1:]):
            ctx[a:b] = [p + n for n in ctx[a:b]]
        s["cu_groups"], s["prefix_len"] = whole(s["groups"]), whole(s["prefix"])
    have = [-(-(n + m) // PAGE) for n, m in zip(ctx, rows)]
    ids = torch.randperm(sum(have) + 5, generator=g, device="cuda").int()
    tables = torch.full((R, max(have) + 2), -1, dtype=torch.int32, device="cuda")
    for i, first in enumerate(offsets(have)[:-1]):
        tables[i, :have[i]] = ids[first:first + have[i]]
    if op == "prefix":
        for p, a, b in zip(s["prefix"], s["groups"], s["groups"][1:]):
            tables[a:b, :p // PAGE] = tables[a, :p // PAGE].clone()
    parent = parents(g, rows, c["tree"])
    N, blocks = cu[-1], ids.numel()
    s.update(ctx=ctx, rows=rows, cu=cu, parent=parent, tables=tables, lens=whole(ctx), cu_rows=whole(cu),
             parents=whole(parent), max_rows=max(rows))
    if op in ("bounds", "sparse", "prefix"):
        s["k_cache"] = keys(g, blocks, c)
    elif op == "score":  # the pages themselves are not read
        s["k_cache"] = torch.empty(blocks, K, PAGE, D, dtype=torch.bfloat16, device="cuda")
    else:
        s["k_cache"] = torch.empty(blocks, 1, PAGE, 64, dtype=torch.bfloat16, device="cuda").expand(-1, K, -1, -1)
    s["v_cache"] = s["k_cache"]
    if op in ("sparse", "prefix"):
        s["v_cache"] = torch.randn(blocks, K, PAGE, D, generator=g, device="cuda", dtype=torch.bfloat16)
    if op in ("score", "sparse", "prefix"):
        s["q"] = torch.randn(N, H, D, generator=g, device="cuda").mul_(1.5).bfloat16()
        s["scale"] = D ** -0.5
    if op == "bounds":
        back = torch.randint(1, max(1, c["last"]) + 1, (R,), generator=g, device="cuda").tolist()
        s["from"] = [max(0, n - b) if c["last"] else 0 for n, b in zip(ctx, back)]
        s["from_len"] = whole(s["from"])
        s["bounds"] = torch.zeros(blocks, K, 2, D, dtype=torch.bfloat16, device="cuda")
    elif op == "score":
        near = keys(g, blocks, {"kv_heads": K, "dim": D})[:, :, :2]  # a page's least and greatest key
        s["bounds"] = torch.stack([near[:, :, 0] - 1.5, near[:, :, 0] + near[:, :, 1].abs() + 1], 2)
        s["out"] = torch.zeros(N, K, max(ctx) // PAGE + 3, device="cuda")
    elif op == "select":
        s["first"], s["last"], s["keep"] = min(1, c["keep"] // 2), min(4, c["keep"] // 2), c["keep"]
        s["scores"] = torch.randn(N, K, max(ctx) // PAGE + 3, generator=g, device="cuda").mul_(9).round_(decimals=1)
        s["out"] = torch.zeros(N, K, c["keep"], dtype=torch.int32, device="cuda")
    elif op == "sparse":
        s["pages"] = chosen(g, c, s)
        s["out"] = torch.zeros_like(s["q"])
    else:
        s["out"] = torch.zeros_like(s["q"])
    if own:
        s["call"] = bind(s)
    return s


def chosen(g, c, s):
    """Page lists of rows whose choices overlap: three quarters of a list are the
    request's, the rest the row's own, half of them its neighbour's too."""
    K, keep = c["kv_heads"], c["keep"]
    out = torch.full((s["cu"][-1], K, keep), -1, dtype=torch.int32, device="cuda")
    for i, (n, m) in enumerate(zip(s["ctx"], s["rows"])):
        n //= PAGE
        if n <= keep:
            out[s["cu"][i]:s["cu"][i + 1], :, :n] = torch.arange(n, device="cuda").int()
            continue
        deal = torch.rand(K, n, generator=g, device="cuda").argsort(1)
        base, each = keep - keep // 4, keep // 4
        at = torch.arange(keep, device="cuda").repeat(m, 1)
        at[:, base:] += (torch.arange(m, device="cuda") * ((each + 1) // 2))[:, None]
        at[:, base:] = base + (at[:, base:] - base) % (n - base)
        out[s["cu"][i]:s["cu"][i + 1]] = deal[:, at].sort(-1).values.permute(1, 0, 2).int()
    return out


# ------------------------------------------------- the framework's own calls --

def bind(s):
    from speculative_decoding_verification_padding_gb300 import api
    k = s["k_cache"].contiguous()
    kv = api.PagedKV(k, k if s["v_cache"] is s["k_cache"] else s["v_cache"], s["tables"], s["lens"])
    batch = api.Batch(s["cu_rows"], s["parents"], torch.zeros_like(s["parents"]), s["max_rows"])
    if s["op"] == "bounds":
        return api.bind_bound_pages(kv, s["bounds"], from_len=s["from_len"])
    if s["op"] == "score":
        return api.bind_score_pages(kv, batch, s["q"], s["bounds"], s["out"])
    if s["op"] == "select":
        return api.bind_select_pages(kv, batch, s["scores"], s["out"], n_first=s["first"], n_last=s["last"])
    heads = s["q"].shape[1]
    if s["op"] == "sparse":
        ws = api.workspace(api.sv_page_attend_workspace(batch, kv, heads, s["pages"].shape[2]))
        return api.bind_page_attend(kv, batch, s["q"], s["scale"], s["pages"], s["out"], ws)
    shared = api.SharedPrefix(s["cu_groups"], s["prefix_len"])
    ws = api.workspace(api.sv_prefix_attend_workspace(batch, kv, shared, heads))
    return api.bind_prefix_attend(kv, batch, shared, s["q"], s["scale"], s["out"], ws)


# -------------------------------------------------------------------- run --

def run(s):
    if own:
        s["call"]()
    else:
        PLAIN[s["op"]](s)
    return {"bounds": s["bounds"]} if s["op"] == "bounds" else {"out": s["out"]}


def plain_bounds(s):
    for i, (a, n) in enumerate(zip(s["from"], s["ctx"])):
        ids = s["tables"][i, a // PAGE:n // PAGE].long()
        if ids.numel():
            page = s["k_cache"][ids].float()
            s["bounds"][ids] = torch.stack([page.amin(2), page.amax(2)], 2).bfloat16()


def plain_score(s):
    N, H, D = s["q"].shape
    K = s["bounds"].shape[1]
    q = s["q"].float().view(N, K, H // K, D)
    up, down = q.clamp(min=0), q.clamp(max=0)
    for i, n in enumerate(s["ctx"]):
        a, b, n = s["cu"][i], s["cu"][i + 1], n // PAGE
        lo, hi = s["bounds"][s["tables"][i, :n].long()].float().permute(2, 1, 3, 0)  # [heads][dim][pages]
        s["out"][a:b, :, :n] = (up[a:b] @ hi + down[a:b] @ lo).amax(2)


def plain_select(s):
    keep = s["keep"]
    for i, n in enumerate(s["ctx"]):
        a, b, n = s["cu"][i], s["cu"][i + 1], n // PAGE
        x = s["scores"][a:b, :, :n].clone()
        x[..., :s["first"]] = math.inf
        x[..., max(0, n - s["last"]):] = math.inf
        best = x.sort(dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
        s["out"][a:b] = -1
        s["out"][a:b, :, :best.shape[-1]] = best.int()


def plain_reach(s, i):
    """[rows][rows]: whether the second node is the first or one of its ancestors."""
    n = s["rows"][i]
    up = torch.eye(n, device="cuda")
    own_parent = s["parents"][s["cu"][i]:s["cu"][i + 1]].long()
    up[torch.arange(1, n, device="cuda"), own_parent[1:]] = 1
    for _ in range(max(1, (n - 1).bit_length())):
        up = (up @ up).clamp(max=1)
    return up > 0


def plain_softmax(x):
    e = (x - x.amax(-1, keepdim=True)).exp()
    return e / e.sum(-1, keepdim=True)


def plain_sparse(s):
    N, H, D = s["q"].shape
    K = s["k_cache"].shape[1]
    q = s["q"].float().view(N, K, H // K, D) * s["scale"]
    head = torch.arange(K, device="cuda")[:, None]
    for i, ctx in enumerate(s["ctx"]):
        a, b, n = s["cu"][i], s["cu"][i + 1], ctx // PAGE
        table = s["tables"][i].long()
        last = torch.arange(n, -(-(ctx + b - a) // PAGE), device="cuda")
        pages = s["pages"][a:b].long()
        pages = torch.cat([pages, last.expand(b - a, K, -1)], 2)
        slot = pages[..., None] * PAGE + torch.arange(PAGE, device="cuda")
        node = (slot - ctx).clamp(0, b - a - 1)
        seen = torch.where(slot < ctx, (pages >= 0)[..., None], False)
        mine = plain_reach(s, i)[torch.arange(b - a, device="cuda")[:, None, None, None], node]
        seen = (seen | (mine & (slot >= ctx) & (slot < ctx + b - a))).flatten(2)
        ids = table[pages.clamp(min=0)]
        k = s["k_cache"][ids, head].float().flatten(2, 3)  # [rows][heads][keys][dim]
        v = s["v_cache"][ids, head].float().flatten(2, 3)
        x = (q[a:b] @ k.transpose(-1, -2)).masked_fill(~seen[:, :, None], -math.inf)
        s["out"][a:b] = (plain_softmax(x) @ v).flatten(1, 2).bfloat16()


def plain_prefix(s):
    N, H, D = s["q"].shape
    K = s["k_cache"].shape[1]
    q = s["q"].float().view(N, K, H // K, D) * s["scale"]
    for p, r0, r1 in zip(s["prefix"], s["groups"], s["groups"][1:]):
        a, b = s["cu"][r0], s["cu"][r1]
        ids = s["tables"][r0, :p // PAGE].long()
        top = torch.empty(b - a, K, H // K, 1, device="cuda")
        total, acc = torch.empty_like(top), torch.empty(b - a, K, H // K, D, device="cuda")
        for h in range(K):  # the prefix, once for the whole group
            x = q[a:b, h].flatten(0, 1) @ s["k_cache"][ids, h].float().flatten(0, 1).T
            m = x.amax(-1, keepdim=True)
            e = x.sub_(m).exp_()
            top[:, h], total[:, h] = m.view(b - a, -1, 1), e.sum(-1).view(b - a, -1, 1)
            acc[:, h] = (e @ s["v_cache"][ids, h].float().flatten(0, 1)).view(b - a, -1, D)
        for i in range(r0, r1):  # what is the request's own
            c, d, ctx = s["cu"][i], s["cu"][i + 1], s["ctx"][i]
            ids_own = s["tables"][i, p // PAGE:-(-(ctx + d - c) // PAGE)].long()
            n = ctx + d - c - p
            k = s["k_cache"][ids_own].float().transpose(1, 2).flatten(0, 1)[:n].permute(1, 2, 0)
            v = s["v_cache"][ids_own].float().transpose(1, 2).flatten(0, 1)[:n].transpose(0, 1)
            x = q[c:d] @ k
            x[..., ctx - p:].masked_fill_(~plain_reach(s, i)[:, None, None], -math.inf)
            m = torch.maximum(x.amax(-1, keepdim=True), top[c - a:d - a])
            e, back = (x - m).exp(), (top[c - a:d - a] - m).exp()
            o = (e @ v + acc[c - a:d - a] * back) / (e.sum(-1, keepdim=True) + total[c - a:d - a] * back)
            s["out"][c:d] = o.flatten(1, 2).bfloat16()


PLAIN = {"bounds": plain_bounds, "score": plain_score, "select": plain_select, "sparse": plain_sparse,
         "prefix": plain_prefix}


# ------------------------------------------------------------------- work --

def work(c):
    R, K, D, H = c["requests"], c["kv_heads"], c["dim"], c["heads"]
    ctx = sizes(c["ctx_lo"], c["ctx_hi"], R, log=True)
    mean_rows = sum(sizes(c["rows_lo"], c["rows_hi"], R)) / R  # rows and lengths are dealt apart
    pages = sum(n // PAGE for n in ctx)
    N = mean_rows * R
    if c["op"] == "bounds":
        if c["last"]:
            pages = R * (c["last"] + 1) / 2 / PAGE
        return {"bytes": pages * (K * D * (2 * PAGE + 4) + 4) + 8 * R, "flops": 2 * pages * K * PAGE * D}
    if c["op"] == "score":
        return {"bytes": pages * (4 * K * D + 4) + 2 * N * H * D + 4 * mean_rows * K * pages,
                "flops": 4 * mean_rows * H * pages * D}
    if c["op"] == "select":
        return {"bytes": 4 * mean_rows * K * pages + 4 * N * K * c["keep"], "flops": mean_rows * K * pages}
    if c["op"] == "sparse":
        keep = c["keep"]
        read = seen = 0
        for n in ctx:
            n //= PAGE
            each = keep // 4
            union = min(n, keep + (mean_rows - 1) * ((each + 1) // 2)) if n > keep else n
            read += union * PAGE + PAGE / 2 + mean_rows
            seen += mean_rows * (min(n, keep) * PAGE + PAGE / 2 + mean_rows / 2)
        return {"bytes": 4 * read * K * D + 4 * N * H * D + 4 * N * K * keep, "flops": 4 * seen * H * D}
    p = sizes(c["prefix_lo"], c["prefix_hi"], c["groups"], log=True)
    read = sum(p) + sum(ctx) + N
    seen = N * (sum(p) / len(p) + sum(ctx) / R + mean_rows / 2)
    return {"bytes": 4 * read * K * D + 4 * N * H * D, "flops": 4 * seen * H * D}


# ------------------------------------------------------------------ exact --

def exact(c, seed):
    s = prepare(c, seed)
    return {"bounds": exact_bounds(s)} if s["op"] == "bounds" else {"out": EXACT[s["op"]](s)}


def exact_bounds(s):
    out = s["bounds"].double()
    for i, table in enumerate(s["tables"].tolist()):
        for block in table[s["from"][i] // PAGE:s["ctx"][i] // PAGE]:
            page = s["k_cache"][block].double()
            low, high = page[:, 0], page[:, 0]
            for k in range(1, PAGE):
                low, high = torch.minimum(low, page[:, k]), torch.maximum(high, page[:, k])
            out[block, :, 0], out[block, :, 1] = low, high
    return out


def exact_score(s):
    out = s["out"].double()
    K, group = s["bounds"].shape[1], s["q"].shape[1] // s["bounds"].shape[1]
    for i, ctx in enumerate(s["ctx"]):
        b = s["bounds"][s["tables"][i, :ctx // PAGE].long()].double()
        for r in range(s["cu"][i], s["cu"][i + 1]):
            best = None
            for h in range(group):
                q = s["q"][r, h::group].double()
                x = torch.maximum(q * b[:, :, 0], q * b[:, :, 1]).sum(-1)
                best = x if best is None else torch.maximum(best, x)
            out[r, :, :ctx // PAGE] = best.T
    return out


def exact_select(s):
    out = torch.full_like(s["out"], -1).cpu()
    scores, keep = s["scores"].cpu().numpy(), s["keep"]
    for i, ctx in enumerate(s["ctx"]):
        n = ctx // PAGE
        for r in range(s["cu"][i], s["cu"][i + 1]):
            for h in range(out.shape[1]):
                x = scores[r, h, :n]
                always = [t for t in range(n) if t < s["first"] or t >= n - s["last"]]
                rest = [t for t in (-x).argsort(kind="stable").tolist() if s["first"] <= t < n - s["last"]]
                pages = sorted(always + rest[:keep - len(always)]) if n > keep else list(range(n))
                out[r, h, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
    return out.cuda()


def exact_rows(s, keys_of):
    """Each row by itself: keys_of(request, row, KV head) are the cached slots it sees."""
    out = s["out"].double()
    N, H, D = s["q"].shape
    K = s["k_cache"].shape[1]
    group = H // K
    for i, ctx in enumerate(s["ctx"]):
        for r in range(s["cu"][i], s["cu"][i + 1]):
            path, j = [], r - s["cu"][i]
            while j >= 0:
                path.append(ctx + j)
                j = s["parent"][s["cu"][i] + j]
            path = torch.tensor(path, device="cuda")
            for h in range(K):
                slot = torch.cat([keys_of(i, r, h), path])
                block = s["tables"][i, slot // PAGE].long()
                k, v = s["k_cache"][block, h, slot % PAGE].double(), s["v_cache"][block, h, slot % PAGE].double()
                x = s["q"][r, h * group:(h + 1) * group].double() @ k.T * s["scale"]
                out[r, h * group:(h + 1) * group] = torch.softmax(x, -1) @ v
    return out


def exact_sparse(s):
    def cached(i, r, h):
        pages = s["pages"][r, h].long()
        pages = pages[pages >= 0]
        whole_pages = (pages[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
        return torch.cat([whole_pages, torch.arange(s["ctx"][i] // PAGE * PAGE, s["ctx"][i], device="cuda")])
    return exact_rows(s, cached)


def exact_prefix(s):
    return exact_rows(s, lambda i, r, h: torch.arange(s["ctx"][i], device="cuda"))


EXACT = {"score": exact_score, "select": exact_select, "sparse": exact_sparse, "prefix": exact_prefix}
