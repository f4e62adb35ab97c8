"""Workloads of the paged cache held in 8 bits, and of its pages:

  append8   a block's new tokens: queries and keys rotated, keys and values written to the pages as 8-bit codes
  attend8   attention of the block's rows over the cached codes, where groups of sequences may share a long prefix
  commit8   after a drafted tree was verified, the accepted path's codes move to consecutive slots, in every layer
  fork      a new batch whose sequences continue old ones (beams, branches, finished requests): full pages are shared, partly filled
            ones copied, pages that nobody holds any more are free, pages for the next block are taken
  compact   the pages in use move to the front of the pool

A code is an e4m3 number; a page has one scale for each key head, a power of two held as its biased exponent (e8m0), for keys and
values apart.  The scale is the smallest that keeps the page's values within 448; a page that an append writes on with larger values
has its earlier codes rounded to the new scale.  `run` computes the plain form where `own` is false and calls the library where it is
true.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
GOLDEN = 0.6180339887498949
E4M3_MAX = 448.0
LOWEST = -120  # least exponent of a scale that an append writes


def listed():
    return [
        # one sequence, four drafted tokens, a short context: what an interactive request costs a layer
        attend_case("attend8 one chain", batch=1, depth=4, longest=1000, shortest=1000),
        # a large serving batch that verifies five drafted tokens for each sequence
        attend_case("attend8 large batch", batch=512, depth=5, longest=2048, shortest=1024),
        # a batch behind one long system prompt: the prompt's part has enough rows to be bound by arithmetic
        attend_case("attend8 shared prompt", batch=64, depth=5, longest=700, shortest=20, groups=1, prefix=32768),
        # a tree of eight branches of seven tokens a sequence, small heads, an odd page size
        attend_case("attend8 trees", batch=16, branches=8, depth=7, longest=4001, shortest=500, heads=24, kv_heads=4, dim=64, page=24),
        # one interactive request's new rows
        append_case("append8 one chain", batch=1, depth=4, longest=1000, shortest=1000),
        # the large batch's new rows; half of each head is rotated, neighbours paired
        append_case("append8 large batch", batch=512, depth=5, longest=200, shortest=30, rotary=64, style="interleaved"),
        # every layer's accepted path after a step over branch-complete trees
        commit_case("commit8 all layers", layers=32, batch=64, branches=8, depth=7, longest=200, shortest=20),
        # one request, one layer, a small tree
        commit_case("commit8 one request", layers=4, batch=1, branches=3, depth=4, longest=500, shortest=500, dim=64),
        # 64 requests of four beams that continue each other, some of them finished
        fork_case("fork beams", dtype="bf16", layers=8, batch=256, children=256, width=4, longest=400, shortest=100),
        # one request that eight drafted branches start from
        fork_case("fork branches", dtype="e4m3", layers=4, batch=1, children=8, width=1, longest=1000, shortest=1000),
        # a pool that is half empty after requests have finished
        compact_case("compact pool", dtype="e4m3", layers=8, batch=128, longest=500, shortest=100, spare=100),
        # a small model's cache
        compact_case("compact small pool", dtype="bf16", layers=2, batch=4, longest=300, shortest=50, kv_heads=2, dim=64, spare=40),
    ]


def attend_case(name=None, dtype="bf16", batch=1, branches=0, depth=4, longest=1000, shortest=1, groups=0, prefix=0, heads=32,
                kv_heads=8, dim=128, page=16):
    c = dict(op="attend8", dtype=dtype, batch=batch, branches=branches, depth=depth, longest=longest, shortest=shortest, groups=groups,
             prefix=prefix, heads=heads, kv_heads=kv_heads, dim=dim, page=page)
    return dict(c, name=name) if name else c


def append_case(name=None, dtype="bf16", batch=1, branches=0, depth=4, longest=1000, shortest=1, heads=32, kv_heads=8, dim=128, page=16,
                rotary=128, style="half"):
    c = dict(op="append8", dtype=dtype, batch=batch, branches=branches, depth=depth, longest=longest, shortest=shortest, groups=0, prefix=0,
             heads=heads, kv_heads=kv_heads, dim=dim, page=page, rotary=rotary, style=style)
    return dict(c, name=name) if name else c


def commit_case(name=None, layers=1, batch=1, branches=1, depth=4, longest=100, shortest=1, kv_heads=8, dim=128, page=16):
    c = dict(op="commit8", dtype="e4m3", layers=layers, batch=batch, branches=branches, depth=depth, longest=longest, shortest=shortest,
             groups=0, prefix=0, kv_heads=kv_heads, dim=dim, page=page)
    return dict(c, name=name) if name else c


def fork_case(name=None, dtype="bf16", layers=1, batch=1, children=1, width=1, longest=100, shortest=1, reserve=6, kv_heads=8, dim=128,
              page=16, spare=0):
    c = dict(op="fork", dtype=dtype, layers=layers, batch=batch, children=children, width=width, longest=longest, shortest=shortest,
             reserve=reserve, kv_heads=kv_heads, dim=dim, page=page, spare=spare)
    return dict(c, name=name) if name else c


def compact_case(name=None, dtype="bf16", layers=1, batch=1, longest=100, shortest=1, kv_heads=8, dim=128, page=16, spare=100):
    """spare: free pages in percent of those in use."""
    c = dict(op="compact", dtype=dtype, layers=layers, batch=batch, longest=longest, shortest=shortest, kv_heads=kv_heads, dim=dim,
             page=page, spare=spare)
    return dict(c, name=name) if name else c


def log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    while True:
        c = draw_any(rng)
        w = work(c)
        if w["bytes"] < 1.6e9 and w["flops"] < (2e11 if c["dtype"] == "bf16" else 1.5e10) and footprint(c) < 8e9:
            return c


def draw_any(rng):
    op = rng.choice(["attend8", "attend8", "attend8", "append8", "commit8", "fork", "compact"])
    batch = log_int(rng, 1, 512)
    page = rng.choice([8, 16, 24, 32, 64, 100])
    branches, depth = rng.choice([(0, 0), (0, rng.randint(1, 32)), (rng.randint(1, 8), rng.randint(1, 16))])
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 80, 96, 128])
    if op == "commit8":
        return commit_case(layers=log_int(rng, 1, 32), batch=min(batch, 64), branches=max(1, branches), depth=max(1, depth) % 16 + 1,
                           longest=log_int(rng, 20, 250), shortest=rng.randint(0, 20), kv_heads=kv, dim=dim, page=page)
    if op == "fork":
        width = rng.choice([1, 2, 4, 5, 8])
        groups = max(1, min(batch, 256) // width)
        return fork_case(dtype=rng.choice(["bf16", "f32", "e4m3"]), layers=log_int(rng, 1, 16), batch=groups * width,
                         children=groups * rng.choice([1, 2, 4, 8]), width=width, longest=log_int(rng, 20, 600), shortest=rng.randint(0, 20),
                         reserve=rng.choice([0, 1, 6, 33]), kv_heads=kv, dim=dim, page=page, spare=log_int(rng, 1, 100))
    if op == "compact":
        return compact_case(dtype=rng.choice(["bf16", "f32", "e4m3"]), layers=log_int(rng, 1, 16), batch=min(batch, 256),
                            longest=log_int(rng, 20, 600), shortest=rng.randint(0, 20), kv_heads=kv, dim=dim, page=page, spare=log_int(rng, 3, 300))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append8":
        return append_case(dtype=dtype, batch=batch, branches=branches, depth=depth, longest=log_int(rng, 20, 250), shortest=rng.randint(0, 20),
                           heads=kv * rng.choice([1, 3, 4, 8]), kv_heads=kv, dim=dim, page=page, rotary=rng.choice([0, dim, dim // 2]),
                           style=rng.choice(["half", "interleaved"]))
    groups = rng.choice([0, 0, 1, 2, 4])
    batch = min(batch, 64) if dtype == "f32" else batch
    batch = groups * max(1, batch // groups) if groups else batch
    longest = log_int(rng, 1, 16384)
    if not groups and dtype == "bf16" and rng.random() < 0.2:   # a prompt's rows, a part at a time
        batch, branches, depth = min(batch, 4), 0, log_int(rng, 100, 1300)
    return attend_case(dtype=dtype, batch=batch, branches=branches, depth=depth, longest=longest, shortest=rng.randint(0, longest),
                       groups=groups, prefix=log_int(rng, page, 32768) // page * page if groups else 0, heads=kv * rng.choice([1, 2, 4, 6, 8]),
                       kv_heads=kv, dim=dim, page=page)


# ---- sizes that a case implies -----------------------------------------------------------------------------------------------

def rows_of(case):
    return case["branches"] * case["depth"] + 1 if case["branches"] else case["depth"] + 1


def own_lengths(case):
    """Cached tokens of each sequence after its shared prefix, spread evenly over [shortest, longest]."""
    span = case["longest"] - case["shortest"] + 1
    return [case["shortest"] + int(span * ((b + 1) * GOLDEN % 1.0)) for b in range(case["batch"])]


def prefix_lengths(case):
    return [case["prefix"]] * case["groups"]


def contexts(case):
    if "groups" not in case:
        return own_lengths(case)
    each = case["batch"] // case["groups"] if case["groups"] else 1
    return [n + (prefix_lengths(case)[b // each] if case["groups"] else 0) for b, n in enumerate(own_lengths(case))]


def accepted(case):
    """Drafted tokens of each sequence that were accepted, from none to the whole branch."""
    return [(5 * b + 2) % (case["depth"] + 1) for b in range(case["batch"])]


def sources(case):
    """The old sequence that each new one continues, -1 for none: one of its request's beams, a few requests finished."""
    width, n = case["width"], case["children"]
    each = n * width // case["batch"]  # new sequences of a request
    return [-1 if (g := j // each) % 11 == 5 else g * width + int(width * ((j + 1) * GOLDEN % 1.0)) for j in range(n)]


def copied_tails(case):
    """Tokens of partly filled pages that a fork copies: all but the first new sequence's of an old one."""
    seen, tokens, ctx = set(), 0, contexts(case)
    for s in sources(case):
        if s >= 0:
            tokens += ctx[s] % case["page"] if s in seen else 0
            seen.add(s)
    return tokens


def held(case):
    """Page table entries that the old sequences hold."""
    return sum(-(-n // case["page"]) for n in contexts(case))


def new_pages(case):
    ctx = contexts(case)
    return sum(-(-(ctx[s] + case["reserve"]) // case["page"]) - ctx[s] // case["page"] for s in sources(case) if s >= 0)


def elem(case):
    return {"bf16": 2, "f32": 4, "e4m3": 1}[case["dtype"]]


def pool_pages(case):
    if case["op"] == "compact":
        return held(case) + max(1, held(case) * case["spare"] // 100)
    return held(case) + new_pages(case) + case["spare"]


def footprint(case):
    """Bytes of the cache."""
    if case["op"] in ("fork", "compact"):
        return 2 * case["layers"] * pool_pages(case) * case["page"] * case["kv_heads"] * case["dim"] * elem(case)
    shared, each = case["prefix"] // case["page"], -(-(case["longest"] + rows_of(case)) // case["page"])
    pages = case["groups"] * shared + case["batch"] * each
    return 2 * case.get("layers", 1) * pages * case["page"] * case["kv_heads"] * case["dim"]


def work(case):
    n = case["batch"]
    if case["op"] == "fork":
        token = case["kv_heads"] * case["dim"] * elem(case)
        return {"bytes": 4 * case["layers"] * copied_tails(case) * token + 4 * (2 * held(case) + 3 * case["children"] + 2 * pool_pages(case)),
                "flops": 0}
    if case["op"] == "compact":
        live, pages = held(case), pool_pages(case)
        moved = live * (pages - live) / pages  # of a scattered pool, as a mean
        per_page = case["page"] * case["kv_heads"] * case["dim"] * elem(case)
        return {"bytes": 4 * case["layers"] * moved * per_page + 8 * live + 8 * pages, "flops": 0}
    rows = rows_of(case)
    code = case["kv_heads"] * case["dim"]
    if case["op"] == "commit8":
        return {"bytes": 4 * case["layers"] * sum(accepted(case)) * code + 12 * n + 4 * n * (rows - 1), "flops": 0}
    size = elem(case)
    if case["op"] == "append8":
        q = case["heads"] * case["dim"] * size
        return {"bytes": n * rows * (2 * q + 2 * code * (size + 1)), "flops": 3 * n * rows * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    inner = rows + case["branches"] * case["depth"] * (case["depth"] + 1) // 2 if case["branches"] else rows * (rows + 1) // 2
    kv = 2 * code * (sum(own_lengths(case)) + sum(prefix_lengths(case)) + n * rows)
    io = n * rows * case["heads"] * (2 * case["dim"] * size + 4)
    seen = sum(rows * c + inner for c in contexts(case))
    return {"bytes": kv + io, "flops": 4 * case["heads"] * case["dim"] * seen}


# ---- inputs -------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16 if dt == DTYPES["e4m3"] else dt)

    def whole(values):
        return torch.tensor(values, device=DEVICE, dtype=torch.int32)

    s = {"case": case}
    page, n = case["page"], case["batch"]
    if case["op"] in ("fork", "compact"):
        # each sequence holds the pages of its tokens, scattered over the pool; entries behind them are empty
        pages = pool_pages(case)
        most = -(-(case["longest"] + case.get("reserve", 0)) // page)
        took = torch.tensor([-(-x // page) for x in contexts(case)], device=DEVICE)
        slot = torch.arange(most, device=DEVICE)[None]
        place = (took.cumsum(0) - took)[:, None] + slot
        pool = torch.randperm(pages, generator=g, device=DEVICE).int()
        s["page_table"] = torch.where(slot < took[:, None], pool[place.clamp(max=pages - 1)], -1).contiguous()
        s["context_len"] = whole(contexts(case))
        s["page_refs"] = torch.zeros(pages, device=DEVICE, dtype=torch.int32)
        s["page_refs"][pool[:held(case)].long()] = 1
        if case["op"] == "fork":
            s["src"] = whole(sources(case))
        fill_cache(s, (case["layers"], pages, page, case["kv_heads"], case["dim"]), normal)
        return s
    if case.get("rotary"):
        i = torch.arange(case["rotary"] // 2, device=DEVICE, dtype=torch.float64)
        s["inv_freq"] = torch.pow(torch.tensor(10000.0, device=DEVICE, dtype=torch.float64), -2.0 * i / case["rotary"]).float()
    rows, groups = rows_of(case), case["groups"]
    if case["branches"]:
        node = torch.arange(case["branches"] * case["depth"], device=DEVICE, dtype=torch.int32)
        s["parents"] = torch.where(node % case["depth"] == 0, 0, node)[None].repeat(n, 1).contiguous()
    # pages: a prefix's pages are shared by its group, the rest belong to one sequence; they lie anywhere in the pool
    shared, each = case["prefix"] // page, -(-(case["longest"] + rows) // page)
    total = groups * shared + n * each
    pool = torch.randperm(total, generator=g, device=DEVICE).int()
    table = pool[groups * shared:].reshape(n, each)
    if groups:
        table = torch.cat([pool[:groups * shared].reshape(groups, shared).repeat_interleave(n // groups, 0), table], 1)
        s["group_start"] = whole([k * (n // groups) for k in range(groups + 1)])
        s["prefix_len"] = whole(prefix_lengths(case))
    s["page_table"] = table.contiguous()
    s["context_len"] = whole(contexts(case))
    shape = (total, page, case["kv_heads"], case["dim"])
    if case["op"] == "commit8":
        shape = (case["layers"],) + shape
        s["accept_len"] = whole(accepted(case))
        branch = torch.randint(0, case["branches"], (n, 1), generator=g, device=DEVICE)
        j = torch.arange(rows - 1, device=DEVICE)[None]
        s["path"] = torch.where(j < s["accept_len"][:, None], branch * case["depth"] + 1 + j, -1).int().contiguous()
    fill_cache(s, shape, normal)
    if case["op"] == "attend8":
        s["q"] = normal(n, rows, case["heads"], case["dim"]) * 2  # scores spread enough for some keys to stand out
    if case["op"] == "append8":
        # the three parts of one projection's output, as a model has them: views with the projection's row stride
        qkv = normal(n, rows, case["heads"] + 2 * case["kv_heads"], case["dim"])
        s["q"], s["k"], s["v"] = qkv.split([case["heads"], case["kv_heads"], case["kv_heads"]], 2)
    return s


def fill_cache(s, shape, normal):
    """Caches of `shape`; codes with their scales where they are held in 8 bits (all but fork and compact hold them so)."""
    case = s["case"]
    if case["op"] in ("fork", "compact") and case["dtype"] != "e4m3":
        s["k_cache"], s["v_cache"] = normal(*shape), normal(*shape)
        return
    for name in ("k", "v"):
        x = normal(*shape)
        # pages and heads of unlike size, as a model's are
        x *= torch.exp2(normal(*shape[:-3], 1, shape[-2], 1).float().round()).to(x.dtype)
        e = exponent(x.abs().amax((-3, -1)).float())
        s[name + "_cache"] = (x * torch.exp2(-e.float())[..., None, :, None].to(x.dtype)).to(torch.float8_e4m3fn)
        s[name + "_scale"] = as_scale(e)


def exponent(most):
    """The smallest exponent, LOWEST at least, of a scale that keeps `most` within 448."""
    m, e = torch.frexp(most.double() / E4M3_MAX)
    return torch.where(most > 0, (e - (m == 0.5).int()).clamp(min=LOWEST), LOWEST).int()


def as_scale(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def of_scale(scale):
    return scale.view(torch.uint8).int() - 127


# ---- one pass ------------------------------------------------------------------------------------------------------------------

def run(state):
    op, s = state["case"]["op"], state
    if own:
        import speculative_decoding_verification_gb300 as sv
        if op in ("fork", "compact"):
            scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if "k_scale" in s else {}
            if op == "fork":
                got = sv.sv_kv_fork(s["k_cache"], s["v_cache"], s["page_refs"], s["context_len"], s["page_table"], s["src"],
                                    reserve=s["case"]["reserve"], **scales)
            else:
                got = sv.sv_kv_compact(s["k_cache"], s["v_cache"], s["page_refs"], s["page_table"], **scales)
            return (*got, *caches(s))
        cache = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["context_len"], s["page_table"]
        if op == "append8":
            return (sv.sv_kv_append8(s["k"], s["v"], *cache, q=s["q"], inv_freq=s.get("inv_freq"), style=s["case"]["style"],
                                     parents=s.get("parents")), *caches(s))
        if op == "commit8":
            return (sv.sv_kv_commit8(*cache, s["accept_len"], s["path"]), *caches(s))
        return sv.sv_kv_attend8(s["q"], *cache, parents=s.get("parents"), group_start=s.get("group_start"),
                                prefix_len=s.get("prefix_len"), lse=True)
    return {"append8": plain_append, "commit8": plain_commit, "attend8": plain_attend, "fork": plain_fork, "compact": plain_compact}[op](s)


def caches(s):
    return tuple(s[name] for name in ("k_cache", "v_cache", "k_scale", "v_scale") if name in s)


def rotated(x, angle, style):
    """x [..., heads, dim] with its first 2 * angle.shape[-1] elements rotated in pairs by angle [..., pairs], in 32 bits."""
    half = angle.shape[-1]
    x = x.float()
    c, s = angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if style == "half":
        a, b = r[..., :half], r[..., half:]
        return torch.cat([a * c - b * s, a * s + b * c, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), rest], -1)


def ancestors(s, rows):
    """[batch or 1, rows, rows]: whether row i sees row j.  For a tree with parent matrix P it is (1 - P)^-1, the sum of P's powers."""
    eye = torch.eye(rows, device=DEVICE)
    if "parents" not in s:
        return torch.ones_like(eye).tril()[None] > 0
    below = torch.zeros(len(s["parents"]), rows, rows, device=DEVICE)
    below[:, 1:].scatter_(2, s["parents"].long()[..., None], 1.0)
    return torch.linalg.solve_triangular(eye - below, eye.expand_as(below), upper=False, unitriangular=True) > 0.5


def places(s, slots):
    """Page and place in it of token numbers slots [batch, n]."""
    page = s["case"]["page"]
    slots = slots.long()
    at = (slots // page).clamp(max=s["page_table"].shape[1] - 1)
    return s["page_table"].long().gather(1, at), slots % page


def requantised(codes, shift):
    """uint8 codes in a scale that is 2^shift times theirs, as uint8 codes."""
    return (codes.view(torch.float8_e4m3fn).float() * torch.exp2(-shift.float())).to(torch.float8_e4m3fn).view(torch.uint8)


def values(s, name, p, o):
    """Cached values at places (p, o), in 32 bits."""
    return s[name + "_cache"].view(torch.uint8)[p, o].view(torch.float8_e4m3fn).float() * torch.exp2(of_scale(s[name + "_scale"])[p].float())[..., None]


def plain_append(s):
    case, rows, page = s["case"], s["k"].shape[1], s["case"]["page"]
    ctx = s["context_len"][:, None]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if case["rotary"]:
        depth = ancestors(s, rows).sum(-1) - 1
        angle = (ctx + depth).double()[..., None] * s["inv_freq"].double()
        q, k = rotated(q, angle, case["style"]), rotated(k, angle, case["style"])
    slot = ctx + torch.arange(rows, device=DEVICE)
    p, o = places(s, slot)
    first, place = places(s, ctx // page * page + torch.arange(page, device=DEVICE))  # the page that holds cached tokens already
    cached = place < ctx % page
    for name, x in (("k", k), ("v", v)):
        old = of_scale(s[name + "_scale"])
        e = old.clone()
        e[p[slot % page == 0]] = LOWEST  # pages that the block begins
        e.index_reduce_(0, p.flatten(), exponent(x.abs().amax(-1)).flatten(0, 1), "amax")
        codes = s[name + "_cache"].view(torch.uint8)
        before = codes[first, place]
        after = requantised(before, (e - old)[first][..., None].expand(before.shape))
        codes[first, place] = torch.where(cached[..., None, None], after, before)
        codes[p, o] = (x * torch.exp2(-e[p].float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_scale"].copy_(as_scale(e))
    return (q.to(s["q"].dtype), *caches(s))


def plain_commit(s):
    ctx, page = s["context_len"][:, None], s["case"]["page"]
    j = torch.arange(s["path"].shape[1], device=DEVICE)[None]
    to = ctx + 1 + j
    took = j < s["accept_len"][:, None]
    sp, so = places(s, torch.where(took, ctx + s["path"], to))  # what was not accepted stays where it is
    dp, do = places(s, to)
    first, place = places(s, (ctx + 1) // page * page + torch.arange(page, device=DEVICE))
    kept = (place <= (ctx + 1) % page - 1) & (s["accept_len"][:, None] > 0)
    for name in ("k", "v"):
        old = of_scale(s[name + "_scale"])
        arrives = torch.where(took[None, :, :, None], old[:, sp], LOWEST - 7)
        e = old.clone().index_reduce_(1, dp.flatten(), arrives.flatten(1, 2), "amax")
        codes = s[name + "_cache"].view(torch.uint8)
        before, came, there = codes[:, first, place], codes[:, sp, so], codes[:, dp, do]
        stay = requantised(before, (e - old)[:, first][..., None].expand(before.shape))
        new = requantised(came, (e[:, dp] - old[:, sp])[..., None].expand(came.shape))
        codes[:, first, place] = torch.where(kept[None, ..., None, None], stay, before)
        codes[:, dp, do] = torch.where(took[None, ..., None, None], new, there)
        s[name + "_scale"].copy_(as_scale(e))
    return (s["context_len"] + 1 + s["accept_len"], *caches(s))


def plain_attend(s):
    case, q = s["case"], s["q"]
    n, rows, heads, dim = q.shape
    kv, page = case["kv_heads"], case["page"]
    groups = max(1, case["groups"])
    q5 = q.float().reshape(n, rows, kv, heads // kv, dim) * dim ** -0.5
    ctx = s["context_len"][:, None].long()
    start = s["prefix_len"].long().repeat_interleave(n // groups)[:, None] if case["groups"] else torch.zeros_like(ctx)
    # each sequence's tokens after the prefix
    slot = start + torch.arange(case["longest"] + rows, device=DEVICE)
    p, o = places(s, slot)
    k, v = values(s, "k", p, o), values(s, "v", p, o)
    score = torch.einsum("bihrd,bjhd->bhrij", q5, k)
    sees = ancestors(s, rows).expand(n, -1, -1)
    new = (slot - ctx)[:, None].expand(-1, rows, -1)
    seen = (new < 0) | ((new < rows) & sees.gather(2, new.clamp(0, rows - 1)))
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    if case["groups"]:
        # the group's prefix, read once for all its sequences
        first = s["page_table"][s["group_start"][:-1].long()].long()
        j = torch.arange(case["prefix"], device=DEVICE)
        pk, pv = (values(s, c, first[:, j // page], j % page) for c in ("k", "v"))
        gq = q5.reshape(groups, n // groups, rows, kv, heads // kv, dim)
        before = torch.einsum("gbihrd,gjhd->gbhrij", gq, pk).reshape(n, kv, heads // kv, rows, -1)
        beyond = j >= s["prefix_len"][:, None]
        before = before.masked_fill(beyond.repeat_interleave(n // groups, 0)[:, None, None, None], -math.inf)
        top = torch.maximum(score.amax(-1, True), before.amax(-1, True))
        wp = (before - top).exp()
        w = (score - top).exp()
        total = w.sum(-1, True) + wp.sum(-1, True)
        out = torch.einsum("gbhrij,gjhd->gbihrd", wp.reshape(groups, n // groups, kv, heads // kv, rows, -1), pv).reshape_as(q5)
        out = out + torch.einsum("bhrij,bjhd->bihrd", w, v)
    else:
        top = score.amax(-1, True)
        w = (score - top).exp()
        total = w.sum(-1, True)
        out = torch.einsum("bhrij,bjhd->bihrd", w, v)
    out = out / total.squeeze(-1).permute(0, 3, 1, 2)[..., None]
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    return out.reshape(q.shape).to(q.dtype), lse.reshape(n, rows, heads).contiguous()


def plain_fork(s):
    case, page, refs = s["case"], s["case"]["page"], s["page_refs"]
    table, src, pages = s["page_table"], s["src"], len(s["page_refs"])
    goes = src >= 0
    of = src.clamp(min=0).long()
    ctx = torch.where(goes, s["context_len"][of], 0)
    theirs = torch.where(goes[:, None], table[of], -1).long()
    full, part = (ctx // page)[:, None], (ctx % page > 0)[:, None]
    need = torch.where(goes, -(-(ctx + case["reserve"]) // page), 0)[:, None]
    col = torch.arange(table.shape[1], device=DEVICE)[None]

    def counted(entries):
        return torch.bincount(torch.where(entries >= 0, entries, pages).long().flatten(), minlength=pages + 1)[:pages]

    shared = torch.where(col < full, theirs, -1)
    left = refs - counted(table)  # holders that are no sequence of the old batch
    after = left + counted(shared)
    # a partly filled page stays with its first new sequence where nobody else holds it
    tail = torch.where((col == full) & part, theirs, -1)
    child = torch.arange(len(src), device=DEVICE)[:, None].expand_as(tail)
    owner = torch.full((pages + 1,), len(src), device=DEVICE)
    owner.scatter_reduce_(0, torch.where(tail >= 0, tail, pages).flatten(), child.flatten(), "amin")
    keeps = (tail >= 0) & (owner[tail] == child) & (after[tail] == 0)
    after = after + counted(torch.where(keeps, tail, -1))
    # the others get the lowest free pages in order
    wants = (col >= full) & (col < need) & ~keeps
    free = after == 0
    listed_free = torch.zeros(pages + 1, device=DEVICE, dtype=torch.long)
    listed_free[torch.where(free, free.cumsum(0) - 1, pages)] = torch.arange(pages, device=DEVICE)
    rank = (wants.flatten().cumsum(0) - 1).reshape(wants.shape)
    gets = torch.where(wants, listed_free[rank.clamp(min=0)], -1)
    after = after + counted(gets)
    new = torch.where(wants, gets, torch.where(keeps, tail, shared)).int()
    # tokens of the partly filled pages
    at = full.clamp(max=table.shape[1] - 1).long()
    place = torch.arange(page, device=DEVICE)[None]
    moves = (wants.gather(1, at) & part & (place < (ctx % page)[:, None])).flatten().nonzero().flatten()
    frm = theirs.gather(1, at).expand(-1, page).flatten()[moves]
    to = new.long().gather(1, at).expand(-1, page).flatten()[moves]
    o = place.expand(len(src), -1).flatten()[moves]
    for c in caches(s):
        c = c.view(torch.uint8) if c.element_size() == 1 else c
        if c.dim() == 5:
            c[:, to, o] = c[:, frm, o]
        else:
            c[:, to] = c[:, frm]
    return new, ctx.int(), after.int(), *caches(s)


def plain_compact(s):
    refs, table = s["page_refs"], s["page_table"]
    pages = len(refs)
    live = refs > 0
    count = live.sum()
    at = torch.arange(pages, device=DEVICE)
    frm = (live & (at >= count)).nonzero().flatten()
    to = (~live & (at < count)).nonzero().flatten()
    where = at.clone()
    where[frm] = to
    for c in caches(s):
        c = c.view(torch.uint8) if c.element_size() == 1 else c
        c[:, to] = c[:, frm]
    after = torch.where(at < count, refs, 0)
    after[to] = refs[frm]
    new = torch.where(table >= 0, where[table.clamp(min=0).long()].int(), table)
    return new, after, count.int().reshape(1), *caches(s)


# ---- the definition in 64 bits ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fork", "compact"):
        return exact_pages(case, s)
    n, page, rows, table = case["batch"], case["page"], rows_of(case), s["page_table"].tolist()
    ctx = s["context_len"].tolist()
    if case["op"] == "commit8":
        return exact_commit(case, s, table, ctx)
    up = [-1] + s["parents"][0].tolist() if "parents" in s else list(range(-1, rows - 1))
    sees = [[False] * rows for _ in range(rows)]
    for i in range(rows):
        j = i
        while j >= 0:
            sees[i][j] = True
            j = up[j]
    if case["op"] == "append8":
        return exact_append(case, s, table, ctx, [sum(r) - 1 for r in sees])
    out = torch.empty(s["q"].shape, device=DEVICE, dtype=torch.float64)
    lse = torch.empty(s["q"].shape[:3], device=DEVICE, dtype=torch.float64)
    rep = case["heads"] // case["kv_heads"]
    sees = torch.tensor(sees, device=DEVICE)
    full = [s[c + "_cache"].double() * s[c + "_scale"].double()[:, None, :, None] for c in ("k", "v")]
    kf, vf = (c.flatten(0, 1) for c in full)
    for b in range(n):
        j = torch.arange(ctx[b] + rows, device=DEVICE)
        at = s["page_table"][b].long()[j // page] * page + j % page
        hide = torch.zeros(rows, ctx[b] + rows, device=DEVICE, dtype=torch.bool)
        hide[:, ctx[b]:] = ~sees
        for h in range(case["kv_heads"]):
            k, v = kf[at, h], vf[at, h]
            mine = slice(h * rep, h * rep + rep)
            x = torch.matmul(s["q"][b, :, mine].double(), k.T) / math.sqrt(case["dim"])
            x = x.masked_fill(hide[:, None], -math.inf)
            lse[b, :, mine] = torch.logsumexp(x, -1)
            out[b, :, mine] = torch.matmul(torch.softmax(x, -1), v)
    return out, lse


def on_grid(x):
    """x, in doubles, rounded to the nearest e4m3 number, ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact_append(case, s, table, ctx, depth):
    page, n, rows = case["page"], case["batch"], rows_of(case)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if case["rotary"]:
        pos = torch.tensor([c + d for c in ctx for d in depth], device=DEVICE)
        q, k = (exact_rotation(x.flatten(0, 1), pos, s["inv_freq"], case["style"]).reshape(x.shape) for x in (q, k))
    got = [q]
    for name, x in (("k", k), ("v", v)):
        codes, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        spans = [(b, i, min(i + page - (ctx[b] + i) % page, rows)) for b in range(n)
                 for i in [0, *(i for i in range(1, rows) if (ctx[b] + i) % page == 0)]]
        most = torch.stack([x[b, i:j].abs().amax((0, 2)) for b, i, j in spans])
        need = torch.exp2(torch.ceil(torch.log2(most / E4M3_MAX)).clamp(min=LOWEST))
        for (b, i, j), e in zip(spans, need):
            p, o = table[b][(ctx[b] + i) // page], (ctx[b] + i) % page
            if o:
                e = torch.maximum(e, scale[p])
                codes[p, :o] = on_grid(codes[p, :o] * (scale[p] / e)[:, None])
            scale[p] = e
            codes[p, o:o + j - i] = on_grid(x[b, i:j] / e[:, None])
        got += [codes, scale]
    return got[0], got[1], got[3], got[2], got[4]


def exact_commit(case, s, table, ctx):
    page, path, took = case["page"], s["path"].tolist(), s["accept_len"].tolist()
    got = []
    for name in ("k", "v"):
        codes, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        for b in range(case["batch"]):
            for j0 in [j for j in range(took[b]) if j == 0 or (ctx[b] + 1 + j) % page == 0]:
                p, o = table[b][(ctx[b] + 1 + j0) // page], (ctx[b] + 1 + j0) % page
                js = range(j0, min(took[b], j0 + page - o))
                frm = [divmod(ctx[b] + path[b][j], page) for j in js]
                sp, so = [table[b][f[0]] for f in frm], [f[1] for f in frm]
                e = torch.maximum(scale[:, p], scale[:, sp].amax(1))
                kept = on_grid(codes[:, p, :o] * (scale[:, p] / e)[:, None, :, None])
                came = on_grid(codes[:, sp, so] * (scale[:, sp] / e[:, None])[..., None])
                codes[:, p, :o], codes[:, p, o:o + len(js)], scale[:, p] = kept, came, e
        got += [codes, scale]
    return None, got[0], got[2], got[1], got[3]


def exact_pages(case, s):
    """Pages moved one at a time, in the order of the definition; the caches as they then are."""
    refs, table, page = s["page_refs"].tolist(), s["page_table"].tolist(), case["page"]
    moves = []
    if case["op"] == "fork":
        ctx, src = s["context_len"].tolist(), s["src"].tolist()
        for row in table:
            for p in row:
                refs[p] -= p >= 0
        for b in src:
            for p in table[b][:ctx[b] // page] if b >= 0 else []:
                refs[p] += 1
        keeps = set()
        for j, b in enumerate(src):
            if b >= 0 and ctx[b] % page and refs[table[b][ctx[b] // page]] == 0:
                refs[table[b][ctx[b] // page]] += 1
                keeps.add(j)
        free = iter([p for p, r in enumerate(refs) if r == 0])
        for j, b in enumerate(src):
            if b < 0:
                continue
            full = ctx[b] // page
            for c in range(full + (j in keeps), -(-(ctx[b] + case["reserve"]) // page)):
                p = next(free)
                if c == full and ctx[b] % page:
                    moves.append((table[b][c], p, ctx[b] % page))
    else:
        live = [p for p, r in enumerate(refs) if r > 0]
        holes = [p for p, r in enumerate(refs[:len(live)]) if r == 0]
        moves = list(zip([p for p in live if p >= len(live)], holes, [page] * len(holes)))
    got = [c.double() for c in caches(s)]
    for frm, to, tokens in moves:
        for c in got:
            if c.dim() == 5:
                c[:, to, :tokens] = c[:, frm, :tokens]
            else:
                c[:, to] = c[:, frm]
    return None, None, None, *got


def exact_rotation(x, pos, inv_freq, style):
    """Pairs as complex numbers, turned by exp(i * position * frequency)."""
    x = x.double().clone()
    r = 2 * inv_freq.numel()
    turn = torch.polar(torch.ones((), device=DEVICE, dtype=torch.float64), pos.double()[:, None] * inv_freq.double())[:, None]
    if style == "half":
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
        x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
        x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
    return x
