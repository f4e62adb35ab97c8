"""Workloads of the target model's side of a speculative-decoding step, over a paged key/value cache:

  rope    rotary positions applied to query or key heads, or their gradient taken back through the rotation
  append  a block's new tokens: queries and keys rotated, keys and values written to the pages of each sequence
  attend  attention of the block's rows over the cached tokens, where groups of sequences may share a long prefix
  commit  after a drafted tree was verified, the accepted path's keys and values move to consecutive slots

A block is what one verification step scores for each sequence: the last committed token and the drafted ones after it, as a
chain (each row sees the rows before it) or as a tree of `branches` paths of `depth` tokens that all start at row 0 (each row
sees its ancestors).  `run` computes the plain form where `own` is false and calls the library where it is true.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GOLDEN = 0.6180339887498949


def listed():
    return [
        # one sequence, four drafted tokens, a short context: what an interactive request costs a layer
        attend_case("attend one chain", batch=1, depth=4, longest=1000, shortest=1000),
        # ordinary decoding in float32 heads of an odd width (a small draft model), one token a sequence, contexts of all lengths
        attend_case("attend single tokens, float32", dtype="f32", batch=64, depth=0, longest=8192, shortest=7, heads=12, kv_heads=3, dim=80, page=20),
        # a large serving batch that verifies five drafted tokens for each sequence
        attend_case("attend large batch", batch=512, depth=5, longest=2048, shortest=1024),
        # four requests whose eight drafted branches each run as sequences of their own over the request's context
        attend_case("attend branches, shared context", batch=32, depth=7, longest=33, shortest=1, groups=4, prefix=16384),
        # a batch behind one long system prompt: the prompt's part has enough rows to be bound by arithmetic
        attend_case("attend shared prompt", batch=64, depth=5, longest=700, shortest=20, groups=1, prefix=32768),
        # a tree of eight branches of seven tokens a sequence, small heads, an odd page size
        attend_case("attend trees", batch=16, branches=8, depth=7, longest=4001, shortest=500, heads=24, kv_heads=4, dim=64, page=24),
        # one interactive request's new rows
        append_case("append one chain", batch=1, depth=4, longest=1000, shortest=1000),
        # the large batch's new rows; half of each head is rotated, neighbours paired
        append_case("append large batch", batch=512, depth=5, longest=200, shortest=30, rotary=64, style="interleaved"),
        # the queries of a long prompt at positions far out
        rope_case("rope long prompt", tokens=8192, heads=32, first=120000),
        # training a drafter: the gradient of a float32 batch
        rope_case("rope gradient", dtype="f32", tokens=1000, heads=12, dim=80, rotary=40, style="interleaved", backward=True),
        # every layer's accepted path after a step over branch-complete trees
        commit_case("commit all layers", layers=32, batch=64, branches=8, depth=7, longest=200, shortest=20),
        # one request, one layer, a small tree
        commit_case("commit one request", layers=4, batch=1, branches=3, depth=4, longest=500, shortest=500, dim=64),
    ]


def attend_case(name=None, dtype="bf16", batch=1, branches=0, depth=4, longest=1000, shortest=1, groups=0, prefix=0, heads=32,
                kv_heads=8, dim=128, page=16):
    c = dict(op="attend", dtype=dtype, batch=batch, branches=branches, depth=depth, longest=longest, shortest=shortest, groups=groups,
             prefix=prefix, heads=heads, kv_heads=kv_heads, dim=dim, page=page)
    return dict(c, name=name) if name else c


def append_case(name=None, dtype="bf16", batch=1, branches=0, depth=4, longest=1000, shortest=1, heads=32, kv_heads=8, dim=128, page=16,
                rotary=128, style="half"):
    c = dict(op="append", dtype=dtype, batch=batch, branches=branches, depth=depth, longest=longest, shortest=shortest, groups=0, prefix=0,
             heads=heads, kv_heads=kv_heads, dim=dim, page=page, rotary=rotary, style=style)
    return dict(c, name=name) if name else c


def rope_case(name=None, dtype="bf16", tokens=1, heads=32, dim=128, rotary=128, style="half", backward=False, first=0):
    c = dict(op="rope", dtype=dtype, tokens=tokens, heads=heads, dim=dim, rotary=rotary, style=style, backward=backward, first=first)
    return dict(c, name=name) if name else c


def commit_case(name=None, dtype="bf16", layers=1, batch=1, branches=1, depth=4, longest=100, shortest=1, kv_heads=8, dim=128, page=16):
    c = dict(op="commit", dtype=dtype, layers=layers, batch=batch, branches=branches, depth=depth, longest=longest, shortest=shortest,
             groups=0, prefix=0, kv_heads=kv_heads, dim=dim, page=page)
    return dict(c, name=name) if name else c


def log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    while True:
        c = draw_any(rng)
        w = work(c)
        if w["bytes"] < 2.5e9 and w["flops"] < (2e11 if c["dtype"] == "bf16" else 1.5e10):
            return c


def draw_any(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "rope", "commit"])
    if op == "rope":
        # angles formed in 32 bits lose a float32 output's last digits at positions in the thousands: float32 stays below
        dtype, dim = rng.choice(["bf16", "f32"]), rng.choice([64, 80, 96, 128])
        return rope_case(dtype=dtype, tokens=log_int(rng, 1, 8192 if dtype == "bf16" else 4000), heads=rng.choice([1, 3, 8, 12, 32]), dim=dim,
                         rotary=rng.choice([dim, dim // 2, dim // 2 - 6]), style=rng.choice(["half", "interleaved"]),
                         backward=rng.random() < 0.4, first=log_int(rng, 1, 120000) if dtype == "bf16" else 0)
    batch = log_int(rng, 1, 512)
    page = rng.choice([8, 16, 24, 32, 64, 100])
    branches, depth = rng.choice([(0, 0), (0, rng.randint(1, 32)), (rng.randint(1, 8), rng.randint(1, 16))])
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 80, 96, 128])
    if op == "commit":
        return commit_case(dtype=rng.choice(["bf16", "f32"]), layers=log_int(rng, 1, 32), batch=min(batch, 64), branches=max(1, branches),
                           depth=max(1, depth) % 16 + 1, longest=log_int(rng, 20, 250), shortest=rng.randint(0, 20), kv_heads=kv, dim=dim, page=page)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        return append_case(dtype=dtype, batch=batch, branches=branches, depth=depth, longest=log_int(rng, 20, 250), shortest=rng.randint(0, 20),
                           heads=kv * rng.choice([1, 3, 4, 8]), kv_heads=kv, dim=dim, page=page, rotary=rng.choice([0, dim, dim // 2]),
                           style=rng.choice(["half", "interleaved"]))
    groups = rng.choice([0, 0, 1, 2, 4])
    batch = min(batch, 64) if dtype == "f32" else batch
    batch = groups * max(1, batch // groups) if groups else batch
    longest = log_int(rng, 1, 16384)
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
    each = case["batch"] // case["groups"] if case["groups"] else 1
    return [n + (prefix_lengths(case)[b // each] if case["groups"] else 0) for b, n in enumerate(own_lengths(case))]


def accepted(case):
    """Drafted tokens of each sequence that were accepted, from none to the whole branch."""
    return [(5 * b + 2) % (case["depth"] + 1) for b in range(case["batch"])]


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"], "flops": 3 * n * case["rotary"]}
    n, rows = case["batch"], rows_of(case)
    token = case["kv_heads"] * case["dim"] * size
    if case["op"] == "commit":
        return {"bytes": 4 * case["layers"] * sum(accepted(case)) * token + 12 * n + 4 * n * (rows - 1), "flops": 0}
    if case["op"] == "append":
        q = case["heads"] * case["dim"] * size
        return {"bytes": 2 * n * rows * (q + 2 * token), "flops": 3 * n * rows * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    inner = rows + case["branches"] * case["depth"] * (case["depth"] + 1) // 2 if case["branches"] else rows * (rows + 1) // 2
    kv = 2 * token * (sum(own_lengths(case)) + sum(prefix_lengths(case)) + n * rows)
    io = n * rows * case["heads"] * (2 * case["dim"] * size + 4)
    seen = sum(rows * c + inner for c in contexts(case))
    return {"bytes": kv + io, "flops": 4 * case["heads"] * case["dim"] * seen}


# ---- inputs -------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE, dtype=dt)

    def whole(values):
        return torch.tensor(values, device=DEVICE, dtype=torch.int32)

    s = {"case": case}
    if case.get("rotary"):
        i = torch.arange(case["rotary"] // 2, device=DEVICE, dtype=torch.float64)
        s["inv_freq"] = torch.pow(torch.tensor(10000.0, device=DEVICE, dtype=torch.float64), -2.0 * i / case["rotary"]).float()
    if case["op"] == "rope":
        s["x"] = normal(case["tokens"], case["heads"], case["dim"])
        s["positions"] = torch.arange(case["first"], case["first"] + case["tokens"], device=DEVICE, dtype=torch.int32)
        return s
    n, rows, page, groups = case["batch"], rows_of(case), case["page"], case["groups"]
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
    if case["op"] == "commit":
        shape = (case["layers"],) + shape
        s["accept_len"] = whole(accepted(case))
        branch = torch.randint(0, case["branches"], (n, 1), generator=g, device=DEVICE)
        j = torch.arange(rows - 1, device=DEVICE)[None]
        s["path"] = torch.where(j < s["accept_len"][:, None], branch * case["depth"] + 1 + j, -1).int().contiguous()
    s["k_cache"], s["v_cache"] = normal(*shape), normal(*shape)
    if case["op"] == "attend":
        s["q"] = normal(n, rows, case["heads"], case["dim"]) * 2  # scores spread enough for some keys to stand out
    if case["op"] == "append":
        # the three parts of one projection's output, as a model has them: views with the projection's row stride
        qkv = normal(n, rows, case["heads"] + 2 * case["kv_heads"], case["dim"])
        s["q"], s["k"], s["v"] = qkv.split([case["heads"], case["kv_heads"], case["kv_heads"]], 2)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import speculative_decoding_verification_gb300 as sv
        if op == "rope":
            return sv.sv_rope(state["x"], state["positions"], state["inv_freq"], style=state["case"]["style"], backward=state["case"]["backward"])
        if op == "append":
            q = sv.sv_kv_append(state["k"], state["v"], state["k_cache"], state["v_cache"], state["context_len"], state["page_table"],
                                q=state["q"], inv_freq=state.get("inv_freq"), style=state["case"]["style"], parents=state.get("parents"))
            return q, state["k_cache"], state["v_cache"]
        if op == "commit":
            context = sv.sv_kv_commit(state["k_cache"], state["v_cache"], state["context_len"], state["page_table"], state["accept_len"],
                                      state["path"])
            return context, state["k_cache"], state["v_cache"]
        return sv.sv_kv_attend(state["q"], state["k_cache"], state["v_cache"], state["context_len"], state["page_table"],
                               parents=state.get("parents"), group_start=state.get("group_start"), prefix_len=state.get("prefix_len"), lse=True)
    return {"rope": plain_rope, "append": plain_append, "commit": plain_commit, "attend": plain_attend}[op](state)


def rotated(x, angle, style, sign=1.0):
    """x [..., heads, dim] with its first 2 * angle.shape[-1] elements rotated in pairs by angle [..., pairs], in 32 bits."""
    half = angle.shape[-1]
    x = x.float()
    c, s = angle.cos()[..., None, :], sign * angle.sin()[..., None, :]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if style == "half":
        a, b = r[..., :half], r[..., half:]
        return torch.cat([a * c - b * s, a * s + b * c, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), rest], -1)


def plain_rope(s):
    angle = s["positions"].float()[:, None] * s["inv_freq"]
    return rotated(s["x"], angle, s["case"]["style"], -1.0 if s["case"]["backward"] else 1.0).to(s["x"].dtype)


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


def plain_append(s):
    case, rows = s["case"], s["k"].shape[1]
    ctx = s["context_len"][:, None]
    q, k = s["q"], s["k"]
    if case["rotary"]:
        depth = ancestors(s, rows).sum(-1) - 1
        angle = (ctx + depth).float()[..., None] * s["inv_freq"]
        q, k = rotated(q, angle, case["style"]).to(q.dtype), rotated(k, angle, case["style"]).to(k.dtype)
    p, o = places(s, ctx + torch.arange(rows, device=DEVICE))
    s["k_cache"][p, o] = k
    s["v_cache"][p, o] = s["v"]
    return q.contiguous(), s["k_cache"], s["v_cache"]


def plain_commit(s):
    j = torch.arange(s["path"].shape[1], device=DEVICE)[None]
    to = s["context_len"][:, None] + 1 + j
    took = j < s["accept_len"][:, None]
    p, o = places(s, torch.where(took, s["context_len"][:, None] + s["path"], to))  # what was not accepted stays where it is
    k, v = s["k_cache"][:, p, o], s["v_cache"][:, p, o]
    p, o = places(s, to)
    s["k_cache"][:, p, o] = k
    s["v_cache"][:, p, o] = v
    return s["context_len"] + 1 + s["accept_len"], s["k_cache"], s["v_cache"]


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
    k, v = s["k_cache"][p, o].float(), s["v_cache"][p, o].float()
    score = torch.einsum("bihrd,bjhd->bhrij", q5, k)
    sees = ancestors(s, rows).expand(n, -1, -1)
    new = (slot - ctx)[:, None].expand(-1, rows, -1)
    seen = (new < 0) | ((new < rows) & sees.gather(2, new.clamp(0, rows - 1)))
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    if case["groups"]:
        # the group's prefix, read once for all its sequences
        first = s["page_table"][s["group_start"][:-1].long()].long()
        j = torch.arange(case["prefix"], device=DEVICE)
        pk, pv = (s[c][first[:, j // page], j % page].float() for c in ("k_cache", "v_cache"))
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


# ---- the definition in 64 bits ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return exact_rotation(s["x"], s["positions"], s["inv_freq"], case["style"], -1 if case["backward"] else 1)
    n, page, rows, table = case["batch"], case["page"], rows_of(case), s["page_table"].tolist()
    ctx = s["context_len"].tolist()
    if case["op"] == "commit":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        path, took = s["path"].tolist(), s["accept_len"].tolist()
        moves = [(b, ctx[b] + path[b][j], ctx[b] + 1 + j) for b in range(n) for j in range(took[b])]
        if moves:
            src, dst = ([table[m[0]][m[i] // page] * page + m[i] % page for m in moves] for i in (1, 2))
            for c in (k, v):
                flat = c.view(c.shape[0], -1, *c.shape[3:])
                flat[:, dst] = flat[:, src].clone()
        return None, k, v
    up = [-1] + s["parents"][0].tolist() if "parents" in s else list(range(-1, rows - 1))
    sees = [[False] * rows for _ in range(rows)]
    for i in range(rows):
        j = i
        while j >= 0:
            sees[i][j] = True
            j = up[j]
    if case["op"] == "append":
        slots = [ctx[b] + i for b in range(n) for i in range(rows)]
        at = [table[b][(ctx[b] + i) // page] * page + (ctx[b] + i) % page for b in range(n) for i in range(rows)]
        q, k = s["q"].double(), s["k"].double()
        if case["rotary"]:
            pos = torch.tensor([ctx[b] + sum(sees[i]) - 1 for b in range(n) for i in range(rows)], device=DEVICE)
            q = exact_rotation(q.flatten(0, 1), pos, s["inv_freq"], case["style"], 1).reshape(q.shape)
            k = exact_rotation(k.flatten(0, 1), pos, s["inv_freq"], case["style"], 1).reshape(k.shape)
        assert len(slots) == len(set(at))
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc.view(-1, *kc.shape[2:])[at] = k.flatten(0, 1)
        vc.view(-1, *vc.shape[2:])[at] = s["v"].double().flatten(0, 1)
        return q, kc, vc
    out = torch.empty(s["q"].shape, device=DEVICE, dtype=torch.float64)
    lse = torch.empty(s["q"].shape[:3], device=DEVICE, dtype=torch.float64)
    rep = case["heads"] // case["kv_heads"]
    sees = torch.tensor(sees, device=DEVICE)
    kf, vf = (s[c].flatten(0, 1) for c in ("k_cache", "v_cache"))
    for b in range(n):
        j = torch.arange(ctx[b] + rows, device=DEVICE)
        at = s["page_table"][b].long()[j // page] * page + j % page
        hide = torch.zeros(rows, ctx[b] + rows, device=DEVICE, dtype=torch.bool)
        hide[:, ctx[b]:] = ~sees
        for h in range(case["kv_heads"]):
            k, v = kf[at, h].double(), vf[at, h].double()
            mine = slice(h * rep, h * rep + rep)
            x = torch.matmul(s["q"][b, :, mine].double(), k.T) / math.sqrt(case["dim"])
            x = x.masked_fill(hide[:, None], -math.inf)
            lse[b, :, mine] = torch.logsumexp(x, -1)
            out[b, :, mine] = torch.matmul(torch.softmax(x, -1), v)
    return out, lse


def exact_rotation(x, pos, inv_freq, style, sign):
    """Pairs as complex numbers, turned by exp(i * position * frequency)."""
    x = x.double().clone()
    r = 2 * inv_freq.numel()
    turn = torch.polar(torch.ones((), device=DEVICE, dtype=torch.float64), sign * pos.double()[:, None] * inv_freq.double())[:, None]
    if style == "half":
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
        x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
        x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
    return x
