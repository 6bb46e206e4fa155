"""A speculative decoding step over the paged cache, as cases that can be measured.

Three operators, each with its plain form in elementary torch operations and
its definition in 64 bits.  A sequence has committed keys in its pages and a
tree of drafted nodes behind them: node 0 is the last token that is certain,
every other node a guess that follows its parent, and node i's K/V rows sit at
the position of the i-th key past the committed ones.

  tree     attention of every node to the committed keys and to the nodes on
           its way to the root, itself included;
  verify   the walk down the tree: siblings are accepted or rejected against
           the target's probabilities from given random numbers, and where no
           child is left the next token is drawn from what remains;
  commit   the accepted nodes' K/V rows move up behind the committed keys, in
           the pools of all layers, and the rows shrink to them.

Whole numbers (accepted counts, paths, tokens, lengths, page counts) are equal
in all forms; sums and products that decide them are taken in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 16
DIM = 128
LEAST_LEFT = 2.0 ** -24  # a draft row's mass that is left counts as this much at least


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one chat with a small tree: latency counts
        dict(name="tree 1", op="tree", seqs=1, n_min=8, n_max=8, arity=2, ctx_min=300,
             ctx_max=301, hq=12, hkv=2, f32=False, lens=1),
        # a small batch of chats, a usual tree each
        dict(name="tree 8", op="tree", seqs=8, n_min=24, n_max=32, arity=4, ctx_min=128,
             ctx_max=4096, hq=12, hkv=2, f32=False, lens=2),
        # continuous batching: short guesses, contexts of very different lengths
        dict(name="tree 64", op="tree", seqs=64, n_min=1, n_max=8, arity=3, ctx_min=1,
             ctx_max=8192, hq=12, hkv=2, f32=False, lens=3),
        # few long contexts, large trees
        dict(name="tree long 4", op="tree", seqs=4, n_min=60, n_max=64, arity=4, ctx_min=32700,
             ctx_max=32768, hq=32, hkv=8, f32=False, lens=4),
        # chains over long contexts, fp32 rows for a reduction that follows
        dict(name="chain long 6", op="tree", seqs=6, n_min=5, n_max=7, arity=1, ctx_min=9001,
             ctx_max=30001, hq=20, hkv=4, f32=True, lens=5),
        # one chat's tree, a small vocabulary
        dict(name="verify 1", op="verify", seqs=1, n_min=8, n_max=8, arity=2, vocab=32000,
             drafts=True, again=False, lens=6),
        # trees of a small batch, siblings drawn with replacement
        dict(name="verify 16", op="verify", seqs=16, n_min=24, n_max=32, arity=4, vocab=128000,
             drafts=True, again=True, lens=7),
        # a full batch at a large vocabulary
        dict(name="verify 64", op="verify", seqs=64, n_min=6, n_max=8, arity=3, vocab=151936,
             drafts=True, again=False, lens=8),
        # guesses looked up in the prompt: no draft probabilities; an odd vocabulary
        dict(name="verify lookup 32", op="verify", seqs=32, n_min=4, n_max=11, arity=1,
             vocab=50021, drafts=False, again=False, lens=9),
        # eight chats, four layers
        dict(name="commit 8", op="commit", seqs=8, n_min=24, n_max=32, arity=4, ctx_min=900,
             ctx_max=1100, layers=4, hkv=2, lens=10),
        # a full batch, 28 layers
        dict(name="commit 64", op="commit", seqs=64, n_min=20, n_max=32, arity=3, ctx_min=100,
             ctx_max=2000, layers=28, hkv=4, lens=11),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "verify", "commit"])
    hi = _log(rng, 1, 64)
    c = dict(op=op, n_min=max(1, rng.randint(hi // 3, hi)), n_max=hi,
             arity=rng.choice([1, 2, 3, 4, 8]), lens=rng.randrange(1 << 20))
    if op == "verify":
        vocab = _log(rng, 100, 160000)
        seqs = max(1, min(_log(rng, 1, 64), 64 * 8 * 151936 // (hi * vocab)))
        return dict(c, seqs=seqs, vocab=vocab, drafts=rng.random() < 0.75,
                    again=rng.random() < 0.3)
    hkv = rng.choice([1, 2, 4, 8])
    if op == "commit":
        ctx = _log(rng, 64, 2000)
        return dict(c, seqs=_log(rng, 1, 64), ctx_min=_log(rng, 64, ctx), ctx_max=ctx,
                    layers=rng.randint(1, 14), hkv=min(hkv, 4))
    group = rng.randint(1, 8)
    ctx = _log(rng, 1, 32768)
    keys = (ctx + hi) * hkv
    seqs = max(1, min(_log(rng, 1, 64), 1048576 // keys, 268435456 // (keys * group * hi)))
    if keys * group * hi > 268435456:  # a single sequence over the largest listed work
        ctx = 268435456 // (hkv * group * hi) - hi
    return dict(c, seqs=seqs, ctx_min=_log(rng, 1, ctx), ctx_max=ctx, hq=hkv * group, hkv=hkv,
                f32=rng.random() < 0.25)


def _shape(case):
    """What the case alone sets: (committed lengths, node counts, parents of every tree)."""
    r = random.Random(case["lens"])
    nodes = [r.randint(case["n_min"], case["n_max"]) for _ in range(case["seqs"])]
    done = []
    if "ctx_min" in case:
        lo, hi = case["ctx_min"], case["ctx_max"]
        log = hi > 10 * lo
        done = [_log(r, lo, hi) if log else r.randint(lo, hi) for _ in nodes]
        if len(done) > 2 and lo == 1:
            done[0], done[1] = 0, 16
    trees = []
    for n in nodes:
        kids, par = [0] * n, [-1]
        for i in range(1, n):
            free = [j for j in range(i) if kids[j] < case["arity"]]
            # the later nodes are the likelier parents: a tree some levels deep
            j = free[max(r.randrange(len(free)), r.randrange(len(free)))]
            kids[j] += 1
            par.append(j)
        trees.append(par)
    return done, nodes, trees


def _pages(n):
    return (n + BLOCK - 1) // BLOCK


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _tables(g, ctx, num_blocks):
    """Every sequence's pages, drawn from a permutation of the pool."""
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    need = [_pages(n) for n in ctx]
    t = torch.full((len(ctx), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = perm[at:at + k]
        at += k
    return t


def prepare(case, seed):
    g = _gen(seed)
    done, nodes, trees = _shape(case)
    cu = [0]
    for n in nodes:
        cu.append(cu[-1] + n)
    s = dict(op=case["op"], case=case, cu=_i32(cu), parents=_i32(sum(trees, [])),
             max_nodes=max(nodes))
    if case["op"] == "verify":
        _probabilities(s, g, case, nodes, trees)
    else:
        ctx = [a + b for a, b in zip(done, nodes)]
        num_blocks = sum(_pages(n) for n in ctx) + 64
        s["tables"], s["ctx"] = _tables(g, ctx, num_blocks), _i32(ctx)
        lead = (case["layers"],) if case["op"] == "commit" else ()
        for name in ("k", "v"):
            pool = torch.empty(lead + (num_blocks, BLOCK, case["hkv"], DIM), dtype=torch.bfloat16,
                               device="cuda")
            for part in (pool if lead else [pool]):
                part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
            s[name] = pool
    if case["op"] == "tree":
        s["q"] = _rows(g, cu[-1], case["hq"], DIM)
        s["scale"] = 1.0 / math.sqrt(DIM)
        s["out"] = torch.empty(s["q"].shape, device="cuda",
                               dtype=torch.float32 if case["f32"] else torch.bfloat16)
    if case["op"] == "commit":
        _accepted(s, seed, trees)
        held = s["tables"][s["tables"] >= 0].long()
        s["refs"] = torch.zeros(num_blocks, dtype=torch.int32, device="cuda")
        s["refs"][held] = 1
        s["new_ctx"], s["new_refs"] = s["ctx"].clone(), s["refs"].clone()
    if own:
        _handles(s)
    return s


def _probabilities(s, g, case, nodes, trees):
    """A target's and a draft's rows that resemble each other, guesses drawn from the draft's
    rows (siblings without replacement unless the case says so), and the random numbers."""
    total, vocab = sum(nodes), case["vocab"]
    s["p"] = torch.empty((total, vocab), device="cuda")
    s["q"] = torch.empty((total, vocab), device="cuda") if case["drafts"] else None
    s["tokens"] = torch.zeros(total, dtype=torch.int32, device="cuda")
    at = 0
    for n, par in zip(nodes, trees):
        z = torch.randn((n, vocab), generator=g, device="cuda")
        other = torch.randn((n, vocab), generator=g, device="cuda")
        s["p"][at:at + n] = torch.softmax(3.0 * z, -1)
        q = torch.softmax(3.0 * (0.95 * z + 0.31 * other), -1)
        if case["drafts"]:
            s["q"][at:at + n] = q
        most = max(par.count(j) for j in range(n)) if n > 1 else 0
        if most:
            if case["again"] and case["drafts"]:
                picks = torch.multinomial(q, most, replacement=True, generator=g)
            elif case["drafts"]:
                u = torch.rand(q.shape, generator=g, device="cuda").clamp_(min=1e-30)
                picks = torch.topk(torch.log(q) - torch.log(-torch.log(u)), min(most, vocab)).indices
            else:
                picks = torch.topk(q, min(most, vocab)).indices
            nth = [par[:i].count(par[i]) % picks.shape[1] for i in range(1, n)]
            s["tokens"][at + 1:at + n] = picks[par[1:], nth].to(torch.int32)
        at += n
    s["u"] = torch.rand(total, generator=g, device="cuda")
    s["u_last"] = torch.rand(len(nodes), generator=g, device="cuda")


def _accepted(s, seed, trees):
    """Paths as a verification leaves them: from the root down, each a while."""
    r = random.Random(seed)
    path = torch.full((len(trees), s["max_nodes"]), -1, dtype=torch.int32)
    count = []
    for b, par in enumerate(trees):
        way = [0]
        while True:
            kids = [i for i in range(len(par)) if par[i] == way[-1]]
            if not kids or r.random() < 0.2:
                break
            way.append(r.choice(kids))
        path[b, :len(way)] = torch.tensor(way, dtype=torch.int32)
        count.append(len(way))
    s["path"], s["count"] = path.cuda(), _i32(count)


def _handles(s):
    """What a program that uses the framework keeps between calls."""
    from paged_kv_continuous_gb300 import ops
    if s["op"] == "tree":
        s["call"] = ops.DecodeTreeCall(s["q"], s["cu"], s["parents"], s["k"], s["v"], s["tables"],
                                       s["ctx"], s["scale"], s["max_nodes"], s["out"])
    elif s["op"] == "verify":
        s["call"] = ops.VerifyTreeCall(s["tokens"], s["parents"], s["cu"], s["p"], s["u"],
                                       s["u_last"], s["max_nodes"], draft_probs=s["q"],
                                       with_replacement=s["case"]["again"])
    else:
        pools = ops.PagePools([layer for pool in (s["k"], s["v"]) for layer in pool])
        s["call"] = ops.CommitTreeCall(pools, s["cu"], s["tables"], s["new_ctx"], s["path"],
                                       s["count"], ref_counts=s["new_refs"])


# ---- one pass ---------------------------------------------------------------

def run(s):
    if s["op"] == "tree":
        return s["call"]() if own else _plain_tree(s)
    if s["op"] == "verify":
        count, path, tokens = s["call"]() if own else _plain_verify(s)
        return {"accepted": count, "path": path, "tokens": tokens}
    # the lengths and page counts that this step began with
    s["new_ctx"].copy_(s["ctx"])
    s["new_refs"].copy_(s["refs"])
    if own:
        s["call"]()
    else:
        _plain_commit(s)
    return {"k": s["k"], "v": s["v"], "ctx": s["new_ctx"], "refs": s["new_refs"]}


# ---- plain forms ------------------------------------------------------------

def _grid(s):
    """(first node, count) of each tree and its nodes' places in the packed arrays."""
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    j = torch.arange(s["max_nodes"], device="cuda")
    return cu[:-1], n, (cu[:-1, None] + j).clamp(max=max(0, s["parents"].shape[0] - 1))


def _plain_tree(s):
    case, M = s["case"], s["max_nodes"]
    hq, hkv = case["hq"], case["hkv"]
    first, n, at = _grid(s)
    ctx = s["ctx"].long()
    B, L = ctx.shape[0], s["tables"].shape[1] * BLOCK
    j = torch.arange(M, device="cuda")
    there = j < n[:, None]
    # who is on whose way to the root: the parent relation and the identity, squared
    par = torch.where(there, s["parents"].long()[at], -1)
    way = ((par[:, :, None] == j) | (j[:, None] == j)).float()
    for _ in range(max(1, M - 1).bit_length()):
        way = (torch.matmul(way, way) > 0).float()
    key = torch.arange(L, device="cuda")
    node = key[None] - (ctx - n)[:, None]  # of each key; below 0: committed
    on = way.gather(2, node.clamp(0, M - 1)[:, None].expand(B, M, L)) > 0
    seen = (node < 0)[:, None] | (on & (node < n[:, None])[:, None])
    seen &= there[:, :, None]
    pages = s["tables"].clamp(min=0).long()
    dead = (key[None] >= ctx[:, None])[:, :, None, None]
    k = s["k"][pages].reshape(B, L, hkv, DIM).float().masked_fill(dead, 0.0)
    v = s["v"][pages].reshape(B, L, hkv, DIM).float().masked_fill(dead, 0.0)
    q = s["q"][at].float().reshape(B, M, hkv, hq // hkv, DIM).permute(0, 2, 3, 1, 4)
    sc = torch.matmul(q.reshape(B, hkv, -1, DIM), k.permute(0, 2, 3, 1)) * s["scale"]
    sc = sc.reshape(B, hkv, hq // hkv, M, L).masked_fill(~seen[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True).clamp(min=-3.0e38)
    w = torch.exp(sc - top)
    den = w.sum(-1).clamp(min=1e-38)
    o = torch.matmul(w.reshape(B, hkv, -1, L), v.permute(0, 2, 1, 3))
    o = o.reshape(B, hkv, hq // hkv, M, DIM) / den[..., None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, M, hq, DIM)
    row = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.bucketize(row, s["cu"][1:].long(), right=True)
    return o[b, row - first[b]].to(s["out"].dtype)


def _plain_verify(s):
    """All sequences at once.  A node's children come after it and in their order, so one scan
    over the nodes is the walk: a node is tried where its parent is where the walk stands."""
    first, n, _ = _grid(s)
    B, M, dev = n.shape[0], s["max_nodes"], "cuda"
    last = s["parents"].shape[0] - 1
    b = torch.arange(B, device=dev)
    p, q = s["p"], s["q"]
    f64 = dict(dtype=torch.float64, device=dev)
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    count = (n > 0).long()
    path = torch.full((B, M), -1, dtype=torch.long, device=dev)
    path[:, 0] = torch.where(n > 0, 0, -1)
    tokens = torch.full((B, M), -1, dtype=torch.long, device=dev)
    beta, gone, mass = torch.zeros(B, **f64), torch.zeros(B, **f64), torch.ones(B, **f64)
    out = torch.zeros((B, p.shape[1]), dtype=torch.bool, device=dev)  # looked-up guesses rejected
    for j in range(1, M):
        at = (first + j).clamp(max=last)
        row = (first + cur).clamp(max=last)
        kid = (j < n) & (s["parents"].long()[at] == cur)
        tok = s["tokens"].long()[at]
        px, u = p[row, tok].double(), s["u"].double()[at]
        if q is None:
            w = torch.where(out[b, tok], 0.0, px)
            ok = kid & (u * mass < w)
        else:
            qx, left = q[row, tok].double(), (1 - gone).clamp(min=LEAST_LEFT)
            ok = kid & (u * (qx / left) * mass < px - beta * qx)
        no = kid & ~ok
        if q is None:
            mass = torch.where(no, (mass - w).clamp(min=0.0), mass)
            out[b, tok] |= no
            out &= ~ok[:, None]
        else:
            beta = torch.where(no, beta + mass / left, beta)
            if not s["case"]["again"]:
                gone = torch.where(no, gone + qx, gone)
            rest = (p[row].double() - beta[:, None] * q[row].double()).clamp(min=0.0).sum(-1)
            mass = torch.where(no, rest, mass)
        path[b, count.clamp(max=M - 1)] = torch.where(ok, j, path[b, count.clamp(max=M - 1)])
        tokens[b, (count - 1).clamp(min=0)] = torch.where(ok, tok, tokens[b, (count - 1).clamp(min=0)])
        count += ok
        cur = torch.where(ok, j, cur)
        beta, gone = torch.where(ok, 0.0, beta), torch.where(ok, 0.0, gone)
        mass = torch.where(ok, 1.0, mass)
    row = (first + cur).clamp(max=last)
    w = p[row].double()
    if q is None:
        w = w.masked_fill(out, 0.0)
    else:
        w = (w - beta[:, None] * q[row].double()).clamp(min=0.0)
    # nothing left, by rounding alone: the target's row itself
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p[row].double())
    upto = torch.cumsum(w, -1)
    pick = (upto <= s["u_last"].double()[:, None] * upto[:, -1:]).sum(-1)
    ids = torch.arange(w.shape[1], device=dev)
    pick = torch.minimum(pick, torch.where(w > 0, ids, 0).amax(-1))
    tokens[b, (count - 1).clamp(min=0)] = torch.where(n > 0, pick, -1)
    return count.to(torch.int32), path.to(torch.int32), tokens.to(torch.int32)


def _plain_commit(s):
    first, n, _ = _grid(s)
    ctx, count = s["new_ctx"].long(), s["count"].long()
    done = (ctx - n)[:, None]
    i = torch.arange(s["path"].shape[1], device="cuda")[None]
    move = i < count[:, None]
    src, dst = done + s["path"].long(), done + i
    t = s["tables"].long()
    b = torch.arange(t.shape[0], device="cuda")[:, None].expand_as(src)[move]
    src, dst = src[move], dst.expand_as(move)[move]
    for pool in (s["k"], s["v"]):
        rows = pool[:, t[b, src // BLOCK], src % BLOCK]
        pool[:, t[b, dst // BLOCK], dst % BLOCK] = rows
    new = done[:, 0] + count
    e = torch.arange(t.shape[1], device="cuda")[None]
    drop = (e >= ((new + BLOCK - 1) // BLOCK)[:, None]) & (e < ((ctx + BLOCK - 1) // BLOCK)[:, None])
    s["new_refs"].scatter_add_(0, t.clamp(min=0).reshape(-1), -drop.reshape(-1).to(torch.int32))
    s["new_ctx"].copy_(new.to(torch.int32))


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    done, nodes, trees = _shape(case)
    total = sum(nodes)
    if case["op"] == "tree":
        hq, hkv = case["hq"], case["hkv"]
        kv = sum((a + n) * hkv * DIM * 4 + _pages(a + n) * 4 for a, n in zip(done, nodes))
        seen = 0
        for a, par in zip(done, trees):
            deep = []
            for j in par:
                deep.append(1 if j < 0 else deep[j] + 1)
            seen += a * len(par) + sum(deep)
        row = total * hq * DIM * (2 + (4 if case["f32"] else 2))
        return {"bytes": kv + row + 4 * total, "flops": 4.0 * DIM * hq * seen}
    if case["op"] == "verify":
        # the rows of the node where the walk ends, at the least: the token drawn there depends on
        # all of its target's row (and its draft's, once a child was rejected)
        rows = case["seqs"] * case["vocab"] * 4
        return {"bytes": rows * (2 if case["drafts"] else 1) + 12 * total, "flops": 3.0 * rows / 4}
    # every accepted node behind the root, all but those in place already (at most)
    deep = [max(1, min(len(par), 4)) for par in trees]
    moves = sum(deep) - len(deep)
    return {"bytes": 2 * moves * case["hkv"] * DIM * 2 * 2 * case["layers"] + 12 * total, "flops": 0}


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_tree(s):
    case = s["case"]
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    cu, ctx, parents = s["cu"].tolist(), s["ctx"].tolist(), s["parents"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(ctx):
        a, e = cu[b], cu[b + 1]
        hidden = torch.ones((e - a, n), dtype=torch.bool)
        hidden[:, :n - (e - a)] = False
        for i in range(e - a):
            j = i
            while j >= 0:
                hidden[i, n - (e - a) + j] = False
                j = parents[a + j]
        hidden = hidden.cuda()
        pages = s["tables"][b, :_pages(n)].long()
        for h in range(hkv):
            kh = s["k"][pages, :, h].reshape(-1, DIM)[:n].double()
            vh = s["v"][pages, :, h].reshape(-1, DIM)[:n].double()
            for x in range(h * g, (h + 1) * g):
                sc = (s["q"][a:e, x].double() @ kh.T) * s["scale"]
                out[a:e, x] = torch.softmax(sc.masked_fill(hidden, -math.inf), -1) @ vh
    return out


def _exact_verify(s):
    """One sequence after the other, by the distributions themselves."""
    cu, par, tok = s["cu"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    u, u_last = s["u"].double().tolist(), s["u_last"].double().tolist()
    B, M = len(cu) - 1, s["max_nodes"]
    count = [0] * B
    path = [[-1] * M for _ in range(B)]
    tokens = [[-1] * M for _ in range(B)]
    for b in range(B):
        a, n = cu[b], cu[b + 1] - cu[b]
        if not n:
            continue
        way, node = [0], 0
        while True:
            target = s["p"][a + node].double()
            drawn, gone, mass = None, 0.0, 1.0
            if s["q"] is not None:
                drawn = s["q"][a + node].double()
            found = None
            for i in range(node + 1, n):
                if par[a + i] != node:
                    continue
                x = tok[a + i]
                if drawn is None:
                    # a guess without probabilities stands for itself alone
                    if u[a + i] * mass < float(target[x]):
                        found = i
                        break
                    mass = max(0.0, mass - float(target[x]))
                    target[x] = 0.0
                    continue
                now = drawn / max(1.0 - gone, LEAST_LEFT)
                if u[a + i] * float(now[x]) < float(target[x]):
                    found = i
                    break
                rest = torch.relu(target - now)
                if not float(rest.sum()) > 0:
                    target = s["p"][a + node].double()
                    break
                target = rest / rest.sum()
                if not s["case"]["again"]:
                    gone += float(s["q"][a + node, x])
            if found is None:
                break
            tokens[b][len(way) - 1] = tok[a + found]
            way.append(found)
            node = found
        upto = torch.cumsum(target, 0)
        pick = int(torch.searchsorted(upto, u_last[b] * upto[-1:], right=True))
        tokens[b][len(way) - 1] = min(pick, int(torch.nonzero(target)[-1]))
        path[b][:len(way)] = way
        count[b] = len(way)
    return {"accepted": _i32(count), "path": _i32(path), "tokens": _i32(tokens)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "verify":
        return _exact_verify(s)
    return None  # whole numbers and moved rows: no computed values
