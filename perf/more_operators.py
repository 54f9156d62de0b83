"""Timed cases of the operators around drafted tokens and the paged cache.

Seven kinds of case, each with a plain form (elementary torch operations) and
the calls a user makes of the framework:

    rotate        bsp.bsp_rotary: rotary positions of Q and K before attention
    rotate_train  bsp.rotary and its gradient; returns both outputs and both gradients
    tree          bsp.bsp_draft_tree and bsp.bsp_paged_tree_attention: a ragged batch of trees of
                  drafted tokens over the cache; returns positions, the trees' bits, O, log-sum-exp
    verify        bsp.bsp_draft_verify: drafted tokens against the target's probabilities; returns
                  the accepted nodes, their number and the next token of each sequence
    keep          bsp.bsp_paged_append and bsp.bsp_paged_keep: the trees' rows into the cache, then
                  the accepted ones next to each other; returns both caches
    turn          bsp.bsp_pages_free, bsp_pages_fork, bsp_pages_reserve, bsp_paged_copy: a turn of a
                  search over beams; returns the bookkeeping, the pairs of pages and both caches
    compact       bsp.bsp_pages_compact and bsp.bsp_paged_copy: the pages in use to the front

A tree's node 0 is the sequence's last known token, parent[0] = -1; the nodes
stand at the last n positions of the sequence.  Node i sees node a when a is i
or one of its ancestors; its position is that of the first node plus its depth.
"""

import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # positions of a serving batch's next tokens, far into long contexts: latency
        dict(name="rotate_decode", kind="rotate", Z=1, S=64, Hq=32, Hkv=8, D=128, rot=128, pairs=False, rows_first=True,
             far=1000000, scaling="parts", factor=16.0, amplitude=1.2772588722239782, dtype="bf16"),
        # a batch of long prompts in full precision, a quarter of the head rotated
        dict(name="rotate_prompt", kind="rotate", Z=2, S=4099, Hq=12, Hkv=12, D=80, rot=20, pairs=True, rows_first=False,
             far=0, scaling="none", factor=1.0, amplitude=1.0, dtype="f32"),
        # a training step's positions, projections' own order, shared KV heads
        dict(name="rotate_train", kind="rotate_train", Z=4, S=8192, Hq=32, Hkv=8, D=128, rot=128, pairs=False,
             rows_first=True, far=0, scaling="linear", factor=4.0, amplitude=1.0, dtype="bf16"),
        # one user's drafted tokens: latency
        dict(name="tree_one", kind="tree", nodes="13", kv="1013", Hq=16, Hkv=4, D=128, page=16, window=0, sinks=0,
             dtype="f16"),
        # drafted trees of a serving batch over ragged histories: the cache's bandwidth
        dict(name="tree_batch", kind="tree", nodes=_spread(64, 12, 32, 5), kv=_spread(64, 2048, 8192, 6), Hq=32, Hkv=8,
             D=128, page=64, window=0, sinks=0, dtype="bf16"),
        # wide trees in full precision, window and sinks, a head size between the powers of two
        dict(name="tree_f32", kind="tree", nodes=_spread(16, 5, 70, 7), kv=_spread(16, 300, 6000, 8), Hq=6, Hkv=2, D=80,
             page=32, window=1024, sinks=4, dtype="f32"),
        # one user's chain of four drafted tokens: latency
        dict(name="verify_one", kind="verify", nodes="5", V=32000, branch=1, drawn=True, dtype="f32"),
        # chains of a serving batch, a large vocabulary
        dict(name="verify_chain", kind="verify", nodes=_text([8] * 64), V=128000, branch=1, drawn=True, dtype="f32"),
        # trees whose children are the draft's likeliest tokens, an odd vocabulary
        dict(name="verify_tree", kind="verify", nodes=_spread(32, 10, 40, 9), V=50001, branch=3, drawn=False, dtype="bf16"),
        # a serving batch's drafted rows in, the accepted ones kept
        dict(name="keep_batch", kind="keep", nodes=_spread(64, 12, 32, 5), kv=_spread(64, 1000, 4000, 10), Hkv=8, D=128,
             page=64, dtype="bf16"),
        # a turn of 24 searches of 4 beams each
        dict(name="turn_beams", kind="turn", searches=24, beams=4, kv=_spread(24, 300, 3000, 11), grow=64, Hkv=8, D=128,
             page=64, dtype="bf16"),
        # a cache of many short sequences, a third of its pages free here and there
        dict(name="compact_cache", kind="compact", n_pages=4999, used=0.66, n_seq=200, Hkv=8, D=128, page=32, dtype="bf16"),
    ]


def _spread(n, lo, hi, seed):
    """n whole numbers between lo and hi, spread over their logarithm."""
    r = random.Random(seed)
    return _text(_log_int(r, lo, hi) for _ in range(n))


def _text(numbers):
    """The sequences' numbers as a case holds them: one text."""
    return " ".join(str(n) for n in numbers)


def _ints(text):
    return [int(n) for n in text.split()]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["kind"], (0, 0))
        most[c["kind"]] = max(b, w["bytes"]), max(f, w["flops"])
    while True:
        kind = rng.choice(("rotate", "rotate_train", "tree", "tree", "tree", "verify", "verify", "keep", "turn", "compact"))
        dtype = rng.choice(("bf16", "bf16", "f16", "f16", "f32"))
        D = rng.choice((16, 32, 48, 64, 64, 80, 96, 112, 128, 128, 128))
        Hkv = rng.choice((1, 2, 3, 4, 8, 16))
        page = rng.choice((16, 32, 64, 128))
        if kind in ("rotate", "rotate_train"):
            scaling = rng.choice(("none", "linear", "base", "parts"))
            factor = 1.0 if scaling == "none" else rng.choice((2.0, 4.0, 7.5))
            case = dict(kind=kind, Z=rng.choice((1, 1, 2, 3)), S=_log_int(rng, 1, 16384),
                        Hq=Hkv * rng.choice((1, 1, 2, 3, 4, 5, 8)), Hkv=Hkv, D=D,
                        rot=rng.choice((D, D, D // 2, D // 4 // 2 * 2, 2 * rng.randint(2, D // 2))), pairs=rng.random() < 0.5,
                        rows_first=rng.random() < 0.5, far=rng.choice((0, 0, _log_int(rng, 1000, 10000000))),
                        scaling=scaling, factor=factor,
                        amplitude=0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0, dtype=dtype)
        elif kind == "verify":
            n, wide = _log_int(rng, 1, 64), rng.choice((4, 9, 20, 40))
            case = dict(kind=kind, nodes=_text(rng.randint(1, wide) for _ in range(n)), V=_log_int(rng, 1000, 160000),
                        branch=rng.choice((1, 1, 2, 3, 5)), drawn=rng.random() < 0.6, dtype=dtype)
            if sum(_ints(case["nodes"])) * case["V"] > 8 * 64 * 128000:
                continue
        elif kind == "compact":
            case = dict(kind=kind, n_pages=_log_int(rng, 20, 8000), used=rng.choice((0.1, 0.4, 0.5, 0.66, 0.9)),
                        n_seq=_log_int(rng, 1, 300), Hkv=Hkv, D=D, page=page, dtype=dtype)
        elif kind == "turn":
            n = _log_int(rng, 1, 64)
            case = dict(kind=kind, searches=n, beams=rng.randint(1, 8), kv=_text(_log_int(rng, 1, 4000) for _ in range(n)),
                        grow=_log_int(rng, 1, 400), Hkv=Hkv, D=D, page=page, dtype=dtype)
        else:
            n, wide = _log_int(rng, 1, 64), rng.choice((3, 9, 30, 90))
            nodes = [rng.randint(1, wide) for _ in range(n)]
            case = dict(kind=kind, nodes=_text(nodes), kv=_text(q + _log_int(rng, 1, 16384) - 1 for q in nodes), Hkv=Hkv, D=D,
                        page=page, dtype=dtype)
            if kind == "tree":
                case.update(Hq=Hkv * rng.choice((1, 1, 2, 3, 4, 5, 8)), window=rng.choice((0, 0, _log_int(rng, 16, 4096))),
                            sinks=rng.choice((0, 4, 40)))
        w = work(case)
        limit = most[kind]
        if kind == "tree" and dtype == "f32":  # on the CUDA cores: the fp32 listed case bounds it
            f32 = work(next(c for c in listed() if c["name"] == "tree_f32"))
            limit = 4 * f32["bytes"], 4 * f32["flops"]
        if w["bytes"] <= limit[0] and w["flops"] <= limit[1]:
            return case


# ------------------------------------------------------------------ work --

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    kind = case["kind"]
    if kind in ("rotate", "rotate_train"):
        x = case["Z"] * case["S"] * (case["Hq"] + case["Hkv"])
        times = 2 if kind == "rotate_train" else 1
        return {"bytes": times * 2 * e * x * case["D"], "flops": times * 3 * x * case["rot"]}
    if kind == "verify":
        # one of the target's rows and, where tokens are drawn from it, one of the draft's
        rows = len(_ints(case["nodes"])) * (2 if case["drawn"] else 1)
        return {"bytes": e * rows * case["V"], "flops": 2 * rows * case["V"]}
    if kind == "compact":
        live = int(case["used"] * case["n_pages"])
        moved = int(live * (1 - case["used"]))
        return {"bytes": 4 * e * moved * case["page"] * case["Hkv"] * case["D"] + 12 * case["n_pages"], "flops": 0}
    if kind == "turn":
        pages = case["searches"] * (case["beams"] - 1)
        return {"bytes": 4 * e * pages * case["page"] * case["Hkv"] * case["D"] + 4 * case["searches"] * case["beams"],
                "flops": 0}
    nodes, kvs = _ints(case["nodes"]), _ints(case["kv"])
    D, Hkv, T = case["D"], case["Hkv"], sum(nodes)
    if kind == "keep":
        return {"bytes": 4 * e * T * Hkv * D, "flops": 0}
    Hq, pairs, keys = case["Hq"], 0, 0
    for n, kv in zip(nodes, kvs):
        ctx = kv - n
        near = min(ctx, case["window"]) if case["window"] else ctx
        seen = near + min(ctx - near, case["sinks"])
        keys += seen + n
        pairs += n * (seen + min(n, 4))  # of the tree, a few ancestors each
    return {"bytes": e * (2 * T * Hq * D + 2 * keys * Hkv * D) + 4 * T * Hq, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- inputs --

def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    R, f = case["rot"], case["factor"]
    i = np.arange(R // 2, dtype=np.float64)
    base = 10000.0
    if case["scaling"] == "base" and R > 2:
        base *= f ** (R / (R - 2))
    w = base ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "parts":
        # pairs that turn often over the original 4096 positions keep their frequency
        turns = 4096 * w / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        w = w * keep + w / f * (1 - keep)
    return w


def _parents(n, branch, r):
    """Parents of a tree's nodes: node 0 the root, the others below recent nodes with room."""
    out, kids = [-1], [0]
    for i in range(1, n):
        room = [a for a in range(i) if kids[a] < branch][-6:]
        a = r.choice(room) if branch > 1 else i - 1
        out.append(a)
        kids.append(0)
        kids[a] += 1
    return out


def _path(parent, r):
    """A root-to-somewhere path through the tree."""
    path = [0]
    while True:
        kids = [i for i, a in enumerate(parent) if a == path[-1]]
        if not kids or r.random() < 0.2:
            return path
        path.append(r.choice(kids))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    r = random.Random(seed * 7919 + 5)
    dt = _DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def starts(n):
        return ints([sum(n[:i]) for i in range(len(n) + 1)])

    def pages(kvs, spare):
        """Pages of a ragged batch in random order."""
        used = [-(-kv // case["page"]) for kv in kvs]
        order = list(range(sum(used) + spare))
        r.shuffle(order)
        table = torch.zeros(len(used), max(used), dtype=torch.int32)
        at = 0
        for i, n in enumerate(used):
            table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        return sum(used) + spare, table.cuda()

    def caches(n):
        return dict(k_cache=randn(n, case["Hkv"], case["page"], case["D"]), v_cache=randn(n, case["Hkv"], case["page"], case["D"]))

    kind, s = case["kind"], dict(case=case)
    if kind in ("rotate", "rotate_train"):
        def heads(H):
            if case["rows_first"]:  # as a projection leaves them
                return randn(case["Z"], case["S"], H, case["D"]).transpose(1, 2)
            return randn(case["Z"], H, case["S"], case["D"])

        s.update(q=heads(case["Hq"]), k=heads(case["Hkv"]))
        first = torch.tensor([r.randrange(case["far"] + 1) for _ in range(case["Z"] * case["S"])]) if kind == "rotate" and \
            case["far"] else torch.arange(case["S"]).repeat(case["Z"]) + case["far"]
        s["pos"] = first.to(torch.int32).view(case["Z"], case["S"]).cuda()
        if kind == "rotate_train":
            s.update(dq=heads(case["Hq"]), dk=heads(case["Hkv"]))
            if own:
                s["q"].requires_grad_()
                s["k"].requires_grad_()
        s["freq"] = _frequencies(case)
    elif kind in ("tree", "keep"):
        nodes, kvs = _ints(case["nodes"]), _ints(case["kv"])
        T = sum(nodes)
        trees = [_parents(n, 3, r) for n in nodes]
        n_pages, table = pages(kvs, 3)
        s.update(caches(n_pages), table=table, q_start=starts(nodes), kv_len=ints(kvs),
                 parent=ints([p for t in trees for p in t]))
        if kind == "tree":
            s.update(q=randn(T, case["Hq"], case["D"]), scale=1.0 / math.sqrt(case["D"]))
        else:
            paths = [_path(t, r) for t in trees]
            s.update(k_new=randn(T, case["Hkv"], case["D"]), v_new=randn(T, case["Hkv"], case["D"]),
                     path=ints([x for p, n in zip(paths, nodes) for x in p + [-1] * (n - len(p))]),
                     count=ints([len(p) for p in paths]))
    elif kind == "verify":
        nodes, V = _ints(case["nodes"]), case["V"]
        T = sum(nodes)
        first = [sum(nodes[:i]) for i in range(len(nodes))]
        trees = [_parents(n, case["branch"], r) for n in nodes]
        logits = torch.randn(T, V, generator=g, device="cuda").mul_(3.0)
        s["target"] = torch.softmax(logits, -1).to(dt)
        draft = torch.softmax(logits.add_(torch.randn(T, V, generator=g, device="cuda"), alpha=0.8), -1).to(dt)
        # each node's token is of its parent's row of the draft: drawn, or its likeliest by rank among siblings
        row = [f + max(a, 0) for f, t in zip(first, trees) for a in t]
        rank = [t[:i].count(a) for t in trees for i, a in enumerate(t)]
        if case["drawn"]:
            tokens = torch.empty(T, dtype=torch.int64, device="cuda")
            for a in range(0, T, 64):
                tokens[a:a + 64] = torch.multinomial(draft[row[a:a + 64]].float(), 1, generator=g)[:, 0]
        else:
            top = torch.topk(draft.float(), max(rank) + 1, dim=-1).indices
            tokens = top[torch.tensor(row).cuda(), torch.tensor(rank).cuda()]
        s.update(draft=draft if case["drawn"] else None, tokens=tokens.to(torch.int32), q_start=starts(nodes),
                 parent=ints([p for t in trees for p in t]), accept=torch.rand(T, generator=g, device="cuda"),
                 sample=torch.rand(len(nodes), generator=g, device="cuda"))
    elif kind == "turn":
        # beam 0 of each search goes on, and beams 1.. fork off an earlier one
        page, beams, lens = case["page"], case["beams"], _ints(case["kv"])
        n_seq = case["searches"] * beams
        kvs = [kv for kv in lens for _ in range(beams)]
        most = max(-(-(kv + case["grow"]) // page) for kv in lens) + 1
        n_pages, table = pages(kvs, n_seq * (case["grow"] // page + 2))
        full = torch.full((n_seq, most), -1, dtype=torch.int32)
        table = table.cpu()
        for i, kv in enumerate(kvs):
            full[i, :-(-kv // page)] = table[i, :-(-kv // page)]
        refs = torch.bincount(full[full >= 0].long(), minlength=n_pages).to(torch.int32)
        parent = [b * beams + (0 if j == 0 else r.choice((0, 0, j))) for b in range(case["searches"]) for j in range(beams)]
        s.update(caches(n_pages), table=full.cuda(), refs=refs.cuda(), kv_len=ints(kvs), parent=ints(parent),
                 want=ints([kv + case["grow"] for kv in kvs]))
    else:
        n_pages, n_seq = case["n_pages"], case["n_seq"]
        live = int(case["used"] * n_pages)
        order = list(range(n_pages))
        r.shuffle(order)
        sizes = random.Random(n_pages)  # the sequences' lengths are the case's own
        cut = sorted(sizes.randint(0, live) for _ in range(n_seq - 1))
        cut = [0] + cut + [live]
        table = torch.full((n_seq, max(b - a for a, b in zip(cut, cut[1:])) or 1), -1, dtype=torch.int32)
        for i, (a, b) in enumerate(zip(cut, cut[1:])):
            table[i, :b - a] = torch.tensor(order[a:b], dtype=torch.int32)
        refs = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
        s.update(caches(n_pages), table=table.cuda(), refs=refs.cuda())
    if own:
        from sparse_attention_layout_gb300 import bsp
        if kind in ("rotate", "rotate_train"):
            s["R"] = bsp.bsp_rotary_create(s["freq"], amplitude=case["amplitude"], interleaved=case["pairs"])
        else:
            s["W"] = bsp.bsp_window_create(window=case.get("window", 0), sinks=case.get("sinks", 0))
    return s


def run(state):
    kind = state["case"]["kind"]
    if not own:
        return {"rotate": _plain_rotate, "rotate_train": _plain_rotate_train, "tree": _plain_tree, "verify": _plain_verify,
                "keep": _plain_keep, "turn": _plain_turn, "compact": _plain_compact}[kind](state)
    from sparse_attention_layout_gb300 import bsp
    s = state
    c = s["case"]
    if kind == "rotate":
        return bsp.bsp_rotary(s["R"], s["q"], s["k"], s["pos"])
    if kind == "rotate_train":
        q, k = bsp.rotary(s["R"], s["q"], s["k"], s["pos"])
        return (q.detach(), k.detach(), *torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"])))
    if kind == "tree":
        pos, bits = bsp.bsp_draft_tree(s["W"], s["q_start"], s["kv_len"], s["parent"], max(_ints(c["nodes"])))
        return (pos, bits, *bsp.bsp_paged_tree_attention(s["W"], s["q"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_len"],
                                                         s["table"], pos, bits, scale=s["scale"]))
    if kind == "verify":
        return bsp.bsp_draft_verify(s["W"], s["target"], s["draft"], s["tokens"], s["q_start"], s["parent"], s["accept"],
                                    s["sample"])
    if kind == "keep":
        bsp.bsp_paged_append(s["W"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_len"], s["table"])
        bsp.bsp_paged_keep(s["W"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_len"], s["table"], s["path"], s["count"])
        return s["k_cache"], s["v_cache"]
    if kind == "turn":
        bsp.bsp_pages_free(s["W"], s["refs"], s["table"], s["kv_len"], c["page"])
        bsp.bsp_pages_fork(s["W"], s["refs"], s["table"], s["kv_len"], s["parent"], c["page"])
        src, dst = bsp.bsp_pages_reserve(s["W"], s["refs"], s["table"], s["kv_len"], s["want"], c["page"])
        bsp.bsp_paged_copy(s["W"], s["k_cache"], s["v_cache"], src, dst)
        return s["refs"], s["table"], s["kv_len"], src, dst, s["k_cache"], s["v_cache"]
    refs, table, src, dst = bsp.bsp_pages_compact(s["W"], s["refs"], s["table"])
    bsp.bsp_paged_copy(s["W"], s["k_cache"], s["v_cache"], src, dst)
    return refs, table, src, dst, s["k_cache"], s["v_cache"]


# ------------------------------------------------------------ plain forms --

def _plain_turned(x, s, back=False):
    """Rotated x [Z, H, S, D]: angles in 64 bits, products in 32."""
    c = s["case"]
    R = c["rot"]
    phi = s["pos"].double()[:, None, :, None] * torch.from_numpy(s["freq"]).cuda()
    cos, sin = (torch.cos(phi) * c["amplitude"]).float(), (torch.sin(phi) * c["amplitude"]).float()
    if back:
        sin = -sin
    y = x.float().clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if c["pairs"] else (slice(0, R // 2), slice(R // 2, R))
    xa, xb = x[..., a].float(), x[..., b].float()
    y[..., a] = xa * cos - xb * sin
    y[..., b] = xb * cos + xa * sin
    out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    out.copy_(y)
    return out


def _plain_rotate(s):
    return _plain_turned(s["q"], s), _plain_turned(s["k"], s)


def _plain_rotate_train(s):
    return (*_plain_rotate(s), _plain_turned(s["dq"], s, True), _plain_turned(s["dk"], s, True))


def _sequences(s):
    """(first row, nodes, parents) of each sequence's tree."""
    at, out = 0, []
    parent = s["parent"].tolist()
    for n in _ints(s["case"]["nodes"]):
        out.append((at, n, parent[at:at + n]))
        at += n
    return out


def _slots(s, i, positions):
    """Pages and slots of key positions of sequence i."""
    page = s["case"]["page"]
    return s["table"][i][positions // page].long(), positions % page


def _plain_tree(s):
    c = s["case"]
    q = s["q"]
    G = c["Hq"] // c["Hkv"]
    T = q.shape[0]
    words = -(-max(_ints(c["nodes"])) // 32)
    O, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    pos, bits = torch.empty(T, dtype=torch.int32), torch.zeros(T, words, dtype=torch.int64)
    for i, ((t, n, parent), kv) in enumerate(zip(_sequences(s), _ints(c["kv"]))):
        ctx = kv - n
        tree = torch.zeros(n, n, dtype=torch.bool)
        depth = [0] * n
        for a in range(n):
            if parent[a] >= 0:
                depth[a] = depth[parent[a]] + 1
                tree[a] = tree[parent[a]]
            tree[a, a] = True
        depth = torch.tensor(depth)
        if c["window"]:
            tree &= (depth[:, None] - depth[None, :] < c["window"]) | (ctx + depth[None, :] < c["sinks"])
        pos[t:t + n] = (ctx + depth).int()
        for w in range(words):
            some = tree[:, 32 * w:32 * w + 32].long()
            bits[t:t + n, w] = (some << torch.arange(some.shape[1])).sum(-1)
        p = (ctx + depth).cuda()[:, None]
        j = torch.arange(ctx, device=q.device)[None, :]
        keep = torch.ones(n, ctx, dtype=torch.bool, device=q.device)
        if c["window"]:
            keep = (p - j < c["window"]) | (j < c["sinks"])
        keep = torch.cat([keep, tree.cuda()], 1)
        pg, sl = _slots(s, i, torch.arange(kv, device=q.device))
        kf, vf = s["k_cache"][pg, :, sl].float(), s["v_cache"][pg, :, sl].float()  # [kv, Hkv, D]
        for h in range(c["Hkv"]):
            hs = slice(h * G, (h + 1) * G)
            x = (q[t:t + n, hs].float().transpose(0, 1) @ kf[:, h].T) * s["scale"]
            x = x.masked_fill(~keep, -math.inf)
            m = x.amax(-1, keepdim=True)
            e = torch.exp(x - m)
            l = e.sum(-1, keepdim=True)
            O[t:t + n, hs] = ((e / l) @ vf[:, h]).transpose(0, 1).to(q.dtype)
            lse[t:t + n, hs] = (m + torch.log(l))[..., 0].transpose(0, 1)
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits)
    return pos.cuda(), bits.to(torch.int32).cuda(), O, lse


def _plain_verify(s):
    """Sums in 64 bits: a token is chosen by the border that its number falls next to."""
    target, draft, tokens = s["target"], s["draft"], s["tokens"].long()
    trees = _sequences(s)
    row = torch.tensor([t + max(a, 0) for t, _, parent in trees for a in parent]).cuda()
    px = target[row, tokens].double().tolist()
    qx = draft[row, tokens].double().tolist() if draft is not None else [1.0] * len(px)
    accept, tok = s["accept"].double().tolist(), tokens.tolist()
    path = torch.full((tokens.shape[0],), -1, dtype=torch.int32)
    count, nxt = [], []
    for i, (t, n, parent) in enumerate(trees):
        node, taken = 0, [0]
        while True:
            kids = [a for a in range(node + 1, n) if parent[a] == node]
            r, mass, chosen = None, 1.0, -1
            for a in kids:
                have = px[t + a] if r is None else r[tok[t + a]].item()
                if accept[t + a] * qx[t + a] * mass < have:
                    chosen = a
                    break
                if r is None:
                    r = target[t + node].double()
                if draft is not None:
                    r = torch.clamp(r - mass * draft[t + node].double(), min=0.0)
                else:
                    r = r.clone()
                    r[tok[t + a]] = 0.0
                mass = r.sum().item()
            if chosen < 0:
                break
            node = chosen
            taken.append(node)
        if r is None or mass <= 0.0:
            r = target[t + node].double()
        total = torch.cumsum(r, 0)
        above = total > s["sample"][i].double() * total[-1]
        nxt.append(int(torch.argmax(above.int()).item()))
        path[t:t + len(taken)] = torch.tensor(taken, dtype=torch.int32)
        count.append(len(taken))
    return path.cuda(), torch.tensor(count, dtype=torch.int32).cuda(), torch.tensor(nxt, dtype=torch.int32).cuda()


def _plain_keep(s):
    c = s["case"]
    count = s["count"].tolist()
    for i, ((t, n, _), kv) in enumerate(zip(_sequences(s), _ints(c["kv"]))):
        pg, sl = _slots(s, i, torch.arange(kv - n, kv, device="cuda"))
        took = s["path"][t:t + count[i]].long()
        for cache, new in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])):
            cache[pg, :, sl] = new[t:t + n]
            cache[pg[:count[i]], :, sl[:count[i]]] = cache[pg[took], :, sl[took]]
    return s["k_cache"], s["v_cache"]


def _plain_moved(s, src, dst):
    on = src >= 0
    for cache in (s["k_cache"], s["v_cache"]):
        cache[dst[on].long()] = cache[src[on].long()]


def _plain_turn(s):
    page = s["case"]["page"]
    refs, table, kv_len = s["refs"], s["table"], s["kv_len"]
    n_seq, most = table.shape
    j = torch.arange(most, device="cuda")[None, :]

    def let_go(which):
        refs.index_add_(0, table[which].long(), torch.full((int(which.sum()),), -1, dtype=torch.int32, device="cuda"))

    # pages behind the sequences' ends
    held = (kv_len[:, None] + page - 1) // page
    behind = (j >= held) & (table >= 0)
    let_go(behind)
    table[behind] = -1
    # forks share their parents' pages
    parent = s["parent"].long()
    other = parent != torch.arange(n_seq, device="cuda")
    rows = table[parent].masked_fill(j >= held[parent], -1)
    let_go(other[:, None] & (table >= 0))
    table[other] = rows[other]
    kv_len.copy_(kv_len[parent])
    new = table[other[:, None] & (table >= 0)].long()
    refs.index_add_(0, new, torch.ones(len(new), dtype=torch.int32, device="cuda"))
    # pages of the positions to be written: missing ones, and copies of shared ones
    write = (j >= kv_len[:, None] // page) & (j < (s["want"][:, None] + page - 1) // page)
    have = write & (table >= 0)
    item = torch.arange(n_seq * most, device="cuda").view(n_seq, most)
    users = torch.bincount(table[have].long(), minlength=len(refs))
    first = torch.full((len(refs),), n_seq * most, device="cuda").scatter_reduce_(0, table[have].long(), item[have], "amin")
    at = table.clamp(min=0).long()
    keeps = (users[at] == refs[at]) & (first[at] == item)
    leave = have & (refs[at] > 1) & ~keeps
    need = leave | (write & (table < 0))
    let_go(leave)
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    old = table.clone()
    table[need] = free[:int(need.sum())]
    refs[table[need].long()] = 1
    copied = leave & (j == kv_len[:, None] // page) & (kv_len[:, None] % page != 0)
    src = torch.where(copied, old, -1).amax(-1).to(torch.int32)
    dst = torch.where(copied, table, -1).amax(-1).to(torch.int32)
    _plain_moved(s, src, dst)
    return refs, table, kv_len, src, dst, s["k_cache"], s["v_cache"]


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    n = len(refs)
    used = refs > 0
    live = int(used.sum())
    high = torch.nonzero(used[live:])[:, 0] + live
    low = torch.nonzero(~used[:live])[:, 0]
    src, dst = (torch.full((n // 2,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    src[:len(high)], dst[:len(low)] = high.int(), low.int()
    place = torch.arange(n, device="cuda", dtype=torch.int32)
    place[high] = low.int()
    moved = torch.where(table >= 0, place[table.clamp(min=0).long()], table)
    counts = refs.clone()
    counts[low], counts[high] = refs[high], 0
    _plain_moved(s, src, dst)
    return counts, moved, src, dst, s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------ exact --
# The definitions in 64 bits: rotations as products of complex numbers, trees
# and tables walked one entry at a time on the host.

def _exact_rotate(x, s, sign):
    c = s["case"]
    R = c["rot"]
    x = x.detach().double()
    angle = s["pos"].double().unsqueeze(-1) * torch.as_tensor(s["freq"], device="cuda") * sign
    turn = torch.polar(torch.full_like(angle, c["amplitude"]), angle)[:, None]
    head = x[..., :R]
    z = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) if c["pairs"] else \
        torch.complex(head[..., :R // 2].contiguous(), head[..., R // 2:].contiguous())
    z = z * turn
    head = torch.stack([z.real, z.imag], -1).flatten(-2) if c["pairs"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x[..., R:]], -1)


def _exact_tree(s):
    c = s["case"]
    G, D, page = c["Hq"] // c["Hkv"], c["D"], c["page"]
    table, flat = s["table"].tolist(), {}
    for name in ("k_cache", "v_cache"):
        flat[name] = s[name].transpose(1, 2).reshape(-1, c["Hkv"], D)
    O = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i, ((t, n, parent), kv) in enumerate(zip(_sequences(s), _ints(c["kv"]))):
        ctx = kv - n
        at = torch.tensor([table[i][x // page] * page + x % page for x in range(kv)], device="cuda")
        k, v = flat["k_cache"][at].double(), flat["v_cache"][at].double()
        for a in range(n):
            line = [a]  # the node and its ancestors, upwards
            while parent[line[-1]] >= 0:
                line.append(parent[line[-1]])
            p = ctx + len(line) - 1
            low, head = (max(p - c["window"] + 1, 0), min(c["sinks"], ctx)) if c["window"] else (0, 0)
            tree = [ctx + b for up, b in enumerate(line) if not c["window"] or up < c["window"] or p - up < c["sinks"]]
            idx = torch.cat([torch.arange(min(head, low)), torch.arange(min(low, ctx), ctx), torch.tensor(tree)]).cuda()
            q = s["q"][t + a].double().view(c["Hkv"], G, D)
            x = torch.einsum("hgd,mhd->hgm", q, k[idx]) * s["scale"]
            lse[t + a] = torch.logsumexp(x, -1).reshape(-1)
            O[t + a] = torch.einsum("hgm,mhd->hgd", torch.softmax(x, -1), v[idx]).reshape(-1, D)
    return None, None, O, lse


def _exact_verify(s):
    out = [-1] * s["tokens"].shape[0]
    counts, drawn = [], []
    tok, u = s["tokens"].tolist(), s["accept"].double().cpu().numpy()

    def line(x, at):
        return x[at].double().cpu().numpy()

    for i, (t, n, parent) in enumerate(_sequences(s)):
        v, depth = 0, 0
        while True:
            out[t + depth] = v
            p = line(s["target"], t + v)
            left, weight, after = p.copy(), 1.0, None
            for a in range(n):
                if a <= v or parent[a] != v:
                    continue
                x = tok[t + a]
                if s["draft"] is None:
                    if u[t + a] * weight < left[x]:
                        after = a
                        break
                    left[x] = 0.0
                else:
                    q = line(s["draft"], t + v)
                    if u[t + a] * q[x] * weight < left[x]:
                        after = a
                        break
                    left = np.maximum(left - weight * q, 0.0)
                weight = float(np.sum(left))
            if after is None:
                break
            v, depth = after, depth + 1
        if weight <= 0.0:
            left = p
        run_sum = np.cumsum(left)
        drawn.append(int(np.searchsorted(run_sum, float(s["sample"][i].double()) * run_sum[-1], side="right")))
        counts.append(depth + 1)
    return torch.tensor(out, dtype=torch.int32), torch.tensor(counts, dtype=torch.int32), torch.tensor(drawn, dtype=torch.int32)


def _exact_keep(s):
    c = s["case"]
    page, table = c["page"], s["table"].tolist()
    path, count = s["path"].tolist(), s["count"].tolist()
    to, new = [], []
    for i, ((t, n, _), kv) in enumerate(zip(_sequences(s), _ints(c["kv"]))):
        for d in range(n):
            x = kv - n + d
            to.append(table[i][x // page] * page + x % page)
            new.append(t + (path[t + d] if d < count[i] else d))
    to, new = torch.tensor(to, device="cuda"), torch.tensor(new, device="cuda")
    out = []
    for cache, rows in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])):
        flat = cache.double().transpose(1, 2).reshape(-1, c["Hkv"], c["D"])
        flat.index_copy_(0, to, rows.double()[new])
        out.append(flat.view(-1, page, c["Hkv"], c["D"]).transpose(1, 2))
    return tuple(out)


def _exact_moved(s, src, dst):
    out = []
    for cache in (s["k_cache"], s["v_cache"]):
        x = cache.double()
        pairs = [(a, b) for a, b in zip(src, dst) if a >= 0]
        if pairs:
            a, b = (torch.tensor(v, device="cuda") for v in zip(*pairs))
            x.index_copy_(0, b, cache.double()[a])
        out.append(x)
    return out


def _exact_turn(s):
    page = s["case"]["page"]
    refs, table, kv, parent, want = (s[n].tolist() for n in ("refs", "table", "kv_len", "parent", "want"))

    def held(n):
        return -(-n // page)

    for i, row in enumerate(table):
        for j in range(held(kv[i]), len(row)):
            if row[j] >= 0:
                refs[row[j]] -= 1
                row[j] = -1
    before, lens = [list(row) for row in table], list(kv)
    for i, a in enumerate(parent):
        if a == i:
            continue
        for x in before[i]:
            if x >= 0:
                refs[x] -= 1
        table[i] = [x if j < held(lens[a]) else -1 for j, x in enumerate(before[a])]
        for x in table[i]:
            if x >= 0:
                refs[x] += 1
        kv[i] = lens[a]
    asked = [(i, j) for i in range(len(table)) for j in range(kv[i] // page, held(want[i]))]
    users, first = {}, {}
    for i, j in asked:
        x = table[i][j]
        if x >= 0:
            users[x] = users.get(x, 0) + 1
            first.setdefault(x, (i, j))
    was = list(refs)
    give = []
    for i, j in asked:
        x = table[i][j]
        if x < 0:
            give.append((i, j))
        elif was[x] > 1 and not (users[x] == was[x] and first[x] == (i, j)):
            give.append((i, j))
            refs[x] -= 1
    free = [x for x, n in enumerate(refs) if n == 0]
    src, dst = [-1] * len(table), [-1] * len(table)
    for (i, j), x in zip(give, free):
        if table[i][j] >= 0 and j == kv[i] // page and kv[i] % page:
            src[i], dst[i] = table[i][j], x
        table[i][j] = x
        refs[x] = 1
    return (*(torch.tensor(x, dtype=torch.int32) for x in (refs, table, kv, src, dst)), *_exact_moved(s, src, dst))


def _exact_compact(s):
    refs, table = s["refs"].tolist(), s["table"].tolist()
    live = sum(n > 0 for n in refs)
    high = [x for x in range(live, len(refs)) if refs[x] > 0]
    low = [x for x in range(live) if refs[x] == 0]
    to = dict(zip(high, low))
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
    table = [[to.get(x, x) for x in row] for row in table]
    rest = [-1] * (len(refs) // 2 - len(high))
    src, dst = high + rest, low + rest
    return (*(torch.tensor(x, dtype=torch.int32) for x in (refs, table, src, dst)), *_exact_moved(s, src, dst))


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kind = case["kind"]
    if kind == "rotate":
        return _exact_rotate(s["q"], s, 1), _exact_rotate(s["k"], s, 1)
    if kind == "rotate_train":
        return (*(_exact_rotate(s[n], s, 1) for n in "qk"), *(_exact_rotate(s[n], s, -1) for n in ("dq", "dk")))
    return {"tree": _exact_tree, "verify": _exact_verify, "keep": _exact_keep, "turn": _exact_turn,
            "compact": _exact_compact}[kind](s)
