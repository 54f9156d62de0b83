"""Timed cases of the windowed and paged attention operators.

Four kinds of case, each with a plain form (elementary torch operations in
32 bits) and the call a user makes of the framework:

    window  bsp.bsp_window_attention: causal attention with a sliding window
            and sink tokens; returns O and the rows' log-sum-exp
    train   bsp.window_attention and its gradient; returns O, dQ, dK, dV
    append  bsp.bsp_paged_append: the K and V rows of new tokens into a paged
            cache; returns both caches
    paged   bsp.bsp_paged_attention: a ragged batch of new tokens over the
            cache; returns O and the rows' log-sum-exp

A key j is visible to the query at position p when j <= p and (p - j < window
or j < sinks); window 0 stands for no limit.
"""

import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # the latency of one short prompt through a small layer
        dict(name="window_small", kind="window", Z=1, Hq=4, Hkv=4, S=256, D=64, window=64, sinks=4,
             dtype="bf16", rows_first=False),
        # the banded workload's sizes as a causal window: a batch of long documents
        dict(name="window_band", kind="window", Z=4, Hq=16, Hkv=16, S=8192, D=128, window=512, sinks=4,
             dtype="bf16", rows_first=False),
        # the strided workload's sizes with shared KV heads: one long prompt, wide window
        dict(name="window_long", kind="window", Z=1, Hq=32, Hkv=8, S=16384, D=128, window=4096, sinks=64,
             dtype="f16", rows_first=True),
        # a training step's attention, shared KV heads, projections' own [Z, S, H, D] order
        dict(name="train_gqa", kind="train", Z=1, Hq=32, Hkv=8, S=8192, D=128, window=1024, sinks=4,
             dtype="bf16", rows_first=True),
        # fine-tuning on short odd lengths, a head size between the powers of two
        dict(name="train_odd", kind="train", Z=2, Hq=6, Hkv=2, S=1037, D=80, window=200, sinks=3,
             dtype="f16", rows_first=False),
        # the BigBird workload's sizes, full precision training
        dict(name="train_f32", kind="train", Z=2, Hq=12, Hkv=12, S=4096, D=64, window=512, sinks=16,
             dtype="f32", rows_first=False),
        # one user's next token: latency
        dict(name="decode_one", kind="paged", new="1", kv="1000", Hq=16, Hkv=4, D=128, page=16, window=0, sinks=0,
             dtype="f16"),
        # next tokens of a serving batch over ragged histories: the cache's bandwidth
        dict(name="decode_batch", kind="paged", new=_text([1] * 64), kv=_spread(64, 2048, 8192, 5), Hq=32, Hkv=8, D=128,
             page=64, window=0, sinks=0, dtype="bf16"),
        # chunks of prompts over what is cached of them
        dict(name="chunk", kind="paged", new="512 512 512 512", kv="4608 9001 16384 12345", Hq=32, Hkv=8,
             D=128, page=128, window=0, sinks=0, dtype="bf16"),
        # one chunk joined by other users' next tokens, window and sinks
        dict(name="mixed", kind="paged", new=_text([1000] + [1] * 31), kv="2500 " + _spread(31, 300, 6000, 9), Hq=24, Hkv=8,
             D=128, page=32, window=1024, sinks=4, dtype="f16"),
        # a prompt batch's keys and values into the cache
        dict(name="append_prompt", kind="append", new=_spread(8, 700, 1400, 3), kv=_spread(8, 1400, 2800, 4), Hkv=8,
             D=128, page=16, dtype="bf16"),
        # a serving batch's next tokens into the cache
        dict(name="append_decode", kind="append", new=_text([1] * 64), kv=_spread(64, 100, 1000, 6), Hkv=8, D=128, page=64,
             dtype="f16"),
    ]


def _spread(n, lo, hi, seed):
    """n whole numbers between lo and hi, spread over their logarithm."""
    r = random.Random(seed)
    return _text(_log_int(r, lo, hi) for _ in range(n))


def _text(numbers):
    """The sequences' lengths as a case holds them: one text."""
    return " ".join(str(n) for n in numbers)


def _numbers(case):
    """New tokens and lengths (the new tokens included) of each sequence."""
    return [int(n) for n in case["new"].split()], [int(n) for n in case["kv"].split()]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {kind: max(work(c)["flops"] for c in listed() if c["kind"] == kind) for kind in ("window", "train", "paged")}
    bytes_most = {kind: max(work(c)["bytes"] for c in listed() if c["kind"] == kind)
                  for kind in ("window", "train", "paged", "append")}
    while True:
        kind = rng.choice(("window", "window", "train", "train", "paged", "paged", "paged", "append"))
        dtype = rng.choice(("bf16", "bf16", "f16", "f16", "f32"))
        D = rng.choice((16, 32, 48, 64, 64, 80, 96, 112, 128, 128, 128))
        Hkv = rng.choice((1, 2, 3, 4, 8, 16))
        Hq = Hkv * rng.choice((1, 1, 2, 3, 4, 5, 8))
        if kind in ("window", "train"):
            S = _log_int(rng, 64, 16384)
            case = dict(kind=kind, Z=rng.choice((1, 1, 2, 3, 4)), Hq=Hq, Hkv=Hkv, S=S, D=D,
                        window=rng.choice((0, _log_int(rng, 16, 4096), _log_int(rng, 16, 4096))),
                        sinks=rng.choice((0, 1, 4, 16, 130)), dtype=dtype, rows_first=rng.random() < 0.5)
        else:
            n = _log_int(rng, 1, 64)
            page = rng.choice((16, 32, 64, 128))
            shape = rng.choice(("decode", "chunk", "mixed"))
            new = [1 if shape == "decode" or (shape == "mixed" and rng.random() < 0.8) else _log_int(rng, 2, 1000)
                   for _ in range(n)]
            kv = [q + _log_int(rng, 1, 16384) - 1 for q in new]
            case = dict(kind=kind, new=_text(new), kv=_text(kv), Hkv=Hkv, D=D, page=page, dtype=dtype)
            if kind == "paged":
                case.update(Hq=Hq, window=rng.choice((0, 0, _log_int(rng, 16, 4096))), sinks=rng.choice((0, 4, 40)))
        w = work(case)
        # the fp32 kernels run on the CUDA cores: the fp32 listed case bounds them
        limit = most.get(kind, 0) / (16 if dtype == "f32" else 1)
        if (kind == "append" or w["flops"] <= limit) and w["bytes"] <= bytes_most[kind]:
            return case


# ------------------------------------------------------------------ work --

def _pairs(first, count, window, sinks):
    """Visible (query, key) pairs of the queries at positions first .. first + count - 1."""
    p = np.arange(first, first + count, dtype=np.int64)
    p = p[p >= 0]
    lo = np.maximum(p - window + 1, 0) if window else np.zeros_like(p)
    return int(np.sum(p - lo + 1 + np.minimum(lo, sinks)))


def _visible_keys(kv, new, window, sinks):
    """Keys that some of the `new` last queries see."""
    lo = max(kv - new - window + 1, 0) if window else 0
    return kv - lo + min(lo, sinks)


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    D, Hkv = case["D"], case["Hkv"]
    if case["kind"] == "append":
        return {"bytes": 4 * e * sum(_numbers(case)[0]) * Hkv * D, "flops": 0}
    Hq = case["Hq"]
    if case["kind"] == "paged":
        new, kvs = _numbers(case)
        T = sum(new)
        keys = sum(_visible_keys(kv, q, case["window"], case["sinks"]) for q, kv in zip(new, kvs))
        pairs = sum(_pairs(kv - q, q, case["window"], case["sinks"]) for q, kv in zip(new, kvs))
        return {"bytes": e * (2 * T * Hq * D + 2 * keys * Hkv * D) + 4 * T * Hq, "flops": 4 * D * Hq * pairs}
    q = case["Z"] * Hq * case["S"] * D
    k = case["Z"] * Hkv * case["S"] * D
    pairs = case["Z"] * Hq * _pairs(0, case["S"], case["window"], case["sinks"])
    if case["kind"] == "window":
        return {"bytes": e * (2 * q + 2 * k) + 4 * case["Z"] * Hq * case["S"], "flops": 4 * D * pairs}
    # Q, K, V, dO in; O, dQ, dK, dV out; two products forward, five backward
    return {"bytes": e * (4 * q + 4 * k), "flops": 14 * D * pairs}


# ---------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    dt = _DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = dict(case=case, scale=1.0 / math.sqrt(case["D"]))
    if case["kind"] in ("window", "train"):
        def heads(H):
            if case["rows_first"]:  # as a projection leaves them
                return randn(case["Z"], case["S"], H, case["D"]).transpose(1, 2)
            return randn(case["Z"], H, case["S"], case["D"])

        s.update(q=heads(case["Hq"]), k=heads(case["Hkv"]), v=heads(case["Hkv"]))
        if case["kind"] == "train":
            s["do"] = heads(case["Hq"])
            if own:
                for name in "qkv":
                    s[name].requires_grad_()
        window, sinks = case["window"], case["sinks"]
    else:
        new, kvs = _numbers(case)
        T, page, D, Hkv = sum(new), case["page"], case["D"], case["Hkv"]
        used = [-(-kv // page) for kv in kvs]
        n_pages = sum(used) + 3
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = torch.zeros(len(used), max(used), dtype=torch.int32)
        at = 0
        for i, n in enumerate(used):
            table[i, :n] = order[at:at + n]
            at += n
        s.update(k_cache=randn(n_pages, Hkv, page, D), v_cache=randn(n_pages, Hkv, page, D), table=table.cuda(),
                 q_start=torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda(),
                 kv_len=torch.tensor(kvs, dtype=torch.int32).cuda())
        if case["kind"] == "paged":
            s["q"] = randn(T, case["Hq"], D)
        else:
            s.update(k_new=randn(T, Hkv, D), v_new=randn(T, Hkv, D))
        window, sinks = case.get("window", 0), case.get("sinks", 0)
    if own:
        from sparse_attention_layout_gb300 import bsp
        s["W"] = bsp.bsp_window_create(window=window, sinks=sinks)
    return s


def run(state):
    kind = state["case"]["kind"]
    if not own:
        return {"window": _plain_window, "train": _plain_train, "append": _plain_append, "paged": _plain_paged}[kind](state)
    from sparse_attention_layout_gb300 import bsp
    s = state
    if kind == "window":
        return bsp.bsp_window_attention(s["W"], s["q"], s["k"], s["v"], scale=s["scale"])
    if kind == "train":
        o = bsp.window_attention(s["W"], s["q"], s["k"], s["v"], s["scale"])
        return (o.detach(), *torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"]))
    if kind == "append":
        bsp.bsp_paged_append(s["W"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_len"],
                             s["table"])
        return s["k_cache"], s["v_cache"]
    return bsp.bsp_paged_attention(s["W"], s["q"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_len"], s["table"],
                                   scale=s["scale"])


# ------------------------------------------------------------ plain forms --
# The scores of one KV head's query heads are formed for at most this many
# query rows at a time, so that the largest case fits beside its inputs.
_ROWS = 2048


def _keep(p, j, window, sinks):
    """[len(p), len(j)] truth values: key position j is visible to query position p."""
    p, j = p[:, None], j[None, :]
    keep = j <= p
    if window:
        keep = keep & ((p - j < window) | (j < sinks))
    return keep


def _plain_rows(q, k, v, first, scale, window, sinks):
    """q [G, n, D] at positions first .., k and v [Sk, D] (fp32) -> P [G, n, Sk], O, lse."""
    n, Sk = q.shape[1], k.shape[0]
    p = torch.arange(first, first + n, device=q.device)
    s = (q @ k.T) * scale
    s = s.masked_fill(~_keep(p, torch.arange(Sk, device=q.device), window, sinks), -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    P = e / l
    return P, P @ v, (m + torch.log(l))[..., 0]


def _plain_window(s):
    c = s["case"]
    q, k, v = s["q"], s["k"], s["v"]
    G = c["Hq"] // c["Hkv"]
    O = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    for z in range(c["Z"]):
        for h in range(c["Hkv"]):
            hs = slice(h * G, (h + 1) * G)
            kf, vf = k[z, h].float(), v[z, h].float()
            for a in range(0, c["S"], _ROWS):
                b = min(a + _ROWS, c["S"])
                _, o, l = _plain_rows(q[z, hs, a:b].float(), kf[:b], vf[:b], a, s["scale"], c["window"], c["sinks"])
                O[z, hs, a:b], lse[z, hs, a:b] = o.to(q.dtype), l
    return O, lse


def _plain_train(s):
    c = s["case"]
    q, k, v, do = s["q"], s["k"], s["v"], s["do"]
    G = c["Hq"] // c["Hkv"]
    O = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dQ, dK, dV = torch.empty_like(O), torch.empty(k.shape, dtype=k.dtype, device=k.device), \
        torch.empty(v.shape, dtype=v.dtype, device=v.device)
    for z in range(c["Z"]):
        for h in range(c["Hkv"]):
            hs = slice(h * G, (h + 1) * G)
            kf, vf = k[z, h].float(), v[z, h].float()
            dk, dv = torch.zeros_like(kf), torch.zeros_like(vf)
            for a in range(0, c["S"], _ROWS):
                b = min(a + _ROWS, c["S"])
                qf, dof = q[z, hs, a:b].float(), do[z, hs, a:b].float()
                P, o, _ = _plain_rows(qf, kf[:b], vf[:b], a, s["scale"], c["window"], c["sinks"])
                dP = dof @ vf[:b].T
                dS = P * (dP - (P * dP).sum(-1, keepdim=True)) * s["scale"]
                dv[:b] += (P.transpose(1, 2) @ dof).sum(0)
                dk[:b] += (dS.transpose(1, 2) @ qf).sum(0)
                O[z, hs, a:b], dQ[z, hs, a:b] = o.to(q.dtype), (dS @ kf[:b]).to(q.dtype)
            dK[z, h], dV[z, h] = dk.to(k.dtype), dv.to(v.dtype)
    return O, dQ, dK, dV


def _slots(s, i, positions):
    """Pages and slots of key positions of sequence i."""
    page = s["case"]["page"]
    return s["table"][i][positions // page].long(), positions % page


def _plain_append(s):
    c = s["case"]
    t = 0
    for i, (n, kv) in enumerate(zip(*_numbers(c))):
        pg, sl = _slots(s, i, torch.arange(kv - n, kv, device="cuda"))
        s["k_cache"][pg, :, sl] = s["k_new"][t:t + n]
        s["v_cache"][pg, :, sl] = s["v_new"][t:t + n]
        t += n
    return s["k_cache"], s["v_cache"]


def _plain_paged(s):
    c = s["case"]
    q = s["q"]
    G = c["Hq"] // c["Hkv"]
    O = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    t = 0
    for i, (n, kv) in enumerate(zip(*_numbers(c))):
        pg, sl = _slots(s, i, torch.arange(kv, device=q.device))
        kf, vf = s["k_cache"][pg, :, sl].float(), s["v_cache"][pg, :, sl].float()  # [kv, Hkv, D]
        for h in range(c["Hkv"]):
            hs = slice(h * G, (h + 1) * G)
            _, o, l = _plain_rows(q[t:t + n, hs].float().transpose(0, 1), kf[:, h], vf[:, h], kv - n, s["scale"],
                                  c["window"], c["sinks"])
            O[t:t + n, hs], lse[t:t + n, hs] = o.transpose(0, 1).to(q.dtype), l.transpose(0, 1)
        t += n
    return O, lse


# ------------------------------------------------------------------ exact --
# The definition in 64 bits, a few query rows at a time over the keys they can
# see: the sinks' columns and the window's, gathered by their indices.

def _exact_block(q, k, v, rows, first, scale, window, sinks, do=None):
    """q [G, n, D] of the rows `rows` (positions first + row); k, v [Sk, D].
    Returns O, lse, and with do also (columns, dQ, dK and dV at them)."""
    p = (torch.as_tensor(rows, device=q.device) + first).double()
    hi = int(p[-1].item())
    lo = max(int(p[0].item()) - window + 1, 0) if window else 0
    cols = torch.cat([torch.arange(min(sinks, lo), device=q.device), torch.arange(lo, hi + 1, device=q.device)])
    kc, vc = k[cols], v[cols]
    dist = p[:, None] - cols[None, :].double()
    hidden = dist < 0
    if window:
        hidden |= (dist >= window) & (cols[None, :] >= sinks)
    x = torch.einsum("gnd,md->gnm", q, kc) * scale
    x[:, hidden] = -math.inf
    lse = torch.logsumexp(x, -1)
    P = torch.exp(x - lse[..., None])
    O = torch.einsum("gnm,md->gnd", P, vc)
    if do is None:
        return O, lse
    dP = torch.einsum("gnd,md->gnm", do, vc)
    dS = P * (dP - torch.einsum("gnd,gnd->gn", do, O)[..., None])
    return (O, lse, cols, torch.einsum("gnm,md->gnd", dS, kc) * scale, torch.einsum("gnm,gnd->md", dS, q) * scale,
            torch.einsum("gnm,gnd->md", P, do))


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["kind"] == "append":
        new, kvs = _numbers(case)
        table, page = s["table"].cpu().tolist(), case["page"]
        owner = [(i, kv - n + r) for i, (n, kv) in enumerate(zip(new, kvs)) for r in range(n)]
        at = torch.tensor([table[i][p // page] * page + p % page for i, p in owner], device="cuda")
        out = []
        for cache, rows in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])):
            flat = cache.double().transpose(1, 2).reshape(-1, case["Hkv"], case["D"])
            flat.index_copy_(0, at, rows.double())
            out.append(flat.view(-1, page, case["Hkv"], case["D"]).transpose(1, 2))
        return tuple(out)
    G = case["Hq"] // case["Hkv"]
    step = 256
    if case["kind"] == "paged":
        T = sum(_numbers(case)[0])
        O = torch.zeros(T, case["Hq"], case["D"], dtype=torch.float64, device="cuda")
        lse = torch.zeros(T, case["Hq"], dtype=torch.float64, device="cuda")
        t = 0
        for i, (n, kv) in enumerate(zip(*_numbers(case))):
            pos = np.arange(kv)
            pages = s["table"][i].cpu().numpy()[pos // case["page"]].astype(np.int64)
            rows = torch.from_numpy(pages * case["page"] + pos % case["page"]).cuda()
            for h in range(case["Hkv"]):
                k = s["k_cache"][:, h].reshape(-1, case["D"])[rows].double()
                v = s["v_cache"][:, h].reshape(-1, case["D"])[rows].double()
                for a in range(0, n, step):
                    r = range(a, min(a + step, n))
                    q = s["q"][t + a:t + r[-1] + 1, h * G:(h + 1) * G].double().transpose(0, 1)
                    o, l = _exact_block(q, k, v, r, kv - n, s["scale"], case["window"], case["sinks"])
                    O[t + a:t + r[-1] + 1, h * G:(h + 1) * G] = o.transpose(0, 1)
                    lse[t + a:t + r[-1] + 1, h * G:(h + 1) * G] = l.transpose(0, 1)
            t += n
        return O, lse
    train = case["kind"] == "train"
    q, k, v = (s[n].double() for n in "qkv")
    O, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    dQ, dK, dV = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    do = s["do"].double() if train else None
    for z in range(case["Z"]):
        for h in range(case["Hkv"]):
            hs = slice(h * G, (h + 1) * G)
            for a in range(0, case["S"], step):
                b = min(a + step, case["S"])
                got = _exact_block(q[z, hs, a:b], k[z, h], v[z, h], range(a, b), 0, s["scale"], case["window"],
                                   case["sinks"], do[z, hs, a:b] if train else None)
                O[z, hs, a:b], lse[z, hs, a:b] = got[0], got[1]
                if train:
                    cols = got[2]
                    dQ[z, hs, a:b] = got[3]
                    dK[z, h].index_add_(0, cols, got[4])
                    dV[z, h].index_add_(0, cols, got[5])
    return (O, dQ, dK, dV) if train else (O, lse)
