"""Plain fp64 windowed attention, its gradient, and entry-wise error bounds
for kernels that take the same inputs, sum in fp32 and round P, dS and the
outputs to the inputs' type.

Bounds.  u = half a step of the type relative to the value (gpu_util.U); ab =
half the spacing of its subnormals, which P and dS of fp16 meet (0 otherwise).
A score's error is at most gamma(D) scale sum |q||k| (fp32 sums) plus 2^-23 |s|
(its scaling), so exp(s - lse) is off by the factor e^(2 es), es the largest
such error of the row, beside EXP_ERR.  Let ep = u + 2 es + 4 EXP_ERR:
    O:  u |O| + (ep + gamma(n)) P|V| + ab sum |V|
    dV: u |dV| + (ep + gamma(n)) P^T |dO| + ab sum |dO|
    dS: E = P (gamma(D) |dO||V|^T + ed) + ep |dS| + ab, ed = the error of
        delta = dO . O, whose O was rounded: (2 u + gamma(D)) |dO| . |O| + the
        error of O times |dO|
    dQ: u |dQ| + scale (E |K| + gamma(n) |dS||K|), dK alike with |Q|
n is the number of terms.  Each bound is doubled where a rounded value enters
a second rounding (2 u in assert_close's |r| term)."""

import torch

from gpu_util import EXP_ERR, U, gamma

AB = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def keep_mask(p, j, window, sinks):
    p, j = p[:, None], j[None, :]
    k = j <= p
    if window:
        k = k & ((p - j < window) | (j < sinks))
    return k


def head(q, k, v, first, scale, window, sinks, dtype, do=None):
    """One query head: q [n, D] at positions first .., k, v [Sk, D], all fp64.
    dict of values and bounds."""
    n, D = q.shape
    Sk = k.shape[0]
    u, ab = U[dtype], AB[dtype]
    keep = keep_mask(torch.arange(first, first + n, device=q.device), torch.arange(Sk, device=q.device), window, sinks)
    s = ((q @ k.T) * scale).masked_fill(~keep, float("-inf"))
    lse = torch.logsumexp(s, -1)  # -inf where nothing is visible
    P = torch.exp(s - lse[:, None].masked_fill(torch.isinf(lse)[:, None], 0.0))
    P = P.masked_fill(~keep, 0.0)
    O = P @ v
    mags = ((q.abs() @ k.abs().T) * scale * keep)
    mags = torch.cat([mags, torch.zeros(n, 1, dtype=mags.dtype, device=q.device)], 1)  # no key at all: no error
    es = (gamma(D) * mags).amax(-1, keepdim=True) + 2.0 ** -23 * mags.amax(-1, keepdim=True)
    ep = u + 2 * es + 4 * EXP_ERR
    cnt = keep.sum(-1, keepdim=True)
    eO_in = (ep + gamma(1) + cnt * 2.0 ** -22) * (P @ v.abs()) + ab * (keep.double() @ v.abs())
    out = dict(O=O, lse=lse, eO=u * O.abs() + eO_in + ab,
               else_=(2 * es[:, 0] + 8 * EXP_ERR + 2.0 ** -22 * (lse.abs().nan_to_num(posinf=0.0) + 1)
                      + cnt[:, 0] * 2.0 ** -22))
    if do is None:
        return out
    dP = do @ v.T
    delta = (do * O).sum(-1, keepdim=True)
    dS = P * (dP - delta)
    ed = (2 * u + gamma(D)) * (do.abs() * O.abs()).sum(-1, keepdim=True) + (do.abs() * eO_in).sum(-1, keepdim=True)
    E = P * (gamma(D) * (do.abs() @ v.abs().T) + ed) + ep * dS.abs() + ab * keep
    rows = keep.sum(0)[:, None]
    out.update(dQ=scale * (dS @ k), dK=scale * (dS.T @ q), dV=P.T @ do,
               eQ=scale * (E @ k.abs() + cnt * 2.0 ** -22 * (dS.abs() @ k.abs())),
               eK=scale * (E.T @ q.abs() + rows * 2.0 ** -22 * (dS.abs().T @ q.abs())),
               eV=(P * ep).T @ do.abs() + rows * 2.0 ** -22 * (P.T @ do.abs()) + ab * (keep.double().T @ do.abs()))
    return out


def dense(Q, K, V, scale, window, sinks, dO=None):
    """Values and bounds for [Z, H, S, D] tensors."""
    Z, Hq, Sq, D = Q.shape
    Hkv, Sk = K.shape[1], K.shape[2]
    G = Hq // Hkv
    dt = Q.dtype
    q, k, v = Q.double(), K.double(), V.double()
    do = None if dO is None else dO.double()
    o = dict(O=torch.zeros_like(q), eO=torch.zeros_like(q), lse=torch.zeros(Q.shape[:3], dtype=torch.float64, device=Q.device))
    o["else_"] = torch.zeros_like(o["lse"])
    if dO is not None:
        o.update(dQ=torch.zeros_like(q), eQ=torch.zeros_like(q), dK=torch.zeros_like(k), eK=torch.zeros_like(k),
                 dV=torch.zeros_like(v), eV=torch.zeros_like(v))
    for z in range(Z):
        for h in range(Hq):
            r = head(q[z, h], k[z, h // G], v[z, h // G], Sk - Sq, scale, window, sinks, dt,
                     None if do is None else do[z, h])
            for name in ("O", "eO", "lse", "else_"):
                o[name][z, h] = r[name]
            if dO is not None:
                o["dQ"][z, h], o["eQ"][z, h] = r["dQ"], r["eQ"] + U[dt] * r["dQ"].abs()
                for name in ("dK", "eK", "dV", "eV"):  # the heads that share a KV head add up
                    o[name][z, h // G] += r[name]
    if dO is not None:
        o["eK"] += U[dt] * o["dK"].abs()
        o["eV"] += U[dt] * o["dV"].abs()
        for name in ("eQ", "eK", "eV"):
            o[name] += AB[dt]
    return o


def check(got, want, bound, what):
    g = got.double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    same = (g == want) | ((g - want).abs() <= bound)
    if not bool(same.all()):
        bad = (~same).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {len(bad)} of {g.numel()} entries off, first at {i}: {g[i].item()} for "
                             f"{want[i].item()}, bound {bound.expand_as(want)[i].item()}")
