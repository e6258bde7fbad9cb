"""The losses of the RQ-coded head in 64 bits, from their definition, and the
error bounds that the GPU results are held to.  Plain torch on the CPU or the
GPU; shares nothing with the library."""
import math

import torch

F64 = torch.float64


def rows(C, codes):
    """E [V, D] in 64 bits from C [M, L, K, ds] and codes [V, M, L] (int64,
    codes >= K as the library takes them)."""
    M, L, K, ds = C.shape
    c = codes.long()
    c = c % K if K & (K - 1) == 0 else c.clamp(max=K - 1)
    E = torch.zeros(c.shape[0], M, ds, dtype=F64, device=C.device)
    for l in range(L):
        E += C[torch.arange(M, device=C.device), l, c[:, :, l]].to(F64)
    return E.view(c.shape[0], M * ds), c


def probabilities(V, ids, val, T):
    """q [N, V] of a target list (val None) or a teacher's, and which rows have one."""
    ids = ids.long().view(ids.shape[0], -1)
    ok = (ids >= 0) & (ids < V)
    if val is None:
        w = ok.to(F64)
    else:
        t = (val.to(F64) / T).masked_fill(~ok, -math.inf)
        ok = t > -math.inf
        w = torch.softmax(t, 1).nan_to_num(0.0)
    q = torch.zeros(ids.shape[0], V, dtype=F64, device=ids.device)
    q.scatter_add_(1, ids.clamp(0, V - 1), torch.where(ok, w, 0.0))
    return q, ok.any(1), torch.where(ok, w, 0.0)


def losses(h, C, codes, ids, val=None, T=1.0, cap=30.0, weight=None):
    """dict of loss, lse, dh, dC, and the sizes the bounds are made of."""
    E, c = rows(C, codes)
    V, (M, L, K, ds) = E.shape[0], C.shape
    hd = h.to(F64)
    z = hd @ E.t()
    y = cap * torch.tanh(z / cap) if cap > 0 else z
    lse = torch.logsumexp(y / T, 1)
    q, some, w = probabilities(V, ids, val, T)
    ce = (q * (lse[:, None] - y / T)).sum(1)
    ent = torch.xlogy(w, w).sum(1) if val is not None else 0.0
    loss = T * T * (ce + ent) * some
    p = torch.exp(y / T - lse[:, None])
    f = (torch.ones_like(loss) if weight is None else weight.to(F64)) * T * some
    slope = 1 - (y / cap) ** 2 if cap > 0 else torch.ones_like(y)
    dz = f[:, None] * (p - q) * slope

    def by_code(dE):
        out = torch.zeros(M, L, K, ds, dtype=F64, device=C.device)
        for l in range(L):
            at = (torch.arange(M, device=C.device) * K + c[:, :, l]).view(-1)
            out[:, l] = torch.zeros(M * K, ds, dtype=F64, device=C.device).index_add_(
                0, at, dE.reshape(-1, ds)).view(M, K, ds)
        return out

    mag = f.abs()[:, None] * (p + q) * slope         # what dz is the difference of
    # how far a logit can be off: see bounds()
    size = (hd.abs() @ E.abs().t()).max().item() if V * h.shape[0] else 0.0
    return {"loss": loss, "lse": lse, "dh": dz @ E, "dC": by_code(dz.t() @ hd),
            "dh_mag": mag @ E.abs(), "dC_mag": by_code(mag.t() @ hd.abs()), "size": size,
            "top": y.abs().max().item() / T, "T": T, "cap": cap,
            "list": 0.0 if val is None else (val.abs().nan_to_num(0.0, 0.0, 0.0).max().item() / T)}


def bounds(r, bf16):
    """Elementwise bounds for loss, lse, dh, dC.

    A logit's product h E is a sum of D terms.  On the tensor cores each is
    formed from fp16 hi / lo parts, 3 * 2^-22 of |h E| lost (two split
    remainders and the dropped lo lo product), and added in chains of at most
    48 MMAs that may lose 2^-22 of the chain's magnitude each step (truncation,
    in the last of 24 bits and one guard), joined by fp32 additions (2^-24
    each, at most 128).  The tables of the few-token path add 768 or fewer
    fp32 terms in chunks, each at most 2^-24 of the magnitude: at most
        dz <= (3 + 48 + 32) 2^-22 * max sum |h E|.
    The softcap (slope at most 1, tanhf within 2 ulp of at most cap) and the
    scale 1 / T add 4 * 2^-23 of the largest |y| / T.  With d = that in units
    of y / T, exp(y / T - lse) is off by the factor 2 d (both terms) plus 4
    ulp, and the slope 1 - (y / cap)^2 by 2 dz / cap of 1.
    Sums over the vocabulary or the tokens: the same splits and chains, at
    most (3 + 48 + 32) 2^-22 of the sum of magnitudes.
    """
    prod = 83 * 2.0 ** -22
    d_y = prod * r["size"]
    d = d_y / r["T"] + 8 * 2.0 ** -23 * (1 + r["top"])
    p_rel = 2 * d + 2 * d_y / (r["cap"] if r["cap"] > 0 else math.inf) + 2.0 ** -20
    # the teacher's softmax: its logits' scaling and exp
    q_rel = 8 * 2.0 ** -23 * (1 + r["list"])
    k = 2 * (p_rel + q_rel) + prod
    loss = r["T"] ** 2 * (2 * d + 2 * q_rel * (1 + r["top"] + r["list"]) + 2.0 ** -21 * (1 + r["top"] + r["list"]))
    out = {"loss": torch.full_like(r["loss"], loss), "lse": torch.full_like(r["lse"], 2 * d),
           "dh": k * r["dh_mag"], "dC": k * r["dC_mag"]}
    if bf16:       # the high planes alone (2^-12 each side), and bf16's rounding
        out["dh"] = out["dh"] + 2.0 ** -11 * r["dh_mag"] + 2.0 ** -8 * r["dh"].abs()
    tiny = 2.0 ** -38      # the lo planes' absolute floor, of the largest element
    for g in ("dh", "dC"):
        out[g] = out[g] + tiny * r[g + "_mag"].max()
    return out
