"""Cases of the loss operators on an RQ-coded output head.

The head of a residual-product-quantized embedding is trained and scored
without its logits being kept: softmax cross entropy against target ids
(``xent``) and distillation from a teacher's top logits (``distill``), each
as a loss alone (scoring: perplexity, log-probabilities, the distance from a
teacher) and as a training step (the loss, then the gradients with respect
to the hidden states and the codebooks).

    E[v]   = sum_l C[m][l][code[v][m][l]]            row v, subspace by subspace
    y[n,v] = cap * tanh(<h_n, E_v> / cap)            (cap = 0: the plain product)
    lse_n  = log sum_v exp(y[n,v] / T)
    xent     loss_n = lse_n - y[n, target_n]                         (T = 1)
    distill  q_n = softmax(teacher_n / T) over its listed ids,
             loss_n = T^2 sum_j q_nj (log q_nj - y[n, id_nj] / T + lse_n)
    dy[n,v] = w_n T (exp(y[n,v] / T - lse_n) - q_n[v])
    dh = (dy (1 - (y / cap)^2)) E,   dE = (dy (1 - (y / cap)^2))^T h,
    dC[m][l][k] = sum over the rows v with code[v][m][l] = k of dE[v], subspace m

A target or a teacher's id below 0 stands for none: a row without any has
loss 0 and no gradient.
"""
import math

import torch

own = False

# The artifact of the Gemma-2 shaped workload and the small one of the tests.
_G2 = {"V": 256000, "M": 384, "ds": 6, "L": 2, "K": 1024}
_TINY = {"V": 4096, "M": 32, "ds": 6, "L": 2, "K": 256}


def _case(op, shape, N, h, fmt, k=0, T=1.0, cap=30.0):
    return {"op": op, **shape, "N": N, "h": h, "fmt": fmt, "k": k, "T": T, "cap": cap}


def listed():
    f32, bf16 = "float32", "bfloat16"
    cases = {
        # the log-probability of one chosen token beside a small head: launch latency
        "xent_tiny_n1": _case("xent", _TINY, 1, f32, "u16"),
        # the same on the full head: scoring while decoding token by token
        "xent_g2_n1": _case("xent", _G2, 1, f32, "u16"),
        # scoring a decoding batch
        "xent_g2_n32": _case("xent", _G2, 32, f32, "u16"),
        # perplexity of a window of text, an odd length, on the 10-bit artifact
        "xent_g2_n1000_bf16": _case("xent", _G2, 1000, bf16, "packed10"),
        # a training step of a small head with one byte per code
        "xent_step_tiny_n33": _case("xent_step", _TINY, 33, f32, "u8"),
        # a step on a few tokens (online adaptation)
        "xent_step_g2_n4": _case("xent_step", _G2, 4, f32, "u16"),
        # a micro-batch in 32 bits, not a multiple of any tile
        "xent_step_g2_n500": _case("xent_step", _G2, 500, f32, "u16"),
        # a training batch with bf16 activations: the largest
        "xent_step_g2_n2048_bf16": _case("xent_step", _G2, 2048, bf16, "u16"),
        # the distance of a small head from its teacher on three tokens
        "distill_tiny_n3_k8": _case("distill", _TINY, 3, f32, "u16", 8, 2.0),
        # the distance of the compressed head from its teacher on a held-out batch
        "distill_g2_n64_k50": _case("distill", _G2, 64, f32, "u16", 50, 1.0),
        # codebooks tuned towards the uncompressed head, 10-bit artifact
        "distill_step_g2_n256_k50": _case("distill_step", _G2, 256, f32, "packed10", 50, 2.0),
        # another artifact: five dims a subspace, three levels, K no power of two, no softcap
        "distill_step_odd": _case("distill_step", {"V": 50021, "M": 128, "ds": 5, "L": 3, "K": 200}, 77, bf16, "u8",
                                  16, 1.5, 0.0),
    }
    return [{"name": n, **c} for n, c in cases.items()]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent", "xent_step", "distill", "distill_step"])
    if rng.random() < 0.4:
        shape = {**_G2, "V": _log_int(rng, 32000, 256000)}
    else:
        ds, L = rng.choice([2, 3, 4, 5, 6, 6, 8]), rng.choice([1, 2, 2, 3])
        M = min(_log_int(rng, 16, 384), 768 // L, 2304 // ds)
        shape = {"V": _log_int(rng, 1000, 256000), "M": M, "ds": ds, "L": L,
                 "K": rng.choice([16, 64, 100, 256, 500, 1000, 1024])}
    fmts = ["u16"] + (["u8"] if shape["K"] <= 256 else []) + (["packed10"] if shape["M"] * shape["L"] % 4 == 0 else [])
    distill = op.startswith("distill")
    return _case(op, shape, _log_int(rng, 1, 2048), rng.choice(["float32", "bfloat16"]), rng.choice(fmts),
                 _log_int(rng, 1, 128) if distill else 0, rng.choice([0.7, 1.0, 1.5, 2.0, 4.0]) if distill else 1.0,
                 rng.choice([30.0, 30.0, 50.0, 0.0]))


def _pack(codes, fmt):
    """int16 codes [V, P] in the layout `fmt`."""
    if fmt == "u16":
        return codes.view(torch.uint16)
    if fmt == "u8":
        return codes.to(torch.uint8)
    c = codes.view(codes.shape[0], -1, 4).to(torch.int32)          # four codes fill five bytes
    b = torch.stack([c[..., 0], c[..., 0] >> 8 | c[..., 1] << 2, c[..., 1] >> 6 | c[..., 2] << 4,
                     c[..., 2] >> 4 | c[..., 3] << 6, c[..., 3] >> 2], -1) & 255
    return b.to(torch.uint8).view(codes.shape[0], -1)


def prepare(case, seed):
    V, M, ds, L, K, N, k = (case[x] for x in ("V", "M", "ds", "L", "K", "N", "k"))
    D, dev = M * ds, "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    # rows of about unit norm, each further level a quarter of the one before
    sigma = 0.02 * math.sqrt(2304.0 / D) * 0.25 ** torch.arange(L, device=dev, dtype=torch.float32)
    C = torch.randn(M, L, K, ds, generator=g, device=dev) * sigma.view(1, L, 1, 1)
    codes = torch.randint(0, K, (V, M * L), generator=g, device=dev, dtype=torch.int16)
    s = {"case": case, "C": C, "codes": _pack(codes, case["fmt"])}

    def rows(ids):
        at = codes[ids].long() + torch.arange(M * L, device=dev) * K
        return C.view(-1, ds)[at].view(len(ids), M, L, ds).sum(2).view(len(ids), D)

    def ids(*shape):      # frequent ids and rare ones, with repeats
        return (float(V) ** torch.rand(*shape, generator=g, device=dev)).long().clamp_(max=V) - 1

    # hidden states that favour their target by anything from nothing to almost certainty
    lead = 1.15 * math.log(V) * torch.rand(N, 1, generator=g, device=dev)
    h = torch.randn(N, D, generator=g, device=dev) * 0.83
    masked = torch.rand(N, generator=g, device=dev) < 0.05           # padding in the batch
    masked[0] = False
    if k:
        # a teacher's top logits, descending, over distinct ids; some rows list fewer
        t = (torch.rand(N, 1, generator=g, device=dev) * V).long()
        t = (t + torch.arange(k, device=dev) * max(1, (V - 1) // k)) % V
        val = 14.0 - 2.0 * torch.log1p(torch.arange(k, device=dev, dtype=torch.float32))
        val = (val + 0.5 * torch.randn(N, k, generator=g, device=dev)).sort(1, descending=True).values
        h += lead * rows(t[:, 0]) + 0.5 * lead * rows(t[:, k // 2])
        short = torch.randint(1, 2 * k + 1, (N, 1), generator=g, device=dev)
        t = torch.where((torch.arange(k, device=dev) < short) & ~masked[:, None], t, -1)
        s["val"], s["idx"] = val, t.int()
    else:
        t = ids(N)
        h += lead * rows(t)
        s["target"] = torch.where(masked, -1, t).int()
    s["h"] = h.to(getattr(torch, case["h"]))
    s["weight"] = torch.full((N,), 1.0 / N, device=dev)              # the mean over the batch
    if own:
        import lut_logits_serving_b200 as rq
        s["d"] = rq.dims(V, D, M, L, K)
        s["code_fmt"] = {"u16": rq.U16, "u8": rq.U8, "packed10": rq.PACKED10}[case["fmt"]]
        step = case["op"].endswith("_step")
        s["index"] = rq.rq_prepare_grad(s["codes"], s["code_fmt"], s["d"]) if step else None
        s["ws"] = torch.empty(rq.rq_loss_workspace_bytes(s["d"], N, s["code_fmt"], k, step), dtype=torch.uint8,
                              device=dev)
    return s


def _run_own(s):
    import lut_logits_serving_b200 as rq
    c, head = s["case"], (s["h"], s["C"], s["codes"], s["code_fmt"], s["d"])
    kw = {"softcap": c["cap"], "ws": s["ws"]}
    if c["k"]:
        teacher = (s["val"], s["idx"])
        loss, lse, _ = rq.rq_distill(*head, *teacher, temperature=c["T"], **kw)
    else:
        loss, lse, _ = rq.rq_xent(*head, s["target"], **kw)
    out = {"loss": loss, "lse": lse}
    if c["op"].endswith("_step"):
        kw |= {"weight": s["weight"], "index": s["index"]}
        if c["k"]:
            out["dh"], out["dC"], _ = rq.rq_distill_grad(*head, *teacher, lse, temperature=c["T"], **kw)
        else:
            out["dh"], out["dC"], _ = rq.rq_xent_grad(*head, s["target"], lse, **kw)
    return out


def _unpack(codes, fmt, P):
    """The codes [V, P] as int64."""
    if fmt == "u16":
        return codes.view(torch.int16).long()
    if fmt == "u8":
        return codes.long()
    bit = torch.arange(P, device=codes.device) * 10
    b = codes.int()
    return ((b[:, bit // 8] | b[:, bit // 8 + 1] << 8) >> (bit % 8).int() & 1023).long()


def run(s):
    if own:
        return _run_own(s)
    c, C = s["case"], s["C"]
    V, M, L, K, ds, T, cap = c["V"], c["M"], c["L"], c["K"], c["ds"], c["T"], c["cap"]
    at = _unpack(s["codes"], c["fmt"], M * L) + torch.arange(M * L, device=C.device) * K
    E = C.view(-1, ds)[at].view(V, M, L, ds).sum(2).view(V, M * ds)
    h = s["h"].float()
    y = h @ E.t()
    if cap > 0:
        y = cap * torch.tanh(y / cap)
    top = y.amax(1, keepdim=True) / T
    lse = (torch.exp(y / T - top).sum(1, keepdim=True).log() + top)
    if c["k"]:
        ids, listed_ = s["idx"].long(), s["idx"] >= 0
        some = listed_.any(1)
        t = torch.where(listed_, s["val"] / T, -torch.inf)
        e = torch.exp(t - torch.where(some, t.amax(1), 0.0)[:, None])
        q = e / torch.where(some, e.sum(1), 1.0)[:, None]
        log_q = torch.where(q > 0, q, 1.0).log()
        loss = T * T * (q * (log_q - y.gather(1, ids.clamp(min=0)) / T + lse)).sum(1)
    else:
        ids, some = s["target"].long()[:, None], s["target"] >= 0
        q = some.float()[:, None]
        loss = torch.where(some, (lse - y.gather(1, ids.clamp(min=0)))[:, 0], 0.0)
    out = {"loss": loss, "lse": lse[:, 0]}
    if c["op"].endswith("_step"):
        dy = torch.exp(y / T - lse)
        dy.scatter_add_(1, ids.clamp(min=0), -q)
        dy *= (some * s["weight"] * T)[:, None]
        if cap > 0:
            dy *= 1.0 - (y / cap) ** 2
        # the sum over the vocabulary in blocks: one chain of V products loses bits in 32
        n, block = -(-V // 4096), 4096
        pad = torch.nn.functional.pad
        parts = pad(dy, (0, n * block - V)).view(-1, n, block).transpose(0, 1) @ pad(E, (0, 0, 0, n * block - V)).view(
            n, block, -1)
        out["dh"] = parts.sum(0).to(s["h"].dtype)
        dE = (dy.t() @ h).view(V, M, 1, ds).expand(V, M, L, ds).reshape(-1, ds)
        out["dC"] = torch.zeros_like(C).view(-1, ds).index_add_(0, at.view(-1), dE).view_as(C)
    return out


def work(case):
    V, M, ds, L, K, N, k = (case[x] for x in ("V", "M", "ds", "L", "K", "N", "k"))
    D, hb = M * ds, 4 if case["h"] == "float32" else 2
    codes = V * (-(-10 * M * L // 8) if case["fmt"] == "packed10" else M * L * (2 if case["fmt"] == "u16" else 1))
    books = M * L * K * ds * 4
    read = codes + books + N * D * hb + N * (8 * k if k else 4)
    if case["op"].endswith("_step"):
        return {"bytes": read + 4 * N + 8 * N + N * D * hb + books, "flops": 6 * N * V * D}
    return {"bytes": read + 8 * N, "flops": 2 * N * V * D}


def exact(case, seed):
    """The definition in 64 bits, by blocks of the vocabulary."""
    s = prepare(case, seed)
    V, M, L, K, ds, N, T, cap = (case[x] for x in ("V", "M", "L", "K", "ds", "N", "T", "cap"))
    dev, f64 = s["C"].device, torch.float64
    C, h = s["C"].to(f64), s["h"].to(f64)
    block = 16384

    def codes_of(v0, v1):
        c = s["codes"][v0:v1]
        if case["fmt"] == "u16":
            return c.view(torch.int16).long()
        if case["fmt"] == "u8":
            return c.long()
        bits = (c.long()[:, :, None] >> torch.arange(8, device=dev) & 1).view(v1 - v0, -1)[:, :10 * M * L]
        return (bits.view(v1 - v0, M * L, 10) << torch.arange(10, device=dev)).sum(2)

    def block_of(v0):
        v1 = min(V, v0 + block)
        c = codes_of(v0, v1).view(v1 - v0, M, L)
        E = torch.zeros(v1 - v0, M, ds, dtype=f64, device=dev)
        for m in range(L):
            E += C[torch.arange(M, device=dev), m, c[:, :, m]]
        z = h @ E.view(v1 - v0, M * ds).t()
        return v1, c, E.view(v1 - v0, M * ds), cap * torch.tanh(z / cap) if cap > 0 else z

    # the teacher's (or the target's) probabilities, entry by entry
    if case["k"]:
        ids = s["idx"].long()
        q = torch.softmax((s["val"].to(f64) / T).masked_fill(ids < 0, -math.inf), 1).nan_to_num(0.0)
    else:
        ids = s["target"].long()[:, None]
        q = (ids >= 0).to(f64)
    has = (ids >= 0).any(1).to(f64)
    lse = torch.full((N,), -math.inf, dtype=f64, device=dev)
    at_ids = torch.zeros_like(q)
    for v0 in range(0, V, block):
        v1, _, _, y = block_of(v0)
        lse = torch.logaddexp(lse, torch.logsumexp(y / T, 1))
        here = (ids >= v0) & (ids < v1)
        at_ids = torch.where(here, y.gather(1, (ids - v0).clamp(0, v1 - v0 - 1)), at_ids)
    loss = T * T * (torch.xlogy(q, q) - q * (at_ids / T - lse[:, None])).sum(1)
    out = {"loss": loss, "lse": lse}
    if case["op"].endswith("_step"):
        dh, dC = torch.zeros_like(h), torch.zeros_like(C)
        f = has * s["weight"].to(f64) * T
        for v0 in range(0, V, block):
            v1, c, E, y = block_of(v0)
            here = (ids >= v0) & (ids < v1)
            dy = torch.exp(y / T - lse[:, None])
            dy.scatter_add_(1, (ids - v0).clamp(0, v1 - v0 - 1), -q * here)
            dz = dy * f[:, None] * (1 - (y / cap) ** 2 if cap > 0 else 1)
            dh += dz @ E
            dE = (dz.t() @ h).view(v1 - v0, M, ds)
            for m in range(L):
                at = (torch.arange(M, device=dev) * K + c[:, :, m]).view(-1)
                dC[:, m] += torch.zeros(M * K, ds, dtype=f64, device=dev).index_add_(
                    0, at, dE.reshape(-1, ds)).view(M, K, ds)
        out["dh"], out["dC"] = dh, dC
    return out
