"""GPU tests of the losses on the RQ-coded head (rq_xent, rq_distill) and their
gradients against the definition in 64 bits, elementwise, within bounds derived
in tests/loss_ref.py: both paths (few tokens, tensor cores), every code layout,
odd shapes, masks that leave rows empty, streams, graphs and repeats."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lut_logits_serving_b200 as rq  # noqa: E402
from tests import loss_ref  # noqa: E402

FMT = {"u16": rq.U16, "u8": rq.U8, "packed10": rq.PACKED10, "sched": rq.SCHED, "rot10": rq.ROT10}


class Head:
    """An artifact and hidden states that favour some ids."""

    def __init__(self, V, M, ds, L, K, N, dtype=torch.float32, fmt="u16", seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        D = M * ds
        self.g, self.N, self.V, self.k = g, N, V, 0
        self.d = rq.dims(V, D, M, L, K)
        sig = (1.0 / D) ** 0.5 * 0.25 ** torch.arange(L, device="cuda", dtype=torch.float32)
        self.C = torch.randn(M, L, K, ds, generator=g, device="cuda") * sig.view(1, L, 1, 1)
        self.codes = torch.randint(0, K, (V, M, L), generator=g, device="cuda")
        u16 = self.codes.to(torch.int16).view(torch.uint16).view(V, M * L)
        self.fmt = FMT[fmt]
        self.packed = {"u16": lambda: u16, "u8": lambda: rq.rq_pack8(u16, self.d),
                       "packed10": lambda: rq.rq_pack10(u16, self.d),
                       "sched": lambda: rq.rq_prepare_sched(u16, self.d),
                       "rot10": lambda: rq.rq_prepare_rot10(u16, self.d)}[fmt]()
        self.target = torch.randint(0, V, (N,), generator=g, device="cuda").int()
        E, _ = loss_ref.rows(self.C, self.codes)
        lead = 8 * torch.rand(N, 1, generator=g, device="cuda")
        h = torch.randn(N, D, generator=g, device="cuda") * 0.8 + lead * E[self.target.long()].float()
        self.h = h.to(dtype)
        self.weight = torch.rand(N, generator=g, device="cuda") - 0.3
        self.index = rq.rq_prepare_grad(self.packed, self.fmt, self.d)

    def teacher(self, k):
        self.k = k
        self.idx = torch.randint(0, self.V, (self.N, k), generator=self.g, device="cuda").int()
        self.val = 4 * torch.randn(self.N, k, generator=self.g, device="cuda")
        return self

    def args(self):
        return (self.h, self.C, self.packed, self.fmt, self.d)

    def run(self, T=1.0, cap=30.0, weight=None, grad=True, **kw):
        if self.k:
            loss, lse, ws = rq.rq_distill(*self.args(), self.val, self.idx, temperature=T,
                                          softcap=cap, **kw)
        else:
            loss, lse, ws = rq.rq_xent(*self.args(), self.target, softcap=cap, **kw)
        out = {"loss": loss, "lse": lse}
        if grad:
            kw2 = dict(weight=weight, softcap=cap, **kw)
            if self.k:
                out["dh"], out["dC"], _ = rq.rq_distill_grad(*self.args(), self.val, self.idx, lse,
                                                             self.index, temperature=T, **kw2)
            else:
                out["dh"], out["dC"], _ = rq.rq_xent_grad(*self.args(), self.target, lse,
                                                          self.index, **kw2)
        return out

    def check(self, T=1.0, cap=30.0, weight=None, **kw):
        got = self.run(T, cap, weight, **kw)
        ids, val = (self.idx, self.val) if self.k else (self.target, None)
        ref = loss_ref.losses(self.h, self.C, self.codes, ids, val, T, cap, weight)
        compare(got, ref, self.h.dtype == torch.bfloat16)
        return got, ref


def compare(got, ref, bf16):
    lim = loss_ref.bounds(ref, bf16)
    torch.cuda.synchronize()
    for name, x in got.items():
        if x is None:
            continue
        y = ref[name].view(x.shape)
        off = (x.to(torch.float64) - y).abs()
        bad = ~(off <= lim[name].view(x.shape))
        assert not bad.any(), (name, int(bad.sum()), off.max().item(), y.abs().max().item(),
                               torch.nonzero(bad)[0].tolist(), x[bad][0].item(), y[bad][0].item(),
                               lim[name].view(x.shape)[bad][0].item())
    assert rq.rq_device_error() == 0


@pytest.fixture(autouse=True)
def _clear():
    rq.rq_device_error()
    yield


# V, M, ds, L, K, N, dtype, fmt, T, cap
FEW = [
    (4096, 32, 6, 2, 256, 1, "f", "u16", 1.0, 30.0),
    (1, 4, 2, 1, 1, 1, "f", "u16", 1.0, 30.0),
    (37, 8, 6, 2, 7, 2, "f", "u16", 1.0, 0.0),
    (8192, 16, 3, 1, 100, 3, "b", "u8", 0.7, 30.0),
    (8193, 32, 5, 2, 64, 4, "f", "packed10", 2.0, 50.0),
    (20011, 64, 2, 3, 1000, 5, "b", "u16", 1.0, 30.0),
    (5000, 32, 6, 2, 1024, 16, "f", "sched", 1.0, 30.0),
    (5000, 32, 6, 2, 512, 7, "f", "rot10", 1.5, 30.0),
    (3000, 3, 40, 5, 4096, 2, "f", "u16", 1.0, 10.0),
    (40000, 67, 8, 3, 64, 4, "b", "u16", 1.5, 30.0),
    (33000, 21, 8, 1, 500, 20, "f", "packed10", 1.0, 30.0),
    (1, 1, 1, 1, 1, 3, "f", "u8", 1.0, 30.0),
]
MANY = [
    (4096, 32, 6, 2, 256, 33, "f", "u8", 1.0, 30.0),
    (4099, 32, 6, 2, 1024, 65, "f", "u16", 1.0, 30.0),
    (32768, 24, 8, 2, 100, 128, "b", "u16", 1.0, 30.0),
    (40961, 16, 5, 3, 200, 129, "f", "u16", 1.3, 0.0),
    (1, 4, 2, 1, 1, 70, "f", "u16", 1.0, 30.0),
    (300, 7, 3, 1, 16, 200, "b", "u16", 4.0, 30.0),
    (9000, 64, 6, 2, 1024, 300, "f", "packed10", 1.0, 30.0),
    (5000, 32, 6, 2, 1024, 90, "f", "sched", 1.0, 30.0),
    (5000, 32, 6, 2, 512, 80, "b", "rot10", 1.5, 30.0),
    (700, 3, 40, 5, 4096, 66, "f", "u16", 1.0, 10.0),
    (2000, 2, 350, 1, 30, 20, "f", "u16", 1.0, 30.0),
    (66000, 16, 4, 2, 500, 257, "f", "u16", 1.0, 30.0),
]


def _head(c, seed=0):
    V, M, ds, L, K, N, t, fmt, T, cap = c
    return Head(V, M, ds, L, K, N, torch.float32 if t == "f" else torch.bfloat16, fmt, seed), T, cap


@pytest.mark.parametrize("c", FEW + MANY)
def test_xent(c):
    x, _, cap = _head(c)
    x.check(cap=cap)
    x.check(cap=cap, weight=x.weight)


@pytest.mark.parametrize("c", FEW + MANY)
def test_distill(c):
    x, T, cap = _head(c, 1)
    x.teacher(min(x.V, 9)).check(T, cap, weight=x.weight)


@pytest.mark.parametrize("N", [3, 70])
def test_long_lists_with_repeats(N):
    """k = 1024 of 1500 ids: many listed twice; lists as rq_topk_sample gives them."""
    x = Head(1500, 16, 6, 2, 64, N)
    x.teacher(1024).check(1.5)
    y = torch.randn(N, 1500, device="cuda")
    x.val, x.idx, _ = rq.rq_topk_sample(y, 50)
    x.k = 50
    x.check(2.0)


@pytest.mark.parametrize("N", [5, 100])
def test_empty_rows(N):
    """Masked targets, padded lists, -inf entries; a whole batch of none."""
    x = Head(3000, 16, 6, 2, 100, N, seed=3)
    x.target[::2] = -1
    x.target[0] = -2147483648
    got, ref = x.check(weight=x.weight)
    assert (got["loss"][::2] == 0).all() and (got["dh"][::2] == 0).all()
    x.teacher(7)
    x.idx[1] = -1
    x.val[2] = -torch.inf
    x.val[3, 1:] = -torch.inf
    x.idx[4, ::2] = -1
    x.val[4, 0] = torch.nan          # beside an id that stands for none
    got, ref = x.check(1.3)
    for n in (1, 2):
        assert got["loss"][n] == 0 and (got["dh"][n] == 0).all()
    x.idx[:] = -1
    got, ref = x.check()
    assert (got["dC"] == 0).all() and (got["dh"] == 0).all() and (got["loss"] == 0).all()


@pytest.mark.parametrize("N", [2, 66])
def test_ids_past_the_vocabulary(N):
    x = Head(500, 8, 6, 2, 32, N)
    x.target[1] = 500
    x.run()
    torch.cuda.synchronize()
    assert rq.rq_device_error() == 2
    want = dict(x.run())
    rq.rq_device_error()
    x.target[1] = -1
    got = x.run()
    for n in got:
        assert torch.equal(got[n], want[n])


@pytest.mark.parametrize("N", [4, 80])
@pytest.mark.parametrize("K", [100, 64])
def test_codes_past_the_codebook(N, K):
    x = Head(600, 8, 6, 2, K, N)
    x.codes[::3] += K
    x.packed = x.codes.to(torch.int16).view(torch.uint16).view(x.V, -1)
    x.index = rq.rq_prepare_grad(x.packed, x.fmt, x.d)
    x.check()


@pytest.mark.parametrize("N", [4, 80])
def test_one_code_for_every_row(N):
    """All rows share a codeword: one list with every row, the others empty."""
    x = Head(20000, 8, 6, 2, 256, N)
    x.codes[:] = 17
    x.packed = x.codes.to(torch.int16).view(torch.uint16).view(x.V, -1)
    x.index = rq.rq_prepare_grad(x.packed, x.fmt, x.d)
    x.check()


@pytest.mark.parametrize("K,skew", [(40, 0.0), (600, 0.0), (600, 0.5), (3, 0.9)])
def test_index(K, skew):
    """The index lists each row once per column, under its code, in order."""
    R, cap, P = 8192, 32, 3
    x = Head(R + 77, P, 2, 1, K, 1)
    codes = x.codes.view(x.V, P)
    codes[torch.rand(x.V, P, generator=x.g, device="cuda") < skew] = K // 2
    x.packed = codes.to(torch.int16).view(torch.uint16)
    raw = rq.rq_prepare_grad(x.packed, rq.U16, x.d).cpu().numpy()
    up = lambda n, a: (n + a - 1) // a * a  # noqa: E731
    g = 1
    while g < 32 and K * g < 1024:
        g *= 2
    ns = (K * g + 31) // 32
    code_at = up(2 * ns + 2, 16)
    over_at = code_at + up(2 * K, 16)
    entry_at = up(over_at + 2 * (R // (g * (cap - 1) + 1) + 2), 128)
    unit = entry_at + up(2 * (R + 32 * cap + (64 if g > 1 else 32) * ns), 128)
    assert raw.size == 2 * P * unit == rq.rq_grad_index_bytes(x.d)
    codes = codes.cpu().numpy()
    for b, n in ((0, R), (1, 77)):
        for p in range(P):
            u = raw[(b * P + p) * unit:][:unit].view(np.uint16)
            off, code, over = u[:ns + 1].astype(int), u[code_at // 2:][:K], u[over_at // 2:]
            entry = u[entry_at // 2:] // 4
            assert (u[entry_at // 2:][:64 * off[ns]] % 4 == 0).all()
            assert sorted(code) == list(range(K)) and off[0] == 0
            seen = 0
            for s in range(K):
                lanes = []
                for vl in range(s * g, s * g + g):
                    sl = vl // 32
                    lane = entry[64 * off[sl]:64 * off[sl + 1]].reshape(-1, 32, 2)[:, vl % 32].reshape(-1)
                    lanes.append(lane[lane < R])
                    assert (lane[len(lanes[-1]):] == R).all()
                got = np.full(g * max(map(len, lanes)) if lanes else 0, R)
                for i, lane in enumerate(lanes):
                    got[i::g][:len(lane)] = lane
                got = got[got < R]
                if s < over[0]:
                    rest = entry[64 * off[ns]:][over[1 + s]:over[2 + s]]
                    got = np.concatenate([got, rest])
                want = np.nonzero(codes[b * R:b * R + n, p] == code[s])[0]
                assert np.array_equal(got, want)
                seen += len(got)
            assert seen == n


@pytest.mark.parametrize("N", [3, 150])
def test_extreme_sizes_of_values(N):
    """Hidden states and codebooks far from 1, rows of very different size, a
    zero row, weights of 0 and far apart, no softcap."""
    x = Head(2000, 16, 6, 2, 64, N, seed=5)
    x.h *= 1e-6
    x.h[0] = 0
    x.h[1] *= 1e5
    x.C *= 1e4
    x.weight[::2] = 0
    x.weight[1] = 1e3
    x.check(cap=0.0, weight=x.weight)
    x.C.zero_()
    x.check(weight=x.weight)


@pytest.mark.parametrize("N", [4, 130])
def test_one_gradient_alone_and_repeats(N):
    x = Head(9000, 16, 6, 2, 256, N, seed=6)
    a = x.run()
    b = x.run()
    for n in a:
        assert torch.equal(a[n], b[n])
    dh, none, _ = rq.rq_xent_grad(*x.args(), x.target, a["lse"], x.index, want_dC=False)
    assert none is None and torch.equal(dh, a["dh"])
    none, dC, _ = rq.rq_xent_grad(*x.args(), x.target, a["lse"], x.index, want_dh=False)
    assert none is None and torch.equal(dC, a["dC"])
    # outputs and workspace of NaN: everything is written
    ws = torch.full((rq.rq_loss_workspace_bytes(x.d, N, x.fmt, 1, True) // 4 + 1,), torch.nan,
                    device="cuda")
    dh, dC = torch.full_like(a["dh"], torch.nan), torch.full_like(a["dC"], torch.nan)
    rq.rq_xent_grad(*x.args(), x.target, a["lse"], x.index, dh=dh, dC=dC, ws=ws)
    assert torch.equal(dh, a["dh"]) and torch.equal(dC, a["dC"])


@pytest.mark.parametrize("N", [3, 90])
def test_streams_and_graphs(N):
    """Another stream; a captured loss and gradient, replayed on new inputs;
    two at once, each with its own workspace."""
    x, y = Head(9000, 16, 6, 2, 256, N, seed=7), Head(9000, 16, 6, 2, 256, N, seed=8)
    want, want2 = x.run(), y.run()
    torch.cuda.synchronize()
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got, got2 = x.run(stream=s), y.run(stream=s2)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]) and torch.equal(got2[n], want2[n])
    ws = torch.empty(rq.rq_loss_workspace_bytes(x.d, N, x.fmt, 1, True), dtype=torch.uint8,
                     device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = x.run(ws=ws)
    g.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(out[n], want[n])
    x.h.copy_(y.h)
    x.target.copy_(y.target)
    x.C.copy_(y.C)
    x.packed.copy_(y.packed)
    x.index.copy_(y.index)
    g.replay()
    torch.cuda.synchronize()
    for n in want2:
        assert torch.equal(out[n], want2[n])


@pytest.mark.parametrize("N", [4, 70])
def test_against_differences(N):
    """The gradients against central differences of the loss in 64 bits."""
    x = Head(700, 8, 6, 2, 32, N, seed=9).teacher(5)
    got, ref = x.check(2.0, weight=x.weight)
    g = torch.Generator("cuda").manual_seed(1)
    for name in ("h", "C"):
        v = getattr(x, name)
        u = torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float64)
        u /= u.norm()
        step = 1e-4

        def at(e):
            w = {"h": x.h.double(), "C": x.C.double()}
            w[name] = w[name] + e * u
            r = loss_ref.losses(w["h"], w["C"], x.codes, x.idx, x.val, 2.0, 30.0)
            return (x.weight.double() * r["loss"]).sum()

        diff = (at(step) - at(-step)).item() / (2 * step)
        grad = got["d" + name].double()
        # third derivatives of these losses are below 1e3: 1e-4^2 / 6 of that,
        # and fp32's part of the gradient's length
        assert abs((grad * u).sum().item() - diff) <= 2e-6 + 1e-5 * grad.norm().item()


def test_calls_in_a_row():
    """A run of the calls as they are used: encode rows, take the uncompressed
    head's top logits, distil, step the codebooks, score again.  The step
    along the gradient changes the loss as the gradient says."""
    from lut_logits_serving_b200 import synth
    V, M, ds, L, K, N, k = 3000, 16, 6, 2, 64, 80, 20
    D = M * ds
    X = torch.from_numpy(synth.rows(V, D, D ** -0.5, 4)).cuda()
    C = torch.from_numpy(synth.codebooks(M, L, K, ds, (D ** -0.5, 0.4 * D ** -0.5), 0)).cuda()
    d = rq.dims(V, D, M, L, K)
    codes = rq.rq_encode(X, C, d)
    index = rq.rq_prepare_grad(codes, rq.U16, d)
    h = torch.from_numpy(synth.hidden(N, D, 3.0, 2)).cuda()
    teacher = 30 * torch.tanh(h @ X.t() / 30)
    val, idx, _ = rq.rq_topk_sample(teacher, k)
    loss, lse, ws = rq.rq_distill(h, C, codes, rq.U16, d, val, idx)
    _, dC, _ = rq.rq_distill_grad(h, C, codes, rq.U16, d, val, idx, lse, index, want_dh=False)
    step = 1e-3 / dC.norm()
    after, _, _ = rq.rq_distill(h, C - step * dC, codes, rq.U16, d, val, idx, ws=ws)
    want = -(step * dC.double().square().sum()).item()
    moved = (after.double().sum() - loss.double().sum()).item()
    # the second derivative along the step is below 1e3 |h|^2-scaled units: a
    # tenth of the first-order change at this step
    assert abs(moved - want) <= 0.1 * abs(want) + 1e-4
    y, am, _ = rq.rq_logits_from_hidden(h, C, codes, rq.U16, d, 30.0, want_argmax=True)
    assert torch.allclose(torch.logsumexp(y.double(), 1), lse.double(), atol=1e-4)


JUNK = (float("nan"), float("inf"), -3e38, 1e30, -float("inf"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [3, 20, 100])
def test_padding_may_hold_anything(N, dtype):
    """Rows without a target: their hidden states, weights and lse, finite or
    not, reach no other row and no gradient."""
    x = Head(3000, 16, 6, 2, 100, N, dtype, seed=11)
    pad = torch.arange(N, device="cuda") % 5 != 2
    pad[0] = True
    junk = torch.tensor(JUNK, device="cuda")[torch.arange(N, device="cuda") % 5]
    clean = x.h.masked_fill(pad[:, None], 0)
    x.h = torch.where(pad[:, None], junk[:, None].to(dtype), x.h)
    x.h[::2, 1::3] = clean[::2, 1::3]
    x.weight[pad] = junk[pad]
    for k in (0, 6):
        if k:
            x.teacher(k)
            x.idx[pad] = -1
            x.val[pad] = junk[pad, None]
        else:
            x.target[pad] = -1
        got = x.run(1.3 if k else 1.0, weight=x.weight)
        w = x.weight.masked_fill(pad, 1)
        ids, val = (x.idx, x.val.masked_fill(pad[:, None], 0)) if k else (x.target, None)
        ref = loss_ref.losses(clean, x.C, x.codes, ids, val, 1.3 if k else 1.0, 30.0, w)
        assert (got["loss"][pad] == 0).all() and (got["dh"][pad] == 0).all()
        got["lse"] = torch.where(pad, ref["lse"].float(), got["lse"])
        compare(got, ref, dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [4, 24, 130])
def test_rows_keep_their_own_precision(N, dtype):
    """Rows and weights twelve orders of magnitude apart: each row's loss, lse
    and dh within the bounds of that row alone."""
    x = Head(2500, 16, 6, 2, 64, N, dtype, seed=12)
    n = torch.arange(N, device="cuda")
    x.h = (x.h.float() * 10.0 ** (3 * (n % 5) - 6.0)[:, None]).to(dtype)
    x.weight = 10.0 ** (3 * (n // 5 % 5) - 8.0)
    got = x.run(weight=x.weight)
    for i in range(N):
        s = slice(i, i + 1)
        ref = loss_ref.losses(x.h[s], x.C, x.codes, x.target[s], None, 1.0, 30.0, x.weight[s])
        compare({m: got[m][s] for m in ("loss", "lse", "dh")}, ref, dtype == torch.bfloat16)
    ref = loss_ref.losses(x.h, x.C, x.codes, x.target, None, 1.0, 30.0, x.weight)
    compare({"dC": got["dC"]}, ref, dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [4099, 8192])
def test_several_sweeps_of_tokens(N, dtype):
    """More tokens than one sweep over the vocabulary takes; a short last one."""
    x = Head(500, 4, 6, 2, 32, N, dtype, seed=13)
    x.target[::7] = -1
    x.check(weight=x.weight)
    x.teacher(3).check(2.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [3, 77])
def test_unaligned_tensors(N, dtype):
    """Every float tensor an element past a 16-byte boundary: the same bits."""
    x = Head(2100, 8, 6, 2, 64, N, dtype, seed=14)
    x.teacher(5)
    want = x.run(weight=x.weight)

    def off(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.reshape(-1)
        return b[1:].view(t.shape)

    for name in ("h", "C", "weight", "val", "idx"):
        setattr(x, name, off(getattr(x, name)))
    got = x.run(weight=x.weight)
    for name in want:
        assert torch.equal(got[name], want[name]), name
    dh, dC = off(want["dh"]), off(want["dC"])
    rq.rq_distill_grad(*x.args(), x.val, x.idx, off(want["lse"]), x.index, temperature=1.0,
                       weight=x.weight, dh=dh, dC=dC)
    assert torch.equal(dh, want["dh"]) and torch.equal(dC, want["dC"])


@pytest.mark.parametrize("c", [
    (5, 6, 2, 100, "u16"), (6, 6, 2, 64, "u8"), (8, 5, 1, 50, "packed10"), (16, 2, 2, 300, "packed10"),
    (13, 2, 3, 40, "u16"), (22, 2, 1, 40, "u16"), (9, 8, 3, 30, "u8"), (12, 8, 3, 30, "u8"),
    (16, 3, 2, 70, "packed10"), (24, 4, 3, 33, "u8"), (32, 5, 3, 200, "u8"), (64, 3, 1, 20, "u8"),
    (64, 4, 1, 20, "packed10"), (32, 6, 1, 1000, "packed10"), (32, 3, 2, 300, "sched"),
    (64, 4, 1, 512, "rot10"), (10, 7, 2, 60, "u16"), (3, 16, 4, 20, "u8"), (7, 6, 2, 4000, "u16")])
def test_decoding(c):
    """Rows rebuilt for the tensor cores from codes in words of 16 and 4 bytes
    and one by one, units of subspaces that end early, columns filled up."""
    M, ds, L, K, fmt = c
    x = Head(777, M, ds, L, K, 66, fmt=fmt, seed=15)
    x.check()


@pytest.mark.parametrize("c", [
    (30005, 256, 6, 2, 32, "u16"), (30001, 256, 6, 2, 32, "u8"), (20003, 96, 8, 2, 40, "u16"),
    (20003, 96, 8, 3, 40, "u8"), (31001, 256, 4, 1, 20, "packed10"), (61000, 256, 2, 3, 25, "u8"),
    (125000, 128, 3, 2, 30, "u8")])
def test_decoding_many_rows(c):
    """The same where codes are fetched many rows ahead, with chunks that end
    unevenly and a second piece."""
    V, M, ds, L, K, fmt = c
    x = Head(V, M, ds, L, K, 66, fmt=fmt, seed=16)
    x.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_same_bits_every_time(dtype):
    """Copies that run ahead of their readers meet none of them: a head whose
    codes come rows ahead, forty calls."""
    x = Head(70001, 256, 6, 2, 1024, 200, dtype, seed=17)
    want = x.run()
    for _ in range(40):
        got = x.run()
        for n in want:
            assert torch.equal(got[n], want[n]), n
