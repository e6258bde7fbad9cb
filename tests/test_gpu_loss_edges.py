"""GPU tests of the losses on the RQ-coded head at the ends of their ranges:
large codebooks, wide subspaces, rows of E with a common part, values of any
size, lists of a teacher that hold the type's lowest value or NaN.  References
and heads as in test_gpu_loss.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lut_logits_serving_b200 as rq  # noqa: E402
from tests import loss_ref  # noqa: E402
from tests.test_gpu_loss import Head, compare  # noqa: E402


@pytest.fixture(autouse=True)
def _clear():
    rq.rq_device_error()
    yield


# V, M, ds, L, K, N
BOOKS = [
    (9001, 2, 2, 1, 3840, 4), (9001, 2, 2, 1, 3841, 4), (9001, 2, 2, 2, 3841, 70),
    (70001, 4, 3, 2, 4096, 5), (70001, 4, 3, 2, 4096, 70),       # shares of the blocks, an odd dim
    (25001, 400, 2, 1, 4096, 66),                                # several units a CTA, blocks each
    (25001, 75, 4, 3, 4000, 66), (8192, 5, 8, 2, 4096, 3), (8193, 3, 1, 1, 4096, 20),
    (150001, 2, 4, 1, 4096, 66),                                 # a second piece
]


@pytest.mark.parametrize("c", BOOKS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_codebooks(c, dtype):
    """Up to 4096 codewords on more rows than one block of the index has."""
    V, M, ds, L, K, N = c
    Head(V, M, ds, L, K, N, dtype, seed=20).check()


@pytest.mark.parametrize("N", [4, 70])
def test_large_codebooks_of_few_used_codewords(N):
    """A quarter of the rows share a codeword: lists that go on past their lanes."""
    x = Head(20001, 3, 4, 2, 4096, N, seed=21)
    x.codes[::4] = 4095
    x.packed = x.codes.to(torch.int16).view(torch.uint16).view(x.V, -1)
    x.index = rq.rq_prepare_grad(x.packed, x.fmt, x.d)
    a, _ = x.check()
    for _ in range(5):
        b = x.run()
        for n in a:
            assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("k", [0, 12])
@pytest.mark.parametrize("N", [80, 300])
def test_bf16_gradient_of_rows_with_a_common_part(N, k):
    """Rows of E that share a component 200 times their spread.  dz sums to zero
    over the vocabulary without a softcap, so dh holds none of it: what is lost
    of dz or E shows.  Within the bounds of float operands and one rounding to
    bf16."""
    x = Head(3000, 16, 6, 2, 100, N, torch.bfloat16, seed=22)
    g = torch.Generator("cuda").manual_seed(1)
    # 200 x the spread of an element (1 / sqrt(D) and a quarter of that)
    x.C[:, 0] += 200 * (1.0 / x.d.D) ** 0.5 * torch.randn(16, 1, 6, generator=g, device="cuda").sign()
    x.h = (1e-4 * x.h.float()).bfloat16()
    ids, val = x.target, None
    if k:
        x.teacher(k)
        x.val /= 4
        ids, val = x.idx, x.val
    got = x.run(cap=0.0)
    ref = loss_ref.losses(x.h, x.C, x.codes, ids, val, 1.0, 0.0)
    lim = loss_ref.bounds(ref, False)["dh"] + 2.0 ** -8 * ref["dh"].abs()
    off = (got["dh"].double() - ref["dh"]).abs()
    assert (off <= lim).all(), (off / lim).max().item()


@pytest.mark.parametrize("c", [
    (600, 1, 2050, 1, 4, 66, "u16"),       # codebooks in shared memory
    (600, 1, 2050, 2, 40, 2, "u8"),        # too large for it
    (500, 2, 1025, 1, 16, 66, "u16"), (500, 2, 1025, 2, 10, 66, "packed10"),
    (300, 3, 1025, 2, 300, 67, "u16"), (300, 5, 1027, 3, 7, 3, "u8"),
    (130, 1, 6145, 1, 9, 70, "u16"), (130, 2, 4098, 4, 5, 70, "u8")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_subspaces(c, dtype):
    """More pairs of dims in a group of subspaces than a CTA has threads."""
    V, M, ds, L, K, N, fmt = c
    Head(V, M, ds, L, K, N, dtype, fmt, seed=23).check()


@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
@pytest.mark.parametrize("N", [3, 70])
def test_teacher_of_lowest_and_largest_values(N, T):
    """Finite logits that the temperature takes out of float's range: only their
    differences count.  (-inf alone stands for no entry.)"""
    low = torch.finfo(torch.float32).min
    x = Head(900, 8, 6, 2, 32, N, seed=24).teacher(6)
    same = x.val.clone()
    x.val[0], same[0] = low, 0.0                       # a row of it: all alike
    x.val[1], same[1] = -low, 0.0
    x.val[2, 1:], same[2, 1:] = low, -torch.inf        # beside another: nothing
    got = x.run(T, weight=x.weight)
    ref = loss_ref.losses(x.h, x.C, x.codes, x.idx, same, T, 30.0, x.weight)
    compare(got, ref, False)


@pytest.mark.parametrize("N", [3, 70])
def test_teacher_of_nan(N):
    """A list with NaN gives NaN in its row, one of nothing but NaN too, and in
    no other row."""
    x = Head(900, 8, 6, 2, 32, N, seed=25).teacher(6)
    ref = loss_ref.losses(x.h, x.C, x.codes, x.idx, x.val, 1.3, 30.0)
    x.val[0] = torch.nan
    x.val[1, 3] = torch.nan
    x.idx[1, :2] = -1
    got = x.run(1.3)
    assert got["loss"][:2].isnan().all() and got["dC"].isnan().any()
    assert got["dh"][:2].isnan().all()
    ok = {n: got[n][2:] for n in ("loss", "dh")}
    compare(ok | {"lse": got["lse"][2:]}, {n: ref[n][2:] if n in ("loss", "lse", "dh", "dh_mag") else ref[n]
                                           for n in ref}, False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [4, 24, 90])
def test_powers_of_two(N, dtype):
    """Hidden states up and codebooks down by a power of two, and weights by
    one: the same bits of the loss, gradients times the power."""
    x = Head(2500, 16, 6, 2, 64, N, dtype, seed=26)
    h, C = x.h, x.C
    want = x.run(weight=x.weight)
    for e in (83, -83, 30):
        s = 2.0 ** e
        x.h, x.C = (h.float() * s).to(dtype), C / s
        got = x.run(weight=x.weight)
        for n, f in (("loss", 1.0), ("lse", 1.0), ("dh", 1 / s), ("dC", s)):
            assert torch.equal(got[n].double(), want[n].double() * f), (e, n)
    x.h, x.C = h, C
    for e in (-60, 40, 80):
        s = 2.0 ** e
        got = x.run(weight=x.weight * s)
        for n in ("dh", "dC"):
            assert torch.equal(got[n].double(), want[n].double() * s), (e, n)


# V, M, ds, L, K: lists shared by lanes, by level, three unit buffers, one value buffer
@pytest.mark.parametrize("c", [(9000, 16, 6, 2, 256), (9000, 5, 3, 2, 40), (9001, 160, 4, 2, 1024),
                               (9001, 2, 4, 1, 4096), (700, 8, 6, 1, 64)])
@pytest.mark.parametrize("N", [4, 70])
def test_index_of_other_sizes(c, N):
    """An index that is none of these codes': an error, and the next call as ever."""
    V, M, ds, L, K = c
    x = Head(V, M, ds, L, K, N, seed=27)
    want, mine = x.run(), x.index
    other = Head(V, M, ds, L, 2 * K if K < 4096 else K // 2, 1, seed=28).index
    n = mine.numel()
    g = torch.Generator("cuda").manual_seed(2)
    for name, index in (("ones", torch.full_like(mine, 255)),
                        ("noise", torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8)),
                        ("other", torch.cat([other, mine])[:n].contiguous()),
                        ("shifted", torch.roll(mine, 2)), ("zeros", torch.zeros_like(mine))):
        x.index = index
        got = x.run()
        torch.cuda.synchronize()
        err = rq.rq_device_error()
        assert err in ((4,) if name in ("ones", "noise") else (0, 4)), (name, err)
        assert torch.equal(got["loss"], want["loss"])
    x.index = mine
    got = x.run()
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert rq.rq_device_error() == 0
