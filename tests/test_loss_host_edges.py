"""Host-only checks of the losses at the ends of their ranges (no GPU): sizes
that every accepted shape has to fit, refusals before any launch, and that a
refused call leaves the caller's device and arguments alone."""
import pytest

import lut_logits_serving_b200 as rq


@pytest.mark.parametrize("V", [1, 3000, 8191, 8192, 256000])
def test_every_accepted_codebook_has_room(V):
    """The sums by code keep two units of the index, the values of a block of
    8192 rows and a column's sums in shared memory (226 KB)."""
    blocks = (V + 8191) // 8192
    for K in range(1, 4097):
        unit = rq.rq_grad_index_bytes(rq.dims(V, 1, 1, 1, K)) // blocks
        assert 0 < 2 * unit + (2 * 8192 + 4) * 4 + 8 * K <= 226 * 1024, K
    assert rq.rq_grad_index_bytes(rq.dims(V, 1, 1, 1, 4097)) == 0


@pytest.mark.parametrize("N,V", [(63, 227000), (48, 75000), (40, 120000), (33, 20000), (33, 256000)])
def test_logits_of_33_to_63_tokens_are_not_priced_as_one_group(N, V):
    """The serving kernels take 64 tokens in one pass, 33 to 63 in two, which
    is slower than one product; a call on the serving kernels' logits needs
    little more workspace than those, one on products the decoded rows."""
    d = rq.dims(V, 2304, 384, 2, 1024)
    planes = 4 * 2304 * min(V, 131072)
    assert rq.rq_loss_workspace_bytes(d, N, rq.U16) > planes
    one = rq.dims(256000, 2304, 384, 2, 1024)
    assert rq.rq_loss_workspace_bytes(one, 32, rq.U16) < 4 * 2304 * 131072


class _OnDevice:
    """What a tensor or a stream of another GPU says of itself."""
    is_cuda = True

    def __init__(self, index, N=3, D=192):
        import torch
        self.device, self.shape, self.dtype = torch.device("cuda", index), (N, D), torch.float32
        self.cuda_stream = 0

    def dim(self):
        return 2


@pytest.fixture
def devices(monkeypatch):
    """torch.cuda's current device and stream without a GPU; the list of devices
    entered and left."""
    torch = pytest.importorskip("torch")
    log = []

    class Context:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            log.append(("enter", self.what))

        def __exit__(self, *exc):
            log.append(("leave", self.what))

    monkeypatch.setattr(torch.cuda, "device", lambda d: Context(str(d)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: Context("stream of " + str(s.device)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return log


def test_a_stream_of_another_device_leaves_the_current_one(devices):
    """The refusal comes before the tensors' device is made current: no context
    is left behind by a call that raises."""
    call = rq._LossCall.__new__(rq._LossCall)
    call.h, call.stream, call.stack = _OnDevice(1), _OnDevice(0), None
    call.device = call.h.device
    with pytest.raises(ValueError, match="stream on cuda:0, h on cuda:1"):
        with call:
            raise AssertionError("entered")
    assert devices == []
    call.stream = _OnDevice(1)
    with call:
        pass
    assert [what for what, _ in devices] == ["enter", "enter", "leave", "leave"]


def test_prepare_grad_on_a_stream_of_another_device(devices, monkeypatch):
    torch = pytest.importorskip("torch")
    d = rq.dims(3, 192, 32, 2, 64)

    class Codes(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", 1)

    def codes():
        return torch.zeros((3, 64), dtype=torch.uint16).as_subclass(Codes)

    launched = []
    monkeypatch.setattr(rq, "_on_device", lambda t: True)
    monkeypatch.setattr(rq, "_stream", lambda s: None)
    monkeypatch.setattr(rq, "_check", lambda name, status: launched.append(name))
    out = torch.zeros(rq.rq_grad_index_bytes(d), dtype=torch.uint8).as_subclass(Codes)
    with pytest.raises(ValueError, match="stream on cuda:0, codes on cuda:1"):
        rq.rq_prepare_grad(codes(), rq.U16, d, out=out, stream=_OnDevice(0))
    assert devices == [] and launched == []
    with pytest.raises(ValueError, match="codes: expected a torch.Tensor"):
        rq.rq_prepare_grad([1, 2], rq.U16, d)
    with pytest.raises(ValueError, match="index: expected a torch.Tensor"):
        rq.rq_prepare_grad(codes(), rq.U16, d, out=[0])
    with pytest.raises(ValueError, match="out: on cpu, codes on cuda:1"):
        rq.rq_prepare_grad(codes(), rq.U16, d, out=torch.zeros_like(torch.empty(out.shape, dtype=torch.uint8)))
    assert launched == []


@pytest.mark.parametrize("wrong", [None, [0, 1], 3.0])
def test_arguments_that_are_no_tensors_are_named(wrong, monkeypatch):
    torch = pytest.importorskip("torch")
    d, N, k = rq.dims(4096, 192, 32, 2, 256), 3, 4
    f32, i32 = torch.float32, torch.int32
    good = {"h": torch.zeros(N, d.D), "C": torch.zeros(32, 2, 256, 6),
            "codes": torch.zeros((d.V, 64), dtype=torch.uint16), "teacher_val": torch.zeros(N, k),
            "teacher_idx": torch.zeros(N, k, dtype=i32), "lse": torch.zeros(N, dtype=f32),
            "index": torch.zeros(rq.rq_grad_index_bytes(d), dtype=torch.uint8)}
    monkeypatch.setattr(rq, "_on_device", lambda x: True)
    for name in good:
        a = dict(good)
        a[name] = wrong
        head = (a["h"], a["C"], a["codes"], rq.U16, d, a["teacher_val"], a["teacher_idx"])
        with pytest.raises(ValueError, match=f"{name}: expected a torch.Tensor"):
            rq.rq_distill_grad(*head, a["lse"], a["index"])
        if name not in ("lse", "index"):
            with pytest.raises(ValueError, match=f"{name}: expected a torch.Tensor"):
                rq.rq_distill(*head)
    if wrong is not None:
        a = good
        with pytest.raises(ValueError, match="ws: expected a torch.Tensor"):
            rq.rq_distill(a["h"], a["C"], a["codes"], rq.U16, d, a["teacher_val"], a["teacher_idx"],
                          ws=wrong)


def test_current_stream_without_torch_s_private_name(monkeypatch):
    torch = pytest.importorskip("torch")
    stream = _OnDevice(0)
    stream.cuda_stream = 0x1230
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x4560, raising=False)
    assert rq._stream(None).value == 0x4560
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert rq._stream(None).value == 0x1230 and rq._stream(stream).value == 0x1230


def test_softcaps_without_a_finite_value_are_refused():
    """cap tanh(z / cap) of an infinite cap is infinity times 0, of one whose
    reciprocal is infinite a NaN at z = 0; none or a negative one is off."""
    import ctypes
    a, null = ctypes.c_void_p(0x100000), ctypes.c_void_p(None)
    d = rq.dims(4096, 192, 32, 2, 256)

    def xent(cap):
        return rq.lib().rq_xent(a, 0, a, a, 0, d, 8, cap, a, a, a, null, 0, null)

    def xent_grad(cap):
        return rq.lib().rq_xent_grad(a, 0, a, a, 0, d, 8, cap, a, a, null, a, a, a, null, 0, null)

    for f in (xent, xent_grad):
        assert f(float("inf")) == 1 and f(1e-39) == 1
        for cap in (30.0, 0.0, -1.0, -float("inf"), 1e-37, 3e38):
            assert f(cap) == 3, cap                     # on to the missing workspace
