"""Host-only checks of the losses' C calls and binding (no GPU, no kernel
launched): malformed arguments are refused before any CUDA call, sizes add up,
the binding names what is wrong."""
import ctypes

import pytest

import lut_logits_serving_b200 as rq

G2 = rq.dims(256000, 2304, 384, 2, 1024)
TINY = rq.dims(4096, 192, 32, 2, 256)
INV, UNS, WS, MIS = 1, 2, 3, 5
BIG = 1 << 40


def _p(x):
    return ctypes.c_void_p(x)


A, S, NULL = _p(0x100000), _p(None), _p(None)     # never dereferenced: every call returns early


def xent(h=A, bf=0, C=A, codes=A, fmt=0, d=G2, N=8, cap=30.0, target=A, loss=A, lse=A, ws=A,
         n=BIG):
    return rq.lib().rq_xent(h, bf, C, codes, fmt, d, N, cap, target, loss, lse, ws, n, S)


def xent_grad(h=A, bf=0, C=A, codes=A, fmt=0, d=G2, N=8, target=A, lse=A, w=NULL, index=A, dh=A,
              dC=A, ws=A, n=BIG):
    return rq.lib().rq_xent_grad(h, bf, C, codes, fmt, d, N, 30.0, target, lse, w, index, dh, dC,
                                 ws, n, S)


def distill(val=A, idx=A, k=5, T=1.0, d=G2, N=8, ws=A, n=BIG):
    return rq.lib().rq_distill(A, 0, A, A, 0, d, N, 30.0, val, idx, k, T, A, A, ws, n, S)


def distill_grad(val=A, idx=A, k=5, T=1.0, d=G2, N=8, index=A, ws=A, n=BIG):
    return rq.lib().rq_distill_grad(A, 0, A, A, 0, d, N, 30.0, val, idx, k, T, A, NULL, index, A,
                                    A, ws, n, S)


def test_null_pointers_and_values():
    for name in ("h", "C", "codes", "target", "loss", "lse"):
        assert xent(**{name: NULL}) == INV, name
    for name in ("h", "C", "codes", "target", "lse", "index"):
        assert xent_grad(**{name: NULL}) == INV, name
    assert xent_grad(dh=NULL, dC=NULL) == INV          # nothing asked for
    assert xent(N=0) == INV and xent(N=-3) == INV and xent(bf=2) == INV
    assert xent(fmt=9) == INV and xent(fmt=-1) == INV
    assert xent(d=rq.dims(10, 7, 2, 1, 4)) == INV      # D % M != 0
    assert distill(val=NULL) == INV and distill(idx=NULL) == INV
    for k in (0, -1):
        assert distill(k=k) == INV
    assert distill(k=11, d=rq.dims(10, 12, 2, 1, 4)) == INV          # more than V
    for T in (0.0, -1.0, float("inf"), float("nan"), 1e-45):
        assert distill(T=T) == INV, T
        assert distill_grad(T=T) == INV, T
    assert distill_grad(val=NULL) == INV and distill_grad(index=NULL) == INV


def test_unsupported():
    assert distill(k=1025) == UNS
    assert xent(fmt=rq.U8) == UNS                                     # K > 256
    assert xent(fmt=rq.SCHED, d=rq.dims(10, 48, 24, 1, 64)) == UNS    # M L % 32
    big = rq.dims(1000, 64, 8, 1, 5000)
    assert rq.rq_grad_index_bytes(big) == 0
    assert xent_grad(d=big) == UNS
    assert rq.lib().rq_prepare_grad(A, 0, big, _p(0x900000000), S) == UNS


def test_alignment():
    for name, off in (("h", 2), ("C", 2), ("codes", 8), ("target", 2), ("loss", 2), ("lse", 1),
                      ("ws", 128)):
        assert xent(**{name: _p(0x100000 + off)}) == MIS, name
    assert xent(h=_p(0x100002), bf=1, ws=NULL) == WS                  # bf16: 2 bytes will do
    for name, off in (("lse", 2), ("w", 2), ("index", 8), ("dh", 2), ("dC", 2)):
        assert xent_grad(**{name: _p(0x100000 + off)}) == MIS, name


def _apart(**kw):
    """Arguments 64 GB apart, so that none meets another."""
    return {n: _p((i + 1) << 36) for i, n in enumerate(kw)} | {n: v for n, v in kw.items() if v}


def test_outputs_meet_nothing():
    """Before any launch: an output or the workspace on an input or on another output."""
    f = dict.fromkeys(("h", "C", "codes", "target", "loss", "lse", "ws"))
    a = _apart(**f)
    for x, y, off in (("loss", "lse", 28), ("loss", "target", -28), ("lse", "h", 64), ("ws", "C", 256),
                      ("C", "ws", 256), ("loss", "ws", 1024), ("codes", "lse", -16)):
        assert xent(**_apart(**f | {x: _p(a[y].value + off)})) == INV, (x, y)
    f = dict.fromkeys(("h", "C", "codes", "target", "lse", "w", "index", "dh", "dC", "ws"))
    a = _apart(**f)
    for x, y in (("dh", "h"), ("dC", "C"), ("dC", "dh"), ("dh", "index"), ("dC", "ws"), ("dh", "w"),
                 ("ws", "codes"), ("dC", "lse")):
        assert xent_grad(**_apart(**f | {x: a[y]})) == INV, (x, y)


@pytest.mark.parametrize("d", [G2, TINY, rq.dims(1, 1, 1, 1, 1), rq.dims(50021, 640, 128, 3, 200)])
@pytest.mark.parametrize("N", [1, 4, 20, 64, 65, 5000])
def test_workspace(d, N):
    need = rq.rq_loss_workspace_bytes(d, N, rq.U16)
    both = rq.rq_loss_workspace_bytes(d, N, rq.U16, 1, True)
    assert 0 < need <= both
    assert rq.rq_loss_workspace_bytes(d, N, rq.U16, 0) == need        # cross entropy: k 0 or 1
    assert xent(d=d, N=N, n=need - 1) == WS and xent(d=d, N=N, ws=NULL) == WS
    assert xent_grad(d=d, N=N, ws=NULL) == WS and xent_grad(d=d, N=N, n=0) == WS
    # logits of every token are never kept for more than a few of them
    assert both < 8e9


def test_sizes():
    assert rq.rq_loss_workspace_bytes(G2, 0, 0) == 0
    assert rq.rq_loss_workspace_bytes(G2, 8, 7) == 0
    assert rq.rq_loss_workspace_bytes(G2, 8, rq.U8) == 0
    assert rq.rq_loss_workspace_bytes(G2, 8, 0, 1025) == 0
    assert rq.rq_loss_workspace_bytes(rq.dims(10, 7, 2, 1, 4), 8, 0) == 0
    assert rq.rq_loss_workspace_bytes(rq.dims(10, 12, 2, 1, 4), 8, 0, 11) == 0
    # two bytes a code, padding and tables: below twice the codes for the full head
    codes = rq.rq_codes_bytes(G2, rq.U16)
    assert codes < rq.rq_grad_index_bytes(G2) < 2 * codes
    assert rq.rq_grad_index_bytes(rq.dims(0, 12, 2, 1, 4)) == 0


def test_prepare_grad_refuses():
    f = rq.lib().rq_prepare_grad
    far = _p(0x900000000)
    assert f(NULL, 0, TINY, far, S) == INV and f(A, 0, TINY, NULL, S) == INV
    assert f(A, 5, TINY, far, S) == INV and f(A, rq.U8, G2, far, S) == UNS
    assert f(_p(0x100008), 0, TINY, far, S) == MIS and f(A, 0, TINY, _p(0x900000008), S) == MIS
    assert f(A, 0, TINY, _p(0x100000 + 4096), S) == INV               # overlap


def test_binding_names_what_is_wrong(monkeypatch):
    torch = pytest.importorskip("torch")
    real = rq.lib()

    class NoLaunch:
        def __getattr__(self, name):
            if name.endswith("_bytes") or name in ("rq_lut_token_stride", "rq_status_string"):
                return getattr(real, name)

            def reached(*a):
                raise RuntimeError(f"{name} reached")
            return reached

    d, N, k = TINY, 3, 4
    h = torch.zeros(N, d.D)
    C = torch.zeros(d.M, d.L, d.K, d.D // d.M)
    codes = torch.zeros((d.V, d.M * d.L), dtype=torch.uint16)
    t = torch.zeros(N, dtype=torch.int32)
    lse = torch.zeros(N)
    val, idx = torch.zeros(N, k), torch.zeros(N, k, dtype=torch.int32)
    index = torch.zeros(rq.rq_grad_index_bytes(d), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        rq.rq_xent(h, C, codes, rq.U16, d, t)
    monkeypatch.setattr(rq, "lib", lambda: NoLaunch())
    monkeypatch.setattr(rq, "_on_device", lambda x: True)
    monkeypatch.setattr(rq, "_stream", lambda s: ctypes.c_void_p(None))

    def refused(fn, *a, match, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)

    def reaches(fn, *a, **kw):
        with pytest.raises(RuntimeError, match="reached"):
            fn(*a, **kw)

    head = (h, C, codes, rq.U16, d)
    reaches(rq.rq_xent, *head, t)
    reaches(rq.rq_xent, h.bfloat16(), C, codes, rq.U16, d, t)
    reaches(rq.rq_xent, h[0], C, codes, rq.U16, d, t[:1])             # one token
    refused(rq.rq_xent, h.half(), *head[1:], t, match="h: dtype")
    refused(rq.rq_xent, h[:, :-1], *head[1:], t, match="h: shape")
    refused(rq.rq_xent, torch.zeros(d.D, N).t(), *head[1:], t, match="h: must be contiguous")
    refused(rq.rq_xent, h, C[:-1], *head[2:], t, match="C: .* bytes")
    refused(rq.rq_xent, h, C, codes[:-1], rq.U16, d, t, match="codes: .* bytes")
    refused(rq.rq_xent, *head, t.long(), match="target: dtype")
    refused(rq.rq_xent, *head, t[:-1], match="target: .* bytes")
    refused(rq.rq_xent, *head, t, loss=torch.zeros(N - 1), match="loss: .* bytes")
    refused(rq.rq_xent, *head, [0, 1, 2], match="target: expected")
    reaches(rq.rq_distill, *head, val, idx)
    refused(rq.rq_distill, *head, val[:, :-1], idx, match="teacher_val, teacher_idx")
    refused(rq.rq_distill, *head, val, idx[:-1], match="teacher_val, teacher_idx")
    refused(rq.rq_distill, *head, val.double(), idx, match="teacher_val: dtype")
    reaches(rq.rq_xent_grad, *head, t, lse, index)
    refused(rq.rq_xent_grad, *head, t, lse[:-1], index, match="lse: .* bytes")
    refused(rq.rq_xent_grad, *head, t, lse, index[:-1], match="index: .* bytes")
    refused(rq.rq_xent_grad, *head, t, lse, index, weight=lse.double(), match="weight: dtype")
    refused(rq.rq_xent_grad, *head, t, lse, index, dh=torch.zeros(N, d.D).bfloat16(),
            match="dh: dtype")
    refused(rq.rq_xent_grad, *head, t, lse, index, dC=C[:-1], match="dC: .* bytes")
    reaches(rq.rq_distill_grad, *head, val, idx, lse, index)
    refused(rq.rq_distill_grad, *head, val, idx.long(), lse, index, match="teacher_idx: dtype")
    refused(rq.rq_prepare_grad, codes[:-1], rq.U16, d, match="codes_?.*bytes")
    reaches(rq.rq_prepare_grad, codes, rq.U16, d)
