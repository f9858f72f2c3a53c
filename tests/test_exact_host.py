"""The exact operators' entry points refuse bad arguments on the host, before
anything is launched (no GPU needed), and the rotation's frequencies follow
their formulas."""
import ctypes
import math

import pytest
import torch

import adaptive_vector_quantized_b200 as avq

P = ctypes.byref
FAKE = [0x100000000 * i for i in range(1, 12)]  # 16-byte aligned, never dereferenced
BAD = avq.AVQ_ERR_INVALID_ARG


def qk(**kw):
    d = dict(B=2, N=10, Hq=4, Hk=2, d=64, rot=64, axes=1, pos_batch=0, layout=0, norm=avq.AVQ_NORM_RMS, eps=1e-6,
             mscale=1.0)
    d.update(kw)
    return avq.avq_qk_dims(*(d[n] for n, _ in avq.avq_qk_dims._fields_))


def dense(B, H, N, d):
    return avq.avq_strides(H * N * d, N * d, d)


QS, KS = dense(2, 4, 10, 64), dense(2, 2, 10, 64)


def norm(dims=None, dt=avq.AVQ_BF16, Q=FAKE[0], qs=QS, K=FAKE[1], ks=KS, w=None, pos=None, f=FAKE[2], Yq=FAKE[3],
         Yk=FAKE[4]):
    return avq.lib().avq_qk_norm(P(dims or qk()), dt, Q, P(qs) if qs else None, K, P(ks) if ks else None, w, None,
                                 None, None, pos, f, Yq, Yk, None)


@pytest.mark.parametrize("kw, status", [
    (dict(dims=qk(B=0)), BAD), (dict(dims=qk(N=0)), BAD), (dict(dims=qk(Hq=0)), BAD), (dict(dims=qk(Hk=-1)), BAD),
    (dict(dims=qk(d=96)), avq.AVQ_ERR_UNSUPPORTED), (dict(dims=qk(B=1 << 15, N=1 << 15)), avq.AVQ_ERR_UNSUPPORTED),
    (dict(dims=qk(rot=4)), BAD), (dict(dims=qk(rot=72)), BAD), (dict(dims=qk(rot=-8)), BAD),
    (dict(dims=qk(rot=8, axes=2)), BAD), (dict(dims=qk(axes=3)), BAD), (dict(dims=qk(layout=2)), BAD),
    (dict(dims=qk(norm=3)), BAD), (dict(dims=qk(norm=0)), BAD), (dict(dims=qk(eps=-1.0)), BAD),
    (dict(dims=qk(eps=math.nan)), BAD), (dict(dims=qk(mscale=math.inf)), BAD), (dict(dt=7), BAD),
    (dict(Q=None), BAD), (dict(Q=FAKE[0] + 8), BAD), (dict(K=None), BAD), (dict(qs=None), BAD),
    (dict(qs=avq.avq_strides(2560, 640, 60)), BAD), (dict(qs=avq.avq_strides(-8, 640, 64)), BAD),
    (dict(w=FAKE[5] + 2), BAD), (dict(pos=FAKE[5] + 2), BAD), (dict(f=None), BAD), (dict(f=FAKE[2] + 4), BAD),
    (dict(Yq=None), BAD), (dict(Yk=None), BAD), (dict(Yq=FAKE[0] + 16), BAD), (dict(Yk=FAKE[3] + 16), BAD),
])
def test_qk_norm_refuses(kw, status):
    assert norm(**kw) == status, avq.last_error()
    assert avq.last_error()


def test_rotary_refuses():
    L = avq.lib()

    def call(dims, f=FAKE[2]):
        return L.avq_rotary(P(dims), avq.AVQ_F32, FAKE[0], P(QS), FAKE[1], P(KS), None, f, 0, FAKE[3], FAKE[4], None)

    assert call(qk()) == BAD and "AVQ_NORM_NONE" in avq.last_error()
    assert call(qk(norm=0), None) == BAD and "freqs" in avq.last_error()
    assert L.avq_rotary(None, 0, FAKE[0], P(QS), None, P(KS), None, FAKE[2], 0, FAKE[3], None, None) == BAD


def test_qk_norm_backward_refuses():
    L = avq.lib()
    need = L.avq_qk_norm_workspace_size(P(qk()), avq.AVQ_BF16)
    assert need > 0 and need % 256 == 0

    def call(dims=None, dQ=FAKE[5], ws=FAKE[8], n=need, dw=FAKE[7], dYq=FAKE[0]):
        return L.avq_qk_norm_backward(P(dims or qk()), avq.AVQ_BF16, dYq, P(QS), FAKE[1], P(KS), FAKE[2], P(QS),
                                      FAKE[3], P(KS), None, None, None, FAKE[4], dQ, FAKE[6], dw, None, None, None,
                                      ws, n, None)

    assert call(ws=None) == avq.AVQ_ERR_WORKSPACE
    assert call(n=need - 1) == avq.AVQ_ERR_WORKSPACE
    assert call(ws=FAKE[8] + 16) == BAD
    assert call(dQ=FAKE[2]) == BAD and "overlaps" in avq.last_error()
    assert call(dw=FAKE[7] + 4) == BAD
    assert call(dYq=None) == BAD
    assert call(qk(norm=0)) == BAD


def cd(**kw):
    d = dict(B=2, Bk=2, Hq=4, Hk=2, Nq=10, Nk=20, d=64, scale=0.125)
    d.update(kw)
    return avq.avq_cross_dims(*(d[n] for n, _ in avq.avq_cross_dims._fields_))


CQ, CK = dense(2, 4, 10, 64), dense(2, 2, 20, 64)


def cross(dims=None, dt=avq.AVQ_BF16, Q=FAKE[0], qs=CQ, K=FAKE[1], ks=CK, V=FAKE[2], O=FAKE[3], os_=CQ, lens=None,
          lse=None, ws=FAKE[9], n=1 << 40):
    return avq.lib().avq_cross_attention(P(dims or cd()), dt, Q, P(qs), K, P(ks), V, P(ks), lens, None, O, P(os_), lse,
                                         ws, n, None)


@pytest.mark.parametrize("kw, status", [
    (dict(dims=cd(B=0)), BAD), (dict(dims=cd(B=3)), BAD), (dict(dims=cd(Hq=3)), BAD), (dict(dims=cd(Nq=0)), BAD),
    (dict(dims=cd(Nk=-1)), BAD), (dict(dims=cd(d=80)), avq.AVQ_ERR_UNSUPPORTED),
    (dict(dims=cd(Nq=1 << 28)), avq.AVQ_ERR_UNSUPPORTED), (dict(dims=cd(Nk=1 << 28)), avq.AVQ_ERR_UNSUPPORTED),
    (dict(dims=cd(scale=0.0)), BAD), (dict(dims=cd(scale=-1.0)), BAD), (dict(dims=cd(scale=math.inf)), BAD),
    (dict(dims=cd(scale=math.nan)), BAD), (dict(dt=2), BAD), (dict(Q=None), BAD), (dict(K=None), BAD),
    (dict(V=FAKE[2] + 2), BAD), (dict(O=None), BAD), (dict(O=FAKE[1] + 64), BAD), (dict(lens=FAKE[4] + 2), BAD),
    (dict(lse=FAKE[4] + 4), BAD), (dict(qs=avq.avq_strides(2560, 640, 65)), BAD),
    (dict(qs=avq.avq_strides(2560, 640, 0)), BAD), (dict(ks=avq.avq_strides(2560, 1280, 0)), BAD),
    (dict(os_=avq.avq_strides(2560, 0, 64)), BAD), (dict(os_=avq.avq_strides(2560, 640, 32)), BAD),
])
def test_cross_attention_refuses(kw, status):
    assert cross(**kw) == status, avq.last_error()
    assert avq.last_error()


def test_cross_attention_workspace_is_checked():
    L = avq.lib()
    for dims, dt in ((cd(Nk=20000), avq.AVQ_BF16), (cd(Nk=20000), avq.AVQ_F32), (cd(Nq=300, Nk=20000), avq.AVQ_BF16)):
        need = L.avq_cross_workspace_size(P(dims), dt, 0)
        assert need > 0 and need % 256 == 0  # few rows, many keys: split
        ks, qs = dense(2, 2, 20000, 64), dense(2, 4, dims.Nq, 64)
        assert cross(dims, dt, qs=qs, os_=qs, ks=ks, ws=None, n=0) == avq.AVQ_ERR_WORKSPACE
        assert cross(dims, dt, qs=qs, os_=qs, ks=ks, n=need - 1) == avq.AVQ_ERR_WORKSPACE
        assert cross(dims, dt, qs=qs, os_=qs, ks=ks, ws=FAKE[9] + 16) == BAD
    assert L.avq_cross_workspace_size(P(cd(B=3)), avq.AVQ_BF16, 0) == 0


def test_cross_attention_backward_refuses():
    L = avq.lib()
    need = L.avq_cross_workspace_size(P(cd()), avq.AVQ_BF16, 1)
    assert need > 0

    def call(dO=FAKE[0], lse=FAKE[5], dQ=FAKE[6], dK=FAKE[7], dV=FAKE[8], ws=FAKE[9], n=need):
        return L.avq_cross_attention_backward(P(cd()), avq.AVQ_BF16, dO, P(CQ), FAKE[1], P(CQ), FAKE[2], P(CK),
                                              FAKE[3], P(CK), FAKE[4], P(CQ), lse, None, None, dQ, dK, dV, ws, n,
                                              None)

    assert call(dO=None) == BAD
    assert call(lse=None) == BAD
    assert call(dK=None) == BAD
    assert call(dQ=FAKE[3]) == BAD and "overlaps" in avq.last_error()
    assert call(dV=FAKE[7]) == BAD and "overlap" in avq.last_error()
    assert call(ws=None) == avq.AVQ_ERR_WORKSPACE
    assert call(n=need - 1) == avq.AVQ_ERR_WORKSPACE


def test_injected_failures(monkeypatch):
    for entry, call in (("qk_norm", norm), ("cross_attention", cross)):
        monkeypatch.setenv("AVQ_FAULT", entry)
        assert call() == avq.AVQ_ERR_CUDA and "injected" in avq.last_error()


def test_tensors_are_checked():
    x = torch.zeros(1, 2, 3, 64)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):  # not on a GPU
        avq.avq_cross_attention(x, x, x)
    with pytest.raises(ValueError):
        avq.avq_rotary(x, freqs=f)
    with pytest.raises(ValueError):
        avq.avq_rotary(x)
    with pytest.raises(ValueError):
        avq.avq_qk_norm(x, norm="batch")
    with pytest.raises(ValueError):
        avq.avq_qk_norm(x, x[:, :, :2])


def test_rotary_freqs():
    f, m = avq.avq_rotary_freqs(64)
    assert m == 1.0 and f.dtype == torch.float64
    want = [10000.0 ** (-i / 32) for i in range(32)]
    assert torch.allclose(f, torch.tensor(want, dtype=torch.float64), rtol=1e-14)
    # two axes: each with the frequencies of a rotation of half the elements
    g, _ = avq.avq_rotary_freqs(64, axes=2)
    h, _ = avq.avq_rotary_freqs(32)
    assert torch.equal(g, torch.cat([h, h]))
    lin, _ = avq.avq_rotary_freqs(64, scaling="linear", factor=4.0)
    assert torch.allclose(lin * 4, f, rtol=1e-14)
    # the fastest pair is kept, the slowest divided by the factor
    ntk, _ = avq.avq_rotary_freqs(64, scaling="ntk", factor=4.0)
    assert ntk[0] == f[0] and abs(ntk[-1] * 4 / f[-1] - 1) < 1e-12 and (ntk[1:] < f[1:]).all()
    y, m = avq.avq_rotary_freqs(64, scaling="yarn", factor=8.0, trained=4096)
    assert abs(m - (0.1 * math.log(8.0) + 1)) < 1e-7
    turns = 4096 * f / (2 * math.pi)
    ratio = f / y
    lo, hi = int((turns > 32).nonzero().max()), int((turns < 1).nonzero().min())
    assert torch.allclose(ratio[:lo + 1], torch.ones(lo + 1, dtype=torch.float64), rtol=1e-12)
    assert torch.allclose(ratio[hi:], torch.full_like(ratio[hi:], 8.0), rtol=1e-12)
    inner = ratio[lo:hi + 1]
    assert (inner[1:] >= inner[:-1]).all()
    same, _ = avq.avq_rotary_freqs(64, scaling="yarn", factor=1.0)
    assert torch.allclose(same, f, rtol=1e-14)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=12), dict(rot=8, axes=2), dict(rot=64, axes=3),
                                dict(rot=64, base=1.0), dict(rot=64, factor=0.5), dict(rot=64, factor=math.nan),
                                dict(rot=64, scaling="yarn", trained=0),
                                dict(rot=64, scaling="yarn", turns_low=2.0, turns_high=1.0)])
def test_rotary_freqs_refuses(kw):
    with pytest.raises(avq.AVQError):
        avq.avq_rotary_freqs(**kw)


def test_cross_refuses_outputs_that_overlap_themselves(monkeypatch):
    S = avq.avq_strides
    monkeypatch.setenv("AVQ_FAULT", "cross_attention")
    for st in (S(2560, 640, 64), S(2560, 64, 256), S(64, 1280, 128), S(640, 1280, 64), S(10240, 64, 512)):
        assert cross(os_=st) == avq.AVQ_ERR_CUDA and "injected" in avq.last_error()  # every order of the dimensions
    for st in (S(64, 64, 128), S(640, 640, 64), S(2560, 576, 64), S(2560, 64, 192), S(2496, 64, 256), S(32, 640, 64)):
        assert cross(os_=st) == BAD and "must not overlap" in avq.last_error()


def test_cross_refuses_an_lse_inside_another_tensor():
    for t in (FAKE[0], FAKE[1], FAKE[2], FAKE[3] + 64):
        assert cross(lse=t) == BAD and "lse overlaps" in avq.last_error()
