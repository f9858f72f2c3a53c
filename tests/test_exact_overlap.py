"""Outputs of the exact operators that share memory with an input, with another
output or with the workspace are refused on the host (no GPU needed)."""
import ctypes

import pytest

import adaptive_vector_quantized_b200 as avq

P = ctypes.byref
BAD = avq.AVQ_ERR_INVALID_ARG
AT = {n: 0x100000000 * (i + 1) for i, n in enumerate(
    "Q K V dYq dYk dO O wq wk bq bk pos freqs lse lens mask Yq Yk dQ dK dV dwq dwk dbq dbk ws".split())}
B, N, HQ, HK, D = 2, 10, 4, 2, 64
NK = 20


@pytest.fixture(autouse=True)
def nothing_is_launched(monkeypatch):
    monkeypatch.setenv("AVQ_FAULT", "all")


def st(h, n):
    return P(avq.avq_strides(h * n * D, n * D, D))


def qk(norm, hk=HK):
    return avq.avq_qk_dims(B, N, HQ, hk, D, 32, 1, 1, 0, norm, 1e-6, 1.0)


def rotary(m):
    return avq.lib().avq_rotary(P(qk(0)), avq.AVQ_BF16, m["Q"], st(HQ, N), m["K"], st(HK, N), m["pos"], m["freqs"], 0,
                                m["Yq"], m["Yk"], None)


def norm(m):
    return avq.lib().avq_qk_norm(P(qk(1)), avq.AVQ_BF16, m["Q"], st(HQ, N), m["K"], st(HK, N), m["wq"], m["wk"], m["bq"],
                                 m["bk"], m["pos"], m["freqs"], m["Yq"], m["Yk"], None)


def norm_backward(m, hk=HK):
    return avq.lib().avq_qk_norm_backward(
        P(qk(2, hk)), avq.AVQ_BF16, m["dYq"], st(HQ, N), m["dYk"], st(HK, N), m["Q"], st(HQ, N), m["K"], st(HK, N),
        m["wq"], m["wk"], m["pos"], m["freqs"], m["dQ"], m["dK"], m["dwq"], m["dwk"], m["dbq"], m["dbk"], m["ws"], 1 << 30,
        None)


def cd():
    return avq.avq_cross_dims(B, B, HQ, HK, 300, NK, D, 0.125)


def cross(m, dims=None):
    return avq.lib().avq_cross_attention(P(dims or cd()), avq.AVQ_BF16, m["Q"], st(HQ, 300), m["K"], st(HK, NK), m["V"],
                                         st(HK, NK), m["lens"], m["mask"], m["O"], st(HQ, 300), m["lse"], m["ws"], 1 << 30,
                                         None)


def cross_backward(m):
    return avq.lib().avq_cross_attention_backward(
        P(cd()), avq.AVQ_BF16, m["dO"], st(HQ, 300), m["Q"], st(HQ, 300), m["K"], st(HK, NK), m["V"], st(HK, NK), m["O"],
        st(HQ, 300), m["lse"], m["lens"], m["mask"], m["dQ"], m["dK"], m["dV"], m["ws"], 1 << 30, None)


Q_BYTES, K_BYTES = B * HQ * N * D * 2, B * HK * N * D * 2
# call, its outputs and their bytes, its inputs and theirs
CALLS = {
    "rotary": (rotary, dict(Yq=Q_BYTES, Yk=K_BYTES), dict(Q=Q_BYTES, K=K_BYTES, pos=B * N * 4, freqs=16 * 8)),
    "norm": (norm, dict(Yq=Q_BYTES, Yk=K_BYTES),
             dict(Q=Q_BYTES, K=K_BYTES, wq=D * 2, wk=D * 2, bq=D * 2, bk=D * 2, pos=B * N * 4, freqs=16 * 8)),
    "norm_backward": (norm_backward, dict(dQ=Q_BYTES, dK=K_BYTES, dwq=D * 4, dwk=D * 4, dbq=D * 4, dbk=D * 4, ws=256),
                      dict(dYq=Q_BYTES, dYk=K_BYTES, Q=Q_BYTES, K=K_BYTES, wq=D * 2, wk=D * 2, pos=B * N * 4, freqs=16 * 8)),
    "cross_backward": (cross_backward, dict(dQ=B * HQ * 300 * D * 2, dK=B * HK * NK * D * 2, dV=B * HK * NK * D * 2, ws=256),
                       dict(dO=B * HQ * 300 * D * 2, Q=B * HQ * 300 * D * 2, K=B * HK * NK * D * 2, V=B * HK * NK * D * 2,
                            O=B * HQ * 300 * D * 2, lse=B * HQ * 300 * 4, lens=B * 4, mask=B * NK)),
    "cross": (cross, dict(O=B * HQ * 300 * D * 2, lse=B * HQ * 300 * 4),
              dict(Q=B * HQ * 300 * D * 2, K=B * HK * NK * D * 2, V=B * HK * NK * D * 2, lens=B * 4, mask=B * NK)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_apart_are_taken(name):
    call, outs, ins = CALLS[name]
    assert call(AT) == avq.AVQ_ERR_CUDA and "injected" in avq.last_error()
    # one right behind the other
    for o, size in outs.items():
        for i in ins:
            if o != "ws":
                assert call(dict(AT, **{i: AT[o] + size})) == avq.AVQ_ERR_CUDA, avq.last_error()


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_that_overlap_are_refused(name):
    call, outs, ins = CALLS[name]
    for o in outs:
        for i, size in ins.items():
            # at the input's first bytes and inside its last 256 (the workspace's alignment), 16 (theirs)
            for at in {AT[i], AT[i] + (size - 1) // (256 if o == "ws" else 16) * (256 if o == "ws" else 16)}:
                assert call(dict(AT, **{o: at})) == BAD and "overlaps" in avq.last_error(), (o, i, avq.last_error())
        for p, size in outs.items():
            if p != o:
                assert call(dict(AT, **{o: AT[p]})) == BAD and "overlaps" in avq.last_error(), (o, p)


def test_cross_workspace_apart():
    """Long keys, so that the forward call needs a workspace."""
    dims = avq.avq_cross_dims(B, B, HQ, HK, 300, 20000, D, 0.125)
    assert avq.avq_cross_workspace_size(dims, avq.AVQ_BF16) > 0

    def call(**kw):
        m = dict(AT, **kw)
        return avq.lib().avq_cross_attention(P(dims), avq.AVQ_BF16, m["Q"], st(HQ, 300), m["K"], st(HK, 20000), m["V"],
                                             st(HK, 20000), m["lens"], m["mask"], m["O"], st(HQ, 300), m["lse"], m["ws"],
                                             1 << 30, None)

    assert call() == avq.AVQ_ERR_CUDA
    for t in ("Q", "K", "V", "lens", "mask", "O", "lse"):
        assert call(ws=AT[t]) == BAD and "overlaps" in avq.last_error(), t


def test_sums_of_absent_keys_are_not_looked_at():
    m = dict(AT, K=None, dYk=None, dK=None, dwk=AT["Q"], dbk=AT["Q"] + 4)
    assert norm_backward(m, 0) == avq.AVQ_ERR_CUDA, avq.last_error()
