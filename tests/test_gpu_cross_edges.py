"""Exact attention where its arithmetic degenerates: one key to a row, scores
and inputs that are not finite, gradients of keys that are left out."""
import pytest
import torch

import adaptive_vector_quantized_b200 as avq
from tests import exact_ref as ref
from tests.test_gpu_cross import DT, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["bf16", "bf16_cuda_cores", "f32"])
def family(request):
    """The element type, on the kernels that it is computed by."""
    old = avq.avq_set_path(avq.AVQ_PATH_SIMT if request.param == "bf16_cuda_cores" else avq.AVQ_PATH_AUTO)
    yield DT[request.param.split("_")[0]]
    avq.avq_set_path(old)


# ---- one key -------------------------------------------------------------------------------
# The softmax over one key is 1 whatever its score, so dQ and dK are 0 by
# definition: dO V^T and rowsum(dO O) are one number, whose two forms in fp32
# must not leave their difference behind.


# B, Bk, Hq, Hk, Nq, Nk, lens, the keys that a mask leaves of each encoder sequence
LONE = {
    "nk_1": (2, 1, 4, 2, 130, 1, None, None),
    "nk_1_many_rows": (1, 1, 2, 1, 5000, 1, None, None),
    "lens": (3, 3, 2, 2, 70, 40, [1, 40, 0], None),
    "mask": (4, 2, 4, 2, 90, 300, None, [[170], [0, 299]]),
    "mask_and_lens": (2, 2, 2, 2, 33, 500, [260, 500], [[257, 260, 499], [3]]),
    "mask_one_tile": (2, 2, 2, 2, 200, 77, None, [[76], [0, 76]]),
    "mask_long": (1, 1, 2, 2, 64, 5000, None, [[4990]]),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", list(LONE))
def test_one_key_has_no_gradient_through_the_softmax(case, d, family):
    B, Bk, Hq, Hk, Nq, Nk, lens, seen = LONE[case]
    Q, K, V, dO, _ = inputs(B, Bk, Hq, Hk, Nq, Nk, d, family, 31)
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    mask = None
    if seen is not None:
        mask = torch.zeros(Bk, Nk, dtype=torch.bool)
        for i, keys in enumerate(seen):
            mask[i, keys] = True
    kw = dict(kv_lens=None if lens is None else lens.cuda(), key_mask=None if mask is None else mask.cuda())
    O, lse = avq.avq_cross_attention(Q, K, V, lse=True, **kw)
    grads = avq.avq_cross_attention_backward(dO, Q, K, V, O, lse, **kw)
    want = ref.cross(Q, K, V, lens, mask, dO=dO, O_given=O)
    for n, t in zip(("dQ", "dK", "dV"), grads):
        ref.check(n, t, want[n], want[n + "_tol"] * 2)  # lse as the kernel wrote it
    alone = ref.keep_mask(Bk, Nk, lens, mask).sum(1) == 1
    assert alone.any()
    assert (grads[0].cpu()[alone.repeat_interleave(B // Bk)] == 0).all()
    assert (grads[1].cpu()[alone] == 0).all()
    if not alone.all() and case != "lens":
        assert (grads[0].cpu()[~alone.repeat_interleave(B // Bk)] != 0).any()


# ---- scores that are not finite --------------------------------------------------------------


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("Nq", [3, 200])
@pytest.mark.parametrize("key", [*range(8), 131, 134, 255])
def test_an_infinite_score_is_not_hidden(key, Nq, masked, family):
    """exp(inf - inf): every row that sees the key is NaN, the other heads are as they were."""
    Q, K, V, _, _ = inputs(1, 1, 2, 2, Nq, 256, 64, family, 32)
    Q[..., 0] = 1.0
    mask = None
    if masked:
        mask = torch.ones(1, 256, dtype=torch.bool, device="cuda")
        mask[0, [11, 140]] = False
    want, wl = avq.avq_cross_attention(Q, K, V, key_mask=mask, lse=True)
    K[0, 1, key, 0] = float("inf")
    O, lse = avq.avq_cross_attention(Q, K, V, key_mask=mask, lse=True)
    assert torch.isnan(O[0, 1]).all() and torch.isnan(lse[0, 1]).all()
    assert torch.equal(O[0, 0], want[0, 0]) and torch.equal(lse[0, 0], wl[0, 0])


@pytest.mark.parametrize("Nq", [3, 200])
@pytest.mark.parametrize("Nk", [64, 256, 700, 5000])
def test_scores_of_minus_infinity_weigh_nothing(Nk, Nq, family):
    """All of a row's: as a row without keys.  Those of its first keys: as if they were left out."""
    Q, K, V, _, _ = inputs(1, 1, 2, 2, Nq, Nk, 64, family, 33)
    Q[..., 0] = 1e25  # finite: the product overflows
    K[..., 0] = 0.0
    K[0, 0, :, 0] = -1e25
    first = Nk // 2 + 1
    K[0, 1, :first, 0] = -1e25
    O, lse = avq.avq_cross_attention(Q, K, V, lse=True)
    assert (O[0, 0] == 0).all() and (lse[0, 0] == float("-inf")).all()
    Q[..., 0] = 0.0
    rest = torch.arange(Nk, device="cuda")[None] >= first
    want = ref.cross(Q, K, V, key_mask=rest)
    ref.check("O", O[:, 1:], want["O"][:, 1:], want["O_tol"][:, 1:])
    ref.check("lse", lse[:, 1:], want["lse"][:, 1:], want["lse_tol"][:, 1:])


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("Nk, d", [(77, 64), (300, 64), (300, 128)])
@pytest.mark.parametrize("row", [*range(8), 134, 199])
def test_a_nan_query_reaches_every_gradient(row, Nk, d, masked, family):
    """Of its row's dQ, and of dK and dV of every key that the row sees; nothing else changes."""
    Q, K, V, dO, _ = inputs(1, 1, 2, 2, 200, Nk, d, family, 34)
    mask = None
    if masked:
        mask = torch.ones(1, Nk, dtype=torch.bool, device="cuda")
        mask[0, [5, 70]] = False
    O, lse = avq.avq_cross_attention(Q, K, V, key_mask=mask, lse=True)
    want = avq.avq_cross_attention_backward(dO, Q, K, V, O, lse, key_mask=mask)
    Q[0, 1, row, 7] = float("nan")
    O, lse = avq.avq_cross_attention(Q, K, V, key_mask=mask, lse=True)
    dQ, dK, dV = avq.avq_cross_attention_backward(dO, Q, K, V, O, lse, key_mask=mask)
    seen = slice(None) if mask is None else mask[0]
    for n, t in (("dK", dK), ("dV", dV)):
        assert torch.isnan(t[0, 1][seen]).all(), n
    rows = torch.arange(200, device="cuda") != row
    assert torch.isnan(dQ[0, 1, row]).all() and torch.equal(dQ[0, 1, rows], want[0][0, 1, rows])
    assert all(torch.equal(a[0, 0], b[0, 0]) for a, b in zip((dQ, dK, dV), want))


@pytest.mark.parametrize("Nk, d", [(77, 64), (128, 128), (300, 64), (300, 128)])
def test_scores_of_minus_infinity_have_no_gradient(Nk, d, family):
    """A row all of whose scores are -inf has no part in any gradient."""
    Q, K, V, dO, _ = inputs(1, 1, 2, 2, 200, Nk, d, family, 35)
    Q[..., 0] = 0.0
    K[..., 0] = 1e25
    rows = torch.tensor([0, 3, 6, 7, 134, 199])
    Q[0, 1, rows, 0] = -1e25
    O, lse = avq.avq_cross_attention(Q, K, V, lse=True)
    assert (lse[0, 1, rows] == float("-inf")).all()
    dQ, dK, dV = avq.avq_cross_attention_backward(dO, Q, K, V, O, lse)
    assert (dQ[0, 1, rows] == 0).all()
    others = torch.ones(200, dtype=torch.bool)
    others[rows] = False
    want = ref.cross(Q[:, 1:, others], K[:, 1:], V[:, 1:], dO=dO[:, 1:, others], O_given=O[:, 1:, others])
    ref.check("dQ", dQ[:, 1:, others], want["dQ"], want["dQ_tol"] * 2)
    ref.check("dK", dK[:, 1:], want["dK"], want["dK_tol"] * 2)
    ref.check("dV", dV[:, 1:], want["dV"], want["dV_tol"] * 2)


# ---- keys that are left out ------------------------------------------------------------------


@pytest.mark.parametrize("Nk, d", [(77, 64), (300, 64), (300, 128)])
def test_keys_left_out_get_zero_whatever_the_rows_hold(Nk, d, family):
    Q, K, V, dO, _ = inputs(2, 2, 2, 1, 200, Nk, d, family, 36)
    lens = torch.tensor([Nk - 9, Nk], dtype=torch.int32, device="cuda")
    mask = torch.ones(2, Nk, dtype=torch.bool, device="cuda")
    mask[1, [0, 33, 70]] = False
    keep = ref.keep_mask(2, Nk, lens, mask)
    O, lse = avq.avq_cross_attention(Q, K, V, kv_lens=lens, key_mask=mask, lse=True)
    Q[:, 0, 100, 3] = float("nan")
    dO[:, 1, 150, 5] = float("inf")
    _, dK, dV = avq.avq_cross_attention_backward(dO, Q, K, V, O, lse, kv_lens=lens, key_mask=mask)
    for t in (dK, dV):
        out = t.cpu()[:, 0]
        assert (out[~keep] == 0).all()
        assert not torch.isfinite(out[keep]).all(-1).any()


# ---- steep scores ----------------------------------------------------------------------------


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_over_dense_inputs_and_rising_scores(d, family):
    """Dense tensors, and keys ordered so that a row's scores rise by 60: nearly all keys weigh next to nothing."""
    Q, K, V, dO, _ = inputs(1, 1, 2, 2, 160, 1000, d, family, 4, packed=False)
    Q[..., 0] = 1.0
    K[..., 0] = torch.linspace(0.0, 60.0, 1000).to(family).cuda()
    want = ref.cross(Q, K, V, scale=1.0)
    O, lse = want["O"].to(family).cuda(), want["lse"].float().cuda()
    want = ref.cross(Q, K, V, scale=1.0, dO=dO, O_given=O)
    got = avq.avq_cross_attention_backward(dO, Q, K, V, O, lse, scale=1.0)
    for n, t in zip(("dQ", "dK", "dV"), got):
        ref.check(n, t, want[n], want[n + "_tol"])


@pytest.mark.parametrize("Nk, d", [(77, 64), (300, 64), (300, 128)])
def test_masks_of_calls_in_a_row_share_a_workspace(Nk, d, family):
    """Calls with one key and with many after one another, eager and captured, and two streams side by side."""
    Q, K, V, dO, g = inputs(2, 2, 4, 2, 200, Nk, d, family, 37)
    few = torch.zeros(2, Nk, dtype=torch.bool, device="cuda")
    few[0, Nk - 1] = few[1, 5] = True
    masks = [few, (torch.rand(2, Nk, generator=g) < 0.5).cuda(), few.flip(0).contiguous()]
    sets = []
    for m in masks:
        O, lse = avq.avq_cross_attention(Q, K, V, key_mask=m, lse=True)
        sets.append(((dO, Q, K, V, O, lse), dict(key_mask=m)))
    want = []
    for a, kw in sets:
        torch.cuda.synchronize()
        want.append(avq.avq_cross_attention_backward(*a, **kw))
    assert (want[0][0] == 0).all() and (want[1][0] != 0).any() and (want[2][1] == 0).all()
    dims = avq.avq_cross_dims(2, 2, 4, 2, 200, Nk, d, d ** -0.5)
    size = avq.avq_cross_workspace_size(dims, avq.AVQ_F32 if family == torch.float32 else avq.AVQ_BF16, True)
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
    order = (0, 1, 2, 1, 0, 2)

    def run():
        return [avq.avq_cross_attention_backward(*sets[i][0], ws=ws, **sets[i][1]) for i in order]

    def same(got):
        return all(torch.equal(a, b) for i, g in zip(order, got) for a, b in zip(g, want[i]))

    assert same(run())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        got = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(got)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [avq.avq_cross_attention_backward(*sets[i][0], stream=streams[k % 2], **sets[i][1])
           for k, i in enumerate(order * 4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for k, g in enumerate(got) for a, b in zip(g, want[(order * 4)[k]]))
    avq.avq_check_device()
