"""Exact attention over another sequence and its gradients against the 64-bit
definition: one row to many, one key to many, shared key heads and encoder
states, lengths, masks, rows with no key, views, both types and kernel
families."""
import pytest
import torch

import adaptive_vector_quantized_b200 as avq
from tests import exact_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(B, Bk, Hq, Hk, Nq, Nk, d, dt, seed=0, packed=True, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    if packed:
        Q = (spread * torch.randn(B, Nq, Hq, d, generator=g)).to(dt).cuda().transpose(1, 2)
        kv = torch.randn(Bk, Nk, 2, Hk, d, generator=g).to(dt).cuda()
        K, V = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    else:
        Q = (spread * torch.randn(B, Hq, Nq, d, generator=g)).to(dt).cuda()
        K, V = (torch.randn(Bk, Hk, Nk, d, generator=g).to(dt).cuda() for _ in range(2))
    dO = torch.randn(B, Hq, Nq, d, generator=g).to(dt).cuda()
    return Q, K, V, dO, g


def run_case(B, Bk, Hq, Hk, Nq, Nk, d, dtype, lens=None, mask=None, seed=0, packed=True, scale=None, spread=1.5):
    """Forward and backward against the definition; garbage where keys are left out."""
    dt = DT[dtype]
    Q, K, V, dO, g = inputs(B, Bk, Hq, Hk, Nq, Nk, d, dt, seed, packed, spread)
    kv_lens = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    key_mask = None
    if mask is not None:
        key_mask = torch.rand(Bk, Nk, generator=g) < mask
    keep = ref.keep_mask(Bk, Nk, kv_lens, key_mask)
    if Nk and not keep.all():
        out = (~keep)[:, None, :, None].cuda()
        # infinities and NaN in the places that are left out
        K.masked_fill_(out, float("nan"))
        V.masked_fill_(out, float("inf"))
    kw = dict(kv_lens=None if lens is None else kv_lens.cuda(), key_mask=None if mask is None else key_mask.cuda(),
              scale=scale)
    O, lse = avq.avq_cross_attention(Q, K, V, lse=True, **kw)
    kernels = avq.last_kernels()
    want = ref.cross(Q, K, V, kv_lens, key_mask, scale)
    ref.check("O", O, want["O"], want["O_tol"])
    ref.check("lse", lse, want["lse"], want["lse_tol"])
    empty = torch.isinf(want["lse"])
    if empty.any():
        assert (O.cpu()[empty] == 0).all()
    # gradients from the definition's O and lse, rounded as the forward pass keeps them
    Og, lg = want["O"].to(dt).cuda(), want["lse"].float().cuda()
    wg = ref.cross(Q, K, V, kv_lens, key_mask, scale, dO=dO, O_given=Og)
    dQ, dK, dV = avq.avq_cross_attention_backward(dO, Q, K, V, Og, lg, **kw)
    for n, t in (("dQ", dQ), ("dK", dK), ("dV", dV)):
        ref.check(n, t, wg[n], wg[n + "_tol"])
    again = avq.avq_cross_attention_backward(dO, Q, K, V, Og, lg, **kw)
    assert all(torch.equal(a, b) for a, b in zip((dQ, dK, dV), again))  # no order of sums left to chance
    # a run of both, as training does it
    own = avq.avq_cross_attention_backward(dO, Q, K, V, O, lse, **kw)
    wo = ref.cross(Q, K, V, kv_lens, key_mask, scale, dO=dO, O_given=O)
    # lse as the kernel wrote it scales a row's probabilities by its error
    for n, t in zip(("dQ", "dK", "dV"), own):
        ref.check(n + " of the run", t, wo[n], wo[n + "_tol"] * 2)
    avq.avq_check_device()
    return kernels


# B, Bk, Hq, Hk, Nq, Nk, d, lens, mask
CASES = {
    "one_row_one_key": (1, 1, 1, 1, 1, 1, 64, None, None),
    "one_row": (2, 2, 4, 4, 1, 77, 64, None, None),
    "one_row_shared_heads": (3, 3, 8, 2, 1, 300, 128, [300, 0, 131], None),
    "one_row_long": (1, 1, 4, 1, 1, 5000, 64, [4097], None),
    "few_rows": (2, 2, 6, 2, 5, 515, 128, [515, 33], 0.7),
    "beams": (12, 3, 4, 2, 1, 200, 64, [200, 64, 0], None),
    "beams_rows": (6, 2, 4, 4, 40, 130, 128, [130, 129], None),
    "text": (2, 2, 3, 3, 400, 77, 64, [77, 9], None),
    "text_wide": (2, 2, 2, 1, 257, 77, 128, [0, 77], None),
    "one_key": (2, 1, 2, 2, 130, 1, 64, None, None),
    "tile_edges": (1, 1, 2, 2, 128, 128, 64, None, None),
    "past_tile_edges": (1, 1, 2, 1, 129, 129, 128, None, None),
    "row_pairs": (1, 1, 1, 1, 256, 256, 64, None, 0.5),
    "odd": (2, 2, 3, 1, 333, 517, 128, [517, 260], 0.8),
    "long_keys": (1, 1, 2, 2, 200, 3000, 64, None, None),
    "long_rows": (1, 1, 2, 1, 3001, 190, 64, [150], None),
    "mask_leaves_nothing": (2, 2, 2, 2, 70, 200, 64, None, 0.0),
    "mask_few": (2, 2, 2, 2, 150, 400, 128, None, 0.01),
    "lens_out_of_range": (3, 3, 2, 2, 140, 100, 64, [-5, 1000, 100], None),
    "no_keys": (2, 2, 2, 1, 20, 0, 64, None, None),
    "shared_by_all": (5, 1, 2, 2, 150, 140, 64, [139], None),
}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", list(CASES))
def test_cross(case, dtype):
    *dims, lens, mask = CASES[case]
    run_case(*dims, dtype, lens, mask)


@pytest.mark.parametrize("case", ["one_row_shared_heads", "beams_rows", "text", "odd", "long_keys", "no_keys"])
def test_cross_bf16_on_the_cuda_cores(case):
    *dims, lens, mask = CASES[case]
    old = avq.avq_set_path(avq.AVQ_PATH_SIMT)
    try:
        assert "simt" in run_case(*dims, "bf16", lens, mask)
    finally:
        avq.avq_set_path(old)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("spread, scale", [(8.0, None), (1.5, 1.0), (0.05, 0.02)])
def test_cross_peaked_and_flat(dtype, spread, scale):
    """Logits up to a hundred, where one key takes all, and next to none."""
    run_case(1, 1, 2, 2, 200, 300, 64, dtype, None, None, seed=3, spread=spread, scale=scale)


@pytest.mark.parametrize("dtype", list(DT))
def test_cross_dense_inputs_and_rising_maximum(dtype):
    """Dense tensors, and keys ordered so that a row's maximum grows in every tile."""
    dt = DT[dtype]
    Q, K, V, dO, _ = inputs(1, 1, 2, 2, 160, 1000, 64, dt, 4, packed=False)
    ramp = torch.linspace(0.0, 60.0, 1000).cuda()
    unit = torch.zeros(64, device="cuda")
    unit[0] = 8.0
    Q[..., 0] = 1.0
    K[..., 0] = (ramp / 1.0).to(dt)
    want = ref.cross(Q, K, V, scale=1.0, dO=dO)
    O, lse = avq.avq_cross_attention(Q, K, V, scale=1.0, lse=True)
    ref.check("O", O, want["O"], want["O_tol"])
    ref.check("lse", lse, want["lse"], want["lse_tol"])


def test_cross_given_views_streams_and_graph():
    """O into a view of the next projection's input, a stream of the caller's, and a graph of both directions."""
    B, H, Nq, Nk, d = 2, 4, 300, 150, 64
    Q, K, V, dO, _ = inputs(B, B, H, H, Nq, Nk, d, torch.bfloat16, 6)
    want, wl = avq.avq_cross_attention(Q, K, V, lse=True)
    wd = avq.avq_cross_attention_backward(dO, Q, K, V, want, wl)
    rows = torch.full((B, Nq + 3, H * d + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    O = rows[:, :Nq, :H * d].unflatten(-1, (H, d)).transpose(1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, none = avq.avq_cross_attention(Q, K, V, O=O, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert none is None and got is O
    assert torch.equal(O, want)
    assert (rows[:, Nq:] == 7).all() and (rows[..., H * d:] == 7).all()  # what lies behind stays
    strided = torch.empty(B, Nq, H, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2).copy_(dO)
    got = avq.avq_cross_attention_backward(strided, Q, K, V, O, wl)
    assert all(torch.equal(a, b) for a, b in zip(got, wd))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = avq.avq_cross_attention(Q, K, V, lse=True)
        g = avq.avq_cross_attention_backward(dO, Q, K, V, o, l)
    Q.mul_(0.5)  # replays read the inputs anew
    want, wl = avq.avq_cross_attention(Q, K, V, lse=True)
    wd = avq.avq_cross_attention_backward(dO, Q, K, V, want, wl)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(l, wl)
    assert all(torch.equal(a, b) for a, b in zip(g, wd))


def test_cross_two_streams_at_once():
    """Two split calls with workspaces of their own, side by side."""
    a = inputs(1, 1, 4, 4, 1, 6000, 64, torch.bfloat16, 7)[:3]
    b = inputs(2, 2, 4, 2, 3, 5000, 128, torch.bfloat16, 8)[:3]
    want = [avq.avq_cross_attention(*x)[0] for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, x in enumerate((a, b)):
            got[i].append(avq.avq_cross_attention(*x, stream=streams[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_cross_repeated_inputs():
    """K and V repeated over batch and heads by a stride of 0 give what the shared form gives."""
    Q, K, V, dO, _ = inputs(4, 1, 6, 1, 90, 210, 64, torch.bfloat16, 9)
    want = avq.avq_cross_attention(Q, K, V)[0]
    Ke, Ve = K.expand(4, 6, 210, 64), V.expand(4, 6, 210, 64)
    got = avq.avq_cross_attention(Q, Ke, Ve)[0]
    ref_ = ref.cross(Q, K, V)
    ref.check("O", got, ref_["O"], ref_["O_tol"])
    ref.check("O", want, ref_["O"], ref_["O_tol"])


def test_cross_gradient_by_differences():
    """Directional differences of the fp32 forward pass."""
    Q, K, V, dO, g = inputs(2, 1, 2, 1, 20, 30, 64, torch.float32, 10, packed=False, spread=1.0)
    mask = (torch.rand(1, 30, generator=g) < 0.7).cuda()
    O, lse = avq.avq_cross_attention(Q, K, V, key_mask=mask, lse=True)
    grads = avq.avq_cross_attention_backward(dO, Q, K, V, O, lse, key_mask=mask)
    h = 2.0 ** -6
    for i, x in enumerate((Q, K, V)):
        way = torch.randn(x.shape, generator=g).cuda()
        way /= way.norm()
        ins = [[Q, K, V], [Q, K, V]]
        ins[0][i], ins[1][i] = x - h * way, x + h * way
        lo, hi = (avq.avq_cross_attention(*t, key_mask=mask)[0].double() for t in ins)
        diff = ((hi - lo) * dO.double()).sum().item() / (2 * h)
        got = (grads[i].double() * way.double()).sum().item()
        # the step's third order (logits move by less than h along a unit vector) and the fp32 steps of O over 2h
        tol = h * h * dO.norm().item() + 2.0 ** -20 * dO.abs().sum().item() ** 0.5 * 4 / (2 * h)
        assert abs(diff - got) <= tol, (i, diff, got, tol)


def test_cross_refuses():
    Q, K, V, dO, _ = inputs(2, 2, 4, 2, 10, 20, 64, torch.float32, 0, packed=False)
    with pytest.raises(ValueError):
        avq.avq_cross_attention(Q[:, :3], K, V)
    with pytest.raises(ValueError):
        avq.avq_cross_attention(Q, K, V[:, :, :10])
    with pytest.raises(TypeError):
        avq.avq_cross_attention(Q, K.bfloat16(), V)
    with pytest.raises(TypeError):
        avq.avq_cross_attention(Q, K, V, kv_lens=torch.tensor([1, 2]).cuda())
    with pytest.raises(ValueError):
        avq.avq_cross_attention(Q, K, V, kv_lens=torch.tensor([1, 2], dtype=torch.int32))
    with pytest.raises(TypeError):
        avq.avq_cross_attention(Q, K, V, key_mask=torch.ones(2, 20).cuda())
    with pytest.raises(avq.AVQError):
        avq.avq_cross_attention(Q, K, V, scale=0.0)
    with pytest.raises(avq.AVQError):
        avq.avq_cross_attention(Q, K, V, O=Q)
    with pytest.raises(ValueError):
        avq.avq_cross_attention_backward(dO, Q, K, V, Q, None)
    with pytest.raises(ValueError):
        avq.avq_cross_attention(Q, K.transpose(2, 3), V)
    with pytest.raises(avq.AVQError):  # repeated tokens
        avq.avq_cross_attention(Q, K[:, :, :1].expand(2, 2, 20, 64), V)
    O, lse = avq.avq_cross_attention(Q, K, V, lse=True)
    with pytest.raises(avq.AVQError):
        avq.avq_cross_attention_backward(dO[:, :, :1].expand(2, 4, 10, 64), Q, K, V, O, lse)
    old = avq.avq_set_path(avq.AVQ_PATH_TC)
    try:
        with pytest.raises(avq.AVQError):  # no tensor-core kernel for fp32
            avq.avq_cross_attention(Q, K, V)
    finally:
        avq.avq_set_path(old)


def test_cross_repeated_inputs_backward():
    """Repeated K and V (stride 0) have a gradient for every place; their sum is the shared form's."""
    Q, K, V, dO, _ = inputs(4, 1, 6, 1, 90, 110, 64, torch.bfloat16, 9)
    want = ref.cross(Q, K, V, dO=dO)
    O, lse = want["O"].to(torch.bfloat16).cuda(), want["lse"].float().cuda()
    Ke, Ve = K.expand(4, 6, 110, 64), V.expand(4, 6, 110, 64)
    each = ref.cross(Q, Ke, Ve, dO=dO, O_given=O)
    dQ, dK, dV = avq.avq_cross_attention_backward(dO, Q, Ke, Ve, O, lse)
    for n, t in (("dQ", dQ), ("dK", dK), ("dV", dV)):
        ref.check(n, t, each[n], each[n + "_tol"])
    # a gradient that repeats over batch and heads
    ones = dO[:1, :1].expand(4, 6, 90, 64)
    flat = ref.cross(Q, K, V, dO=ones, O_given=O)
    got = avq.avq_cross_attention_backward(ones, Q, K, V, O, lse)
    for n, t in zip(("dQ", "dK", "dV"), got):
        ref.check(n, t, flat[n], flat[n + "_tol"])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("Nq, Nk", [(1, 700), (150, 300)])
def test_cross_nan_reaches_its_rows_alone(dtype, Nq, Nk):
    """NaN in one query gives NaN in its row, infinity in a value that is looked at is not hidden, nothing else changes."""
    Q, K, V, _, _ = inputs(2, 2, 3, 3, Nq, Nk, 64, DT[dtype], 11)
    want = avq.avq_cross_attention(Q, K, V)[0]
    Q[1, 2, Nq - 1, 5] = float("nan")
    V[0, 1, Nk // 2, 7] = float("inf")
    got = avq.avq_cross_attention(Q, K, V)[0]
    assert torch.isnan(got[1, 2, Nq - 1]).all()
    assert torch.isinf(got[0, 1, :, 7]).all()
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[1, 2, Nq - 1] = True
    hit[0, 1, :, 7] = True
    assert torch.equal(got[~hit], want[~hit])


def rand_cases(n, seed):
    """Shapes across the kernels' rules: rows from one to several tiles, keys from none to many tiles."""
    import random

    r = random.Random(seed)
    out = []
    for _ in range(n):
        Hk, Bk = r.choice([1, 2, 3]), r.choice([1, 2, 3])
        Nk = r.choice([1, 2, 63, 64, 65, 77, 127, 128, 129, r.randint(1, 128), r.randint(129, 1500)])
        Nq = r.choice([1, 2, 7, 17, 33, 127, 128, 129, 255, 257, r.randint(1, 600)])
        lens = [r.choice([0, Nk, r.randint(0, Nk)]) for _ in range(Bk)] if r.random() < 0.6 else None
        mask = r.choice([None, None, 0.5, 0.95])
        out.append((Bk * r.choice([1, 2, 3]), Bk, Hk * r.choice([1, 2, 4]), Hk, Nq, Nk, r.choice([64, 128]), lens, mask,
                    r.random() < 0.5))
    return out


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("i", range(24))
def test_cross_shapes_across_the_rules(i, dtype):
    B, Bk, Hq, Hk, Nq, Nk, d, lens, mask, packed = rand_cases(24, 77)[i]
    run_case(B, Bk, Hq, Hk, Nq, Nk, d, dtype, lens, mask, seed=i, packed=packed)


def test_cross_full_rounds_and_a_split_last():
    """More items than SMs: those of the last round are split over keys, the others not."""
    Q, K, V, _, _ = inputs(2, 2, 40, 40, 512, 1100, 64, torch.bfloat16, 12)  # 160 pairs of row tiles
    O, lse = avq.avq_cross_attention(Q, K, V, lse=True)
    assert avq.last_kernels() == "cross_tc cross_join"
    want = ref.cross(Q, K, V)
    ref.check("O", O, want["O"], want["O_tol"])
    ref.check("lse", lse, want["lse"], want["lse_tol"])
    again = avq.avq_cross_attention(Q, K, V)[0]
    assert torch.equal(again, O)


def test_cross_offsets_past_32_bits():
    """One token over encoder states of more than 2^32 bytes each and 2^31 elements."""
    Nk, d = (1 << 25) + 4097, 64  # 2^31 elements and more in K and in V
    kv = torch.zeros((1, Nk, 2, 1, d), dtype=torch.bfloat16, device="cuda")
    K, V = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    Q = torch.zeros((1, 2, 1, d), dtype=torch.bfloat16, device="cuda")
    Q[..., 0] = 16.0
    # keys behind the 2^31st element carry all the weight: logits of 16 against 0
    far = [Nk - 1, Nk - 4000, (1 << 25) + 5]
    for i, j in enumerate(far):
        K[0, 0, j, 0] = 16.0
        V[0, 0, j, i] = 1.0
    O, lse = avq.avq_cross_attention(Q, K, V, scale=1.0 / 8, lse=True)  # e^32 against Nk ones
    e = torch.tensor(32.0, dtype=torch.float64).exp()
    z = 3 * e + (Nk - 3)
    want = torch.zeros(1, 2, 1, d, dtype=torch.float64)
    want[..., :3] = e / z
    ref.check("O", O, want, 2 * 2.0 ** -8 * want.abs() + 2e-4 * want.abs() + 1e-30)
    ref.check("lse", lse, torch.full((1, 2, 1), z.log().item(), dtype=torch.float64), torch.full((1, 2, 1), 3e-4))


def test_layer_as_it_is_used():
    """A layer's run: joint projection -> norm and rotation -> quantised self attention, and attention over
    text states, with the gradients back to the projection, each step against its definition."""
    g = torch.Generator().manual_seed(21)
    B, H, N, d, Nt = 2, 4, 784, 64, 77
    qkv = torch.randn(B, N, 3, H, d, generator=g).bfloat16().cuda()
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    text = torch.randn(B, Nt, 2, H, d, generator=g).bfloat16().cuda()
    tk, tv = text[:, :, 0].transpose(1, 2), text[:, :, 1].transpose(1, 2)
    lens = torch.tensor([77, 20], dtype=torch.int32).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda()
    t = avq.avq_gilbert_order(28, 28).long()
    pos = torch.stack([t // 28, t % 28], -1).int()
    freqs, m = avq.avq_rotary_freqs(64, axes=2, base=100.0)
    turn = dict(freqs=freqs.cuda(), positions=pos.cuda(), axes=2, mscale=m)
    Qn, Kn = avq.avq_qk_norm(q, k, w, w, norm="layer", eps=1e-5, **turn)
    ang = ref.angles(pos, freqs, 2, B, N)
    for x, y in ((q, Qn), (k, Kn)):
        want = ref.norm_forward(x.cpu(), w.cpu(), None, "layer", 1e-5, ang, "half", m)
        ref.check("norm", y, want, ref.row_bound(want, torch.bfloat16))
    # quantised self attention on the result
    par = Kn[0, :, ::49].contiguous()  # 16 codewords per head, no children
    assign, vsum, counts = avq.avq_quantize(Kn, v.contiguous(), par, None)
    O, _, _ = avq.avq_attention(Qn, par, None, vsum, counts, P=0)
    P = par.cpu().double()
    dist = ((P * P).sum(-1)[None, :, None, :] - 2 * Kn.cpu().double() @ P.transpose(-1, -2)[None])
    got = assign.cpu().long()
    best = dist.min(-1).values
    assert (dist.gather(-1, got[..., None])[..., 0] - best <= 1e-5 * (best.abs() + 200)).all()  # nearest, up to near ties
    onehot = torch.nn.functional.one_hot(got, par.shape[1]).double()
    vs = onehot.transpose(-1, -2) @ v.cpu().double()
    n = onehot.sum(2)
    S = Qn.cpu().double() @ P.transpose(-1, -2)[None] * d ** -0.5
    E = torch.where(n[:, :, None] > 0, (S - S.amax(-1, keepdim=True)).exp(), torch.zeros_like(S))
    want = (E @ vs) / (E * n[:, :, None]).sum(-1, keepdim=True)
    assert (O.cpu().double() - want).abs().max() <= 2e-2 * v.abs().max().item()
    # text, and back to the projection
    X, lse = avq.avq_cross_attention(Qn, tk, tv, kv_lens=lens, lse=True)
    ref_x = ref.cross(Qn, tk, tv, lens.cpu())
    ref.check("X", X, ref_x["O"], ref_x["O_tol"])
    dX = torch.randn(B, H, N, d, generator=g).bfloat16().cuda()
    dQn, dtk, dtv = avq.avq_cross_attention_backward(dX, Qn, tk, tv, X, lse, kv_lens=lens)
    wb = ref.cross(Qn, tk, tv, lens.cpu(), dO=dX, O_given=X)
    for name, got_ in (("dQ", dQn), ("dK", dtk), ("dV", dtv)):
        ref.check(name, got_, wb[name], 2 * wb[name + "_tol"])
    dq, _, dw, _, _, _ = avq.avq_qk_norm_backward(dQn, None, q, None, w, norm="layer", eps=1e-5, **turn)
    dx, dww, _ = ref.norm_backward(dQn.cpu(), q.cpu(), w.cpu(), "layer", 1e-5, ang, "half", m)
    size = dx.abs().amax(-1, keepdim=True) + dQn.cpu().double().abs().amax(-1, keepdim=True) * 8
    ref.check("dq", dq, dx, ref.row_bound(dx, torch.bfloat16, size))
    ref.check("dw", dw, dww, 4096 * ref.U32 * dQn.cpu().double().abs().sum((0, 1, 2)) * 8 + 1e-30)
    avq.avq_check_device()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dims, lens, mask", [
    ((2, 2, 4, 4, 1, 1), None, None),
    ((4, 2, 6, 2, 1, 15), [15, 1], None),
    ((2, 2, 8, 1, 4, 17), [0, 17], None),
    ((1, 1, 2, 2, 31, 2049), None, 0.5),
    ((6, 1, 5, 1, 1, 4100), [4099], 0.02),
    ((3, 3, 2, 2, 32, 700), [700, 63, 0], None),
    ((1, 1, 2, 2, 33, 700), [64], None),
    ((2, 2, 4, 2, 3, 0), None, None),
])
def test_cross_f32_few_rows(dims, lens, mask, d):
    B, Bk, Hq, Hk, Nq, Nk = dims
    kernels = run_case(B, Bk, Hq, Hk, Nq, Nk, d, "f32", lens, mask, packed=B % 2 == 0)
    assert ("cross_few_f32" in kernels) == (B // Bk * (Hq // Hk) * Nq <= 24)


def test_cross_f32_few_rows_captured():
    Q, K, V, _, _ = inputs(2, 2, 4, 2, 1, 3333, 128, torch.float32)
    want, _ = avq.avq_cross_attention(Q, K, V)
    O = torch.empty_like(want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        avq.avq_cross_attention(Q, K, V, O=O)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        avq.avq_cross_attention(Q, K, V, O=O)
    V.neg_()
    O.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, -want)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("dims", [
    (2, 2, 8, 8, 300, 300, 128),    # both gradient kernels side by side
    (1, 1, 4, 2, 200, 1500, 64),    # dQ split
    (2, 1, 4, 2, 1500, 200, 128),   # dK and dV split
    (4, 4, 8, 8, 500, 700, 64),     # neither fits beside the other
    (2, 2, 4, 4, 600, 77, 64),      # one key tile
])
def test_cross_backward_calls_in_a_row_share_a_workspace(dims, dtype):
    sets = []
    for seed in (1, 2):
        Q, K, V, dO, _ = inputs(*dims, DT[dtype], seed)
        O, lse = avq.avq_cross_attention(Q, K, V, lse=True)
        sets.append((dO, Q, K, V, O, lse))
    want = []
    for s in sets:
        torch.cuda.synchronize()
        want.append([t.clone() for t in avq.avq_cross_attention_backward(*s)])
    d = avq.avq_cross_dims(*dims, dims[-1] ** -0.5)
    size = avq.avq_cross_workspace_size(d, avq.AVQ_BF16 if dtype == "bf16" else avq.AVQ_F32, True)
    ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")

    def round_():
        return [avq.avq_cross_attention_backward(*sets[i], ws=ws) for i in (0, 1, 0, 1, 1, 0)]

    torch.cuda.synchronize()
    for k in range(3):
        ws.fill_(255)
        got = round_()
        for i, g in zip((0, 1, 0, 1, 1, 0), got):
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        got = round_()
    for k in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for i, g in zip((0, 1, 0, 1, 1, 0), got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
    avq.avq_check_device()
