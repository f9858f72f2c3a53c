"""Rotation of queries and keys by position and their norms, with the gradients,
against the 64-bit definition: layouts, parts of the head, axes, positions,
strided inputs, one token to many, both types."""
import pytest
import torch

import adaptive_vector_quantized_b200 as avq
from tests import exact_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def heads(g, B, Hq, Hk, N, d, dt, packed):
    """Q, K as views of one projection's output, or dense."""
    if packed:
        x = torch.randn(B, N, (Hq + Hk) * d, generator=g).to(dt).cuda()
        return (x[..., :Hq * d].view(B, N, Hq, d).transpose(1, 2),
                x[..., Hq * d:].view(B, N, Hk, d).transpose(1, 2) if Hk else None)
    return (torch.randn(B, Hq, N, d, generator=g).to(dt).cuda(),
            torch.randn(B, Hk, N, d, generator=g).to(dt).cuda() if Hk else None)


def positions(kind, B, N, g):
    if kind == "none":
        return None, 1
    if kind == "far":  # each sequence from a far place of its own, backwards too
        return (torch.tensor([(1 << 22) - 5 * i for i in range(B)])[:, None] - torch.arange(N) * 37).to(torch.int32), 1
    if kind == "grid":
        t = torch.arange(N)
        return torch.stack([t // 28, t % 28], -1).to(torch.int32), 2
    if kind == "grid_batch":
        return torch.randint(-100, 100, (B, N, 2), generator=g).to(torch.int32), 2
    return torch.randint(0, 5000, (N,), generator=g).to(torch.int32), 1


# B, Hq, Hk, N, d, rot, layout, positions, packed, mscale
SHAPES = [
    (1, 1, 0, 1, 64, 64, "half", "none", False, 1.0),
    (3, 4, 2, 1, 128, 128, "interleaved", "far", True, 1.0),
    (2, 12, 12, 784, 64, 64, "half", "grid", True, 1.0),
    (2, 3, 1, 77, 128, 64, "half", "perm", True, 1.2),
    (1, 5, 5, 333, 64, 16, "interleaved", "grid_batch", False, 1.0),
    (2, 2, 2, 50, 128, 96, "half", "far", False, 0.7),
    (1, 40, 3, 9, 64, 8, "half", "perm", True, 1.0),
    (1, 2, 1, 5000, 64, 48, "interleaved", "far", True, 1.0),
]
IDS = ["-".join(map(str, s[:8])) for s in SHAPES]


def setup(shape, dt, seed=0):
    B, Hq, Hk, N, d, rot, layout, kind, packed, mscale = shape
    g = torch.Generator().manual_seed(seed)
    Q, K = heads(g, B, Hq, Hk, N, d, dt, packed)
    pos, axes = positions(kind, B, N, g)
    freqs, _ = avq.avq_rotary_freqs(rot, axes=axes, base=500.0) if rot % (8 * axes) == 0 else (None, 1.0)
    ang = ref.angles(pos, freqs, axes, B, N)
    kw = dict(freqs=freqs.cuda(), positions=None if pos is None else pos.cuda(), layout=layout, mscale=mscale, axes=axes)
    return g, Q, K, kw, ang


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_rotary(shape, dtype):
    layout, mscale = shape[6], shape[9]
    _, Q, K, kw, ang = setup(shape, DT[dtype])
    for inverse in (False, True):
        got = avq.avq_rotary(Q, K, inverse=inverse, **kw)
        assert avq.last_kernels() == "rotary"
        for name, x, y in zip("QK", (Q, K), got):
            if x is None:
                assert y is None
                continue
            want = ref.rotate(x.cpu().double(), ang, layout, mscale, inverse)
            ref.check(name, y, want, ref.row_bound(want, DT[dtype]))
            assert torch.equal(y[..., ang.shape[-1] * 2:], x[..., ang.shape[-1] * 2:])  # the rest is copied
    avq.avq_check_device()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_norm_and_gradients(shape, norm, dtype):
    dt = DT[dtype]
    B, Hq, Hk, N, d = shape[:5]
    layout, mscale = shape[6], shape[9]
    g, Q, K, kw, ang = setup(shape, dt, 1)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dt).cuda() for _ in range(2)]
    b = [(0.3 * torch.randn(d, generator=g)).to(dt).cuda() for _ in range(2)]
    eps = 1e-5
    got = avq.avq_qk_norm(Q, K, w[0], w[1], b[0], b[1], norm=norm, eps=eps, **kw)
    for i, (x, y) in enumerate(zip((Q, K), got)):
        if x is None:
            continue
        want = ref.norm_forward(x.cpu(), w[i].cpu(), b[i].cpu(), norm, eps, ang, layout, mscale)
        ref.check("y", y, want, ref.row_bound(want, dt))
    dY = [None if x is None else torch.randn(x.shape, generator=g).to(dt).cuda() for x in (Q, K)]
    out = avq.avq_qk_norm_backward(dY[0], dY[1], Q, K, w[0], w[1], norm=norm, eps=eps, bias=True, **kw)
    again = avq.avq_qk_norm_backward(dY[0], dY[1], Q, K, w[0], w[1], norm=norm, eps=eps, bias=True, **kw)
    for a, c in zip(out, again):  # fixed order of the sums
        assert (a is None and c is None) or torch.equal(a, c)
    for i, x in enumerate((Q, K)):
        if x is None:
            assert out[i] is None and out[2 + i] is None and out[4 + i] is None
            continue
        dx, dw, db = ref.norm_backward(dY[i].cpu(), x.cpu(), w[i].cpu(), norm, eps, ang, layout, mscale)
        _, r = ref.normalise(x.cpu().double(), norm, eps)
        z = ref.rotate(dY[i].cpu().double(), ang, layout, mscale, True)
        # each term of dx is a difference of numbers up to r |g| (1 + |u|^2 ...): the row's largest of them
        size = r * (z.abs().amax(-1, keepdim=True) * 2 * w[i].cpu().double().abs().max() * 4)
        ref.check("dx", out[i], dx, ref.row_bound(dx, dt, size))
        # sums over rows * heads terms in fp32, blocks of them added in turn
        n = B * x.shape[1] * N
        u, _ = ref.normalise(x.cpu().double(), norm, eps)
        few = (min(n, 4096) + d + 64) * ref.U32
        ref.check("dw", out[2 + i], dw, few * (z * u).abs().sum((0, 1, 2)) + few * z.abs().sum((0, 1, 2)) + 1e-30)
        ref.check("db", out[4 + i], db, few * 2 * z.abs().sum((0, 1, 2)) + 1e-30)
    avq.avq_check_device()


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_norm_alone_and_gradient_by_differences(norm):
    """Without rotation, weights or biases; the gradient against central
    differences of the kernel's own forward pass in fp32."""
    g = torch.Generator().manual_seed(5)
    Q = torch.randn(1, 2, 3, 64, generator=g).cuda()
    dY = torch.randn(1, 2, 3, 64, generator=g).cuda()
    y, none = avq.avq_qk_norm(Q, norm=norm, eps=1e-6)
    assert none is None
    want = ref.norm_forward(Q.cpu(), None, None, norm, 1e-6, None, "half", 1.0)
    ref.check("y", y, want, ref.row_bound(want, torch.float32))
    dQ = avq.avq_qk_norm_backward(dY, None, Q, norm=norm, eps=1e-6)[0]
    h = 2.0 ** -7
    for at in [(0, 0, 0, 0), (0, 1, 2, 63), (0, 1, 0, 17)]:
        p, m = Q.clone(), Q.clone()
        p[at] += h
        m[at] -= h
        lo, hi = (avq.avq_qk_norm(t, norm=norm, eps=1e-6)[0].double() for t in (m, p))
        diff = ((hi - lo) * dY.double()).sum().item() / (2 * h)
        # third derivative of the norm is below 3 / sd^3 per unit of dY: h^2/6 of it, and the fp32 steps of y over 2h
        tol = h * h * dY.abs().sum().item() + 64 * 4 * ref.U32 * dY.abs().max().item() * 4 / (2 * h)
        assert abs(diff - dQ[at].item()) <= tol, (at, diff, dQ[at].item(), tol)


def test_unrotated_elements_meet_no_infinity():
    """Elements past the rotated part are copied whatever their neighbours hold."""
    x = torch.randn(1, 1, 2, 64).cuda()
    x[0, 0, 0, 40] = float("inf")
    x[0, 0, 1, 63] = float("nan")
    f, _ = avq.avq_rotary_freqs(32, device="cuda")
    y, _ = avq.avq_rotary(x, freqs=f)
    bad = ~torch.isfinite(y)
    assert bad.sum() == 2 and bad[0, 0, 0, 40] and bad[0, 0, 1, 63]


def test_constant_and_zero_heads():
    """A head of equal elements has no deviation: LayerNorm gives the bias, and with eps > 0 all stays finite."""
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16).cuda()
    x[0, 1] = 3.0
    b = torch.full((64,), 0.5, dtype=torch.bfloat16).cuda()
    y, _ = avq.avq_qk_norm(x, q_bias=b, norm="layer", eps=1e-5)
    assert torch.equal(y, torch.full_like(y, 0.5))
    y, _ = avq.avq_qk_norm(x, norm="rms", eps=1e-5)
    assert torch.equal(y[0, 0], torch.zeros_like(y[0, 0]))
    dq = avq.avq_qk_norm_backward(torch.ones_like(x), None, x, norm="layer", eps=1e-5)[0]
    assert torch.isfinite(dq).all()


def test_given_outputs_other_stream_and_graph():
    """Outputs into given tensors, on a stream of the caller's, and replayed from a graph."""
    g = torch.Generator().manual_seed(2)
    Q, K = heads(g, 2, 4, 4, 100, 64, torch.bfloat16, True)
    f, _ = avq.avq_rotary_freqs(64, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16).cuda()
    want = avq.avq_qk_norm(Q, K, w, w, freqs=f)
    Yq, Yk = torch.empty_like(want[0]), torch.empty_like(want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    avq.avq_qk_norm(Q, K, w, w, freqs=f, Yq=Yq, Yk=Yk, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(Yq, want[0]) and torch.equal(Yk, want[1])
    dY = torch.randn_like(Q.contiguous())
    grads = avq.avq_qk_norm_backward(dY, dY, Q, K, w, w, freqs=f)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = avq.avq_qk_norm(Q, K, w, w, freqs=f)
        d = avq.avq_qk_norm_backward(dY, dY, Q, K, w, w, freqs=f)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    for a, b in zip(d, grads):
        assert (a is None and b is None) or torch.equal(a, b)


def test_refuses_overlap_and_wrong_tensors():
    x = torch.randn(1, 2, 8, 64).cuda()
    f, _ = avq.avq_rotary_freqs(64, device="cuda")
    with pytest.raises(avq.AVQError):
        avq.avq_rotary(x, freqs=f, Yq=x)
    with pytest.raises(ValueError):
        avq.avq_rotary(x.transpose(2, 3), freqs=f)
    with pytest.raises(TypeError):
        avq.avq_rotary(x, freqs=f.float())
    with pytest.raises(TypeError):
        avq.avq_rotary(x, freqs=f, positions=torch.arange(8).cuda())
    with pytest.raises(TypeError):
        avq.avq_qk_norm(x, q_weight=torch.ones(64, dtype=torch.bfloat16).cuda())
    with pytest.raises(TypeError):
        avq.avq_rotary(x.half(), freqs=f)
    with pytest.raises(ValueError):
        avq.avq_rotary(x, freqs=f.cpu())
    with pytest.raises(avq.AVQError):
        avq.avq_rotary(x, freqs=torch.cat([f, f]))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last heads and tokens are turned like the first."""
    B, H, N, d = 1, 33, (1 << 20) + 1, 64  # 2.2 billion elements
    x = torch.zeros((B, H, N, d), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(3)
    spots = [(0, 0, 0), (0, H - 1, N - 1), (0, H - 1, 17), (0, 31, N - 2)]
    rows = [torch.randn(d, generator=g).bfloat16() for _ in spots]
    for s, r in zip(spots, rows):
        x[s] = r.cuda()
    f, _ = avq.avq_rotary_freqs(64)
    y, _ = avq.avq_rotary(x, freqs=f.cuda())
    for s, r in zip(spots, rows):
        want = ref.rotate(r.double()[None, None, None], s[2] * f[None, None, None], "half")[0, 0, 0]
        ref.check("y", y[s], want, ref.row_bound(want, torch.bfloat16))
    zero = torch.ones(N, dtype=torch.bool, device="cuda")
    zero[[17, N - 1]] = False
    assert (y[0, H - 1, zero] == 0).all() and (y[0, 15] == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("seed", range(10))
def test_shapes_across_the_rules(seed, dtype):
    """Tokens from one to more than fill the GPU's blocks, heads from one to many, any rotated part."""
    import random

    r = random.Random(seed)
    d = r.choice([64, 128])
    axes = r.choice([1, 2])
    rot = r.choice([x for x in (0, 16, 32, 48, 64, 80, 96, 112, 128) if x <= d])
    B, Hq, Hk, N = r.randint(1, 3), r.randint(1, 9), r.randint(0, 5), r.choice([1, 2, 3, 31, 300, 1023, 4700])
    dt, norm, layout = DT[dtype], r.choice(["rms", "layer"]), r.choice(["half", "interleaved"])
    g = torch.Generator().manual_seed(seed)
    Q, K = heads(g, B, Hq, Hk, N, d, dt, r.random() < 0.5)
    freqs = avq.avq_rotary_freqs(rot, axes=axes, base=1000.0)[0] if rot else None
    shape = ((B, N) if r.random() < 0.5 else (N,)) + ((2,) if axes == 2 else ())
    pos = torch.randint(-(1 << 20), 1 << 20, shape, generator=g).int() if rot else None
    ang = ref.angles(pos, freqs, axes, B, N) if rot else None
    kw = dict(freqs=None if freqs is None else freqs.cuda(), positions=None if pos is None else pos.cuda(), layout=layout,
              axes=axes)
    w = torch.randn(d, generator=g).to(dt).cuda()
    got = avq.avq_qk_norm(Q, K, w, None, None, w, norm=norm, eps=1e-6, **kw)
    for x, y, wt, b in ((Q, got[0], w, None), (K, got[1], None, w)):
        if x is None:
            continue
        want = ref.norm_forward(x.cpu(), None if wt is None else wt.cpu(), None if b is None else b.cpu(), norm, 1e-6, ang,
                                layout, 1.0)
        ref.check("y", y, want, ref.row_bound(want, dt))
    dY = [None if x is None else torch.randn(x.shape, generator=g).to(dt).cuda() for x in (Q, K)]
    out = avq.avq_qk_norm_backward(dY[0], dY[1], Q, K, w, None, norm=norm, eps=1e-6, bias=True, **kw)
    assert out[3] is None  # no weight was given for the keys
    for i, x in enumerate((Q, K)):
        if x is None:
            continue
        wt = w.cpu() if i == 0 else None
        dx, dw, db = ref.norm_backward(dY[i].cpu(), x.cpu(), wt, norm, 1e-6, ang, layout, 1.0)
        u, rs = ref.normalise(x.cpu().double(), norm, 1e-6)
        z = dY[i].cpu().double() if ang is None else ref.rotate(dY[i].cpu().double(), ang, layout, 1.0, True)
        size = rs * (z.abs().amax(-1, keepdim=True) * 8 * (1.0 if wt is None else wt.double().abs().max()))
        ref.check("dx", out[i], dx, ref.row_bound(dx, dt, size))
        few = (4096 + d + 64) * ref.U32
        if i == 0:
            ref.check("dw", out[2], dw, few * (z.abs().sum((0, 1, 2)) + (z * u).abs().sum((0, 1, 2))) + 1e-30)
        ref.check("db", out[4 + i], db, few * 2 * z.abs().sum((0, 1, 2)) + 1e-30)
