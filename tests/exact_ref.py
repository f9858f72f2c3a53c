"""Plain 64-bit forms of the exact operators (rotation by position, norms of
queries and keys, attention over another sequence) and bounds on how far a
kernel that computes in fp32 and rounds to the element type may be from them.

The bounds follow the roundings: u is half a step of a type relative to the
value (bf16 2^-8, fp32 2^-24).  A sum of n products in fp32 is off by at
most n 2^-24 times the sum of their magnitudes.
"""
import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---- rotation and norms ---------------------------------------------------------------


def angles(positions, freqs, axes, B, N):
    """[B or 1, 1, N, rot/2] angles in 64 bits."""
    if positions is None:
        positions = torch.arange(N)
        if axes == 2:
            positions = torch.stack([positions, positions], -1)
    p = positions.double().cpu()
    if p.dim() == (2 if axes == 2 else 1):
        p = p[None]
    f = freqs.double().cpu()
    if axes == 2:
        n = f.numel() // 2
        a = torch.cat([p[..., 0:1] * f[:n], p[..., 1:2] * f[n:]], -1)
    else:
        a = p[..., None] * f
    return a[:, None]


def rotate(x, ang, layout, mscale=1.0, inverse=False):
    if ang is None:
        return x
    if inverse:
        ang = -ang
    n = ang.shape[-1]
    c, s = ang.cos() * mscale, ang.sin() * mscale
    out = x.clone()
    for i in range(n):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        out[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        out[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return out


def normalise(x, norm, eps):
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r, r


def norm_forward(x, w, b, norm, eps, ang, layout, mscale):
    u, _ = normalise(x.double(), norm, eps)
    if w is not None:
        u = u * w.double()
    if b is not None:
        u = u + b.double()
    return rotate(u, ang, layout, mscale)


def norm_backward(dy, x, w, norm, eps, ang, layout, mscale):
    z = rotate(dy.double(), ang, layout, mscale, inverse=True)
    u, r = normalise(x.double(), norm, eps)
    dw, db = (z * u).sum((0, 1, 2)), z.sum((0, 1, 2))
    g = z if w is None else z * w.double()
    dx = g - u * (g * u).mean(-1, keepdim=True)
    if norm == "layer":
        dx = dx - g.mean(-1, keepdim=True)
    return dx * r, dw, db


def row_bound(x, dtype, extra=0.0):
    """A row's elements: one rounding to `dtype` relative to the value, and
    fp32 arithmetic (a handful of operations, a sum of d terms) relative to the
    largest element of the row."""
    d = x.shape[-1]
    return half_step(dtype) * x.abs() + (d + 32) * U32 * (x.abs().amax(-1, keepdim=True) + extra)


# ---- attention over another sequence ----------------------------------------------------


def keep_mask(Bk, Nk, kv_lens, key_mask):
    keep = torch.ones(Bk, Nk, dtype=torch.bool)
    if kv_lens is not None:
        keep &= torch.arange(Nk)[None] < kv_lens.cpu()[:, None]
    if key_mask is not None:
        keep &= key_mask.cpu().bool()
    return keep


def cross(Q, K, V, kv_lens=None, key_mask=None, scale=None, dO=None, O_given=None):
    """Values and bounds: dict with O, lse (and dQ, dK, dV with dO), each with
    a `_tol` of the same shape."""
    dt = Q.dtype
    u = half_step(dt)
    Q, K, V = (t.detach().cpu().double() for t in (Q, K, V))
    B, Hq, Nq, d = Q.shape
    Bk, Hk, Nk, _ = K.shape
    R, G = B // Bk, Hq // Hk
    scale = d ** -0.5 if scale is None else scale
    keep = keep_mask(Bk, Nk, kv_lens, key_mask)
    K = K.masked_fill(~keep[:, None, :, None], 0.0)  # what stands there does not matter
    V = V.masked_fill(~keep[:, None, :, None], 0.0)
    Ke = K.repeat_interleave(R, 0).repeat_interleave(G, 1)
    Ve = V.repeat_interleave(R, 0).repeat_interleave(G, 1)
    on = keep.repeat_interleave(R, 0)[:, None, None, :]
    S = (Q @ Ke.transpose(-1, -2)) * scale
    S = S.masked_fill(~on, float("-inf"))
    m = S.amax(-1, keepdim=True) if Nk else torch.full((B, Hq, Nq, 1), float("-inf"), dtype=torch.float64)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    E = (S - m0).exp()
    z = E.sum(-1, keepdim=True)
    P = E / torch.where(z == 0, torch.ones_like(z), z)
    O = P @ Ve
    out = dict(O=O, lse=(m + z.log()).squeeze(-1))
    # relative error of a probability: the logit's sum of d products and its
    # product with the scale, the exponent's argument (a product and a
    # difference of numbers up to the largest logit), the exponential itself
    # (7.5e-5 on the FMA pipe for bf16, a few steps otherwise), and for bf16
    # the rounding of P to the type of the second product
    mags = (Q.abs() @ Ke.abs().transpose(-1, -2)).amax().item() * scale if Nk else 0.0
    logit = (d + 4) * U32 * mags
    e_p = 2 * logit + 8 * U32 + (1.5e-4 + u if dt == torch.bfloat16 else 0.0)
    sums = (Nk + 16) * U32
    out["O_tol"] = (e_p + sums) * (P @ Ve.abs()) + u * O.abs() + 1e-30
    # e_p bounds each term of the sum, so its logarithm too
    out["lse_tol"] = torch.full_like(out["lse"], e_p + sums) + 4 * U32 * out["lse"].abs().nan_to_num(0, 0, 0)
    if dO is None:
        return out
    g = dO.detach().cpu().double()
    Og = O if O_given is None else O_given.detach().cpu().double()
    dP = g @ Ve.transpose(-1, -2)
    delta = (g * Og).sum(-1, keepdim=True)
    dS = P * (dP - delta) * scale
    dK = (dS.transpose(-1, -2) @ Q).reshape(Bk, R, Hk, G, Nk, d).sum((1, 3))
    dV = (P.transpose(-1, -2) @ g).reshape(Bk, R, Hk, G, Nk, d).sum((1, 3))
    out.update(dQ=dS @ Ke, dK=dK, dV=dV)
    # an element of dS: P's error, the fp32 sums behind dP and delta, and its
    # own rounding to the type of the next product
    sub = (d + 4) * U32 * (g.abs() @ Ve.abs().transpose(-1, -2) + (g * Og).abs().sum(-1, keepdim=True))
    e_ds = P * scale * sub + dS.abs() * (e_p + 8 * U32 + (u if dt == torch.bfloat16 else 0.0))
    # the forward's lse in fp32 shifts all of a row's P alike
    e_lse = 4 * U32 * out["lse"].abs().nan_to_num(0, 0, 0)[..., None]
    e_ds = e_ds + dS.abs() * e_lse
    rows = (R * G * Nq + 16) * U32

    def fold(t):
        return t.reshape(Bk, R, Hk, G, Nk, d).sum((1, 3))

    out["dQ_tol"] = e_ds @ Ke.abs() + sums * (dS.abs() @ Ke.abs()) + u * out["dQ"].abs() + 1e-30
    out["dK_tol"] = fold(e_ds.transpose(-1, -2) @ Q.abs() + rows * (dS.abs().transpose(-1, -2) @ Q.abs())) + u * dK.abs() + 1e-30
    out["dV_tol"] = fold((P * (e_p + e_lse + rows)).transpose(-1, -2) @ g.abs()) + u * dV.abs() + 1e-30
    return out


def check(name, got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    same = (got == want)  # infinities
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert not torch.isnan(err).any(), (name, "NaN")
    assert (err <= tol).all(), (name, "worst error / bound", worst, "largest error", err.max().item())
    return worst
