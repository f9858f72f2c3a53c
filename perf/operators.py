"""The operators of exact attention beside the quantised path, as they are measured.

Three families: the rotation of queries and keys by their positions
(``rotary``), their normalisation per head with that rotation in the same
pass (``norm`` and ``norm_backward``), and attention over another sequence's
keys and values (``cross`` and ``cross_backward``).  With ``own`` false the
operators run in elementary torch operations in 32 bits, with ``own`` true
through the calls of ``adaptive_vector_quantized_b200``.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------------------------


def listed():
    return [
        # one new token of eight sequences, each at its own far position
        dict(name="rotary_token", op="rotary", dtype="bf16", B=8, Hq=16, Hk=4, N=1, d=128, rot=128,
             layout="interleaved", scaling="linear", axes=1, positions="far", packed=True),
        # the first half of each head rotated, in full precision, an odd number of tokens
        dict(name="rotary_part_f32", op="rotary", dtype="f32", B=3, Hq=12, Hk=12, N=4097, d=128, rot=64,
             layout="half", scaling="ntk", axes=1, positions="range", packed=False),
        # the longest sequence of the workloads, positions scaled far beyond the trained range
        dict(name="rotary_long", op="rotary", dtype="bf16", B=1, Hq=16, Hk=16, N=65536, d=64, rot=64,
             layout="half", scaling="yarn", axes=1, positions="range", packed=True),
        # a 28 x 28 patch grid: LayerNorm of queries and keys, rows and columns rotated apart
        dict(name="norm_grid", op="norm", dtype="bf16", B=2, Hq=12, Hk=12, N=784, d=64, rot=64, norm="layer",
             layout="half", scaling="none", axes=2, positions="grid", packed=True),
        # the longest sequence, read out of the joint projection
        dict(name="norm_long", op="norm", dtype="bf16", B=1, Hq=16, Hk=16, N=65536, d=64, rot=64, norm="rms",
             layout="half", scaling="none", axes=1, positions="range", packed=True),
        # the training step of the same with wider heads
        dict(name="norm_backward", op="norm_backward", dtype="bf16", B=1, Hq=8, Hk=8, N=16384, d=128, rot=128,
             norm="rms", layout="interleaved", scaling="none", axes=1, positions="range", packed=True),
        # image tokens over a short text, padded to the batch's longest
        dict(name="cross_text", op="cross", dtype="bf16", B=2, Bk=2, Hq=12, Hk=12, Nq=4096, Nk=77, d=64,
             lens="ragged", mask=False),
        # a long sequence over a long encoder's states
        dict(name="cross_long", op="cross", dtype="bf16", B=1, Bk=1, Hq=8, Hk=8, Nq=16384, Nk=16384, d=128,
             lens="full", mask=False),
        # full precision, odd lengths, keys left out one by one
        dict(name="cross_odd_f32", op="cross", dtype="f32", B=3, Bk=3, Hq=4, Hk=4, Nq=1001, Nk=333, d=64,
             lens="ragged", mask=True),
        # one new token of 32 sequences, shared key heads, encoder states of many lengths
        dict(name="cross_token", op="cross", dtype="bf16", B=32, Bk=32, Hq=16, Hk=4, Nq=1, Nk=8191, d=128,
             lens="ragged", mask=False),
        # training: image tokens over a short text
        dict(name="cross_text_backward", op="cross_backward", dtype="bf16", B=2, Bk=2, Hq=12, Hk=12, Nq=4096,
             Nk=77, d=64, lens="ragged", mask=False),
        # training over a long encoder's states, two query heads to a key head
        dict(name="cross_long_backward", op="cross_backward", dtype="bf16", B=1, Bk=1, Hq=8, Hk=4, Nq=8192,
             Nk=4096, d=128, lens="full", mask=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "norm_backward", "cross", "cross", "cross", "cross_backward", "cross_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    if not op.startswith("cross"):
        axes = rng.choice([1, 1, 2])
        Hk = rng.choice([1, 2, 4, 8])
        c = dict(op=op, dtype=dtype, B=rng.randint(1, 4), Hq=Hk * rng.choice([1, 2, 3]), Hk=Hk, N=1, d=d,
                 rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d]),
                 layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                 axes=axes, positions=rng.choice(["range", "far"]) if axes == 1 else "grid",
                 packed=rng.choice([True, False]))
        if op != "rotary":
            c["norm"] = rng.choice(["rms", "layer"])
        most = 17 * 10 ** 7 // (c["B"] * (c["Hq"] + c["Hk"]) * d * (4 if dtype == "f32" else 2))
        c["N"] = _log(rng, 1, min(65536, most))
        return c
    Hk = rng.choice([1, 2, 3, 4, 8])
    Bk = rng.randint(1, 4)
    c = dict(op=op, dtype=dtype, B=Bk * rng.choice([1, 1, 2, 3]), Bk=Bk, Hq=Hk * rng.choice([1, 1, 2, 4]), Hk=Hk,
             Nq=1, Nk=1, d=d, lens=rng.choice(["full", "ragged"]), mask=rng.choice([False, False, True]))
    c["Nk"] = _log(rng, 1, 16384)
    if op == "cross" and rng.random() < 0.3:
        c["Nq"] = rng.randint(1, 4)
    else:
        scores = 3 * 10 ** 8 if dtype == "bf16" else 3 * 10 ** 7
        c["Nq"] = _log(rng, 1, max(1, min(16384, scores // (c["B"] * c["Hq"] * c["Nk"]))))
    return c


# ---- inputs -----------------------------------------------------------------------------------


def _freqs(case):
    """Angle per position of each rotated pair (64 bits) and the factor on sine and cosine."""
    rot, axes, kind = case["rot"], case["axes"], case["scaling"]
    pairs = rot // 2 // axes
    base, factor, trained = 10000.0, 8.0, 4096
    if kind == "ntk":
        base *= factor ** (pairs / max(pairs - 1, 1))
    f = [base ** (-i / pairs) for i in range(pairs)]
    m = 1.0
    if kind == "linear":
        f = [x / factor for x in f]
    elif kind == "yarn":
        # few turns over the trained range: interpolated; many: kept; a ramp between
        lo = max(math.floor(pairs * math.log(trained / (32.0 * 2 * math.pi)) / math.log(base)), 0)
        hi = min(math.ceil(pairs * math.log(trained / (1.0 * 2 * math.pi)) / math.log(base)), pairs - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(pairs)]
        f = [x * ((1 - r) + r / factor) for x, r in zip(f, ramp)]
        m = 0.1 * math.log(factor) + 1.0
    return f * axes, m


def _lens(case):
    """Keys of each encoder sequence: part of the case, so that its work is known."""
    Bk, Nk = case["Bk"], case["Nk"]
    if case["lens"] == "full":
        return [Nk] * Bk
    r = random.Random(Bk * 1000003 + Nk)
    lens = [r.randint((Nk + 1) // 2, Nk) for _ in range(Bk)]
    lens[0] = Nk
    if Bk >= 3:
        lens[r.randrange(1, Bk)] = 0  # a sequence with no keys: its rows give zero
    return lens


def _heads(g, B, counts, N, d, dt, packed, scale=1.0):
    """Tensors [B, H, N, d]: views of one projection's output [B, N, sum(H) * d], or each by itself."""
    if packed:
        x = torch.randn((B, N, sum(counts) * d), generator=g, device="cuda").mul_(scale).to(dt)
        out, at = [], 0
        for h in counts:
            out.append(x[..., at * d:(at + h) * d].view(B, N, h, d).transpose(1, 2))
            at += h
        return out
    return [torch.randn((B, h, N, d), generator=g, device="cuda").mul_(scale).to(dt) for h in counts]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d = _TYPES[case["dtype"]], case["d"]
    s = dict(case=case)
    if not case["op"].startswith("cross"):
        B, Hq, Hk, N = case["B"], case["Hq"], case["Hk"], case["N"]
        s["Q"], s["K"] = _heads(g, B, [Hq, Hk], N, d, dt, case["packed"])
        if case["positions"] == "far":
            start = torch.randint(0, 1 << 20, (B, 1), generator=g, device="cuda")
            s["positions"] = (start + torch.arange(N, device="cuda")).to(torch.int32)
        elif case["positions"] == "grid":
            side = max(1, math.isqrt(N))
            t = torch.arange(N, device="cuda")
            s["positions"] = torch.stack([t // side, t % side], -1).to(torch.int32)
        else:
            s["positions"] = torch.arange(N, device="cuda", dtype=torch.int32)
        f, s["mscale"] = _freqs(case)
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        if case["op"] != "rotary":
            for n in ("wq", "wk"):
                s[n] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
            for n in ("bq", "bk"):
                s[n] = (0.1 * torch.randn(d, generator=g, device="cuda")).to(dt) if case["norm"] == "layer" else None
            s["eps"] = 1e-6
        if case["op"] == "norm_backward":
            s["dYq"], s["dYk"] = _heads(g, B, [Hq, Hk], N, d, dt, False)
        return s
    B, Bk, Hq, Hk, Nq, Nk = (case[k] for k in ("B", "Bk", "Hq", "Hk", "Nq", "Nk"))
    s["Q"] = _heads(g, B, [Hq], Nq, d, dt, True, 1.5)[0]
    s["K"], s["V"] = _heads(g, Bk, [Hk, Hk], Nk, d, dt, True)
    s["lens"] = None if case["lens"] == "full" else torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    s["mask"] = torch.rand((Bk, Nk), generator=g, device="cuda") < 0.8 if case["mask"] else None
    s["scale"] = d ** -0.5
    if case["op"] == "cross_backward":
        s["dO"] = torch.randn((B, Hq, Nq, d), generator=g, device="cuda").to(dt)
        # what the forward pass kept
        s["O"] = torch.empty((B, Hq, Nq, d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((B, Hq, Nq), dtype=torch.float32, device="cuda")
        for b, h in _units(case):
            o, lse = _attend(s, b, h)
            s["O"][b, h], s["lse"][b, h] = o.to(dt), lse
    return s


# ---- plain forms ------------------------------------------------------------------------------


def _angles(s):
    """Sine and cosine [.., N, rot / 2] in 32 bits, the angles in 64."""
    p, f, axes = s["positions"].double(), s["freqs"], s["case"]["axes"]
    if axes == 2:
        n = f.numel() // 2
        a = torch.cat([p[..., :1] * f[:n], p[..., 1:] * f[n:]], -1)
    else:
        a = p[..., None] * f
    c, n = a.cos() * s["mscale"], a.sin() * s["mscale"]
    if c.dim() == 3:  # one set of positions for each sequence
        c, n = c[:, None], n[:, None]
    return c.float(), n.float()


def _rotate(x, s, cos, sin, back=False):
    rot = s["case"]["rot"]
    if back:
        sin = -sin
    y = x.clone()
    if s["case"]["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    return y


def _normal(x, s):
    """The normalised head, before weight and bias, and 1 / its deviation."""
    if s["case"]["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    return x * r, r


def _norm_plain(s):
    cos, sin = _angles(s)
    out = []
    for x, w, b in ((s["Q"], s["wq"], s["bq"]), (s["K"], s["wk"], s["bk"])):
        y = _normal(x.float(), s)[0] * w.float()
        if b is not None:
            y = y + b.float()
        out.append(_rotate(y, s, cos, sin).to(x.dtype))
    return out


def _norm_backward_plain(s):
    cos, sin = _angles(s)
    dx, dw, db = [], [], []
    for x, g, w in ((s["Q"], s["dYq"], s["wq"]), (s["K"], s["dYk"], s["wk"])):
        g = _rotate(g.float(), s, cos, sin, back=True)
        n, r = _normal(x.float(), s)
        dw.append((g * n).double().sum((0, 1, 2)).float())
        db.append(g.double().sum((0, 1, 2)).float())
        g = g * w.float()
        t = g - n * (g * n).mean(-1, keepdim=True)
        if s["case"]["norm"] == "layer":
            t = t - g.mean(-1, keepdim=True)
        dx.append((t * r).to(x.dtype))
    return dx + dw + (db if s["case"]["norm"] == "layer" else [])


def _units(case):
    """(sequence, head) pairs, a few at a time where the scores are small."""
    B, Hq, scores = case["B"], case["Hq"], case["Nq"] * case["Nk"]
    if Hq * scores <= 1 << 29:
        return [(b, slice(0, Hq)) for b in range(B)]
    return [(b, slice(h, h + 1)) for b in range(B) for h in range(Hq)]


def _key_heads(case, h):
    """Key heads of the query heads h."""
    g = case["Hq"] // case["Hk"]
    return torch.arange(h.start, h.stop, device="cuda") // g


def _probabilities(s, b, h):
    """Scores of sequence b and heads h, the keys left out at -inf."""
    case = s["case"]
    kb, kh = b // (case["B"] // case["Bk"]), _key_heads(case, h)
    K, V = s["K"][kb][kh].float(), s["V"][kb][kh].float()
    Q = s["Q"][b, h].float()
    S = Q @ K.transpose(-1, -2) * s["scale"]
    if s["lens"] is not None or s["mask"] is not None:
        keep = torch.ones(case["Nk"], dtype=torch.bool, device="cuda")
        if s["lens"] is not None:
            keep &= torch.arange(case["Nk"], device="cuda") < s["lens"][kb]
        if s["mask"] is not None:
            keep &= s["mask"][kb]
        S.masked_fill_(~keep, float("-inf"))
    return Q, K, V, S, kb, kh


def _attend(s, b, h):
    Q, K, V, S, _, _ = _probabilities(s, b, h)
    m = S.amax(-1, keepdim=True)
    P = S.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    z = P.sum(-1, keepdim=True)
    O = P @ V / torch.where(z == 0, torch.ones_like(z), z)
    return O, (m + z.log()).squeeze(-1)


def _cross_plain(s):
    case = s["case"]
    O = torch.empty((case["B"], case["Hq"], case["Nq"], case["d"]), dtype=s["Q"].dtype, device="cuda")
    for b, h in _units(case):
        O[b, h] = _attend(s, b, h)[0].to(O.dtype)
    return O


def _cross_backward_plain(s):
    case = s["case"]
    dQ = torch.empty(s["dO"].shape, dtype=s["Q"].dtype, device="cuda")
    dK = torch.zeros(s["K"].shape, dtype=torch.float32, device="cuda")
    dV = torch.zeros_like(dK)
    for b, h in _units(case):
        Q, K, V, S, kb, kh = _probabilities(s, b, h)
        lse = s["lse"][b, h][..., None]
        P = S.sub_(torch.where(lse == float("-inf"), torch.zeros_like(lse), lse)).exp_()
        dO = s["dO"][b, h].float()
        dS = dO @ V.transpose(-1, -2)
        dS.sub_((dO * s["O"][b, h].float()).sum(-1, keepdim=True)).mul_(P).mul_(s["scale"])
        dQ[b, h] = (dS @ K).to(dQ.dtype)
        dK[kb].index_add_(0, kh, dS.transpose(-1, -2) @ Q)
        dV[kb].index_add_(0, kh, P.transpose(-1, -2) @ dO)
    return dQ, dK.to(dQ.dtype), dV.to(dQ.dtype)


# ---- one pass ---------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "rotary":
        cos, sin = _angles(s)
        return [_rotate(x.float(), s, cos, sin).to(x.dtype) for x in (s["Q"], s["K"])]
    return {"norm": _norm_plain, "norm_backward": _norm_backward_plain, "cross": _cross_plain,
            "cross_backward": _cross_backward_plain}[op](s)


def _run_own(s, op):
    import adaptive_vector_quantized_b200 as avq

    case = s["case"]
    if op == "cross":
        return avq.avq_cross_attention(s["Q"], s["K"], s["V"], kv_lens=s["lens"], key_mask=s["mask"],
                                       scale=s["scale"])[0]
    if op == "cross_backward":
        return avq.avq_cross_attention_backward(s["dO"], s["Q"], s["K"], s["V"], s["O"], s["lse"], kv_lens=s["lens"],
                                                key_mask=s["mask"], scale=s["scale"])
    turn = dict(freqs=s["freqs"], positions=s["positions"], layout=case["layout"], mscale=s["mscale"],
                axes=case["axes"])
    if op == "rotary":
        return avq.avq_rotary(s["Q"], s["K"], **turn)
    if op == "norm":
        return avq.avq_qk_norm(s["Q"], s["K"], s["wq"], s["wk"], s["bq"], s["bk"], norm=case["norm"], eps=s["eps"],
                               **turn)
    out = avq.avq_qk_norm_backward(s["dYq"], s["dYk"], s["Q"], s["K"], s["wq"], s["wk"], norm=case["norm"],
                                   eps=s["eps"], bias=case["norm"] == "layer", **turn)
    return [x for x in out if x is not None]


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    e, d = (4 if case["dtype"] == "f32" else 2), case["d"]
    if not case["op"].startswith("cross"):
        rows = case["B"] * (case["Hq"] + case["Hk"]) * case["N"]
        places = case["N"] * case["axes"] * (case["B"] if case["positions"] == "far" else 1)
        moved = 3 if case["op"] == "norm_backward" else 2
        per = {"rotary": 3 * case["rot"], "norm": 3 * case["rot"] + 5 * d, "norm_backward": 3 * case["rot"] + 14 * d}
        # a partly rotated head still has to be given back whole
        return {"bytes": rows * d * e * moved + 4 * places, "flops": rows * per[case["op"]]}
    lens, B, Bk = _lens(case), case["B"], case["Bk"]
    keys = sum(lens)
    rows = B * case["Hq"] * case["Nq"] * d * e
    kv = 2 * keys * case["Hk"] * d * e + (keys if case["mask"] else 0)
    pairs = keys * (B // Bk) * case["Hq"] * case["Nq"]
    if case["op"] == "cross":
        return {"bytes": 2 * rows + kv, "flops": 4 * pairs * d}
    # read dO, Q, O, lse, K, V; write dQ, dK, dV
    return {"bytes": 4 * rows + rows // (d * e) * 4 + kv + 2 * Bk * case["Nk"] * case["Hk"] * d * e,
            "flops": 10 * pairs * d}


# ---- the definition in 64 bits -------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if not case["op"].startswith("cross"):
        return _exact_rows(case, s)
    if case["B"] * case["Hq"] * case["Nq"] * case["Nk"] * case["d"] > 1 << 39:
        return None
    B, Bk, Hq, Hk = case["B"], case["Bk"], case["Hq"], case["Hk"]
    seen = torch.ones((Bk, case["Nk"]), dtype=torch.bool, device="cuda")
    for i, n in enumerate(_lens(case)):
        seen[i, n:] = False
    if s["mask"] is not None:
        seen &= s["mask"]
    wide = torch.float64
    O = torch.zeros((B, Hq, case["Nq"], case["d"]), dtype=wide, device="cuda")
    dQ, dK, dV = torch.zeros_like(O), *(torch.zeros(s["K"].shape, dtype=wide, device="cuda") for _ in "kv")
    for b in range(B):
        i = b * Bk // B
        at = seen[i].nonzero()[:, 0]
        if not len(at):
            continue
        for h in range(Hq):
            j = h * Hk // Hq
            q, k, v = (t.to(wide) for t in (s["Q"][b, h], s["K"][i, j, at], s["V"][i, j, at]))
            logits = torch.einsum("qd,kd->qk", q, k) * s["scale"]
            p = (logits - torch.logsumexp(logits, 1, keepdim=True)).exp()
            del logits
            O[b, h] = torch.einsum("qk,kd->qd", p, v)
            if case["op"] == "cross":
                continue
            g = s["dO"][b, h].to(wide)
            dV[i, j, at] += torch.einsum("qk,qd->kd", p, g)
            t = torch.einsum("qd,kd->qk", g, v)
            t = p * (t - torch.einsum("qk,qk->q", p, t)[:, None]) * s["scale"]
            dQ[b, h] = torch.einsum("qk,kd->qd", t, k)
            dK[i, j, at] += torch.einsum("qk,qd->kd", t, q)
    return O if case["op"] == "cross" else (dQ, dK, dV)


def _exact_rows(case, s):
    """Each pair as a complex number turned by exp(i angle); gradients through the chain rule's own matrix."""
    wide = torch.float64
    pos = s["positions"].to(wide)
    half = case["rot"] // 2
    if case["axes"] == 1:
        ang = pos.unsqueeze(-1) * s["freqs"]
    else:
        ang = pos.repeat_interleave(half // 2, -1) * s["freqs"]
    turn = torch.polar(torch.full_like(ang, s["mscale"]), ang)
    if ang.dim() == 3:
        turn = turn.unsqueeze(1)

    def spin(x, t):
        head, tail = x[..., :case["rot"]], x[..., case["rot"]:]
        if case["layout"] == "half":
            z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * t
            head = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous()) * t
            head = torch.view_as_real(z).flatten(-2)
        return torch.cat([head, tail], -1)

    xs = (s["Q"].to(wide), s["K"].to(wide))
    if case["op"] == "rotary":
        return [spin(x, turn) for x in xs]
    layer = case["norm"] == "layer"
    ys, dxs, dws, dbs = [], [], [], []
    for n, x in zip("qk", xs):
        w = s["w" + n].to(wide)
        mean = x.sum(-1, keepdim=True) / case["d"] if layer else 0.0
        dev = (((x - mean) ** 2).sum(-1, keepdim=True) / case["d"] + s["eps"]).sqrt()
        u = (x - mean) / dev
        if case["op"] == "norm":
            ys.append(spin(u * w + (s["b" + n].to(wide) if layer else 0.0), turn))
            continue
        g = spin(s["dY" + n].to(wide), turn.conj())
        dws.append((g * u).sum((0, 1, 2)))
        dbs.append(g.sum((0, 1, 2)))
        g = g * w
        flat = g.sum(-1, keepdim=True) / case["d"] if layer else 0.0
        dxs.append((g - flat - u * ((g * u).sum(-1, keepdim=True) / case["d"])) / dev)
    return ys if case["op"] == "norm" else dxs + dws + (dbs if layer else [])
