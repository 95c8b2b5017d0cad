"""Measured cases of the training operators: rotary positions of Q and K, and the backward
passes of dense and of block-sparse attention.

A case is a dict of plain values. `prepare` makes what a training or serving program holds
before the call, `run` makes one pass (the plain form in elementary fp32 operations, or with
`own` the library's call), `exact` gives the same outputs in 64 bits from the definitions.

  rope         y = amplitude * R(pos) x: token-major x [B, N, H, d] into the head-major bf16
               tensor [B, H, N, d] that the attention calls read
  rope_bwd     its gradient: head-major bf16 dy back to token-major dx
  dense_bwd    dQ, dK, dV of softmax(Q K^T / sqrt(d)) V from Q, K, V, O, lse and dO
  sparse_bwd   the same over the kept (query group, key group) cells of a route; inputs are
               group-major, the gradients return to the original token order
"""
from __future__ import annotations

import math

import torch

own = False

ROPE_KINDS = ("rope", "rope_bwd")


# ------------------------------------------------------------------------------- cases
def _rope(name, kind, B, H, N, d, layout, widths, dtype="bf16", scaling="none", factor=1.0, start=0, grid=(1, 1)):
    wt, wy, wx = (list(widths) + [0, 0])[:3]
    return {"name": name, "kind": kind, "B": B, "H": H, "N": N, "d": d, "layout": layout, "wt": wt, "wy": wy, "wx": wx,
            "dtype": dtype, "scaling": scaling, "factor": factor, "start": start, "gy": grid[0], "gx": grid[1]}


def _attn(name, kind, B, Hq, Hkv, N, d, G=1, rho=1.0, ragged=False, noise=0.3):
    return {"name": name, "kind": kind, "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "d": d, "G": G, "rho": rho,
            "ragged": ragged, "noise": noise}


def listed():
    return [
        # one new token for each of 8 streams, far into a context extended beyond its trained length
        _rope("rope_token_b8_h32", "rope", 8, 32, 1, 128, "half", (128,), scaling="yarn", factor=8.0, start=250000),
        # queries of one video call (24 heads, grid 13 x 45 x 56), each head split over frame, row and column
        _rope("rope_video_n32760", "rope", 1, 24, 32760, 128, "interleaved", (44, 42, 42), grid=(45, 56)),
        # gradient of the KV heads of a world-model call (grid 21 x 45 x 80), half of each head rotated, fp32 model side
        _rope("rope_bwd_kv_n75600", "rope_bwd", 1, 8, 75600, 128, "half", (64,), dtype="fp32", scaling="linear",
              factor=4.0),
        # a short odd clip at d = 64
        _rope("rope_bwd_odd_n1001", "rope_bwd", 2, 12, 1001, 64, "half", (18, 22, 22), grid=(11, 13)),
        # the tiny call: latency
        _attn("dense_bwd_n1024_d64", "dense_bwd", 1, 2, 2, 1024, 64),
        # grouped queries at an odd length, two samples
        _attn("dense_bwd_gqa_n2311", "dense_bwd", 2, 16, 4, 2311, 128, noise=0.6),
        # the middle call's head count at a quarter of its length
        _attn("dense_bwd_n4096", "dense_bwd", 1, 12, 12, 4096, 128),
        # one layer of the density sweep at its shortest length, every pair
        _attn("dense_bwd_n8192", "dense_bwd", 1, 24, 24, 8192, 128),
        # the tiny call with its 16 x 16 groups
        _attn("sparse_bwd_n1024_d64", "sparse_bwd", 1, 2, 2, 1024, 64, G=16, rho=0.25),
        # grouped queries, uneven groups (empty ones among them) and a query group that keeps no cell
        _attn("sparse_bwd_gqa_n5003", "sparse_bwd", 1, 32, 8, 5003, 128, G=40, rho=0.26, ragged=True, noise=0.6),
        # one layer of the density sweep at its shortest length
        _attn("sparse_bwd_n8192", "sparse_bwd", 1, 24, 24, 8192, 128, G=64, rho=0.22),
        # the middle call
        _attn("sparse_bwd_n16384", "sparse_bwd", 1, 12, 12, 16384, 128, G=64, rho=0.22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rope", "rope_bwd", "dense_bwd", "sparse_bwd"))
    d = rng.choice((64, 128, 128))
    if kind in ROPE_KINDS:
        B, H = rng.choice((1, 1, 2, 4)), rng.choice((2, 4, 8, 12, 24, 32))
        N = _log(rng, 1, min(118800, 24 * 32760 * 128 // (B * H * d)))
        split = rng.choice(("all", "part", "video"))
        if split == "all":
            widths = (d,)
        elif split == "part":
            widths = (2 * rng.randint(1, d // 2 - 1),)
        else:
            side = 2 * rng.randint(1, d // 6)
            widths = (2 * rng.randint(1, (d - 2 * side) // 2), side, side)
        scaling = rng.choice(("none", "linear", "ntk", "yarn"))
        c = _rope("", kind, B, H, N, d, rng.choice(("interleaved", "half")), widths, rng.choice(("bf16", "fp32")),
                  scaling, 1.0 if scaling == "none" else rng.choice((2.0, 4.0, 8.0)), rng.choice((0, 0, _log(rng, 1, 1000000))),
                  (rng.randint(1, 64), rng.randint(1, 96)) if split == "video" else (1, 1))
    else:
        Hkv, g = rng.choice((1, 2, 4, 8, 12)), rng.choice((1, 1, 2, 3, 4))
        B = rng.choice((1, 1, 2))
        top = 24 * 8192 ** 2 if kind == "dense_bwd" else 12 * 16384 ** 2
        hi = int(min(16384, math.sqrt(top / (B * Hkv * g))))
        N = _log(rng, 64, hi)
        if kind == "dense_bwd":
            c = _attn("", kind, B, Hkv * g, Hkv, N, d, noise=rng.choice((0.3, 0.6)))
        else:
            G = _log(rng, 2, max(2, min(256, N // 8)))
            c = _attn("", kind, B, Hkv * g, Hkv, N, d, G, round(rng.uniform(0.1, 1.0), 2), rng.random() < 0.5,
                      rng.choice((0.3, 0.6)))
    del c["name"]
    return c


def work(case):
    c = case
    if c["kind"] in ROPE_KINDS:
        n = c["B"] * c["H"] * c["N"] * c["d"]
        axes = sum(1 for w in _widths(c) if w)
        rotated = sum(_widths(c)) * c["B"] * c["H"] * c["N"]
        return {"bytes": n * ((4 if c["dtype"] == "fp32" else 2) + 2) + 4 * c["B"] * c["N"] * axes, "flops": 3 * rotated}
    nq, nk = c["B"] * c["Hq"] * c["N"] * c["d"], c["B"] * c["Hkv"] * c["N"] * c["d"]
    pairs = float(c["rho"]) * c["N"] ** 2
    return {"bytes": 2 * (4 * nq + 4 * nk) + 4 * c["B"] * c["Hq"] * c["N"], "flops": 10.0 * pairs * c["d"] * c["B"] * c["Hq"]}


# ------------------------------------------------------------------------------- rotary positions
BASE = 10000.0
TRAINED = 32768            # trained length of the contexts that "yarn" extends
BETA_FAST, BETA_SLOW = 32.0, 1.0


def _widths(c):
    return [w for w in (c["wt"], c["wy"], c["wx"]) if w]


def _frequencies(width, scaling, factor):
    """Radians per position step of the width/2 pairs of one axis, in 64 bits."""
    i = torch.arange(width // 2, dtype=torch.float64)
    f = BASE ** (-2.0 * i / width)
    if scaling == "linear":
        return f / factor
    if scaling == "ntk":
        return (BASE * factor ** (width / max(width - 2, 1))) ** (-2.0 * i / width)
    if scaling == "yarn":
        # pairs that turn at least BETA_FAST times within the trained length keep their frequency,
        # those that turn at most BETA_SLOW times are slowed by the factor, a ramp between
        pair = lambda n: width * math.log(TRAINED / (n * 2.0 * math.pi)) / (2.0 * math.log(BASE))  # noqa: E731
        lo, hi = max(math.floor(pair(BETA_FAST)), 0), min(math.ceil(pair(BETA_SLOW)), width - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f / factor * (1.0 - keep) + f * keep
    return f


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0


def _angles(c, pos):
    """[B, N, sum(widths) / 2] angles in 64 bits."""
    parts = [pos[:, :, a, None].double() * _frequencies(w, c["scaling"], c["factor"]).to(pos.device)
             for a, w in enumerate(_widths(c))]
    return torch.cat(parts, dim=2)


def _pair_index(c, device):
    """Indices of the first and the second element of every rotated pair."""
    first, second, at = [], [], 0
    for w in _widths(c):
        i = torch.arange(w // 2, device=device)
        if c["layout"] == "interleaved":
            first.append(at + 2 * i)
            second.append(at + 2 * i + 1)
        else:
            first.append(at + i)
            second.append(at + w // 2 + i)
        at += w
    return torch.cat(first), torch.cat(second)


def _rotate(c, x, pos, sign, dtype):
    """amplitude * R(sign * pos) x for x [B, N, H, d] in `dtype`."""
    ang = _angles(c, pos)
    amp = _amplitude(c)
    cos, sin = (amp * ang.cos()).to(dtype)[:, :, None], (sign * amp * ang.sin()).to(dtype)[:, :, None]
    i, j = _pair_index(c, x.device)
    x = x.to(dtype)
    y = x.clone()
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., i] * sin + x[..., j] * cos
    return y


def _prepare_rope(c, g):
    B, H, N, d = c["B"], c["H"], c["N"], c["d"]
    t = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    n = torch.arange(N, device="cuda")
    frame = c["gy"] * c["gx"]
    pos = torch.stack([n // frame, n // c["gx"] % c["gy"], n % c["gx"]], dim=1).repeat(B, 1, 1)
    if c["start"]:
        # every sample of the batch stands somewhere else in its own context
        pos[:, :, 0] += c["start"] + torch.randint(0, 1000, (B, 1), generator=g, device="cuda")
    pos = pos[:, :, :len(_widths(c))].to(torch.int32).contiguous()
    s = {"case": c, "pos": pos}
    if c["kind"] == "rope":
        # Q and K come out of one fused projection, so x is a slice of a wider row
        fused = torch.randn((B, N, 2 * H, d), generator=g, device="cuda").to(t)
        s["x"] = fused[:, :, :H]
    else:
        s["dy"] = (1e-2 * torch.randn((B, H, N, d), generator=g, device="cuda")).bfloat16()
    if own:
        import free_block_sparse_sparsepr_b200 as spr

        s["rope"] = spr.Rope(d, tuple(_widths(c)), layout=c["layout"], base=BASE, scaling=c["scaling"],
                             factor=c["factor"], trained_length=TRAINED, beta_fast=BETA_FAST, beta_slow=BETA_SLOW)
    return s


def _run_rope(s):
    c = s["case"]
    t = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    if c["kind"] == "rope":
        if own:
            return {"y": s["rope"].forward(s["x"], s["pos"])}
        return {"y": _rotate(c, s["x"], s["pos"], 1.0, torch.float32).transpose(1, 2).contiguous().bfloat16()}
    if own:
        return {"dx": s["rope"].backward(s["dy"], s["pos"], dtype=t)}
    return {"dx": _rotate(c, s["dy"].transpose(1, 2), s["pos"], -1.0, torch.float32).contiguous().to(t)}


# ------------------------------------------------------------------------------- attention
def _features(c, g):
    """Q, K, V in fp32: random-phase Fourier features of the token position plus noise, as video tokens have."""
    B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    uni = lambda *shape: torch.rand(shape, generator=g, device="cuda")  # noqa: E731
    w = max(1, int(math.sqrt(N / 4)))
    n = torch.arange(N, device="cuda", dtype=torch.float32)
    at = torch.stack([n / N, (n / w).floor() % w / w, n % w / w], dim=1)
    omega, theta = 0.5 + 2.5 * uni(B, Hkv, 8, 3), 2.0 * math.pi * uni(B, Hkv, 8)
    G = rnd(B, Hkv, 8, d) / math.sqrt(8.0)
    phi = torch.cos(2.0 * math.pi * torch.einsum("nk,bhfk->bhnf", at, omega) + theta[:, :, None])
    base = 0.8 * phi @ G
    K = base + c["noise"] * rnd(B, Hkv, N, d)
    Q = base.repeat_interleave(Hq // Hkv, dim=1) + c["noise"] * rnd(B, Hq, N, d)
    return Q, K, rnd(B, Hkv, N, d), phi


def _offsets(c, g):
    """Offsets [B * Hkv, G + 1] of uneven groups (with `ragged`, some of them empty)."""
    P, N, G = c["B"] * c["Hkv"], c["N"], c["G"]
    cut = torch.rand((P, G - 1), generator=g, device="cuda")
    even = (torch.arange(1, G, device="cuda", dtype=torch.float32)[None] + (cut - 0.5)) / G
    cuts = (N * (cut if c["ragged"] else even)).round().clamp(0, N)
    if c["ragged"]:
        cuts[:, : G // 8] = 0.0
    ends = torch.tensor([[0.0, float(N)]], device="cuda").expand(P, 2)
    return torch.cat([ends, cuts], dim=1).sort(dim=1).values.to(torch.int32).contiguous()


def _labels(off, N):
    """Group of every group-major position, [P, N]."""
    n = torch.arange(N, device=off.device, dtype=torch.int32).expand(off.shape[0], N).contiguous()
    return torch.searchsorted(off[:, 1:].contiguous(), n, right=True)


def _group_mean(x, off):
    P, N, d = x.shape
    c = torch.cat([torch.zeros((P, 1, d), device=x.device, dtype=torch.float64), x.double().cumsum(1)], dim=1)
    o = off.long()[..., None].expand(-1, -1, d)
    total = c.gather(1, o[:, 1:]) - c.gather(1, o[:, :-1])
    return total / (off[:, 1:] - off[:, :-1]).clamp(min=1)[..., None]


def _prepare_sparse(c, g, s, Q, K, V, phi):
    """Group-major order, offsets, and the cells with the highest mean logits up to the density rho."""
    B, Hq, Hkv, N, d, G = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"], c["G"]
    P, r = B * Hkv, Hq // Hkv
    along = (phi.reshape(P, N, 8) * torch.randn((P, 1, 8), generator=g, device="cuda")).sum(2)
    kperm = along.argsort(dim=1)
    qperm = (along + 0.05 * torch.randn((P, N), generator=g, device="cuda")).argsort(dim=1)
    koff, qoff = _offsets(c, g), _offsets(c, g)
    take = lambda x, p: x.gather(1, p[..., None].expand(-1, -1, d))  # noqa: E731
    Kp, Vp = take(K.reshape(P, N, d), kperm), take(V.reshape(P, N, d), kperm)
    Qp = take(Q.reshape(P * r, N, d), qperm.repeat_interleave(r, dim=0))
    score = _group_mean(Qp.reshape(P, r, N, d).mean(1), qoff) @ _group_mean(Kp, koff).transpose(1, 2)
    ks, qs = (koff[:, 1:] - koff[:, :-1]), (qoff[:, 1:] - qoff[:, :-1])
    cost = (qs[:, :, None].double() * ks[:, None, :].double()).reshape(P, -1)
    score = score.masked_fill(ks[:, None, :] == 0, -math.inf)
    best = torch.zeros_like(score).scatter(2, score.argmax(2, keepdim=True), 1.0) * 1e9
    order = (score + best).reshape(P, -1).argsort(dim=1, descending=True)
    before = cost.gather(1, order).cumsum(1) - cost.gather(1, order)
    keep = torch.zeros((P, G * G), dtype=torch.bool, device="cuda")
    keep.scatter_(1, order, before < float(c["rho"]) * N * N)
    keep = keep.reshape(P, G, G)
    if c["ragged"]:
        keep[:, G // 2] = False          # a query group that keeps no cell
    rowptr = torch.zeros((P, G + 1), dtype=torch.int32, device="cuda")
    rowptr[:, 1:] = keep.sum(2).cumsum(1)
    kg = torch.zeros((P, G * G), dtype=torch.int32, device="cuda")
    z, _, k = keep.nonzero(as_tuple=True)
    count = keep.sum((1, 2))
    kg[z, torch.arange(z.numel(), device="cuda") - (count.cumsum(0) - count)[z]] = k.to(torch.int32)
    s.update(kperm=kperm.to(torch.int32), qperm=qperm.to(torch.int32), koff=koff, qoff=qoff, rowptr=rowptr, kg=kg)
    return Qp.reshape(B, Hq, N, d), Kp.reshape(B, Hkv, N, d), Vp.reshape(B, Hkv, N, d)


def _mask(s):
    """[P, N, N] kept pairs in group-major order, from the route's rows."""
    c = s["case"]
    P, N, G = c["B"] * c["Hkv"], c["N"], c["G"]
    i = torch.arange(G * G, device="cuda", dtype=torch.int32).expand(P, G * G).contiguous()
    row = torch.searchsorted(s["rowptr"][:, 1:].contiguous(), i, right=True)
    keep = torch.zeros((P, G + 1, G), dtype=torch.bool, device="cuda")
    keep[torch.arange(P, device="cuda")[:, None], row, s["kg"].long()] = True
    ql, kl = _labels(s["qoff"], N), _labels(s["koff"], N)
    z = torch.arange(P, device="cuda")[:, None, None]
    return keep[z, ql[:, :, None], kl[:, None, :]]


def _prepare_attn(c, g):
    s = {"case": c}
    Q, K, V, phi = _features(c, g)
    if c["kind"] == "sparse_bwd":
        Q, K, V = _prepare_sparse(c, g, s, Q, K, V, phi)
    Q, K, V = Q.bfloat16(), K.bfloat16(), V.bfloat16()
    B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
    r = Hq // Hkv
    dO = (1e-2 * torch.randn((B, Hq, N, d), generator=g, device="cuda")).bfloat16()
    # what the forward pass leaves: the output and the logarithm of each row's sum of exponentials
    keep = _mask(s) if c["kind"] == "sparse_bwd" else None
    O, lse = torch.empty_like(Q), torch.empty((B, Hq, N), device="cuda")
    for b in range(B):
        for h in range(Hq):
            S = Q[b, h].float() @ K[b, h // r].float().T / math.sqrt(d)
            if keep is not None:
                S.masked_fill_(~keep[b * Hkv + h // r], -math.inf)
            lse[b, h] = torch.logsumexp(S, dim=1)
            O[b, h] = (torch.exp(S - lse[b, h, :, None]).nan_to_num_(0.0) @ V[b, h // r].float()).bfloat16()
    s.update(Q=Q, K=K, V=V, O=O, lse=lse, dO=dO)
    if own:
        import free_block_sparse_sparsepr_b200 as spr

        s["handle"] = spr.SparsePR(B, Hq, Hkv, N, d, Gk=c["G"], Gq=c["G"], flags=spr.FLAG_HARD_DROP_ONLY)
        if c["kind"] == "sparse_bwd":
            s["partition"] = spr.partition_from_tensors({k: s[k] for k in ("kperm", "koff", "qperm", "qoff")})
            s["route"] = spr.route_from_tensors({k: s[k] for k in ("rowptr", "kg")})
    return s


def _run_attn(s):
    c = s["case"]
    sparse = c["kind"] == "sparse_bwd"
    Q, K, V, O, lse, dO = (s[k] for k in ("Q", "K", "V", "O", "lse", "dO"))
    if own:
        h = s["handle"]
        if sparse:
            dq, dk, dv = h.blocksparse_attn_bwd(Q, K, V, s["partition"], s["route"], O, lse, dO)
        else:
            dq, dk, dv = h.dense_attn_bwd(Q, K, V, O, lse, dO)
        return {"dQ": dq, "dK": dk, "dV": dv}
    B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
    r, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    q, o, do = (x.float().reshape(B * Hkv, r, N, d) for x in (Q, O, dO))
    k, v = (x.float().reshape(B * Hkv, 1, N, d) for x in (K, V))
    D = (o * do).sum(-1, keepdim=True)
    P = q @ k.transpose(-1, -2)
    P.mul_(scale).sub_(lse.reshape(B * Hkv, r, N, 1)).exp_()
    if sparse:
        P.masked_fill_(~_mask(s)[:, None], 0.0)
    dv = (P.transpose(-1, -2) @ do).sum(1)
    dS = do @ v.transpose(-1, -2)
    dS.sub_(D).mul_(P).mul_(scale)
    del P
    dq = dS @ k
    dk = (dS.transpose(-1, -2) @ q).sum(1)
    return _finish(s, dq, dk, dv, torch.bfloat16)


def _finish(s, dq, dk, dv, dtype):
    """Rounded gradients; block-sparse ones back in the original token order."""
    c = s["case"]
    B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
    dq, dk, dv = dq.reshape(B * Hq, N, d), dk.reshape(B * Hkv, N, d), dv.reshape(B * Hkv, N, d)
    if c["kind"] == "sparse_bwd":
        back = lambda x, p: torch.empty_like(x).scatter_(1, p.long()[..., None].expand(-1, -1, d), x)  # noqa: E731
        dq = back(dq, s["qperm"].repeat_interleave(Hq // Hkv, dim=0))
        dk, dv = back(dk, s["kperm"]), back(dv, s["kperm"])
    return {"dQ": dq.reshape(B, Hq, N, d).to(dtype), "dK": dk.reshape(B, Hkv, N, d).to(dtype),
            "dV": dv.reshape(B, Hkv, N, d).to(dtype)}


# ------------------------------------------------------------------------------- entry points
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return _prepare_rope(dict(case), g) if case["kind"] in ROPE_KINDS else _prepare_attn(dict(case), g)


def run(state):
    return _run_rope(state) if state["case"]["kind"] in ROPE_KINDS else _run_attn(state)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"] in ROPE_KINDS:
        forward = c["kind"] == "rope"
        x = s["x"] if forward else s["dy"].transpose(1, 2)
        # each pair as a complex number, turned by e^(i angle)
        i, j = _pair_index(c, x.device)
        turn = torch.polar(torch.full_like(_angles(c, s["pos"]), _amplitude(c)), (1 if forward else -1) * _angles(c, s["pos"]))
        y = x.double().clone()
        z = torch.complex(y[..., i], y[..., j]) * turn[:, :, None]
        y[..., i], y[..., j] = z.real, z.imag
        return {"y": y.transpose(1, 2).contiguous()} if forward else {"dx": y.contiguous()}
    B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
    r, sparse = Hq // Hkv, c["kind"] == "sparse_bwd"
    dq = torch.zeros((B, Hq, N, d), dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros((B, Hkv, N, d), dtype=torch.float64, device="cuda") for _ in range(2))
    # kept pairs from the labels of both sides, one row group at a time (apart from the plain form's mask)
    for b in range(B):
        for z in range(Hkv):
            p = b * Hkv + z
            k, v = s["K"][b, z].double(), s["V"][b, z].double()
            if sparse:
                ro, kg = s["rowptr"][p].tolist(), s["kg"][p].tolist()
                cells = torch.tensor([[m in kept for m in range(c["G"])]
                                      for kept in (set(kg[i:j]) for i, j in zip(ro, ro[1:]))], dtype=torch.bool, device="cuda")
                rows = cells.repeat_interleave(s["qoff"][p].long().diff(), dim=0)
                allowed = rows.repeat_interleave(s["koff"][p].long().diff(), dim=1)
            for h in range(z * r, (z + 1) * r):
                q, do = s["Q"][b, h].double(), s["dO"][b, h].double()
                logit = (q @ k.T) / math.sqrt(d) - s["lse"][b, h].double()[:, None]
                if sparse:
                    logit = torch.where(allowed, logit, -math.inf)
                P = logit.exp()
                inner = do @ v.T - (do * s["O"][b, h].double()).sum(1)[:, None]
                dv[b, z] += P.T @ do
                E = P * inner / math.sqrt(d)
                dq[b, h] = E @ k
                dk[b, z] += E.T @ q
    return _finish(s, dq, dk, dv, torch.float64)
