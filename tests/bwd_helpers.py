"""Plain fp64 gradients of dense and block-sparse attention, error bounds of the kernels' arithmetic
against them, and small routed inputs."""
from __future__ import annotations

import math

import torch

U_BF16 = torch.finfo(torch.bfloat16).eps / 2     # a bf16 rounding: at most half a step, 2^-8
E_F32 = torch.finfo(torch.float32).eps           # an fp32 step, 2^-23: a tensor-core sum may truncate


def random_groups(gen, N, G, empty=0):
    """Offsets of G groups over N rows at random cuts, `empty` of them without rows."""
    cuts = torch.randint(0, N + 1, (G - 1,), generator=gen)
    cuts[:empty] = 0
    return torch.cat([torch.tensor([0, N]), cuts]).sort().values.to(torch.int32)


def random_route(gen, P, Gq, Gk, density, empty_rows=()):
    """Kept cells [P, Gq, Gk] and their CSR (rowptr [P, Gq + 1], kg [P, Gq * Gk])."""
    keep = torch.rand((P, Gq, Gk), generator=gen) < density
    for a in empty_rows:
        keep[:, a] = False
    return keep, *csr(keep)


def csr(keep):
    P, Gq, Gk = keep.shape
    rowptr = torch.zeros((P, Gq + 1), dtype=torch.int32)
    rowptr[:, 1:] = keep.sum(2).cumsum(1)
    kg = torch.zeros((P, Gq * Gk), dtype=torch.int32)
    for z in range(P):
        ids = keep[z].nonzero()[:, 1]
        kg[z, : len(ids)] = ids.to(torch.int32)
    return rowptr, kg


def pair_mask(keep, qoff, koff):
    """[N, N] kept pairs of one KV head in group-major order."""
    rows = keep.repeat_interleave(qoff.long().diff(), dim=0)
    return rows.repeat_interleave(koff.long().diff(), dim=1)


def forward_reference(Q, K, V, masks=None):
    """O (fp64) and lse (fp64) of bf16 Q [B, Hq, N, d], K, V [B, Hkv, N, d]; masks[b * Hkv + h] keeps pairs."""
    B, Hq, N, d = Q.shape
    r = Hq // K.shape[1]
    O = torch.zeros((B, Hq, N, d), dtype=torch.float64, device=Q.device)
    lse = torch.full((B, Hq, N), -math.inf, dtype=torch.float64, device=Q.device)
    for b in range(B):
        for h in range(Hq):
            S = Q[b, h].double() @ K[b, h // r].double().T / math.sqrt(d)
            if masks is not None:
                S = S.masked_fill(~masks[b * K.shape[1] + h // r], -math.inf)
            lse[b, h] = torch.logsumexp(S, dim=1)
            O[b, h] = torch.exp(S - lse[b, h, :, None]).nan_to_num(0.0) @ V[b, h // r].double()
    return O, lse


def backward_reference(Q, K, V, O, lse, dO, masks=None):
    """The fp64 gradients, and per gradient a worst-case bound and an rms estimate of the kernels' error.

    The kernels form logits, dO.v and D in fp32 (d products each, at most one step 2^-23 a product),
    P = 2^x with a relative error of the exponent's absolute error plus 2^-18 (a polynomial that is
    2^-18.5 off at most, after roundings of its five terms below 2^-21 together), round P and dS to
    bf16 (2^-8 of their value) as operands, sum in fp32 over n pairs (n steps of the sum of
    magnitudes) and round the result to bf16. The worst case adds all magnitudes; the rms estimate
    adds the squares of the operand roundings, taken at their full half step, so that it holds for
    the 2-norm over a tensor whose roundings are independent."""
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    r, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    out = {n: torch.zeros_like(x, dtype=torch.float64) for n, x in (("dQ", Q), ("dK", K), ("dV", V))}
    worst = {n: torch.zeros_like(x) for n, x in out.items()}
    square = {n: torch.zeros_like(x) for n, x in out.items()}
    n_sum = {"dQ": N, "dK": N * r, "dV": N * r}
    size = {n: torch.zeros_like(x) for n, x in out.items()}
    for b in range(B):
        for h in range(Hq):
            z = h // r
            q, o, do = (x[b, h].double() for x in (Q, O, dO))
            k, v = K[b, z].double(), V[b, z].double()
            ls = lse[b, h].double()[:, None]
            s = q @ k.T * scale
            x = s - ls
            if masks is not None:
                x = torch.where(masks[b * Hkv + z], x, -math.inf)
            P = x.exp()
            D = (do * o).sum(1, keepdim=True)
            dP = do @ v.T
            dS = P * (dP - D)
            # relative error of P; absolute error of dS before its rounding
            finite_ls = torch.where(ls.isfinite(), ls, 0.0)
            eP = scale * d * E_F32 * (q.abs() @ k.abs().T) + 4 * E_F32 * (s.abs() + finite_ls.abs()) + 2.0 ** -18
            eS = P * (eP * (dP - D).abs() + d * E_F32 * (do.abs() @ v.abs().T + (do.abs() * o.abs()).sum(1, keepdim=True)))
            rP, rS = U_BF16 * P, U_BF16 * dS.abs()
            out["dV"][b, z] += P.T @ do
            out["dQ"][b, h] = scale * (dS @ k)
            out["dK"][b, z] += scale * (dS.T @ q)
            worst["dV"][b, z] += (rP + P * eP).T @ do.abs()
            worst["dQ"][b, h] = scale * ((rS + eS) @ k.abs())
            worst["dK"][b, z] += scale * ((rS + eS).T @ q.abs())
            square["dV"][b, z] += (rP ** 2).T @ do ** 2
            square["dQ"][b, h] = scale ** 2 * (rS ** 2 @ k ** 2)
            square["dK"][b, z] += scale ** 2 * ((rS ** 2).T @ q ** 2)
            size["dV"][b, z] += P.T @ do.abs()
            size["dQ"][b, h] = scale * (dS.abs() @ k.abs())
            size["dK"][b, z] += scale * (dS.abs().T @ q.abs())
            # the errors before the operands' rounding enter the estimate at their full size
            square["dV"][b, z] += ((P * eP).T @ do.abs()) ** 2
            square["dQ"][b, h] += (scale * (eS @ k.abs())) ** 2
            square["dK"][b, z] += (scale * (eS.T @ q.abs())) ** 2
    for n in out:
        sums = n_sum[n] * E_F32 * size[n]
        worst[n] += sums + U_BF16 * (out[n].abs() + worst[n] + sums) + 1e-30
        square[n] += sums ** 2 + (U_BF16 * out[n]) ** 2
    return out, worst, square


def check_gradients(got, reference, what=""):
    out, worst, square = reference
    for n, g in zip(("dQ", "dK", "dV"), got):
        if g is None:
            continue
        assert g.dtype == torch.bfloat16 and torch.isfinite(g).all(), f"{what} {n}: not finite"
        e = (g.double() - out[n]).abs()
        over = (e / worst[n]).max().item()
        assert over <= 1.0, f"{what} {n}: {over:.3g} times the worst-case bound"
        rms, allowed = e.norm().item(), square[n].sum().sqrt().item()
        assert rms <= allowed + 1e-30, f"{what} {n}: 2-norm of the error {rms:.4g}, estimate {allowed:.4g}"
