"""dS as two bf16 parts in dQ (FLAG_BWD_SPLIT_DS): dQ as near to fp64 as its own rounding to bf16, dK and dV bit for
bit those of a handle without the flag."""
import math

import pytest

torch = pytest.importorskip("torch")

import free_block_sparse_sparsepr_b200 as spr  # noqa: E402
from bwd_helpers import E_F32, U_BF16, backward_reference, check_gradients, forward_reference  # noqa: E402
from test_attn_bwd import _inputs, _need_gpu, _routed, _structs, _to_original  # noqa: E402

gpu = pytest.mark.gpu


def _handle(B, Hq, Hkv, N, d, G=1, split=True):
    return spr.SparsePR(B, Hq, Hkv, N, d, Gk=G, Gq=G, flags=spr.FLAG_HARD_DROP_ONLY | (spr.FLAG_BWD_SPLIT_DS if split else 0))


def _split_reference(Q, K, V, O, lse, dO, masks=None):
    """backward_reference with dQ's operand rounded at 2^-16 of dS: the first part leaves at most 2^-8 of it, exactly
    formed in fp32, and the second rounds that to bf16, 2^-8 of 2^-8."""
    out, worst, square = backward_reference(Q, K, V, O, lse, dO, masks)
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    r, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    for b in range(B):
        for h in range(Hq):
            z = h // r
            q, o, do, k, v = (x.double() for x in (Q[b, h], O[b, h], dO[b, h], K[b, z], V[b, z]))
            x = q @ k.T * scale - lse[b, h].double()[:, None]
            if masks is not None:
                x = torch.where(masks[b * Hkv + z], x, -math.inf)
            rS = U_BF16 * (x.exp() * (do @ v.T - (do * o).sum(1, keepdim=True))).abs()
            worst["dQ"][b, h] -= (1 - U_BF16) * (1 + U_BF16) * scale * (rS @ k.abs())
            square["dQ"][b, h] -= (1 - U_BF16 ** 2) * scale ** 2 * (rS ** 2 @ k ** 2)
    square["dQ"].clamp_(min=0)       # a difference of sums in 64 bits
    return out, worst, square


def _before_rounding(Q, K, V, O, lse, dO, masks=None):
    """Estimate [B, Hq, N, d] of what dQ is off by before its rounding, as backward_reference has the parts: a pair's
    own errors (logit, exponential, dO.v, the second part of dS) are independent from key to key and add their
    squares; those of D and lse are a row's and go with the row's sum; the sum over the keys takes 16 products a
    step, each step at most two steps of 2^-23 of the magnitudes so far (alignment and addition)."""
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    r, scale, e = Hq // Hkv, 1.0 / math.sqrt(d), E_F32
    total = torch.zeros_like(Q, dtype=torch.float64)
    for b in range(B):
        for h in range(Hq):
            z = h // r
            q, o, do, k, v = (x.double() for x in (Q[b, h], O[b, h], dO[b, h], K[b, z], V[b, z]))
            ls = lse[b, h].double()[:, None]
            s = q @ k.T * scale
            x = s - ls
            if masks is not None:
                x = torch.where(masks[b * Hkv + z], x, -math.inf)
            P = x.exp()
            dS = P * (do @ v.T - (do * o).sum(1, keepdim=True))
            eP = scale * d * e * (q.abs() @ k.abs().T) + 4 * e * s.abs() + 2.0 ** -18 + U_BF16 ** 2
            own = eP * dS.abs() + P * d * e * (do.abs() @ v.abs().T)
            row = d * e * (do.abs() * o.abs()).sum(1, keepdim=True) * (P @ k).abs()
            row = row + 4 * e * torch.where(ls.isfinite(), ls, 0.0).abs() * (dS @ k).abs()
            total[b, h] = scale * ((own ** 2 @ k ** 2).sqrt() + row + N / 8 * e * (dS.abs() @ k.abs()))
    return total


def _check(got, plain, reference, before, what):
    """The bounds, and the 2-norm of dQ's error against that of rounding the exact dQ: equal up to what comes before
    the rounding and 5%, ten standard deviations of a sum of 40000 independent squared roundings and more. One
    bf16 part of dS does not pass."""
    check_gradients(got, reference, what)
    assert torch.equal(got[1], plain[1]) and torch.equal(got[2], plain[2]), what
    out = reference[0]["dQ"]
    rounding = (out.bfloat16().double() - out).norm().item()
    allowed = 1.05 * rounding + before.norm().item()
    e, e_plain = (got[0].double() - out).norm().item(), (plain[0].double() - out).norm().item()
    assert e <= allowed, (what, e, rounding, allowed)
    assert e_plain > allowed, (what, e_plain, rounding, allowed)


DENSE = [(1, 2, 1, 300, 64), (1, 3, 1, 391, 128), (1, 2, 2, 640, 128), (2, 24, 12, 517, 128), (2, 24, 12, 517, 64), (4, 40, 40, 100, 128)]


@gpu
@pytest.mark.parametrize("shape", DENSE, ids=str)
def test_dense(shape):
    _need_gpu()
    B, Hq, Hkv, N, d = shape
    Q, K, V, dO = _inputs(N + d, *shape)
    O, lse = forward_reference(Q, K, V)
    args = (Q, K, V, O.bfloat16(), lse.float(), dO)
    with _handle(*shape) as h, _handle(*shape, split=False) as p:
        got, again = h.dense_attn_bwd(*args), h.dense_attn_bwd(*args)
        plain = p.dense_attn_bwd(*args)
        torch.cuda.synchronize()
        assert h.device_status() == 0
    assert torch.equal(got[0], again[0])
    _check(got, plain, _split_reference(*args), _before_rounding(*args), f"dense {shape}")


ROUTED = [(1, 1, 1, 2600, 64, 20), (1, 8, 1, 700, 128, 12), (2, 40, 40, 260, 128, 20), (2, 8, 4, 900, 128, 24), (4, 40, 20, 400, 64, 4)]


@gpu
@pytest.mark.parametrize("case", ROUTED, ids=str)
def test_routed(case):
    """Shared streams, a tile a group, tiles of two groups; a graph."""
    _need_gpu()
    B, Hq, Hkv, N, d, G = case
    Q, K, V, dO = _inputs(N + d, B, Hq, Hkv, N, d)
    t, masks = _routed(N, B * Hkv, N, G, G, 0.4)
    O, lse = forward_reference(Q, K, V, masks)
    part, route = _structs(t)
    saved = (O.bfloat16(), lse.float(), dO)
    with _handle(B, Hq, Hkv, N, d, G) as h, _handle(B, Hq, Hkv, N, d, G, split=False) as p:
        got = h.blocksparse_attn_bwd(Q, K, V, part, route, *saved)
        dq = h.blocksparse_attn_bwd(Q, K, V, part, route, *saved, need_dkv=False)[0]
        plain = p.blocksparse_attn_bwd(Q, K, V, part, route, *saved)
        out = [torch.zeros_like(x) for x in got]
        ws = torch.empty(h.attn_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h.blocksparse_attn_bwd(Q, K, V, part, route, *saved, *out, workspace=ws)
        graph.replay()
        torch.cuda.synchronize()
        del graph
        assert h.device_status() == 0
    assert torch.equal(got[0], dq) and all(torch.equal(a, b) for a, b in zip(got, out))
    _check(got, plain, _to_original(_split_reference(Q, K, V, *saved, masks), t, Hq // Hkv), _before_rounding(Q, K, V, *saved, masks),
           f"routed {case}")


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_stays_in_its_row(d):
    _need_gpu()
    shape = (1, 1, 1, 200, d)
    Q, K, V, dO = _inputs(8, *shape)
    O, lse = forward_reference(Q, K, V)
    with _handle(*shape) as h:
        clean = h.dense_attn_bwd(Q, K, V, O.bfloat16(), lse.float(), dO)[0]
        for bad in (math.nan, math.inf):
            do = dO.clone()
            do[0, 0, 70, 3] = bad
            dq = h.dense_attn_bwd(Q, K, V, O.bfloat16(), lse.float(), do)[0]
            rest = torch.arange(200, device="cuda") != 70
            assert torch.equal(dq[0, 0, rest], clean[0, 0, rest]) and not torch.isfinite(dq[0, 0, 70]).any()
