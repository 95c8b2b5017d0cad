"""One attention layer's forward and backward as a training program runs them: rotary positions of the
token-major projections, partition and route, the routed (or the dense) attention, and the gradients back
to the projections; every gradient against fp64 autograd of the same function, the route held constant."""
import math

import pytest

torch = pytest.importorskip("torch")

import free_block_sparse_sparsepr_b200 as spr  # noqa: E402
from bwd_helpers import U_BF16, backward_reference, check_gradients, pair_mask  # noqa: E402

pytestmark = pytest.mark.gpu

GRID = (4, 12, 13)
B, HQ, HKV, D, G = 1, 4, 2, 128, 12
N = GRID[0] * GRID[1] * GRID[2]
WIDTHS = (44, 42, 42)


def _projection(seed):
    """The fused token-major Q, K, V projection [B, N, Hq + 2 Hkv, d] and the gradient that reaches O."""
    g = torch.Generator().manual_seed(seed)
    t, y, x = (a.reshape(-1).float() for a in torch.meshgrid(*[torch.arange(n) for n in GRID], indexing="ij"))
    at = torch.stack([t / GRID[0], y / GRID[1], x / GRID[2]], 1)
    phi = torch.cos(2 * math.pi * (at @ (0.5 + torch.rand((3, 8), generator=g))))
    fused = 0.6 * (phi @ torch.randn((8, (HQ + 2 * HKV) * D), generator=g)).reshape(N, -1, D)
    fused = (fused + 0.4 * torch.randn(fused.shape, generator=g))[None].bfloat16().cuda()
    pos = torch.stack([t, y, x], 1).to(torch.int32).cuda()
    return fused, pos, (0.01 * torch.randn((B, HQ, N, D), generator=g)).bfloat16().cuda()


def _turn(x, pos, rope):
    """rope.forward in the dtype of x, differentiable: [B, N, H, d] -> [B, H, N, d]."""
    f = torch.tensor(rope.freq, dtype=torch.float64, device=x.device)
    axis = torch.cat([torch.full((w // 2,), a) for a, w in enumerate(rope.widths)]).cuda()
    ang = (pos.double()[:, axis] * f)[None, :, None]
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * ang.cos() - v * ang.sin(), u * ang.sin() + v * ang.cos()], -1).flatten(-2).transpose(1, 2)


def _autograd(Q, K, V, dO, masks):
    """fp64 O, lse and gradients of sum(dO . O) from the bf16 head-major Q, K, V."""
    q, k, v = (x.double().requires_grad_() for x in (Q, K, V))
    r = HQ // HKV
    S = q @ k.repeat_interleave(r, 1).transpose(-1, -2) / math.sqrt(D)
    if masks is not None:
        S = S.masked_fill(~torch.stack(masks).repeat_interleave(r, 0)[None], -math.inf)
    O = torch.softmax(S, -1) @ v.repeat_interleave(r, 1)
    (O * dO.double()).sum().backward()
    return O.detach(), S.detach(), {"dQ": q.grad, "dK": k.grad, "dV": v.grad}


def _check_projection(dfused, fused, pos, rope, Q, K, V, O, lse, dO, masks):
    """The gradient of the projection against autograd's. Allowed, in the 2-norm: the kernels' own error
    (backward_reference), the change of D = dO.O from O as the forward pass rounded it (its size is
    taken from O itself), and one rounding each of the head-major and the token-major gradient."""
    exact_O, S, grads = _autograd(Q, K, V, dO, masks)
    _, _, square = backward_reference(Q, K, V, O, lse, dO, masks)
    P = torch.softmax(S, -1)
    dD = (dO.double() * (O.double() - exact_O)).sum(-1, keepdim=True)
    r = HQ // HKV
    drift = {"dQ": (P * dD) @ K.double().repeat_interleave(r, 1) / math.sqrt(D),
             "dK": ((P * dD).transpose(-1, -2) @ Q.double() / math.sqrt(D)).reshape(B, HKV, r, N, D).sum(2), "dV": torch.zeros_like(grads["dV"])}
    x = fused.double().requires_grad_()
    (_turn(x[:, :, :HQ], pos, rope) * grads["dQ"]).sum().backward()
    (_turn(x[:, :, HQ:HQ + HKV], pos, rope) * grads["dK"]).sum().backward()
    x.grad[:, :, HQ + HKV:] = grads["dV"].transpose(1, 2)
    for n, lo, hi in (("dQ", 0, HQ), ("dK", HQ, HQ + HKV), ("dV", HQ + HKV, HQ + 2 * HKV)):
        want = x.grad[:, :, lo:hi]
        e = (dfused[:, :, lo:hi].double() - want).norm().item()
        allowed = square[n].sum().sqrt() + drift[n].norm() + 2 * U_BF16 * want.norm()
        assert e <= allowed.item(), (n, e, allowed.item(), want.norm().item())


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spr.load_library()


def _rotate(rope, fused, pos):
    Q, K = rope.forward(fused[:, :, :HQ], pos), rope.forward(fused[:, :, HQ:HQ + HKV], pos)
    # the turned pairs, rounded once, against the same map in fp64
    for got, part in ((Q, fused[:, :, :HQ]), (K, fused[:, :, HQ:HQ + HKV])):
        want = _turn(part.double(), pos, rope)
        assert ((got.double() - want).abs() <= U_BF16 * want.abs() + 2.0 ** -20 * part.double().abs().amax()).all()
    return Q, K, fused[:, :, HQ + HKV:].transpose(1, 2).contiguous()


def _back(rope, dq, dk, dv, pos, fused):
    dfused = torch.empty_like(fused)
    rope.backward(dq, pos, out=dfused[:, :, :HQ])
    rope.backward(dk, pos, out=dfused[:, :, HQ:HQ + HKV])
    dfused[:, :, HQ + HKV:] = dv.transpose(1, 2)
    return dfused


def test_routed_layer():
    rope = spr.Rope(D, WIDTHS, layout="interleaved")
    with spr.SparsePR(B, HQ, HKV, N, D, Gk=G, Gq=G, rho_exec=0.4, flags=spr.FLAG_HARD_DROP_ONLY) as h:
        saved = []
        for layer in range(2):       # two layers on one handle: what the backward pass needs is copied out
            fused, pos, dO = _projection(layer)
            Q, K, V = _rotate(rope, fused, pos)
            part = h.partition(Q, K)
            route = h.route(Q, part)
            Qp, Kp, Vp, Osp, O = (torch.empty_like(x) for x in (Q, K, V, Q, Q))
            lse = torch.empty((B, HQ, N), device="cuda")
            h.permute(Q, K, V, part, Qp, Kp, Vp)
            h.blocksparse_attn(Qp, Kp, Vp, part, route, Osp, lse)
            h.writeback(part, Osp, None, O)
            keep = {k: v.clone() for k, v in {**h.partition_views(part), **h.route_views(route)}.items()
                    if k in ("kperm", "koff", "qperm", "qoff", "kcent", "rowptr", "kg")}
            saved.append((fused, pos, dO, Q, K, V, Qp, Kp, Vp, Osp, lse, O, keep))
        for fused, pos, dO, Q, K, V, Qp, Kp, Vp, Osp, lse, O, keep in reversed(saved):
            part, route = spr.partition_from_tensors(keep), spr.route_from_tensors(keep)
            dOsp = torch.empty_like(dO)
            h.permute(dO, None, None, part, dOsp)
            dq, dk, dv = h.blocksparse_attn_bwd(Qp, Kp, Vp, part, route, Osp, lse, dOsp)
            dfused = _back(rope, dq, dk, dv, pos, fused)
            torch.cuda.synchronize()
            assert h.device_status() == 0
            rowptr, kg = keep["rowptr"].cpu(), keep["kg"].cpu()
            masks, in_order = [], []
            for z in range(B * HKV):
                cells = torch.zeros((G, G), dtype=torch.bool)
                for a in range(G):
                    cells[a, kg[z, rowptr[z, a]:rowptr[z, a + 1]].long()] = True
                m = pair_mask(cells, keep["qoff"][z].cpu(), keep["koff"][z].cpu()).cuda()
                in_order.append(m)
                masks.append(torch.zeros_like(m).index_put_(
                    (keep["qperm"][z].long()[:, None], keep["kperm"][z].long()[None]), m))
            assert 0.3 < torch.stack(masks).double().mean() < 0.5
            lse_o = torch.empty_like(lse)
            for x in range(B * HQ):
                lse_o[0, x, keep["qperm"][x // (HQ // HKV)].long()] = lse[0, x]
            check_gradients((dq, dk, dv), backward_reference(Q, K, V, O, lse_o, dO, masks), "routed layer")
            _check_projection(dfused, fused, pos, rope, Q, K, V, O, lse_o, dO, masks)


def test_dense_layer_in_a_graph():
    """The same with the dense attention, forward and backward captured and replayed on new inputs."""
    rope = spr.Rope(D, WIDTHS, layout="interleaved")
    fused, pos, dO = _projection(3)
    with spr.SparsePR(B, HQ, HKV, N, D, Gk=1, Gq=1, flags=spr.FLAG_HARD_DROP_ONLY) as h:
        lse = torch.empty((B, HQ, N), device="cuda")
        ws = torch.empty(h.attn_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda")

        def step():
            Q, K = rope.forward(fused[:, :, :HQ], pos), rope.forward(fused[:, :, HQ:HQ + HKV], pos)
            V = fused[:, :, HQ + HKV:].transpose(1, 2).contiguous()
            O = h.dense_attn(Q, K, V, lse=lse)
            return Q, K, V, O, _back(rope, *h.dense_attn_bwd(Q, K, V, O, lse, dO, workspace=ws), pos, fused)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        fresh = _projection(4)
        fused.copy_(fresh[0])
        dO.copy_(fresh[2])
        graph.replay()
        torch.cuda.synchronize()
        assert h.device_status() == 0
        captured = [x.clone() for x in out]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
        Q, K, V, O, dfused = eager
        _check_projection(dfused, fused, pos, rope, Q, K, V, O, lse, dO, None)
        del graph
