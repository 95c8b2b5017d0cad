"""Backward passes of dense and block-sparse attention against plain fp64 gradients: head layouts, odd
and tiny lengths, uneven and empty groups, rows without keys, skipped gradients, non-finite
neighbours, streams, graphs, and the refusals (which need no GPU)."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import free_block_sparse_sparsepr_b200 as spr  # noqa: E402
from bwd_helpers import (backward_reference, check_gradients, csr, forward_reference, pair_mask,  # noqa: E402
                         random_groups, random_route)

gpu = pytest.mark.gpu


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spr.load_library()


def _inputs(seed, B, Hq, Hkv, N, d, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda h: torch.randn((B, h, N, d), generator=g)  # noqa: E731
    base = torch.randn((B, Hkv, 1, d), generator=g)
    K = amp * (0.5 * base + rnd(Hkv))
    Q = amp * (0.5 * base.repeat_interleave(Hq // Hkv, 1) + rnd(Hq))
    return [x.bfloat16().cuda() for x in (Q, K, rnd(Hkv), 0.01 * rnd(Hq))]


def _handle(B, Hq, Hkv, N, d, Gk=1, Gq=1):
    return spr.SparsePR(B, Hq, Hkv, N, d, Gk=Gk, Gq=Gq, flags=spr.FLAG_HARD_DROP_ONLY)


def _routed(seed, P, N, Gq, Gk, density, empty=0, empty_rows=()):
    g = torch.Generator().manual_seed(seed)
    keep, rowptr, kg = random_route(g, P, Gq, Gk, density, empty_rows)
    qoff = torch.stack([random_groups(g, N, Gq, empty) for _ in range(P)])
    koff = torch.stack([random_groups(g, N, Gk, empty) for _ in range(P)])
    perm = lambda: torch.stack([torch.randperm(N, generator=g) for _ in range(P)]).to(torch.int32)  # noqa: E731
    masks = [pair_mask(keep[z], qoff[z], koff[z]).cuda() for z in range(P)]
    t = {k: v.cuda() for k, v in dict(qperm=perm(), kperm=perm(), qoff=qoff, koff=koff, rowptr=rowptr, kg=kg).items()}
    return t, masks


def _structs(t):
    return (spr.partition_from_tensors({k: t[k] for k in ("qperm", "kperm", "qoff", "koff")}),
            spr.route_from_tensors({k: t[k] for k in ("rowptr", "kg")}))


def _to_original(grads, t, r):
    """fp64 group-major tensors (dQ, dK, dV in each dict) into the original order."""
    out = []
    for d in grads:
        o = {}
        for n, x in d.items():
            perm = t["qperm"].repeat_interleave(r, 0) if n == "dQ" else t["kperm"]
            flat = x.reshape(-1, *x.shape[2:])
            o[n] = torch.empty_like(flat).scatter_(1, perm.long()[..., None].expand_as(flat), flat).reshape(x.shape)
        out.append(o)
    return out


DENSE = [
    # B, Hq, Hkv, N, d: one token; one row past a tile and one short of it; grouped queries; odd lengths
    (1, 1, 1, 1, 64), (1, 2, 1, 1, 128), (2, 2, 2, 2, 128), (1, 2, 2, 63, 64), (1, 3, 1, 127, 128), (1, 1, 1, 128, 128),
    (1, 4, 2, 129, 64), (2, 4, 1, 257, 128), (1, 6, 2, 391, 64), (1, 2, 2, 640, 128), (3, 5, 5, 1000, 128),
    (1, 8, 1, 1153, 128), (1, 1, 1, 2600, 64),
    # more tiles than SMs, streams longer than the rings
    (4, 16, 8, 1100, 64), (2, 24, 12, 1030, 128),
]


@gpu
@pytest.mark.parametrize("shape", DENSE, ids=str)
def test_dense_gradients(shape):
    _need_gpu()
    B, Hq, Hkv, N, d = shape
    Q, K, V, dO = _inputs(N + d, *shape)
    with _handle(*shape) as h:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device="cuda")
        O = h.dense_attn(Q, K, V, lse=lse)
        got = h.dense_attn_bwd(Q, K, V, O, lse, dO)
        again = h.dense_attn_bwd(Q, K, V, O, lse, dO)
        torch.cuda.synchronize()
        assert h.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "two runs differ"
    # lse: d products of one step 2^-23 each, and the row sum's and logarithm's roundings
    ref_lse = forward_reference(Q, K, V)[1]
    bound = 2.0 ** -23 * (d * (Q.double().abs().sum(-1) * K.double().abs().amax()) / math.sqrt(d) + N + 8 * (1 + ref_lse.abs()))
    assert ((lse.double() - ref_lse).abs() <= bound).all()
    check_gradients(got, backward_reference(Q, K, V, O, lse, dO), f"dense {shape}")


SPARSE = [
    # B, Hq, Hkv, N, d, Gq, Gk, density, empty groups, empty rows
    (1, 1, 1, 1, 64, 1, 1, 1.0, 0, ()),
    (1, 2, 2, 5, 128, 5, 3, 0.6, 0, (0,)),
    (1, 2, 1, 130, 64, 3, 4, 0.5, 0, ()),
    (2, 4, 2, 300, 128, 7, 5, 0.4, 2, (1,)),
    (1, 3, 1, 515, 128, 9, 33, 0.3, 3, (0, 4)),
    (1, 8, 2, 777, 64, 40, 24, 0.25, 8, (5, 6)),
    (1, 2, 2, 1500, 128, 64, 64, 0.15, 4, (7,)),
    (1, 2, 2, 900, 128, 4, 4, 1.0, 0, ()),
    (1, 6, 2, 256, 64, 256, 256, 0.1, 0, ()),      # groups of about one row
    (1, 1, 1, 700, 128, 6, 6, 0.0, 0, ()),         # nothing kept
]


@gpu
@pytest.mark.parametrize("case", SPARSE, ids=str)
def test_blocksparse_gradients(case):
    _need_gpu()
    B, Hq, Hkv, N, d, Gq, Gk, density, empty, empty_rows = case
    P, r = B * Hkv, Hq // Hkv
    Q, K, V, dO = _inputs(7 * N + d, B, Hq, Hkv, N, d)
    t, masks = _routed(N, P, N, Gq, Gk, density, empty, empty_rows)
    part, route = _structs(t)
    O, lse = forward_reference(Q, K, V, masks)
    O, lse = O.bfloat16(), lse.float()
    with _handle(B, Hq, Hkv, N, d, Gk, Gq) as h:
        got = h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO)
        again = h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO)
        torch.cuda.synchronize()
        assert h.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "two runs differ"
    check_gradients(got, _to_original(backward_reference(Q, K, V, O, lse, dO, masks), t, r), f"sparse {case}")


def _routed_by(keep, seed, P, N, empty=0):
    g = torch.Generator().manual_seed(seed)
    _, Gq, Gk = keep.shape
    rowptr, kg = csr(keep)
    qoff = torch.stack([random_groups(g, N, Gq, empty) for _ in range(P)])
    koff = torch.stack([random_groups(g, N, Gk, empty) for _ in range(P)])
    perm = lambda: torch.stack([torch.randperm(N, generator=g) for _ in range(P)]).to(torch.int32)  # noqa: E731
    masks = [pair_mask(keep[z], qoff[z], koff[z]).cuda() for z in range(P)]
    return {k: v.cuda() for k, v in dict(qperm=perm(), kperm=perm(), qoff=qoff, koff=koff, rowptr=rowptr, kg=kg).items()}, masks


# Enough tiles to fill the SMs: tiles may then hold rows of two groups. Neighbours keep much the same groups
# (band: those up to `share` of all away), or groups drawn one by one.
JOINED = [
    # B, Hq, Hkv, N, d, Gq, Gk, band, share, empty groups
    (2, 8, 4, 900, 128, 24, 20, True, 0.2, 2), (2, 8, 4, 900, 128, 24, 20, False, 0.3, 2),
    (1, 12, 12, 1300, 64, 40, 30, True, 0.3, 3), (1, 12, 12, 1300, 64, 40, 30, False, 0.1, 0),
    (1, 10, 10, 517, 128, 2, 16, False, 1.0, 0), (2, 16, 8, 700, 64, 20, 21, False, 0.0, 4),
    (1, 40, 20, 1030, 128, 32, 32, True, 0.06, 16), (1, 24, 24, 2049, 128, 9, 60, True, 0.15, 0),
]


@gpu
@pytest.mark.parametrize("case", JOINED, ids=str)
def test_tiles_of_two_groups(case):
    _need_gpu()
    B, Hq, Hkv, N, d, Gq, Gk, band, share, empty = case
    P, r = B * Hkv, Hq // Hkv
    at = lambda G: (torch.arange(G) + 0.5) / G  # noqa: E731
    keep = ((at(Gq)[:, None] - at(Gk)).abs() < share).expand(P, Gq, Gk) if band else \
        torch.rand((P, Gq, Gk), generator=torch.Generator().manual_seed(N)) < share
    Q, K, V, dO = _inputs(5 * N + d, B, Hq, Hkv, N, d)
    t, masks = _routed_by(keep, N + Gq, P, N, empty)
    part, route = _structs(t)
    O, lse = forward_reference(Q, K, V, masks)
    O, lse = O.bfloat16(), lse.float()
    with _handle(B, Hq, Hkv, N, d, Gk, Gq) as h:
        ws = torch.full((h.attn_bwd_workspace_bytes(),), 0x7B, dtype=torch.uint8, device="cuda")
        got = h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO, workspace=ws)
        dq = h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO, need_dkv=False)[0]
        _, dk, dv = h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO, need_dq=False)
        out = [torch.zeros_like(x) for x in got]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO, *out, workspace=ws)
        graph.replay()
        torch.cuda.synchronize()
        del graph
        assert h.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, (dq, dk, dv))) and all(torch.equal(a, b) for a, b in zip(got, out))
    check_gradients(got, _to_original(backward_reference(Q, K, V, O, lse, dO, masks), t, r), f"joined {case}")


@gpu
def test_non_finite_rows_stay_apart_in_a_tile_of_two_groups():
    _need_gpu()
    B, Hq, Hkv, N, d = 5, 10, 5, 300, 128
    P = B * Hkv
    Q, K, V, dO = _inputs(23, B, Hq, Hkv, N, d)
    off = torch.tensor([[0, 100, 170, 300]], dtype=torch.int32).repeat(P, 1)      # the last two share a tile
    keep = torch.eye(3, dtype=torch.bool).expand(P, 3, 3)
    rowptr, kg = csr(keep)
    ident = torch.arange(N, dtype=torch.int32).repeat(P, 1)
    t = {k: v.cuda() for k, v in dict(qperm=ident, kperm=ident, qoff=off, koff=off, rowptr=rowptr, kg=kg).items()}
    masks = [pair_mask(keep[0], off[0], off[0]).cuda()] * P
    O, lse = forward_reference(Q, K, V, masks)
    O, lse = O.bfloat16(), lse.float()
    part, route = _structs(t)
    with _handle(B, Hq, Hkv, N, d, 3, 3) as h:
        clean = h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO)
        for rows in (slice(0, 100), slice(100, 170), slice(170, 300)):
            for bad in (math.nan, math.inf):
                q, k, v, do, o, l = (x.clone() for x in (Q, K, V, dO, O, lse))
                for x in (q, k, v, do, o, l):
                    x[:, :, rows] = bad
                got = h.blocksparse_attn_bwd(q, k, v, part, route, o, l, do)
                for a, b in zip(got, clean):
                    a, b = a.clone(), b.clone()
                    a[:, :, rows] = b[:, :, rows] = 0
                    assert torch.equal(a, b)


@gpu
def test_out_of_range_ids_are_reported_with_tiles_of_two_groups():
    _need_gpu()
    B, Hq, Hkv, N, d, G = 4, 10, 10, 400, 64, 4
    Q, K, V, dO = _inputs(4, B, Hq, Hkv, N, d)
    t, masks = _routed(4, B * Hkv, N, G, G, 1.0)
    O, lse = forward_reference(Q, K, V, masks)
    args = (O.bfloat16(), lse.float(), dO)
    with _handle(B, Hq, Hkv, N, d, G, G) as h:
        want = h.blocksparse_attn_bwd(Q, K, V, *_structs(t), *args)
        torch.cuda.synchronize()
        assert h.device_status() == 0
        for name, at, value in (("kg", (3, 1), G), ("kg", (0, 2), -3), ("rowptr", (39, 2), 10 ** 6), ("rowptr", (1, 1), -5),
                                ("koff", (0, 2), N + 5), ("qoff", (7, 1), -7), ("kg", (0, 1), 0), ("kg", (0, 0), G - 1),
                                ("qoff", (0, 0), 3), ("koff", (9, G), N - 1), ("koff", (2, 2), 0), ("qoff", (2, 1), 2 ** 31 - 1)):
            bad = {k: v.clone() for k, v in t.items()}
            bad[name][at] = value
            h.blocksparse_attn_bwd(Q, K, V, *_structs(bad), *args)
            torch.cuda.synchronize()
            assert h.device_status() == 6, name
        got = h.blocksparse_attn_bwd(Q, K, V, *_structs(t), *args)
        torch.cuda.synchronize()
        assert h.device_status() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("amp", [1e-3, 4.0, 12.0])
def test_flat_and_peaked_rows(amp):
    """Probabilities from all alike to one key taking the row (logits of several hundred)."""
    _need_gpu()
    shape = (1, 2, 1, 321, 128)
    Q, K, V, dO = _inputs(5, *shape, amp=amp)
    O, lse = forward_reference(Q, K, V)
    O, lse = O.bfloat16(), lse.float()
    with _handle(*shape) as h:
        got = h.dense_attn_bwd(Q, K, V, O, lse, dO)
    check_gradients(got, backward_reference(Q, K, V, O, lse, dO), f"amp {amp}")


@gpu
def test_directional_differences():
    """<dQ, u> and the like against central differences of sum(dO . O) in fp64."""
    _need_gpu()
    B, Hq, Hkv, N, d, G = 1, 4, 2, 200, 64, 6
    Q, K, V, dO = _inputs(3, B, Hq, Hkv, N, d)
    t, masks = _routed(3, B * Hkv, N, G, G, 0.5)
    O, lse = forward_reference(Q, K, V, masks)
    part, route = _structs(t)
    with _handle(B, Hq, Hkv, N, d, G, G) as h:
        got = dict(zip(("dQ", "dK", "dV"), h.blocksparse_attn_bwd(Q, K, V, part, route, O.bfloat16(), lse.float(), dO)))
    bounds = _to_original(backward_reference(Q, K, V, O.bfloat16(), lse.float(), dO, masks), t, Hq // Hkv)
    g = torch.Generator().manual_seed(4)
    for name, i in (("dQ", 0), ("dK", 1), ("dV", 2)):
        x = [Q.double(), K.double(), V.double()]
        u = torch.randn(x[i].shape, generator=g).double().cuda()
        step = 1e-4
        value = []
        for s in (step, -step):
            y = list(x)
            y[i] = x[i] + s * u
            value.append((forward_reference(*y, masks)[0] * dO.double()).sum().item())
        slope = (value[0] - value[1]) / (2 * step)
        u_orig = _to_original([{name: u}], t, Hq // Hkv)[0][name]
        mine = (got[name].double() * u_orig).sum().item()
        # the kernels' own error, and that of D from the bf16 output: P 2^-8 |dO|.|O| a pair
        slack = (bounds[1][name] * u_orig.abs()).sum().item()
        dD = 2.0 ** -8 * (dO.double().abs() * O.abs()).sum(-1)
        amp = {"dQ": (K.double().abs().sum(-1).amax() * u.abs().amax()), "dK": Q.double().abs().amax() * u.abs().amax() * d,
               "dV": torch.zeros((), device="cuda")}[name]
        slack += (dD.sum() * amp / math.sqrt(d)).item()
        assert abs(mine - slope) <= slack + 1e-6 * abs(slope), (name, mine, slope, slack)


@gpu
@pytest.mark.parametrize("shape", [(4, 76, 38, 100, 64), (4, 40, 40, 100, 128), (2, 40, 40, 200, 128)], ids=str)
def test_one_pass_alone_gives_the_same(shape):
    """A little over one CTA of dK and dV an SM: some of dQ are launched before the last of those."""
    _need_gpu()
    B, Hq, Hkv, N, d = shape
    Q, K, V, dO = _inputs(N + Hq, *shape)
    with _handle(*shape) as h:
        lse = torch.empty((B, Hq, N), device="cuda")
        O = h.dense_attn(Q, K, V, lse=lse)
        got = h.dense_attn_bwd(Q, K, V, O, lse, dO)
        dq = h.dense_attn_bwd(Q, K, V, O, lse, dO, need_dkv=False)[0]
        _, dk, dv = h.dense_attn_bwd(Q, K, V, O, lse, dO, need_dq=False)
        torch.cuda.synchronize()
        assert h.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, (dq, dk, dv)))
    check_gradients(got, backward_reference(Q, K, V, O, lse, dO), f"dense {shape}")


@gpu
def test_skipped_gradients_and_own_buffers():
    _need_gpu()
    shape = (1, 4, 2, 200, 128)
    Q, K, V, dO = _inputs(9, *shape)
    with _handle(*shape) as h:
        lse = torch.empty((1, 4, 200), device="cuda")
        O = h.dense_attn(Q, K, V, lse=lse)
        dq, dk, dv = h.dense_attn_bwd(Q, K, V, O, lse, dO)
        only_q = h.dense_attn_bwd(Q, K, V, O, lse, dO, need_dkv=False)
        only_kv = h.dense_attn_bwd(Q, K, V, O, lse, dO, need_dq=False)
        assert only_q[1] is None and only_q[2] is None and only_kv[0] is None
        assert torch.equal(only_q[0], dq) and torch.equal(only_kv[1], dk) and torch.equal(only_kv[2], dv)
        # the caller's buffers and workspace, exactly as large as asked for, the guards around them untouched
        n = h.attn_bwd_workspace_bytes()
        ws = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        wide = torch.full((3, 1, 4, 200, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        got = h.dense_attn_bwd(Q, K, V, O, lse, dO, dQ=wide[1], workspace=ws[256:256 + n])
        assert got[0].data_ptr() == wide[1].data_ptr() and torch.equal(got[0], dq)
        assert (wide[0] == 7).all() and (wide[2] == 7).all()
        assert (ws[:256] == 0x5A).all() and (ws[256 + n:] == 0x5A).all()
        # a workspace that starts on 16 bytes only, on the default stream given by its pointer
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        got = h.dense_attn_bwd(Q, K, V, O, lse, dO, workspace=ws[16:16 + n], stream=0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (dq, dk, dv)))
        assert (ws[:16] == 0x5A).all() and (ws[16 + n:] == 0x5A).all()


@gpu
def test_non_finite_rows_stay_apart():
    """A NaN or infinite row of one group changes nothing in groups that the route keeps apart from it."""
    _need_gpu()
    B, Hq, Hkv, N, d = 1, 2, 1, 300, 128
    Q, K, V, dO = _inputs(21, B, Hq, Hkv, N, d)
    off = torch.tensor([[0, 100, 170, 300]], dtype=torch.int32)
    keep = torch.eye(3, dtype=torch.bool)[None]
    rowptr, kg = csr(keep)
    ident = torch.arange(N, dtype=torch.int32)[None]
    t = {k: v.cuda() for k, v in dict(qperm=ident, kperm=ident, qoff=off, koff=off, rowptr=rowptr, kg=kg).items()}
    masks = [pair_mask(keep[0], off[0], off[0]).cuda()]
    O, lse = forward_reference(Q, K, V, masks)
    O, lse = O.bfloat16(), lse.float()
    part, route = _structs(t)
    with _handle(B, Hq, Hkv, N, d, 3, 3) as h:
        clean = h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO)
        for bad in (math.nan, math.inf):
            q, k, v, do, o, l = (x.clone() for x in (Q, K, V, dO, O, lse))
            for x in (q, k, v, do, o):
                x[:, :, 100:170] = bad
            l[:, :, 100:170] = bad
            got = h.blocksparse_attn_bwd(q, k, v, part, route, o, l, do)
            for a, b in zip(got, clean):
                assert torch.equal(a[:, :, :100], b[:, :, :100]) and torch.equal(a[:, :, 170:], b[:, :, 170:])


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_nan_is_not_lost(d):
    """A NaN in a query reaches every key's gradients, one in a key every query's, wherever in the tile it stands."""
    _need_gpu()
    shape = (1, 1, 1, 200, d)
    Q, K, V, dO = _inputs(8, *shape)
    O, lse = forward_reference(Q, K, V)
    O, lse = O.bfloat16(), lse.float()
    with _handle(*shape) as h:
        for i in list(range(20)) + [63, 64, 100, 127, 128, 199]:
            bad = Q.clone()
            bad[0, 0, i, 3] = math.nan
            dq, dk, dv = h.dense_attn_bwd(bad, K, V, O, lse, dO)
            assert dq[0, 0, i].isnan().all() and dk.isnan().all() and dv.isnan().all(), i
            rest = torch.arange(200) != i
            assert torch.isfinite(dq[0, 0, rest.cuda()]).all(), i
            bad = K.clone()
            bad[0, 0, i, 3] = math.nan
            dq, dk, dv = h.dense_attn_bwd(Q, bad, V, O, lse, dO)
            assert dq.isnan().all() and dk[0, 0, i].isnan().all() and dv[0, 0, i].isnan().all(), i
            assert torch.isfinite(dk[0, 0, rest.cuda()]).all() and torch.isfinite(dv[0, 0, rest.cuda()]).all(), i


@gpu
def test_other_stream_two_calls_at_once_and_graph():
    _need_gpu()
    B, Hq, Hkv, N, d, G = 1, 4, 2, 700, 128, 8
    sets = []
    for seed in (1, 2):
        Q, K, V, dO = _inputs(seed, B, Hq, Hkv, N, d)
        t, masks = _routed(seed, B * Hkv, N, G, G, 0.5)
        O, lse = forward_reference(Q, K, V, masks)
        sets.append((Q, K, V, *_structs(t), O.bfloat16(), lse.float(), dO, t))
    with _handle(B, Hq, Hkv, N, d, G, G) as h:
        want = [h.blocksparse_attn_bwd(*s[:8]) for s in sets]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = [h.blocksparse_attn_bwd(*s[:8], stream=st if i else st.cuda_stream) for i, (s, st) in enumerate(zip(sets, streams))]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        # one graph with both calls, a workspace each; inputs change between replays
        ws = [torch.empty(h.attn_bwd_workspace_bytes(), dtype=torch.uint8, device="cuda") for _ in sets]
        outs = [[torch.zeros_like(x) for x in w] for w in want]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for s, w, o in zip(sets, ws, outs):
                h.blocksparse_attn_bwd(*s[:8], *o, workspace=w)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        sets[0][7].mul_(2.0)      # an exact factor: dS, and with it every gradient, doubles
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, 2 * y) for x, y in zip(outs[0], want[0]))
        assert all(torch.equal(x, y) for x, y in zip(outs[1], want[1]))
        del graph
        assert h.device_status() == 0


@gpu
def test_out_of_range_ids_are_reported():
    """Bad ids and permutation entries are skipped and reported; a clean call follows."""
    _need_gpu()
    B, Hq, Hkv, N, d, G = 1, 1, 1, 300, 64, 4
    Q, K, V, dO = _inputs(2, B, Hq, Hkv, N, d)
    t, masks = _routed(2, 1, N, G, G, 1.0)
    O, lse = forward_reference(Q, K, V, masks)
    args = (O.bfloat16(), lse.float(), dO)
    with _handle(B, Hq, Hkv, N, d, G, G) as h:
        want = h.blocksparse_attn_bwd(Q, K, V, *_structs(t), *args)
        torch.cuda.synchronize()
        assert h.device_status() == 0
        for name, at, value in (("kg", (0, 1), G), ("kg", (0, 2), -3), ("qperm", (0, 5), N), ("kperm", (0, 9), -1),
                                ("rowptr", (0, 2), 10 ** 6), ("koff", (0, 2), N + 5), ("qoff", (0, 1), -7),
                                ("kg", (0, 1), 0), ("kg", (0, 0), G - 1), ("qoff", (0, 0), 3), ("koff", (0, G), N - 1)):
            bad = {k: v.clone() for k, v in t.items()}
            bad[name][at] = value
            h.blocksparse_attn_bwd(Q, K, V, *_structs(bad), *args)
            torch.cuda.synchronize()
            assert h.device_status() == 6, name
        got = h.blocksparse_attn_bwd(Q, K, V, *_structs(t), *args)
        torch.cuda.synchronize()
        assert h.device_status() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_refusals_on_the_device():
    _need_gpu()
    shape = (1, 2, 2, 64, 64)
    Q, K, V, dO = _inputs(1, *shape)
    with _handle(*shape) as h:
        lse = torch.empty((1, 2, 64), device="cuda")
        O = h.dense_attn(Q, K, V, lse=lse)
        bad = [dict(Q=Q.float()), dict(K=K[:, :1]), dict(V=V.transpose(1, 2)), dict(lse=lse.half()), dict(dO=dO.cpu()),
               dict(O=O[..., :32])]
        good = dict(Q=Q, K=K, V=V, O=O, lse=lse, dO=dO)
        for b in bad:
            with pytest.raises(ValueError):
                h.dense_attn_bwd(**{**good, **b})
        with pytest.raises(ValueError):
            h.dense_attn_bwd(**good, need_dq=False, need_dkv=False)
        with pytest.raises(ValueError):
            h.dense_attn_bwd(**good, dQ=torch.empty_like(Q), need_dq=False)
        for kw, code in ((dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), 3), (dict(dQ=Q), 1), (dict(dK=V), 1),
                         (dict(dQ=torch.empty_like(Q), dK=dO), 1)):
            with pytest.raises(spr.SparsePRError) as e:
                h.dense_attn_bwd(**good, **kw)
            assert e.value.code == code
        buf = torch.empty_like(K)
        with pytest.raises(spr.SparsePRError):
            h.dense_attn_bwd(**good, dK=buf, dV=buf)
        torch.cuda.synchronize()
        assert h.device_status() == 0


def test_null_arguments_without_gpu():
    lib = spr.load_library()
    n = ctypes.c_size_t()
    assert lib.sparsepr_attn_bwd_workspace(None, ctypes.byref(n)) == 1
    assert lib.sparsepr_dense_attn_bwd(*[None] * 11, 0, None) == 1
    assert lib.sparsepr_blocksparse_attn_bwd(*[None] * 13, 0, None) == 1
    assert lib.sparsepr_dense_attn_lse(*[None] * 7) == 1


def test_reference_against_autograd():
    """The fp64 formulas that the kernels are held to, against autograd on the same function."""
    g = torch.Generator().manual_seed(0)
    B, Hq, Hkv, N, d = 1, 4, 2, 23, 8
    Q, K, V, dO = (torch.randn((B, h, N, d), generator=g, dtype=torch.float64, requires_grad=True) for h in (Hq, Hkv, Hkv, Hq))
    keep, _, _ = random_route(g, B * Hkv, 3, 3, 0.7)
    keep[:, :, 0] = True
    off = random_groups(g, N, 3)
    masks = [pair_mask(keep[z], off, off) for z in range(B * Hkv)]
    k, v = K.repeat_interleave(2, 1), V.repeat_interleave(2, 1)
    S = (Q @ k.transpose(-1, -2) / math.sqrt(d)).masked_fill(~torch.stack(masks).repeat_interleave(2, 0)[None], -math.inf)
    (torch.softmax(S, -1) @ v * dO).sum().backward()
    with torch.no_grad():
        O, lse = forward_reference(Q, K, V, masks)
        out, _, _ = backward_reference(Q, K, V, O, lse, dO, masks)
    for n, x in (("dQ", Q), ("dK", K), ("dV", V)):
        assert torch.allclose(out[n], x.grad, rtol=1e-10, atol=1e-12), n
