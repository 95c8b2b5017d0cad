"""Backward passes where a call meets what it must leave alone: a timeout that has not been read, rows that bad
offsets leave out, non-finite values in operands that a gradient does not read, rows left out by lse = -inf; and
directional differences along the gradients themselves."""
import ctypes
import math
import time

import pytest

torch = pytest.importorskip("torch")

import free_block_sparse_sparsepr_b200 as spr  # noqa: E402
from bwd_helpers import backward_reference, check_gradients, csr, forward_reference  # noqa: E402
from test_attn_bwd import _handle, _inputs, _need_gpu, _routed, _structs, _to_original  # noqa: E402

gpu = pytest.mark.gpu


def _filled(Q, K, V, value=7.0):
    return [torch.full_like(x, value) for x in (Q, K, V)]


def _workspace(h):
    """A workspace that has been in use: every fp32 word of it is a finite number other than zero."""
    return torch.full((h.attn_bwd_workspace_bytes(),), 0x3B, dtype=torch.uint8, device="cuda")


@gpu
@pytest.mark.parametrize("shape,shared", [((1, 1, 1, 640, 128), True), ((1, 3, 1, 300, 64), True),
                                          ((4, 40, 40, 100, 128), False), ((4, 76, 38, 100, 64), False)], ids=str)
def test_dense_gradients_stay_unwritten_while_a_timeout_stands(shape, shared):
    """`shared`: CTAs share a tile's stream, so that a kernel of its own joins their sums."""
    _need_gpu()
    Q, K, V, dO = _inputs(11, *shape)
    O, lse = forward_reference(Q, K, V)
    O, lse = O.bfloat16(), lse.float()
    B, Hq, Hkv, N, d = shape
    with spr.SparsePR(B, Hq, Hkv, N, d, Gk=1, Gq=1, flags=spr.FLAG_HARD_DROP_ONLY | spr.FLAG_TEST_STALL) as h:
        h.dense_attn(Q, K, V)              # its first wait runs out (about two seconds)
        out, ws = _filled(Q, K, V), _workspace(h)
        for _ in range(3):
            h.dense_attn_bwd(Q, K, V, O, lse, dO, *out, workspace=ws)
        torch.cuda.synchronize()
        assert h.last_launch_count() == (3 if shared else 2)
        assert h.device_status() == 5
        assert all((x == 7).all() for x in out)
        got = h.dense_attn_bwd(Q, K, V, O, lse, dO, *out, workspace=ws)
        torch.cuda.synchronize()
        assert h.device_status() == 0
    check_gradients(got, backward_reference(Q, K, V, O, lse, dO), f"after a timeout {shape}")


@gpu
@pytest.mark.parametrize("density", [0.0, 0.5])
@pytest.mark.parametrize("shape,G,launches", [((1, 1, 1, 2600, 64), 20, 3), ((1, 8, 1, 700, 128), 12, 3),
                                              ((2, 40, 40, 260, 128), 20, 2), ((4, 40, 20, 400, 64), 4, 3)], ids=str)
def test_blocksparse_gradients_stay_unwritten_while_a_timeout_stands(shape, G, launches, density):
    """Joined sums, a tile a group and tiles of two groups; with nothing kept a CTA has nothing to wait for."""
    _need_gpu()
    B, Hq, Hkv, N, d = shape
    Q, K, V, dO = _inputs(12, *shape)
    t, masks = _routed(12, B * Hkv, N, G, G, density)
    O, lse = forward_reference(Q, K, V, masks)
    O, lse = O.bfloat16(), lse.float()
    part, route = _structs(t)
    with spr.SparsePR(B, Hq, Hkv, N, d, Gk=G, Gq=G, flags=spr.FLAG_HARD_DROP_ONLY | spr.FLAG_TEST_STALL) as h:
        h.dense_attn(Q, K, V)
        out, ws = _filled(Q, K, V), _workspace(h)
        for _ in range(3):
            h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO, *out, workspace=ws)
        torch.cuda.synchronize()
        assert h.last_launch_count() == launches
        assert h.device_status() == 5
        assert all((x == 7).all() for x in out)
        got = h.blocksparse_attn_bwd(Q, K, V, part, route, O, lse, dO, *out, workspace=ws)
        torch.cuda.synchronize()
        assert h.device_status() == 0
    check_gradients(got, _to_original(backward_reference(Q, K, V, O, lse, dO, masks), t, Hq // Hkv), f"after a timeout {shape}")


@gpu
@pytest.mark.parametrize("shape,G", [((1, 1, 1, 2600, 64), 20), ((1, 8, 1, 700, 128), 12), ((2, 40, 40, 260, 128), 20),
                                     ((4, 40, 20, 400, 64), 4)], ids=str)
def test_rows_that_no_group_holds_stay_unwritten(shape, G):
    """Bad offsets are reported, and the rows that they leave out keep what they held."""
    _need_gpu()
    B, Hq, Hkv, N, d = shape
    P, r = B * Hkv, Hq // Hkv
    Q, K, V, dO = _inputs(13, *shape)
    t, masks = _routed(13, P, N, G, G, 1.0)
    even = torch.arange(G + 1, dtype=torch.int32, device="cuda") * N // G
    t["qoff"], t["koff"] = even.to(torch.int32).repeat(P, 1), even.to(torch.int32).repeat(P, 1)
    cuts = even.tolist()
    t["qperm"] = t["kperm"] = torch.arange(N, dtype=torch.int32, device="cuda").repeat(P, 1)
    O, lse = forward_reference(Q, K, V)
    args = (O.bfloat16(), lse.float(), dO)
    z = P - 1
    with _handle(B, Hq, Hkv, N, d, G, G) as h:
        ws = _workspace(h)
        good = h.blocksparse_attn_bwd(Q, K, V, *_structs(t), *args, workspace=ws)
        torch.cuda.synchronize()
        assert h.device_status() == 0 and all(torch.isfinite(x).all() for x in good)
        for side in ("qoff", "koff"):
            # the first rows; the last; a group whose end lies past N, and with it the next; one that starts before 0
            for at, value, lost in ((0, 3, (0, 3)), (G, N - 2, (N - 2, N)), (1, N + 5, (0, cuts[2])), (1, -1, (0, cuts[2]))):
                bad = {k: v.clone() for k, v in t.items()}
                bad[side][z, at] = value
                out = _filled(Q, K, V)
                h.blocksparse_attn_bwd(Q, K, V, *_structs(bad), *args, *out, workspace=ws)
                torch.cuda.synchronize()
                assert h.device_status() == 6, (side, at)
                touched = out[:1] if side == "qoff" else out[1:]
                for x in touched:
                    own = x.reshape(P, -1, N, d)[z]
                    held = torch.ones(N, dtype=torch.bool, device="cuda")
                    held[lost[0]:lost[1]] = False
                    assert (own[:, ~held] == 7).all(), (side, at)
                    assert (own[:, held] != 7).any(-1).all(), (side, at)
                    assert (x.reshape(P, -1, N, d)[:z] != 7).any(-1).all(), (side, at)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_dv_does_not_read_the_output(d, bad):
    """dV = P^T dO: a row of O that is not finite reaches dQ of its row and dK, never dV."""
    _need_gpu()
    for shape in ((1, 2, 1, 200, d), (2, 20, 20, 400, d)):
        Q, K, V, dO = _inputs(14, *shape)
        O, lse = forward_reference(Q, K, V)
        O, lse = O.bfloat16(), lse.float()
        with _handle(*shape) as h:
            clean = h.dense_attn_bwd(Q, K, V, O, lse, dO)
            for i in (0, 63, 127, 128, shape[3] - 1):
                o = O.clone()
                o[0, 0, i, 3] = bad
                dq, dk, dv = h.dense_attn_bwd(Q, K, V, o, lse, dO)
                assert torch.equal(dv, clean[2]), i
                assert not torch.isfinite(dq[0, 0, i]).any() and not torch.isfinite(dk[0, 0]).any(), i
                rest = torch.ones(shape[:2] + shape[3:4], dtype=torch.bool, device="cuda")
                rest[0, 0, i] = False
                assert torch.equal(dq[rest], clean[0][rest]), i
                v = V.clone()
                v[0, 0, i] = bad
                assert torch.equal(h.dense_attn_bwd(Q, K, v, O, lse, dO)[2], clean[2]), i


@gpu
@pytest.mark.parametrize("shape", [(1, 2, 1, 200, 64), (1, 2, 1, 200, 128), (4, 40, 40, 100, 128)], ids=str)
def test_rows_left_out_by_their_lse_add_nothing(shape):
    """lse = -inf: P = 0 in every column, so that not even a dO of 1e34 shows."""
    _need_gpu()
    Q, K, V, dO = _inputs(15, *shape)
    O, lse = forward_reference(Q, K, V)
    O, lse = O.bfloat16(), lse.float()
    rows = [0, 5, 64, shape[3] - 1]
    lse[:, :, rows] = -math.inf
    O[:, :, rows] = 0
    big = dO.clone()
    dO[:, :, rows] = 0
    big[:, :, rows] = 1e34
    with _handle(*shape) as h:
        want = h.dense_attn_bwd(Q, K, V, O, lse, dO)
        got = h.dense_attn_bwd(Q, K, V, O, lse, big)
    assert (got[0][:, :, rows] == 0).all()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    kept = torch.ones((shape[3], 1), dtype=torch.bool, device="cuda")
    kept[rows] = False
    masks = [kept] * (shape[0] * shape[2])
    check_gradients(got, backward_reference(Q, K, V, O, lse, dO, masks), f"rows left out {shape}")


def _slopes(Q, K, V, dO, masks, out, step):
    """Central differences of sum(dO . O) in fp64 along each exact gradient's own direction: its norm, and the
    direction."""
    x = [Q.double(), K.double(), V.double()]
    result = {}
    for i, name in enumerate(("dQ", "dK", "dV")):
        u = out[name] / out[name].norm()
        value = []
        for s in (step, -step):
            y = list(x)
            y[i] = x[i] + s * u
            value.append((forward_reference(*y, masks)[0] * dO.double()).sum().item())
        result[name] = ((value[0] - value[1]) / (2 * step), u)
    return result


def _drift(Q, K, O, exact_O, lse, dO, masks):
    """2-norms of what dQ and dK change by when D = dO.O is taken from a rounded O: P dD k and P dD q, dD = dO.(O - exact)."""
    B, Hq, N, d = Q.shape
    r = Hq // K.shape[1]
    dq, dk = torch.zeros_like(Q, dtype=torch.float64), torch.zeros_like(K, dtype=torch.float64)
    for b in range(B):
        for h in range(Hq):
            z = h // r
            S = Q[b, h].double() @ K[b, z].double().T / math.sqrt(d) - lse[b, h, :, None]
            if masks is not None:
                S = S.masked_fill(~masks[b * K.shape[1] + z], -math.inf)
            P = S.exp().nan_to_num(0.0) * (dO[b, h].double() * (O[b, h].double() - exact_O[b, h])).sum(1, keepdim=True)
            dq[b, h] = P @ K[b, z].double() / math.sqrt(d)
            dk[b, z] += P.T @ Q[b, h].double() / math.sqrt(d)
    return {"dQ": dq.norm().item(), "dK": dk.norm().item(), "dV": 0.0}


def _check_slopes(got, Q, K, V, dO, masks, to_original):
    """Along u = grad / |grad| the slope is the gradient's norm, so a gradient that is zero, turned around or scaled
    shows. <got - grad, u> is at most the 2-norm of the error: the kernels' own (backward_reference) and the
    drift of D. The differences add their own: the third derivative, step^2 / 6 of it (1e-8 of the slope at a
    step of 1e-4 along a unit vector), and 2^-53 of the value over the step."""
    exact_O, lse = forward_reference(Q, K, V, masks)
    O = exact_O.bfloat16()
    exact = backward_reference(Q, K, V, exact_O, lse, dO, masks)[0]
    square = backward_reference(Q, K, V, O, lse.float(), dO, masks)[2]
    drift = _drift(Q, K, O, exact_O, lse, dO, masks)
    for name, (slope, u) in _slopes(Q, K, V, dO, masks, exact, 1e-4).items():
        assert abs(slope - exact[name].norm().item()) <= 1e-6 * slope, name       # the formulas against the function
        slack = square[name].sum().sqrt().item() + drift[name]
        assert slack <= 0.1 * slope, (name, slack, slope)
        mine = (got[name].double() * to_original(name, u)).sum().item()
        assert abs(mine - slope) <= slack + 1e-6 * slope, (name, mine, slope, slack)


@gpu
@pytest.mark.parametrize("shape", [(1, 4, 2, 200, 64), (1, 2, 1, 300, 128)], ids=str)
def test_differences_along_the_gradients(shape):
    _need_gpu()
    B, Hq, Hkv, N, d = shape
    G = 6
    Q, K, V, dO = _inputs(3, *shape)
    with _handle(*shape) as h:
        O, lse = forward_reference(Q, K, V)
        got = dict(zip(("dQ", "dK", "dV"), h.dense_attn_bwd(Q, K, V, O.bfloat16(), lse.float(), dO)))
    _check_slopes(got, Q, K, V, dO, None, lambda n, u: u)
    t, masks = _routed(3, B * Hkv, N, G, G, 0.5)
    part, route = _structs(t)
    with _handle(B, Hq, Hkv, N, d, G, G) as h:
        O, lse = forward_reference(Q, K, V, masks)
        got = dict(zip(("dQ", "dK", "dV"), h.blocksparse_attn_bwd(Q, K, V, part, route, O.bfloat16(), lse.float(), dO)))
    _check_slopes(got, Q, K, V, dO, masks, lambda n, u: _to_original([{n: u}], t, Hq // Hkv)[0][n])


def test_the_differences_catch_wrong_gradients():
    """The check above on the CPU, with the fp64 gradients and with spoiled ones."""
    g = torch.Generator().manual_seed(3)
    B, Hq, Hkv, N, d = 1, 2, 1, 40, 16
    rnd = lambda h: torch.randn((B, h, N, d), generator=g)  # noqa: E731
    Q, K, V, dO = (x.bfloat16() for x in (rnd(Hq), rnd(Hkv), rnd(Hkv), 0.01 * rnd(Hq)))
    O, lse = forward_reference(Q, K, V)
    exact = backward_reference(Q, K, V, O, lse, dO)[0]
    same = lambda n, u: u  # noqa: E731
    _check_slopes(exact, Q, K, V, dO, None, same)
    for name in exact:
        for spoiled in (torch.zeros_like(exact[name]), -exact[name], 1.2 * exact[name]):
            with pytest.raises(AssertionError):
                _check_slopes({**exact, name: spoiled}, Q, K, V, dO, None, same)


@gpu
def test_a_dense_call_needs_no_room_for_lists():
    _need_gpu()
    B, Hq, Hkv, N, d, G = 1, 4, 2, 1500, 64, 500
    Q, K, V, dO = _inputs(16, B, Hq, Hkv, N, d)
    with _handle(B, Hq, Hkv, N, d, G, G) as h, _handle(B, Hq, Hkv, N, d) as plain:
        lse = torch.empty((B, Hq, N), device="cuda")
        O = h.dense_attn(Q, K, V, lse=lse)
        n, both = h.attn_bwd_workspace_bytes(dense_only=True), h.attn_bwd_workspace_bytes()
        assert n == plain.attn_bwd_workspace_bytes(dense_only=True) and both > max(n, 2 * Hkv * G * G * 8)
        ws = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        got = h.dense_attn_bwd(Q, K, V, O, lse, dO, workspace=ws[256:256 + n])
        assert (ws[:256] == 0x5A).all() and (ws[256 + n:] == 0x5A).all()
        # without one, no more is taken for the call
        del ws
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        held = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        again = h.dense_attn_bwd(Q, K, V, O, lse, dO)
        own = sum(x.numel() * 2 for x in again)
        assert torch.cuda.max_memory_allocated() - held <= own + n + 4 * 512
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        t, _ = _routed(16, B * Hkv, N, G, G, 0.3)
        with pytest.raises(spr.SparsePRError) as e:
            h.blocksparse_attn_bwd(Q, K, V, *_structs(t), O, lse, dO, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert e.value.code == 3


def test_null_workspace_queries_without_gpu():
    n = ctypes.c_size_t()
    assert spr.load_library().sparsepr_dense_attn_bwd_workspace(None, ctypes.byref(n)) == 1


@gpu
@pytest.mark.parametrize("shape", [(1, 1, 1, 640, 128), (4, 40, 40, 100, 128), (4, 40, 40, 100, 64), (1, 3, 1, 300, 64)], ids=str)
@pytest.mark.parametrize("side", ["both", "dQ", "dK and dV"])
def test_a_wait_of_the_backward_kernel_runs_out(shape, side):
    """The tile that a CTA owns is never loaded: the wait for it gives up after about two seconds, the streamed tiles on
    their way land, every CTA returns, nothing is written, the status says so, and another handle's call runs clean."""
    _need_gpu()
    B, Hq, Hkv, N, d = shape
    Q, K, V, dO = _inputs(17, *shape)
    O, lse = forward_reference(Q, K, V)
    args = (Q, K, V, O.bfloat16(), lse.float(), dO)
    out = _filled(Q, K, V)
    kw = {"both": dict(dQ=out[0], dK=out[1], dV=out[2]), "dQ": dict(dQ=out[0], need_dkv=False),
          "dK and dV": dict(dK=out[1], dV=out[2], need_dq=False)}[side]
    with spr.SparsePR(B, Hq, Hkv, N, d, Gk=1, Gq=1, flags=spr.FLAG_HARD_DROP_ONLY | spr.FLAG_TEST_STALL_BWD) as h:
        t0 = time.perf_counter()
        h.dense_attn_bwd(*args, **kw, workspace=_workspace(h))
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 60.0
        assert h.device_status() == 5 and h.device_status() == 0
    assert all((x == 7).all() for x in out)
    with _handle(*shape) as h:
        got = h.dense_attn_bwd(*args)
        torch.cuda.synchronize()
        assert h.device_status() == 0
    check_gradients(got, backward_reference(*args), f"after a stalled call {shape}")


@gpu
@pytest.mark.parametrize("shape,G", [((1, 8, 1, 700, 128), 12), ((4, 40, 20, 400, 64), 4)], ids=str)
def test_a_wait_of_the_routed_backward_kernel_runs_out(shape, G):
    """Shared streams, and tiles of two groups; every group keeps some cell."""
    _need_gpu()
    B, Hq, Hkv, N, d = shape
    Q, K, V, dO = _inputs(18, *shape)
    t, masks = _routed(18, B * Hkv, N, G, G, 1.0)
    O, lse = forward_reference(Q, K, V, masks)
    out = _filled(Q, K, V)
    with spr.SparsePR(B, Hq, Hkv, N, d, Gk=G, Gq=G, flags=spr.FLAG_HARD_DROP_ONLY | spr.FLAG_TEST_STALL_BWD) as h:
        h.blocksparse_attn_bwd(Q, K, V, *_structs(t), O.bfloat16(), lse.float(), dO, *out, workspace=_workspace(h))
        torch.cuda.synchronize()
        assert h.device_status() == 5
    assert all((x == 7).all() for x in out)
