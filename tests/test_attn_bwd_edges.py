"""Backward passes where a call meets what it must leave alone: a timeout that has not been read, rows that bad
offsets leave out, non-finite values in operands that a gradient does not read, rows left out by lse = -inf; and
directional differences along the gradients themselves."""
import math

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
