"""Rotary positions: the gradient against the forward map along the turned vector itself."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import free_block_sparse_sparsepr_b200 as spr  # noqa: E402
from test_rope import CASES, _case, _config, _need_gpu, _reference  # noqa: E402

gpu = pytest.mark.gpu


def _check_adjoint(x, y, dx, bound):
    """<y, R x> = <R^T y, x> for the rounded y that was handed to the gradient: along y itself the left side is
    |y|^2 up to y's own rounding, so a gradient that is zero, turned around or scaled shows. Allowed, in the
    2-norm: half a step of y against y, half a step of dx and its bound before that against x."""
    a, b = (y.double() ** 2).sum().item(), (dx.double() * x.double()).sum().item()
    eps = lambda t: torch.finfo(t.dtype).eps / 2  # noqa: E731
    # y = R x (1 + e): |R x - y| is at most half a step of y, and what the bound allows before it
    slack = ((eps(y) * y.double().norm() + bound.norm()) * y.double().norm()
             + (eps(dx) * dx.double().norm() + bound.norm()) * x.double().norm()).item()
    assert slack <= 0.1 * a, (slack, a)
    assert abs(a - b) <= slack, (a, b, slack)


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradient_along_the_turned_vector(case):
    _need_gpu()
    rope, pos, x, layout = _case(case)
    y = rope.forward(x, pos)
    bound = _reference(x, pos, rope, layout, 1.0)[1] * max(1.0, abs(rope.amplitude))
    _check_adjoint(x, y, rope.backward(y, pos, dtype=x.dtype), bound)


def test_the_adjoint_check_catches_wrong_gradients():
    """The check above on the CPU, with the fp64 map and with spoiled gradients."""
    rope = spr.Rope(64, (18, 22, 22), layout="half")
    g = torch.Generator().manual_seed(0)
    x = torch.randn((1, 50, 3, 64), generator=g).bfloat16()
    pos = torch.randint(0, 60, (1, 50, 3), generator=g)
    want, bound = _reference(x, pos, rope, "half", 1.0)
    y = want.bfloat16()
    dx = _reference(y, pos, rope, "half", -1.0)[0].bfloat16()
    _check_adjoint(x, y, dx, bound)
    turned = _reference(y, pos, rope, "half", 1.0)[0].bfloat16()       # the map itself in place of its transpose
    for spoiled in (torch.zeros_like(dx), -dx, 1.1 * dx, turned):
        with pytest.raises(AssertionError):
            _check_adjoint(x, y, spoiled, bound)


@pytest.mark.parametrize("factor,amplitude", [(0.25, 1.0), (0.999, 1.0), (1.0, 1.0), (8.0, 1.2079441541679836)])
def test_a_context_that_is_not_extended_keeps_its_amplitude(factor, amplitude):
    """yarn: 0.1 ln(factor) + 1 where the context is extended, 1 where the factor is at most 1."""
    rope = spr.Rope(64, (64,), scaling="yarn", factor=factor, trained_length=4096)
    assert rope.amplitude == pytest.approx(amplitude, rel=1e-15)
    assert spr.Rope(64, (64,), scaling="yarn", factor=factor, trained_length=4096, amplitude=1.5).amplitude == 1.5


def test_positions_inside_the_output_and_huge_amplitudes_are_refused():
    """The kernel would read positions that it has overwritten, or turn pairs by an infinite fp32 amplitude."""
    lib = spr.load_library()
    src, dst = 1 << 20, 1 << 40
    out = 2 * 4 * 64 * 2                       # bytes of [1, 2, 4, 64] bf16 on either side
    for fn in (lib.sparsepr_rope, lib.sparsepr_rope_bwd):
        for pos in (dst, dst + out - 4, dst - 12):
            assert fn(ctypes.byref(_config()), src, pos, dst, None) == 1
        # positions of a second sample, as far away as pos_stride_b says
        c = _config(B=2, stride_b=512, pos_stride_b=100)
        assert fn(ctypes.byref(c), src, dst - 400, dst, None) == 1
        assert fn(ctypes.byref(_config(amplitude=1e39)), src, 1 << 30, dst, None) == 1
