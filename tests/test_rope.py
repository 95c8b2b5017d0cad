"""Rotary positions against fp64: layouts, split and partial heads, scalings, far positions, strides,
one token, gradients, streams, graphs, and the refusals (which need no GPU)."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import free_block_sparse_sparsepr_b200 as spr  # noqa: E402

gpu = pytest.mark.gpu


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spr.load_library()


def _pairs(widths, layout):
    first, second, axis, at = [], [], [], 0
    for a, w in enumerate(widths):
        for i in range(w // 2):
            first.append(at + (2 * i if layout == "interleaved" else i))
            second.append(at + (2 * i + 1 if layout == "interleaved" else w // 2 + i))
            axis.append(a)
        at += w
    return first, second, axis


def _reference(x, pos, rope, layout, sign):
    """fp64 result and bound before the final rounding, for x [B, N, H, d].

    The angle in half turns is one fp32 value (2^-25) cut at 2^-31, from a frequency known to 2^-53
    of its value, as the reference's product is; sin and cos are within 2^-23; amplitude, two products and a sum
    round four times at 2^-24: together under 2^-21 of amplitude (|u| + |v|), plus the far term."""
    first, second, axis = _pairs(rope.widths, layout)
    if pos.dim() == 2:
        pos = pos.expand(x.shape[0], *pos.shape)
    f = torch.tensor(rope.freq, dtype=torch.float64, device=x.device)
    ang = pos.double()[..., axis] * f
    cos, sin = ang.cos()[:, :, None], sign * ang.sin()[:, :, None]
    y = x.double().clone()
    bound = torch.zeros_like(y)
    u, v = x.double()[..., first], x.double()[..., second]
    y[..., first] = rope.amplitude * (u * cos - v * sin)
    y[..., second] = rope.amplitude * (u * sin + v * cos)
    b = abs(rope.amplitude) * (u.abs() + v.abs()) * (2.0 ** -21 + 3 * 2.0 ** -53 * ang.abs())[:, :, None]
    bound[..., first] = b
    bound[..., second] = b
    return y, bound


def _check(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    e = (got.double() - want).abs()
    allowed = bound + half * (want.abs() + bound)
    assert torch.isfinite(got).all() and (e <= allowed).all(), f"{what}: {(e - allowed).max().item():.3g} over the bound"


CASES = [
    # d, widths, layout, B, N, H, dtype, scaling, start
    (64, (64,), "half", 1, 1, 1, torch.bfloat16, {}, 0),
    (128, (128,), "half", 8, 1, 32, torch.bfloat16, dict(scaling="yarn", factor=8.0, trained_length=4096), 250000),
    (128, (128,), "interleaved", 2, 37, 3, torch.float32, dict(scaling="linear", factor=4.0), 100),
    (128, (44, 42, 42), "interleaved", 1, 330, 24, torch.bfloat16, {}, 0),
    (128, (44, 42, 42), "half", 1, 77, 5, torch.bfloat16, dict(scaling="ntk", factor=2.0), 0),
    (128, (16, 56, 56), "half", 2, 130, 8, torch.float32, {}, 3),
    (64, (18, 22, 22), "half", 2, 101, 12, torch.bfloat16, {}, 0),
    (64, (2,), "interleaved", 3, 65, 2, torch.bfloat16, dict(scaling="ntk", factor=4.0), 10),
    (128, (2, 2, 2), "half", 1, 9, 7, torch.float32, dict(scaling="yarn", factor=2.0, trained_length=100), 0),
    (128, (30,), "half", 1, 1025, 4, torch.bfloat16, {}, 10 ** 6),
    (64, (32,), "half", 1, 200, 4, torch.float32, {}, 2 ** 31 - 300),
    (128, (64, 64), "interleaved", 4, 19, 6, torch.bfloat16, {}, -2 ** 31),
    (128, (126,), "half", 1, 4099, 2, torch.bfloat16, {}, 0),
]


def _case(case, seed=0):
    d, widths, layout, B, N, H, dtype, scaling, start = case
    g = torch.Generator().manual_seed(seed)
    rope = spr.Rope(d, widths, layout=layout, **scaling)
    pos = torch.randint(0, 60, (B, N, len(widths)), generator=g)
    pos[:, :, 0] = start + torch.arange(N)
    x = torch.randn((B, N, H, d), generator=g).to(dtype).cuda()
    return rope, pos.to(torch.int32).cuda(), x, layout


@gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradient(case):
    _need_gpu()
    rope, pos, x, layout = _case(case)
    y = rope.forward(x, pos)
    want, bound = _reference(x, pos, rope, layout, 1.0)
    _check(y, want.transpose(1, 2), bound.transpose(1, 2), "forward")
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    dx = rope.backward(dy, pos, dtype=x.dtype)
    want, bound = _reference(dy.transpose(1, 2), pos, rope, layout, -1.0)
    assert dx.dtype == x.dtype and dx.shape == x.shape
    _check(dx, want, bound, "gradient")
    # the map is linear: its gradient against its own difference along x, <dy, R x> = <dx, x>, each
    # product within the roundings of y and dx (half a step of bf16, or of fp32) and the bounds above
    a, b = (dy.double() * y.double()).sum().item(), (dx.double() * x.double()).sum().item()
    slack = 2.0 ** -7 * ((dy.double() * y.double()).abs().sum() + (dx.double() * x.double()).abs().sum()).item()
    assert abs(a - b) <= slack


@gpu
def test_shared_positions_and_strides():
    """Positions shared by the batch; Q, K and V slices of a fused projection read and written in place."""
    _need_gpu()
    B, N, Hq, Hkv, d = 2, 50, 6, 2, 128
    g = torch.Generator().manual_seed(3)
    fused = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).bfloat16().cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[:, None] * 3
    rope = spr.Rope(d, (96,), layout="half")
    q, k = fused[:, :, :Hq], fused[:, :, Hq:Hq + Hkv]
    for x in (q, k, fused.transpose(0, 1)[:, :1].transpose(0, 1), k.expand(B, N, Hkv, d)):
        y = rope.forward(x, pos)
        want, bound = _reference(x, pos, rope, "half", 1.0)
        _check(y, want.transpose(1, 2), bound.transpose(1, 2), "strided forward")
    each = rope.forward(q, pos.expand(B, N, 1).contiguous())
    assert torch.equal(each, rope.forward(q, pos))
    # a broadcast input: every head reads the same row
    one = fused[:, :, :1].expand(B, N, 5, d)
    assert torch.equal(rope.forward(one, pos), rope.forward(one.contiguous(), pos))
    # gradients of the two slices written into one fused gradient, the rest untouched
    dfused = torch.full_like(fused, 5.0)
    dq, dk = (torch.randn((B, h, N, d), generator=g).bfloat16().cuda() for h in (Hq, Hkv))
    rope.backward(dq, pos, out=dfused[:, :, :Hq])
    rope.backward(dk, pos, out=dfused[:, :, Hq:Hq + Hkv])
    assert torch.equal(dfused[:, :, :Hq], rope.backward(dq, pos)) and torch.equal(dfused[:, :, Hq:Hq + Hkv], rope.backward(dk, pos))
    assert (dfused[:, :, Hq + Hkv:] == 5).all()


@gpu
def test_non_finite_elements_stay_in_their_pair():
    _need_gpu()
    rope = spr.Rope(64, (32,), layout="half")
    x = torch.randn((1, 4, 2, 64), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[:, None]
    clean = rope.forward(x, pos)
    x[0, 1, 0, 3], x[0, 2, 1, 40] = math.nan, math.inf
    y = rope.forward(x, pos)
    touched = torch.zeros_like(clean, dtype=torch.bool)
    touched[0, 0, 1, [3, 19]] = True
    touched[0, 1, 2, 40] = True
    assert torch.equal(y[~touched], clean[~touched]) and not torch.isfinite(y[touched]).any()


@gpu
def test_streams_and_graph():
    _need_gpu()
    rope, pos, x, _ = _case(CASES[3])
    want = rope.forward(x, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a, b = rope.forward(x, pos, stream=s), rope.forward(x, pos, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    out, dx = torch.zeros_like(want), torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.forward(x, pos, out=out)
        rope.backward(out, pos, out=dx)
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2 * want) and torch.equal(dx, rope.backward(out, pos))
    del graph


@gpu
def test_refusals_on_the_device():
    _need_gpu()
    rope = spr.Rope(64, (64,))
    x = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    for bx, bp in ((x.half(), pos), (x[..., :32], pos), (x.transpose(2, 3), pos), (x.cpu(), pos.cpu()), (x, pos.long()),
                   (x, pos[:3]), (x, pos.cpu()), (x[0], pos), (x[:, :0], pos[:0])):
        with pytest.raises(ValueError):
            rope.forward(bx, bp)
    wide = torch.zeros((1, 4, 2, 68), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(spr.SparsePRError):          # rows that start on 8 bytes
        rope.forward(wide[..., 4:], pos)
    with pytest.raises(spr.SparsePRError):          # rows 136 bytes apart
        rope.forward(wide[..., :64], pos)
    dy = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(spr.SparsePRError):          # gradient rows on top of one another
        rope.backward(dy, pos, out=x[:, :, :1].expand(1, 4, 2, 64))
    with pytest.raises(spr.SparsePRError):          # in place
        rope.forward(x, pos, out=x.view(1, 2, 4, 64))
    with pytest.raises(ValueError):
        rope.backward(dy, pos, out=x, dtype=torch.float32)
    with pytest.raises(ValueError):
        rope.backward(dy.transpose(1, 2), pos)


def test_plan_refusals():
    for kw in (dict(d=96, widths=(32,)), dict(d=64, widths=(33,)), dict(d=64, widths=(0,)), dict(d=64, widths=(40, 40)),
               dict(d=64, widths=()), dict(d=64, widths=(2, 2, 2, 2)), dict(d=64, widths=(64,), layout="other"),
               dict(d=64, widths=(64,), scaling="other"), dict(d=64, widths=(64,), scaling="yarn", factor=2.0),
               dict(d=64, widths=(64,), factor=0.0), dict(d=64, widths=(64,), base=1.0)):
        with pytest.raises(ValueError):
            spr.Rope(**kw)


def _config(**kw):
    c = spr.RopeConfig()
    c.B, c.H, c.N, c.d, c.layout, c.axes, c.dtype = 1, 2, 4, 64, 0, 1, 0
    c.width[0] = 64
    c.stride_b, c.stride_n, c.stride_h, c.pos_stride_b, c.amplitude = 512, 128, 64, 0, 1.0
    for k, v in kw.items():
        if k == "width":
            c.width[:] = v
        elif k == "freq":
            c.freq[0] = v
        else:
            setattr(c, k, v)
    return c


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(N=0), 1), (dict(d=96), 2), (dict(layout=2), 1), (dict(axes=0), 1), (dict(axes=4), 1),
    (dict(dtype=2), 1), (dict(width=(63, 0, 0)), 1), (dict(width=(64, 2, 0), axes=2), 1), (dict(width=(0, 0, 0)), 1),
    (dict(stride_n=100), 1), (dict(stride_h=-64), 1), (dict(pos_stride_b=-1), 1), (dict(amplitude=float("inf")), 1),
    (dict(freq=float("nan")), 1), (dict(B=1 << 20, H=1 << 10, N=1 << 10), 2), (dict(stride_n=1 << 41), 2),
    (dict(stride_n=1 << 39), 2),
])
def test_c_refusals_without_gpu(kw, code):
    lib = spr.load_library()
    c = _config(**kw)
    for fn in (lib.sparsepr_rope, lib.sparsepr_rope_bwd):
        assert fn(ctypes.byref(c), 1 << 20, 1 << 30, 1 << 40, None) == code


def test_c_pointer_refusals_without_gpu():
    lib = spr.load_library()
    c = _config()
    src, pos, dst = 1 << 20, 1 << 30, 1 << 40
    for fn in (lib.sparsepr_rope, lib.sparsepr_rope_bwd):
        for a in ((None, pos, dst), (src, None, dst), (src, pos, None), (src + 8, pos, dst), (src, pos + 2, dst), (src, pos, dst + 4),
                  (src, pos, src + 512)):
            assert fn(ctypes.byref(c), *a, None) == 1
        assert fn(None, src, pos, dst, None) == 1
    # overlapping gradient rows are refused, overlapping input rows only read
    assert lib.sparsepr_rope_bwd(ctypes.byref(_config(stride_h=0)), src, pos, dst, None) == 1
    assert lib.sparsepr_rope_bwd(ctypes.byref(_config(stride_n=64)), src, pos, dst, None) == 1


def test_frequencies():
    """The four scalings from their definitions."""
    w, base = 64, 10000.0
    plain = [base ** (-2 * i / w) for i in range(w // 2)]
    f = lambda **kw: spr.Rope(128, (w,), base=base, **kw)  # noqa: E731
    assert f().freq == pytest.approx(plain, rel=1e-15) and f().amplitude == 1.0
    assert f(scaling="linear", factor=4.0).freq == pytest.approx([x / 4 for x in plain], rel=1e-15)
    ntk = f(scaling="ntk", factor=8.0).freq
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / 8.0, rel=1e-12)      # the slowest pair by the factor
    y = f(scaling="yarn", factor=8.0, trained_length=4096)
    assert y.amplitude == pytest.approx(0.1 * math.log(8.0) + 1.0)
    ratio = [b / a for a, b in zip(plain, y.freq)]
    turns = [4096 * x / (2 * math.pi) for x in plain]
    assert all(r == pytest.approx(1.0) for r, t in zip(ratio, turns) if t > 45)         # an index past the border at most
    assert all(r == pytest.approx(1 / 8) for r, t in zip(ratio, turns) if t < 0.7)
    assert all(a >= b - 1e-15 for a, b in zip(ratio, ratio[1:]))
    assert spr.Rope(128, (w,), scaling="yarn", factor=8.0, trained_length=4096, amplitude=1.0).amplitude == 1.0
    assert spr.Rope(128, (16, 56, 56)).freq[8:36] == spr.Rope(128, (16, 56, 56)).freq[36:]
