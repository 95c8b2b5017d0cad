"""What the Python entry points refuse before anything reaches the library: handles without a GPU, on a library
that only counts its calls."""
import types

import pytest

torch = pytest.importorskip("torch")

import free_block_sparse_sparsepr_b200 as spr  # noqa: E402


class CountingLibrary:
    """Every entry point returns success and notes its name."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0

        return call


def _handle(B=1, Hq=4, Hkv=2, N=32, d=64):
    h = object.__new__(spr.SparsePR)
    h.lib, h.h, h.device = CountingLibrary(), 1, torch.device("cpu")
    h.cfg = spr.Config(B, Hq, Hkv, N, d)
    return h


def _qkv(B=1, Hq=4, Hkv=2, N=32, d=64):
    return [torch.zeros((B, n, N, d), dtype=torch.bfloat16) for n in (Hq, Hkv, Hkv)]


@pytest.mark.parametrize("lse", [torch.zeros((1, 4, 31)), torch.zeros((1, 2, 32)), torch.zeros((1, 4, 32), dtype=torch.bfloat16),
                                 torch.zeros((1, 4, 32), dtype=torch.float64), torch.zeros((4, 32)), torch.zeros((1, 4, 64))[..., ::2],
                                 torch.zeros((1, 32, 4)).transpose(1, 2), torch.zeros((1, 4, 32), device="meta")],
                         ids=lambda t: f"{tuple(t.shape)} {t.dtype} {t.stride()} {t.device}")
def test_dense_attn_refuses_an_lse_that_the_kernel_would_overrun(lse):
    h = _handle()
    with pytest.raises(ValueError, match="lse"):
        h.dense_attn(*_qkv(), stream=0, lse=lse)
    assert not h.lib.calls


def test_dense_attn_takes_the_lse_that_it_writes():
    h = _handle()
    h.dense_attn(*_qkv(), stream=0, lse=torch.zeros((1, 4, 32)))
    h.dense_attn(*_qkv(), stream=0)
    assert h.lib.calls == ["sparsepr_dense_attn_lse"] * 2


@pytest.mark.parametrize("error", [AssertionError("Torch not compiled with CUDA enabled"), RuntimeError("no CUDA driver")], ids=str)
def test_a_handle_for_host_buffers_needs_no_cuda_in_torch(monkeypatch, error):
    lib = CountingLibrary()

    def current_device():
        raise error

    monkeypatch.setattr(spr, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", current_device)
    with spr.SparsePR(1, 2, 2, 64, 64, Gk=4, Gq=4) as h:
        assert lib.calls[0] == "sparsepr_create" and h.device is None
        with pytest.raises(ValueError, match="Q"):       # no device to hold the gradients' operands against
            q, k, v = _qkv(1, 2, 2, 64, 64)
            h.dense_attn_bwd(q, k, v, q, torch.zeros((1, 2, 64)), q)
    assert "sparsepr_dense_attn_bwd" not in lib.calls


def test_a_stream_of_another_device_is_refused():
    """Work on it would reach this device's tensors from the other's context."""
    h = _handle()
    q, k, v = _qkv()
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=1)
    with pytest.raises(ValueError, match="stream"):
        h.dense_attn_bwd(q, k, v, q, torch.zeros((1, 4, 32)), q, stream=other)
    assert not h.lib.calls
