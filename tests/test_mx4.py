"""The 4-bit weight (MX4) without a GPU: refusals of the C entry points, which launch nothing."""
import ctypes

import pytest
import torch

import orthogonal_equivalence_cnp_b200 as P

A = 1 << 20  # aligned, never dereferenced: validation fails first


def _desc(**kw):
    base = dict(d_in=512, d_out=256, b=64, k=3, dtype=P.POETX_BF16, mode=P.POETX_MEM)
    base.update(kw)
    return P.poetx_desc(*(base[f] for f, _ in P.poetx_desc._fields_))


@pytest.mark.parametrize("args,code", [
    ((2, 4, 64, A, A, A), 1), ((0, -1, 64, A, A, A), 1), ((0, 4, -32, A, A, A), 1), ((0, 4, 48, A, A, A), 2),
    ((0, 4, 64, None, A, A), 1), ((1, 4, 64, A, None, A), 1), ((1, 4, 64, A, A, None), 1), ((0, 4, 64, A + 4, A, A), 3),
    ((0, 4, 64, A, A + 8, A), 3), ((0, 4, 64, A, A, A + 1), 3), ((0, 0, 64, None, None, None), 0),
    ((0, 4, 0, None, None, None), 0),
])
def test_quantize_refusals(args, code):
    assert P.lib().poetx_mx4_quantize(*args, None) == code
    dtype, rows, cols, W, codes, scales = args
    if dtype < 2:
        assert P.lib().poetx_mx4_dequantize(rows, cols, codes, scales, W, None) == code


@pytest.mark.parametrize("args,code", [
    ((2, 1, 64, 64, A, A, A, 2 * A), 1), ((0, -1, 64, 64, A, A, A, 2 * A), 1), ((0, 1, 0, 64, A, A, A, 2 * A), 1),
    ((0, 1, 64, -8, A, A, A, 2 * A), 1), ((0, 1, 48, 64, A, A, A, 2 * A), 2), ((1, 1, 64, 60, A, A, A, 2 * A), 2),
    ((0, 1, 64, 64, None, A, A, 2 * A), 1), ((0, 1, 64, 64, A, None, A, 2 * A), 1), ((0, 1, 64, 64, A, A, None, 2 * A), 1),
    ((0, 1, 64, 64, A, A, A, None), 1), ((0, 1, 64, 64, A + 2, A, A, 2 * A), 3), ((0, 1, 64, 64, A, A, A, 2 * A + 8), 3),
    ((0, 1, 64, 64, A, A, A, A), 1), ((1, 0, 64, 64, None, None, None, None), 0),
])
def test_matmul_refusals(args, code):
    assert P.lib().poetx_mx4_matmul(*args, None) == code


@pytest.mark.parametrize("kw,code", [(dict(mode=P.POETX_FAST), 1), (dict(dtype=P.POETX_F32), 1), (dict(d_in=500), 2),
                                     (dict(b=48), 2)])
def test_layer_refusals(kw, code):
    d, L = _desc(**kw), P.lib()
    ws = 1 << 30
    assert L.poetx_mx4_forward(ctypes.byref(d), 8, A, A, A, A, A, A, A, A, A, ws, None) == code
    assert L.poetx_mx4_backward(ctypes.byref(d), 8, A, A, A, A, A, A, A, A, A, A, A, A, A, A, ws, None) == code
    assert L.poetx_mx4_merge(ctypes.byref(d), A, A, A, A, A, A, A, A, A, A, A, ws, None) == code


def test_layer_pointers_and_workspace():
    d, L = _desc(), P.lib()
    ws = P.poetx_workspace_size(d, 8)
    assert L.poetx_mx4_forward(ctypes.byref(d), 8, A, None, A, A, A, A, A, A, A, ws, None) == 1
    assert L.poetx_mx4_forward(ctypes.byref(d), 8, A, A, A + 8, A, A, A, A, A, A, ws, None) == 3
    assert L.poetx_mx4_forward(ctypes.byref(d), 8, A, A, A, A, A, A, A, A, A, 16, None) == 4
    assert L.poetx_mx4_forward(ctypes.byref(d), 0, A, A, A, A, A, A, A, A, A, ws, None) == 0
    assert L.poetx_mx4_merge(ctypes.byref(d), A, A, A, A, A, A, A, A, A, A, A, 16, None) == 4


def test_binding_checks_types_and_sizes():
    class Fake:
        is_cuda = True

        def __init__(self, n, dtype, dev=0):
            self.n, self.dtype, self.dev = n, dtype, dev

        def numel(self):
            return self.n

        def is_contiguous(self):
            return True

        def get_device(self):
            return self.dev

        def data_ptr(self):
            return A

    bf, u8 = torch.bfloat16, torch.uint8
    good = dict(W=Fake(64 * 4, bf), codes=Fake(64 * 2, u8), scales=Fake(8, u8))
    for kw, word in ((dict(W=Fake(255, bf)), "W"), (dict(W=Fake(256, torch.float32)), "W"), (dict(codes=Fake(127, u8)), "codes"),
                     (dict(codes=Fake(128, torch.int8)), "codes"), (dict(scales=Fake(7, u8)), "scales"),
                     (dict(scales=Fake(8, torch.float32)), "scales"), (dict(codes=Fake(128, u8, 1)), "current device"),
                     (dict(W=torch.zeros(4, 64, dtype=bf)), "CUDA")):
        a = dict(good, **kw)
        with pytest.raises(ValueError, match=word):
            P.poetx_mx4_quantize(P.POETX_BF16, 4, 64, a["W"], a["codes"], a["scales"], 0)
    with pytest.raises(ValueError, match="Y"):
        P.poetx_mx4_matmul(1, 2, 64, 8, Fake(16, bf), Fake(256, u8), Fake(16, u8), Fake(127, bf), 0)


@pytest.mark.parametrize("args,code", [
    ((0, 64, 512, 512, A, A, A, 2 * A, 0, 999_999), 1), ((0, 64, 512, 512, A, A, A, 2 * A, 0, 100_000_001), 1),
    ((0, 64, 512, 512, A, A, A, 2 * A, -1, 1_000_000), 1), ((0, 64, 512, 512, A, A, A, 2 * A, 1 << 30, 1_000_000), 1),
    ((0, 0, 512, 512, A, A, A, 2 * A, 0, 1_000_000), 1), ((0, 64, 500, 512, A, A, A, 2 * A, 0, 1_000_000), 2),
    ((0, 64, 512, 512, A, A, A, A, 0, 1_000_000), 1), ((0, 64, 512, 512, A, A + 8, A, 2 * A, 0, 1_000_000), 3),
])
def test_give_up_probe_refusals(args, code):
    splits = ctypes.c_int()
    assert P.lib().poetx_test_mx4_give_up(*args, ctypes.byref(splits), None) == code
    assert P.lib().poetx_test_mx4_give_up(0, 64, 512, 512, A, A, A, 2 * A, 0, 1_000_000, None, None) == 1


@pytest.mark.parametrize("adjoint", [0, 1])
def test_sizes_that_a_tile_takes_past_31_bits_are_refused(adjoint):
    # The first round-up to a tile past 2^31 - 1 would make every loop over K, or the grid, empty: no result, no error.
    top = 2 ** 31 - 1
    for n, d_in, d_out in ((1, top // 32 * 32, 8), (1, 32, top // 8 * 8), (top, 32, 8), (1, (top - 1024) // 32 * 32 + 32, 8),
                           (1, 32, (top - 1024) // 8 * 8 + 8), (top - 1023, 32, 8)):
        assert P.lib().poetx_mx4_matmul(adjoint, n, d_in, d_out, A, A, A, 2 * A, None) == 2
    # The largest ones get as far as the pointers.
    for n, d_in, d_out in ((1, (top - 1024) // 32 * 32, 8), (1, 32, (top - 1024) // 8 * 8), (top - 1024, 32, 8)):
        assert P.lib().poetx_mx4_matmul(adjoint, n, d_in, d_out, A, A, A, 2 * A + 8, None) == 3


def test_a_torch_without_the_newer_names(monkeypatch):
    # Neither the 4-bit and E8M0 types nor the raw handles: the calls fall back on uint8 and the public interface.
    from types import SimpleNamespace
    old = SimpleNamespace(uint8=torch.uint8, bfloat16=torch.bfloat16, float32=torch.float32, _C=SimpleNamespace(),
                          cuda=SimpleNamespace(is_initialized=lambda: True, current_device=lambda: 3,
                                               current_stream=lambda d: SimpleNamespace(cuda_stream=1000 + d)))
    monkeypatch.setattr(P, "_torch_module", old)
    monkeypatch.setattr(P, "_mx4_types", None)
    assert P._device() == 3 and P._stream(None) == 1003 and P._stream(None, 2) == 1002
    assert P._mx4_setup() == ((torch.uint8,), (torch.uint8,), (torch.bfloat16,), (torch.float32,))
    new = SimpleNamespace(**vars(old), float4_e2m1fn_x2="f4", float8_e8m0fnu="e8")
    monkeypatch.setattr(P, "_torch_module", new)
    assert P._mx4_setup()[:2] == ((torch.uint8, "f4"), (torch.uint8, "e8"))
