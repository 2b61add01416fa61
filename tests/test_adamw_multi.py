"""The many-tensor AdamW step without a GPU: refusals of the C entry point and of MultiAdamW, and the sizes of
the moments it makes."""
import ctypes

import pytest
import torch

import orthogonal_equivalence_cnp_b200 as P
from orthogonal_equivalence_cnp_b200 import optim

A = 1 << 20  # aligned, never dereferenced: validation fails first
GOOD = P.poetx_adamw_cfg(1e-3, 0.5, 0.9, 0.999, 1e-8, 0.01)


def _tensor(**kw):
    base = dict(param=A, grad=A, m=A, v=A, scale=A, n=300, lr_scale=1.0, decay_scale=1.0, param_dtype=P.POETX_F32,
                grad_dtype=P.POETX_BF16, moment=P.POETX_MOMENT_E4M3)
    base.update(kw)
    return P.poetx_adamw_tensor(*(base[f] for f, _ in P.poetx_adamw_tensor._fields_))


def _call(*tensors, cfg=GOOD, t=1, n=None):
    arr = (P.poetx_adamw_tensor * max(1, len(tensors)))(*tensors)
    return P.lib().poetx_adamw_multi_step(ctypes.byref(cfg), len(tensors) if n is None else n, arr, t, 0, None)


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(P.poetx_adamw_tensor) == 72 and P.poetx_adamw_tensor.lr_scale.offset == 48


@pytest.mark.parametrize("kw,code", [
    (dict(param=None), 1), (dict(grad=None), 1), (dict(m=None), 1), (dict(v=None), 1), (dict(scale=None), 1),
    (dict(n=-1), 1), (dict(lr_scale=-1.0), 1), (dict(decay_scale=float("nan")), 1), (dict(param_dtype=2), 1),
    (dict(grad_dtype=-1), 1), (dict(moment=2), 1), (dict(param=A + 4), 3), (dict(grad=A + 8), 3), (dict(m=A + 1), 3),
    (dict(v=A + 2), 3), (dict(scale=A + 4), 3), (dict(n=1 << 60), 2), (dict(n=(1 << 42) + 1), 2),
])
def test_bad_tensors_are_refused(kw, code):
    assert _call(_tensor(**kw)) == code
    assert _call(_tensor(n=0), _tensor(**kw)) == code      # wherever it stands


def test_bad_calls_are_refused_and_empty_ones_do_nothing():
    assert _call(n=-1) == 1 and _call(_tensor(), t=0) == 1
    assert P.lib().poetx_adamw_multi_step(ctypes.byref(GOOD), 1, None, 1, 0, None) == 1
    for bad in (P.poetx_adamw_cfg(1e-3, 0.5, 1.0, 0.999, 1e-8, 0.0), P.poetx_adamw_cfg(1e-3, 0.5, 0.9, 0.999, 0.0, 0.0),
                P.poetx_adamw_cfg(float("nan"), 0.5, 0.9, 0.999, 1e-8, 0.0)):
        assert _call(_tensor(), cfg=bad) == 1
    assert _call() == 0
    assert _call(_tensor(n=0, param=None, grad=None, m=None, v=None, scale=None)) == 0
    with pytest.raises(ValueError, match="exceeds"):
        P.poetx_adamw_multi_step(GOOD, 2, (P.poetx_adamw_tensor * 1)(), 1)


class _Fake:
    """Stands in for a CUDA tensor in the host-side checks."""
    is_cuda = True

    def __init__(self, n, dtype=torch.float32, at=A, contiguous=True, device="cuda:0"):
        self._n, self.dtype, self._at, self._c, self.device = n, dtype, at, contiguous, torch.device(device)

    def numel(self):
        return self._n

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return self._at

    def element_size(self):
        return self.dtype.itemsize


def _five(n=300, **kw):
    d = dict(param=_Fake(n, at=A), grad=_Fake(n, at=2 * A), m=_Fake(n, torch.uint8, 3 * A),
             v=_Fake(n, torch.float8_e4m3fn, 4 * A), scale=_Fake(2 * ((n + 255) // 256), at=5 * A))
    d.update(kw)
    return optim.AdamWTensor(**d)


@pytest.mark.parametrize("kw,word", [
    (dict(grad=_Fake(299, at=2 * A)), "300 elements"), (dict(m=_Fake(300, torch.int32, 3 * A)), "expected"),
    (dict(v=_Fake(300, torch.float32, 4 * A)), "expected"), (dict(scale=_Fake(2, at=5 * A)), "4 elements"),
    (dict(scale=None), "scales"), (dict(param=_Fake(300, torch.float16)), "expected"),
    (dict(param=_Fake(300, contiguous=False)), "contiguous"), (dict(grad=_Fake(300, at=2 * A, device="cuda:1")), "not on"),
    (dict(grad=torch.zeros(300)), "CUDA"), (dict(m=_Fake(300, torch.float32, 3 * A), v=_Fake(300, torch.float32, 4 * A)),
                                            "no scales"),
    (dict(grad=_Fake(300, at=A + 1196)), "overlap"),
])
def test_multi_adamw_checks_its_tensors(kw, word):
    with pytest.raises(ValueError, match=word):
        optim.MultiAdamW([_five(**kw)])


def test_multi_adamw_refuses_a_tensor_given_twice():
    with pytest.raises(ValueError, match="overlap"):
        optim.MultiAdamW([_five(), _five()])
    opt = optim.MultiAdamW([_five(), _five(0, scale=_Fake(0))])
    assert opt._entries[0].n == 300 and opt._entries[1].n == 0 and opt._entries[0].moment == P.POETX_MOMENT_E4M3


def test_new_moments():
    m, v, scale = optim.new_moments(torch.zeros(3, 171))
    assert m.numel() == v.numel() == 513 and m.dtype == torch.float8_e4m3fn and scale.shape == (3, 2)
    m, v, scale = optim.new_moments(torch.zeros(7), "f32")
    assert scale is None and m.dtype == torch.float32
    with pytest.raises(ValueError):
        optim.new_moments(torch.zeros(7), "int8")
    with pytest.raises(ValueError):
        optim.MultiAdamW.from_params([torch.zeros(3)], [])


def test_sqrt_probe_refusals():
    L = P.lib()
    assert L.poetx_test_sqrt(0x0D7FFFFF, 0x3F800000, A, None) == 1 and L.poetx_test_sqrt(0x3F800000, 0x7F800000, A, None) == 1
    assert L.poetx_test_sqrt(2, 1, A, None) == 1 and L.poetx_test_sqrt(0x3F800000, 0x3F800000, None, None) == 1
    assert L.poetx_test_sqrt(0x3F800000, 0x3F800000, A + 4, None) == 3


def test_seeds_of_more_than_64_bits_are_refused():
    # Cut to 64 bits, 2^64 would be 0: to nearest, without a word.
    for seed in (1 << 64, (1 << 64) + 1, 1 << 80):
        with pytest.raises(ValueError, match="64 bits"):
            P.poetx_adamw_multi_step(GOOD, 0, (P.poetx_adamw_tensor * 1)(), 1, seed, 0)
    for seed in (0, 1, (1 << 64) - 1, -1):
        P.poetx_adamw_multi_step(GOOD, 0, (P.poetx_adamw_tensor * 1)(), 1, seed, 0)
