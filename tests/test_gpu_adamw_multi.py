"""The many-tensor AdamW step against the oracle, with fp32 and e4m3 moments.

Tolerances.  A float32 rounding is off by at most 2^-24 of the value (u below).  The first moment takes four (the
decoded old one, two products, the sum): under 4u of beta1 |m| + (1 - beta1) |g|, which cancellation can make much
larger than |m|'s own rounding; v takes five, all of one sign, and its root half of them and one: 3.5u.  The
update is their quotient: the denominator 2u more, the approximate reciprocal 2u, the rate 2u, two products and
the sum with the decay 3u: under 16u of `size`, the update with beta1 |m| + (1 - beta1) |g| in m's place.  The
subtraction adds u of the parameter.  So d = 16u size + 2u |p|.  A bf16 parameter
rounded to nearest is off by half a step of its grid (2^-8 of the value) and d.  Rounded stochastically, both
sides add the same random part r and cut: for x and x' with |x - x'| <= d, cut(x + r) and cut(x' + r) differ by
no more than d and one step (2^-7 of the value); where the parameter nearly cancels its update, d is the
larger part.  They differ at all only if the float32 value's low 16 bits, one or two units off, carry on one side
alone: a chance of 2^-16 per unit.
An e4m3 code differs from the oracle's only where the value before rounding lies within 16u of a rounding
border.  The grid's step is at least 1/16 of the value, so the border's neighbourhood is 2 * 16u * 16 = 3e-5 of a
step: out of n codes, 3e-5 n differ on average, and 5 + 1e-4 n are allowed, each by one step.
"""
import numpy as np
import pytest
import torch

import oracle as O
import orthogonal_equivalence_cnp_b200 as P
import poetx_inputs as I
from helpers import device_clean, rel, to_np
from orthogonal_equivalence_cnp_b200.layer import PoetxLayer, make_desc
from orthogonal_equivalence_cnp_b200.optim import AdamWTensor, MultiAdamW, new_moments

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C = dict(lr=1e-3, gamma=0.5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
F32 = {k: float(np.float32(v)) for k, v in C.items()}  # the settings are 32-bit numbers


def _cfg():
    return P.poetx_adamw_cfg(*(C[k] for k in ("lr", "gamma", "beta1", "beta2", "eps", "weight_decay")))


def _make(rng, n, moments, pdt, gdt, g_scale=1.0):
    p = torch.from_numpy((rng.normal(size=n) * 0.02).astype(np.float32)).cuda().to(pdt)
    g = torch.from_numpy((rng.normal(size=n) * g_scale).astype(np.float32)).cuda().to(gdt)
    m, v, scale = new_moments(p, moments)
    if moments == "f32":
        m.copy_(torch.from_numpy((rng.normal(size=n) * 0.3 * g_scale).astype(np.float32)))
        v.copy_(torch.from_numpy((rng.normal(size=n) * g_scale).astype(np.float32) ** 2))
    elif n:
        codes = rng.integers(0, 127, n).astype(np.uint8)
        m.view(torch.uint8).copy_(torch.from_numpy(codes | (rng.integers(0, 2, n) << 7).astype(np.uint8)))
        v.view(torch.uint8).copy_(torch.from_numpy(rng.integers(40, 127, n).astype(np.uint8)))
        scale.copy_(torch.from_numpy((np.exp(rng.normal(size=tuple(scale.shape))) * g_scale / 448).astype(np.float32)))
    return AdamWTensor(p, g, m, v, scale)


def _expect(x, index, t, seed, lr_scale=1.0, decay_scale=1.0):
    """(p, m values, v or root values, scale) after one step, in 64 bits."""
    f = lambda a: a.float().cpu().numpy().astype(np.float64).ravel()
    p, g, m, v = f(x.param), f(x.grad), f(x.m), f(x.v)
    if x.scale is not None:
        s = np.repeat(x.scale.cpu().numpy().astype(np.float64), 256, axis=0)[:p.size]
        m, v = m * s[:, 0], (v * s[:, 1]) ** 2
    m0, v0 = m, v
    p1, m, v = O.adamw_step(p, g, m, v, t, F32["lr"] * lr_scale, F32["gamma"], F32["beta1"], F32["beta2"], F32["eps"],
                            F32["weight_decay"] * decay_scale)
    size = np.abs(O.adamw_step(-np.abs(p), np.abs(g), np.abs(m0), v0, t, F32["lr"] * lr_scale, F32["gamma"],
                               F32["beta1"], F32["beta2"], F32["eps"], 0.0)[0] + np.abs(p))
    size = size + F32["lr"] * lr_scale * F32["gamma"] * F32["weight_decay"] * decay_scale * np.abs(p)
    h = O.element_bits(p.size, index, seed) if seed else None
    out = dict(p=p1, d=16 * U * size + 2 * U * np.abs(p1), p_bf=O.bf16_stochastic(p1, h) if seed else None)
    if x.scale is None:
        return dict(out, m=m, v=v, scale=None)
    r = np.sqrt(v)
    qm, um = O.e4m3_moments(m, False, None if h is None else (h & np.uint64(0xFFFF)).astype(np.float64))
    qr, ur = O.e4m3_moments(r, True, None if h is None else (h >> np.uint64(16)).astype(np.float64))
    return dict(out, m=qm, v=qr, scale=np.stack([um, ur], 1))


def _check(x, e, seed):
    p = to_np(x.param).ravel()
    if x.param.dtype == torch.float32:
        assert np.all(np.abs(p - e["p"]) <= e["d"] + 1e-44)
    elif seed:
        assert np.all(np.abs(p - e["p_bf"]) <= e["d"] + 2.0 ** -7 * np.abs(e["p_bf"]) + 1e-38)
        assert np.count_nonzero(p != e["p_bf"]) <= 5 + 4 * 2.0 ** -16 * p.size
    else:
        assert np.all(np.abs(p - e["p"]) <= 2.0 ** -8 * (np.abs(e["p"]) + e["d"]) + e["d"])
    if x.scale is None:
        assert np.all(np.abs(to_np(x.m) - e["m"]) <= 8 * U * (np.abs(e["m"]) + np.abs(to_np(x.grad).ravel())))
        assert np.all(np.abs(to_np(x.v) - e["v"]) <= 8 * U * e["v"] + 1e-44)
        return
    np.testing.assert_allclose(x.scale.cpu().numpy(), e["scale"], rtol=16 * U, atol=1e-44)
    for got, want in ((to_np(x.m), e["m"]), (to_np(x.v), e["v"])):
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fine = np.isfinite(want)
        got, want = got[fine], want[fine]
        assert np.all(np.abs(got - want) <= np.maximum(O.e4m3_grid(got), O.e4m3_grid(want)) * (1 + 1e-9))
        assert np.count_nonzero(got != want) <= 5 + 1e-4 * got.size


SIZES = [1, 3, 4, 127, 128, 129, 255, 256, 257, 0, 2047, 2048, 2049, 40003]


@pytest.mark.parametrize("moments", ["e4m3", "f32"])
@pytest.mark.parametrize("pdt,gdt", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                     (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("seed", [0, 77, (5 << 32) + 1])
def test_one_step_of_many_sizes(moments, pdt, gdt, seed):
    rng = np.random.default_rng(3)
    xs = [_make(rng, n, moments, pdt, gdt, 10.0 ** rng.integers(-6, 2)) for n in SIZES]
    xs = [x._replace(lr_scale=1.0 + (i % 3), decay_scale=float(i % 2)) for i, x in enumerate(xs)]
    expect = [_expect(x, i, 5, seed, x.lr_scale, x.decay_scale) for i, x in enumerate(xs)]
    opt = MultiAdamW(xs)
    before = P.poetx_launch_count()
    opt.step(_cfg(), t=5, seed=seed)
    torch.cuda.synchronize()
    assert P.poetx_launch_count() == before + 1 and opt.t == 5
    for x, e in zip(xs, expect):
        _check(x, e, seed)
    device_clean()


@pytest.mark.parametrize("seed", [0, 12])
def test_codes_are_those_of_the_float32_restatement(seed):
    # The header fixes every rounding of the moments, so the same steps in numpy's float32 give the
    # same codes and scales, bit for bit.
    f, n = np.float32, 100 * 256
    x = _make(np.random.default_rng(21), n, "e4m3", torch.float32, torch.float32)
    s = np.repeat(x.scale.cpu().numpy(), 256, axis=0)
    g, m, r = (a.float().cpu().numpy() for a in (x.grad, x.m, x.v))
    b1, b2 = f(C["beta1"]), f(C["beta2"])
    m, r = m * s[:, 0], r * s[:, 1]
    m = b1 * m + (f(1) - b1) * g
    r = np.sqrt(b2 * (r * r) + ((f(1) - b2) * g) * g)
    MultiAdamW([x]).step(_cfg(), t=3, seed=seed)
    torch.cuda.synchronize()
    h = O.element_bits(n, 0, seed) if seed else None
    for k, (w, codes) in enumerate(((m, x.m), (r, x.v))):
        top = np.abs(w).reshape(-1, 256).max(1)
        y = np.abs(w * np.repeat(f(448) * (f(1) / top), 256))
        assert y.dtype == f
        grid = O.e4m3_grid(y.astype(np.float64))
        rnd = None if h is None else (h & np.uint64(0xFFFF) if k == 0 else h >> np.uint64(16)).astype(np.float64)
        q = (np.rint(y / grid) if rnd is None else np.floor(y / grid + rnd / 65536)) * grid
        q = np.minimum(np.maximum(q, 2.0 ** -9 if k else 0), 448) * np.where(w < 0, -1, 1)
        assert np.array_equal(codes.float().cpu().numpy(), q)
        assert np.array_equal(x.scale[:, k].cpu().numpy(), top * (f(1) / f(448)))


def test_more_tensors_than_one_launch_holds():
    rng = np.random.default_rng(4)
    sizes = [int(s) for s in rng.integers(1, 600, 1000)]
    xs = [_make(rng, n, "e4m3" if i % 3 else "f32", torch.float32, torch.float32) for i, n in enumerate(sizes)]
    expect = [_expect(x, i, 9, 31) for i, x in enumerate(xs)]
    before = P.poetx_launch_count()
    MultiAdamW(xs).step(_cfg(), t=9, seed=31)
    torch.cuda.synchronize()
    assert P.poetx_launch_count() == before + 3
    for x, e in zip(xs, expect):
        _check(x, e, 31)


def test_nothing_outside_the_tensors_is_written():
    # A tensor of 300 elements in the middle of larger buffers: the 212 elements behind it in its last
    # block, and everything around, stay as they were.
    for pdt in (torch.float32, torch.bfloat16):
        bufs = [torch.full((1024,), 7.0, device="cuda", dtype=pdt), torch.full((1024,), 3.0, device="cuda"),
                torch.full((1024,), 9, device="cuda", dtype=torch.uint8),
                torch.full((1024,), 50, device="cuda", dtype=torch.uint8), torch.full((8, 2), 0.25, device="cuda")]
        cut = [b[256:556] for b in bufs[:4]] + [bufs[4][1:3]]
        MultiAdamW([AdamWTensor(*cut)]).step(_cfg(), t=3, seed=2)
        torch.cuda.synchronize()
        for b, fill in zip(bufs[:4], (7.0, 3.0, 9, 50)):
            assert bool((b[:256].float() == fill).all()) and bool((b[556:].float() == fill).all())
        assert bool((bufs[4][0] == 0.25).all()) and bool((bufs[4][3:] == 0.25).all())
        assert not bool((bufs[0][256:556].float() == 7.0).all())


def test_zero_gradients_tiny_and_non_finite_values():
    n = 512
    z = MultiAdamW.from_params([torch.ones(n, device="cuda")], [torch.zeros(n, device="cuda")])
    z.step(_cfg())
    x = z.tensors[0]
    # decay alone: 1 - eta * (decay * 1), moments and scales stay zero
    assert not x.m.view(torch.uint8).any() and not x.v.view(torch.uint8).any() and not x.scale.any()
    np.testing.assert_allclose(to_np(x.param), 1 - F32["lr"] * F32["gamma"] * F32["weight_decay"], rtol=2 * U)
    # One element's gradient 10^8 times the others': their roots of v round to nothing and are kept at the
    # smallest code, so with no gradient in the next step they move by m / r, not by m / eps.
    g = torch.full((n,), 1e-4, device="cuda")
    g[5] = 1e4
    y = MultiAdamW.from_params([torch.zeros(n, device="cuda")], [g])
    y.step(_cfg())
    assert int(y.tensors[0].v.view(torch.uint8)[:256].min()) == 1
    before = y.tensors[0].param.clone()
    g.zero_()
    y.step(_cfg())
    assert float((y.tensors[0].param - before).abs().max()) <= F32["lr"] * F32["gamma"] * 10
    # A NaN and an infinite gradient spoil their own elements only.
    g.fill_(1.0)
    g[3], g[260] = float("nan"), float("inf")
    w = MultiAdamW.from_params([torch.zeros(n, device="cuda")], [g])
    w.step(_cfg())
    torch.cuda.synchronize()
    x = w.tensors[0]
    ok = torch.ones(n, dtype=torch.bool, device="cuda")
    ok[3] = ok[260] = False
    assert bool(torch.isfinite(x.param[ok]).all()) and bool(torch.isfinite(x.scale).all())
    assert bool(torch.isnan(x.m.float()[~ok]).all()) and bool(torch.isnan(x.v.float()[~ok]).all())
    assert bool((x.m.float()[ok] == 448).all()) and bool((x.v.float()[ok] == 448).all())
    # Values under the least block maximum are stored as zeros.
    g.fill_(1e-32)
    q = MultiAdamW.from_params([torch.zeros(n, device="cuda")], [g])
    q.step(_cfg())
    assert not q.tensors[0].m.view(torch.uint8).any() and bool(torch.isfinite(q.tensors[0].param).all())


def test_same_bits_again_and_seeds_differ():
    def once(seed):
        x = _make(np.random.default_rng(8), 20000, "e4m3", torch.bfloat16, torch.float32)
        MultiAdamW([x]).step(_cfg(), t=2, seed=seed)
        return [a.view(torch.uint8).cpu() for a in (x.param.view(torch.uint8), x.m, x.v, x.scale.view(torch.uint8))]
    a, b, c = once(5), once(5), once(6)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert not torch.equal(a[0], c[0]) and not torch.equal(a[1], c[1]) and torch.equal(a[3], c[3])


def test_stochastic_rounding_keeps_small_changes():
    # Gradients four times as large as those behind v: with beta2 = 0.999 a step raises sqrt(v) by 0.7 %,
    # less than half a step of the grid wherever the element is not its block's largest.  Rounded to
    # nearest, those stay where they are for good; stochastically they follow the exact value.
    n, steps = 4096, 200
    def run(seeded):
        p, g = torch.zeros(n, device="cuda"), torch.full((n,), 4.0, device="cuda")
        g[::256] = 300.0
        m, v, scale = new_moments(p)
        r0 = torch.ones(n, device="cuda")
        r0[::256] = 300.0
        scale[:, 1] = 300.0 / 448
        v.copy_((r0 / (300.0 / 448)).to(torch.float8_e4m3fn))
        start = (v.float() * (300.0 / 448))[1::256].mean().item()
        opt = MultiAdamW([AdamWTensor(p, g, m, v, scale)])
        for i in range(steps):
            opt.step(_cfg(), t=1000 + i, seed=(i + 1) if seeded else 0)
        live = torch.ones(n, dtype=torch.bool, device="cuda")
        live[::256] = False
        return (v.float() * scale[:, 1].repeat_interleave(256))[live].double().mean().item(), start
    exact_of = lambda r0: np.sqrt(0.999 ** steps * r0 ** 2 + (1 - 0.999 ** steps) * 16)
    got, r0 = run(True)
    # The mean over 4080 elements of a walk of 200 steps with steps of at most 1/8: its spread is under
    # 0.125 * sqrt(200) / sqrt(4080) = 3 % of the value; the bias of r^2 (variance of r) adds under 1 %.
    assert abs(got / exact_of(r0) - 1) < 0.08
    stuck, r0 = run(False)
    assert abs(stuck / r0 - 1) < 0.02 and exact_of(r0) > 1.7 * r0


@pytest.mark.parametrize("how", ["stream", "graph"])
def test_other_stream_and_captured(how):
    xs = [_make(np.random.default_rng(i), 5000 + i, "e4m3", torch.float32, torch.float32) for i in range(3)]
    ys = [AdamWTensor(*(None if a is None else a.clone() for a in x[:5])) for x in xs]
    MultiAdamW(ys).step(_cfg(), t=4, seed=1)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    opt = MultiAdamW(xs)
    if how == "stream":
        with torch.cuda.stream(st):
            opt.step(_cfg(), t=4, seed=1)
    else:
        keep = [tuple(None if a is None else a.clone() for a in x[:5]) for x in xs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            opt.step(_cfg(), t=4, seed=1)
        opt._entries[0].n = 0  # the graph holds its own copy of the table
        for x, k in zip(xs, keep):
            for a, b in zip(x[:5], k):
                if a is not None:
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # capturing ran nothing
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        for a, b in zip(x[:5], y[:5]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_reset_and_step_count():
    p, g = torch.randn(700, device="cuda"), torch.randn(700, device="cuda")
    for moments in ("e4m3", "f32"):
        opt = MultiAdamW.from_params([p], [g], moments)
        opt.step(_cfg(), seed=1)
        opt.step(_cfg(), seed=2)
        assert opt.t == 2 and opt.tensors[0].m.view(torch.uint8).any()
        opt.reset()
        torch.cuda.synchronize()
        x = opt.tensors[0]
        assert opt.t == 0 and not x.m.view(torch.uint8).any() and not x.v.view(torch.uint8).any()
        assert x.scale is None or not x.scale.any()


def test_square_root_of_every_float():
    bad = torch.ones(1, dtype=torch.int64, device="cuda")
    P.poetx_test_sqrt(0x0D800000, 0x7F7FFFFF, bad)
    assert int(bad) == 0


@pytest.mark.parametrize("how", ["stream", "handle", "capture"])
def test_reset_is_ordered_on_the_stream_of_the_step(how):
    # A step held back on another stream, then a reset given the same stream: the reset comes after the step.
    xs = [_make(np.random.default_rng(i), 3000 + i, "e4m3" if i else "f32", torch.float32, torch.float32) for i in range(2)]
    before = [x.param.clone() for x in xs]
    opt = MultiAdamW(xs)
    st = torch.cuda.Stream()
    arg = st.cuda_stream if how == "handle" else st
    torch.cuda.synchronize()
    if how == "capture":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            opt.step(_cfg(), t=4, seed=1, stream=arg)
            opt.reset(stream=arg)
        graph.replay()
    else:
        with torch.cuda.stream(st):
            torch.cuda._sleep(100_000_000)  # about 50 ms
        opt.step(_cfg(), t=4, seed=1, stream=arg)
        opt.reset(stream=arg)
    torch.cuda.synchronize()
    assert opt.t == 0
    for x, p in zip(xs, before):
        assert not torch.equal(x.param, p)
        assert not any(a.view(torch.uint8).any().item() for a in (x.m, x.v))
        assert x.scale is None or not x.scale.any().item()


@pytest.mark.parametrize("seed", [0, 9])
def test_elements_past_32_bits(seed, monkeypatch):
    # A tensor of 2^32 + 1029 elements, zeros but for its last 1285, which start 256 before element 2^32: values and
    # random bits are those of these positions, and the zeros stay.
    n, at = (1 << 32) + 1029, (1 << 32) - 256
    tail = _make(np.random.default_rng(17), n - at, "e4m3", torch.bfloat16, torch.bfloat16)
    zeros = lambda dtype: torch.zeros(n, dtype=dtype, device="cuda")
    m, v = zeros(torch.uint8), zeros(torch.uint8)
    big = AdamWTensor(zeros(torch.bfloat16), zeros(torch.bfloat16), m.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn),
                      torch.zeros((n + 255) // 256, 2, device="cuda"))
    cut = AdamWTensor(*(a[at:] for a in big[:4]), big.scale[at // 256:])
    for a, b in zip(cut[:5], tail[:5]):
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    bits = O.element_bits
    monkeypatch.setattr(O, "element_bits", lambda count, tensor, s: bits(count, tensor, s, start=at))
    expect = _expect(tail, 0, 5, seed)
    MultiAdamW([big]).step(_cfg(), t=5, seed=seed)
    torch.cuda.synchronize()
    device_clean()
    _check(cut, expect, seed)
    for a in (big.param[:at], m[:at], v[:at], big.scale[:at // 256]):
        assert not a.view(torch.int64).any().item()


def test_an_eps_that_is_no_normal_number(monkeypatch):
    # The reciprocal takes subnormal numbers for zero: such an eps counts as 2^-126, and an element that has seen no
    # gradient (0 / eps) stays where it is.
    xs = [_make(np.random.default_rng(5), 3000, moments, torch.float32, torch.float32) for moments in ("f32", "e4m3")]
    for x in xs:
        for a in (x.grad, x.m, x.v):
            a.view(torch.uint8)[:256 * a.element_size()] = 0
    monkeypatch.setitem(F32, "eps", 2.0 ** -126)
    expect = [_expect(x, i, 5, 0) for i, x in enumerate(xs)]
    MultiAdamW(xs).step(P.poetx_adamw_cfg(C["lr"], C["gamma"], C["beta1"], C["beta2"], 1e-42, C["weight_decay"]), t=5)
    torch.cuda.synchronize()
    for x, e in zip(xs, expect):
        assert torch.isfinite(x.param).all().item()
        _check(x, e, 0)


def test_state_saved_and_loaded_goes_on_with_the_same_bits():
    rng = np.random.default_rng(6)
    xs = [_make(rng, n, "e4m3" if n % 2 else "f32", torch.bfloat16, torch.float32) for n in (5001, 300, 77)]
    opt = MultiAdamW(xs)
    for seed in (1, 2):
        opt.step(_cfg(), seed=seed)
    saved = [[None if a is None else a.cpu() for a in x[:5]] for x in opt.tensors]
    ys = [AdamWTensor(*(None if a is None else a.cuda() for a in s)) for s in saved]
    again = MultiAdamW(ys)
    again.t = opt.t
    for o in (opt, again):
        o.step(_cfg(), seed=3)
    for x, y in zip(xs, ys):
        assert all(a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(x[:5], y[:5]))
    opt.reset(stream=0)  # the default stream by its handle
    assert opt.t == 0 and not any(x.m.view(torch.uint8).any().item() for x in xs)
