"""Gradient norm and clipping, and the steps that take the scale, against
64-bit computations.

Tolerances, from the roundings of the kernels (u = 2^-24, half a step of fp32):

* the norm: fp64 squares and sums of n terms, each within n 2^-53, and one
  rounding to fp32: |N - N64| <= (u + n 2^-53) N64, for the sum as for its root;
* the scale: max_norm / (N + eps) in fp64, one rounding: the same bound twice
  over at most (the sum's error and the rounding);
* a clipped entry: the scale's rounding, the product's rounding to fp32 and,
  for a 16-bit output, that type's rounding; below the smallest normal number a
  rounding is half the smallest subnormal instead.

Where two paths of the library must agree (a scaled step, and clipping in
memory followed by the step) the comparison is bit for bit.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import adamw_step_ref, momentum_ref, muon_step_ref, normalize_ref, orient
from tests.gpu_util import rel_fro
from tests.test_gpu_adamw import _bounds
from workloads import ADAMW_WORKLOADS, WORKLOADS, AdamWStream, WorkloadStream

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half of the smallest subnormal
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


@pytest.fixture(scope="module")
def muon():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from newton_schulz_norm_b200 import build
    build.build()
    import newton_schulz_norm_b200 as m
    yield m
    assert m.status() == 0
    assert m.guard_check() == 0


def _grads(sizes, dtypes, seed, offs=None, std=1e-2):
    """Views at the given element offsets into larger buffers, with the buffers."""
    rng = np.random.default_rng(seed)
    views, bases = [], []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        off = offs[i % len(offs)] if offs else 0
        base = torch.full((n + off + 24,), 7.0, dtype=dt, device="cuda")
        view = base[off:off + n]
        view.copy_(torch.from_numpy(rng.standard_normal(n) * std))
        views.append(view)
        bases.append((base, off, n))
    return views, bases


def _guards_hold(bases):
    for base, off, n in bases:
        assert bool((base[:off] == 7.0).all()) and bool((base[off + n:] == 7.0).all())


def _norm64(grads, p):
    xs = [np.abs(g.detach().double().cpu().numpy().ravel()) for g in grads if g.numel()]
    if not xs:
        return 0.0, 0
    x = np.concatenate(xs)
    if p == INF:
        return float(x.max()), x.size
    if p == 1.0:
        return math.fsum(x), x.size
    return math.sqrt(math.fsum(x * x)), x.size


def _norm_ok(got, grads, p):
    want, n = _norm64(grads, p)
    tol = 0.0 if p == INF else (U + n * 2.0 ** -53) * want + 2.0 ** -150
    assert abs(float(got) - want) <= tol, (float(got), want)
    return want, n


def _scale64(want, max_norm, eps):
    return min(1.0, max_norm / (want + eps)) if want + eps > 0 else 1.0


SIZES = [1, 2, 3, 5, 7, 8, 9, 255, 1023, 1024, 1025, 4097, 8191, 8192, 8193, 16383, 16384, 16385, 32769, 100003]


# ---------------------------------------------------------------- the norm

@pytest.mark.parametrize("p", [1.0, 2.0, INF])
@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
def test_norm_of_single_tensors_of_every_edge_size(muon, dtype, p):
    for k, n in enumerate(SIZES):
        (g,), bases = _grads([n], [dtype], seed=k, offs=[k % 8])
        _norm_ok(muon.grad_norm([g], p), [g], p)
        _guards_hold(bases)


@pytest.mark.parametrize("off", range(8))
def test_norm_at_every_alignment(muon, off):
    sizes = [1, 6, 7, 8, 9, 15, 16, 17, 4091, 4100, 9000]
    for dtype in TYPES:
        gs, bases = _grads(sizes, [dtype], seed=off, offs=[off])
        _norm_ok(muon.grad_norm(gs), gs, 2.0)
        _guards_hold(bases)


@pytest.mark.parametrize("p", [1.0, 2.0, INF])
def test_norm_of_a_mixed_list_is_the_same_each_time(muon, p):
    gs, _ = _grads(SIZES + [0, 77777, 0, 300001], TYPES, seed=3, offs=[0, 1, 2, 3, 5])
    group = muon.GradGroup(gs)
    a = group.norm(p)
    _norm_ok(a, gs, p)
    assert a.shape == () and a.dtype == torch.float32
    for _ in range(3):
        assert torch.equal(group.norm(p), a)
    assert torch.equal(muon.grad_norm(gs, p), a)
    norm, scale = group.clip_scale(0.25, p)
    assert torch.equal(norm, a)
    want, n = _norm64(gs, p)
    s = _scale64(want, 0.25, 1e-6)
    assert abs(float(scale) - s) <= 2 * (U + n * 2.0 ** -53) * s


def test_norm_of_a_large_list_takes_several_launches(muon):
    """1300 tensors: three tables of 512; the partial sums of all are joined."""
    rng = np.random.default_rng(4)
    sizes = [int(v) for v in rng.integers(0, 700, 1300)]
    gs, bases = _grads(sizes, TYPES, seed=5, offs=[0, 3, 1])
    for p in (1.0, 2.0, INF):
        _norm_ok(muon.grad_norm(gs, p), gs, p)
    keep = [g.clone() for g in gs]
    norm, scale = muon.clip_scale(gs, 0.5)
    assert torch.equal(muon.clip_grads(gs, 0.5), norm)
    for g, k in zip(gs, keep):
        assert torch.equal(g, (k.float() * scale).to(g.dtype))
    _guards_hold(bases)


def test_norm_of_nothing(muon):
    e = torch.empty(0, device="cuda")
    for gs in ([], [e], [e, e.bfloat16()]):
        norm, scale = muon.clip_scale(gs, 1.0)
        assert float(norm) == 0.0 and float(scale) == 1.0
        assert float(muon.grad_norm(gs, INF)) == 0.0
        assert float(muon.clip_grads(gs, 1.0)) == 0.0
    z = torch.zeros(1000, device="cuda")
    for eps, max_norm, s in ((1e-6, 1.0, 1.0), (0.0, 1.0, 1.0), (0.0, 0.0, 1.0), (1e-6, 0.0, 0.0)):
        norm, scale = muon.clip_scale([z], max_norm, eps=eps)
        assert float(norm) == 0.0 and float(scale) == s


def test_entries_whose_squares_leave_fp32(muon):
    """Squares below and above fp32's range, subnormal entries, and a norm
    above the largest fp32 number."""
    tiny = torch.full((5000,), 1e-30, device="cuda")
    sub = torch.full((333,), 2.0 ** -149, device="cuda")
    huge = torch.full((64,), 1e30, device="cuda")
    for gs in ([tiny], [sub], [huge], [tiny, huge], [sub, tiny]):
        for p in (1.0, 2.0, INF):
            _norm_ok(muon.grad_norm(gs, p), gs, p)
    most = torch.full((9,), 3.0e38, device="cuda")
    assert math.isinf(float(muon.grad_norm([most])))                 # 9e38: no fp32 number
    norm, scale = muon.clip_scale([most], 1.0)
    assert abs(float(scale) - 1 / 9e38) <= 2.0 ** -149               # formed from the unrounded norm
    assert float(muon.grad_norm([most], INF)) == float(most[0])


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
def test_infinity_and_nan(muon, dtype):
    for where in (0, 1, 4096, 9998):
        g = torch.full((9999,), 0.5, device="cuda", dtype=dtype)
        g[where] = -INF
        for p in (1.0, 2.0, INF):
            norm, scale = muon.clip_scale([g], 1.0, p)
            assert math.isinf(float(norm)) and float(scale) == 0.0
        c = g.clone()
        muon.clip_grads([c], 1.0)
        bad = torch.isnan(c)
        assert int(bad.sum()) == 1 and bool(bad[where]) and float(c[~bad].abs().max()) == 0.0
        g[9999 - 1 - where] = float("nan")
        for p in (1.0, 2.0, INF):
            norm, scale = muon.clip_scale([g, torch.full((3,), INF, device="cuda")], 1.0, p)
            assert math.isnan(float(norm)) and math.isnan(float(scale))
        muon.clip_grads([g], 1.0)
        assert bool(torch.isnan(g).all())


def test_a_tensor_of_more_than_2_31_elements(muon):
    """Offsets past 32 bits, in elements and in bytes."""
    n = 2 ** 31 + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, 12345, 2 ** 30 + 1, 2 ** 31 - 1, 2 ** 31, n - 1]
    for k, a in enumerate(at):
        g[a] = 2.0 ** k
    want = math.sqrt(sum(4.0 ** k for k in range(len(at))))
    assert abs(float(muon.grad_norm([g])) - want) <= U * want
    assert float(muon.grad_norm([g], 1.0)) == 63.0 and float(muon.grad_norm([g], INF)) == 32.0
    norm = muon.clip_grads([g], 0.25 * want, eps=0.0)
    assert abs(float(norm) - want) <= U * want
    for k, a in enumerate(at):
        assert float(g[a]) == 2.0 ** (k - 2)
    assert int((g != 0).sum()) == len(at)


# ---------------------------------------------------------------- clipping

def _check_clip(muon, grads, max_norm, p=2.0, eps=1e-6, outs=None):
    before = [g.clone() for g in grads]
    norm, scale = muon.clip_scale(grads, max_norm, p, eps)
    want, n = _norm_ok(norm, before, p)
    s = _scale64(want, max_norm, eps)
    assert abs(float(scale) - s) <= 2 * (U + n * 2.0 ** -53) * s
    got = muon.clip_grads(grads, max_norm, p, eps, out=outs)
    assert torch.equal(got, norm)
    for g, b, o in zip(grads, before, grads if outs is None else outs):
        if outs is not None and o.data_ptr() != g.data_ptr():
            assert torch.equal(g, b)                                 # inputs of another output stay
        assert torch.equal(o, (b.float() * scale).to(o.dtype))
        exact = b.double() * s
        half = HALF_STEP[o.dtype] if o.dtype != torch.float32 else 0.0
        tol = exact.abs() * (2 * (U + n * 2.0 ** -53) + U + half + 3 * U * half) + TINY[o.dtype] + TINY[torch.float32]
        assert bool(((o.double() - exact).abs() <= tol).all())


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("max_norm", [0.0, 0.125, 1.0, 1e6, INF])
def test_clip_in_place(muon, dtype, max_norm):
    gs, bases = _grads(SIZES + [0], [dtype], seed=11, offs=[0, 1, 4, 7])
    _check_clip(muon, gs, max_norm)
    _guards_hold(bases)


@pytest.mark.parametrize("src", TYPES, ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dst", TYPES, ids=["fp32", "bf16", "fp16"])
def test_clip_into_another_type_at_every_alignment(muon, src, dst):
    sizes = [1, 3, 7, 8, 9, 16, 17, 31, 4096, 8192, 12289, 40000]
    for off in range(8):
        gs, _ = _grads(sizes, [src], seed=20 + off, offs=[off])
        outs, bases = _grads(sizes, [dst], seed=40, offs=[(3 * off) % 8, off])
        _check_clip(muon, gs, 0.5, outs=outs)
        _guards_hold(bases)
        _check_clip(muon, gs, 1e9, outs=outs)                        # nothing to clip: a copy
        _guards_hold(bases)


@pytest.mark.parametrize("p", [1.0, 2.0, INF])
def test_clip_by_every_norm(muon, p):
    gs, _ = _grads([4097, 50000, 3], TYPES, seed=30, offs=[1, 0, 2])
    _check_clip(muon, gs, {1.0: 10.0, 2.0: 0.5, INF: 0.01}[p], p)


def test_clip_some_in_place_and_some_elsewhere(muon):
    gs, _ = _grads([5000, 7000, 0, 9000], [torch.float32, torch.bfloat16], seed=31)
    outs = [gs[0], torch.empty(7000, device="cuda"), torch.empty(0, device="cuda"),
            torch.empty(9000, device="cuda", dtype=torch.float16)]
    _check_clip(muon, gs, 1e9, outs=outs)                            # s = 1: the first stays, the rest are copied
    _check_clip(muon, gs, 0.25, outs=outs)


def test_the_same_clip_again_and_again(muon):
    """A clipped list has the bound as its norm; clipping it once more moves
    nothing by more than the scale's distance from one."""
    gs, _ = _grads([30000, 1000], [torch.float32], seed=32)
    group = muon.GradGroup(gs)
    first = group.clip(1.0)
    assert float(first) > 1.0
    for _ in range(3):
        norm = group.clip(1.0)
        assert abs(float(norm) - 1.0) <= 1e-6 + 4 * U


@pytest.mark.parametrize("sizes", [[40_000, 3], [2_500_000, 77], [9_000_001] * 2 + [11] * 600],
                         ids=["cluster", "two_launches", "several_tables"])
def test_writes_before_and_after_are_kept_apart(muon, sizes):
    """Gradients written just before a clip in place and read just after it,
    over and over without a wait: the second launch of the clip begins before
    the first has ended, and must see neither older nor newer values."""
    src = [[torch.randn(n, device="cuda") * (k + 1) for n in sizes] for k in range(3)]
    g = [torch.empty(n, device="cuda") for n in sizes]
    want = []
    for xs in src:
        _, scale = muon.clip_scale(xs, 1.0)
        want.append([x * scale for x in xs])
    group = muon.GradGroup(g)
    bad = torch.zeros((), device="cuda")
    for i in range(60):
        for d, x in zip(g, src[i % 3]):
            d.copy_(x)
        group.clip(1.0)
        for d, w in zip(g[:4], want[i % 3]):
            bad += (d != w).any()
    assert float(bad) == 0.0
    for d, w in zip(g, want[59 % 3]):
        assert torch.equal(d, w)


def test_numbers_of_other_kinds_as_arguments(muon):
    g = [torch.full((500,), 2.0, device="cuda")]
    a = muon.clip_scale(g, 1.0, 2.0)
    for mx, p in ((np.float32(1.0), 2), (torch.tensor(1.0), np.float32(2.0)), (1, "2")):
        b = muon.clip_scale(g, mx, p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert float(muon.grad_norm(g, "inf")) == 2.0


def test_values_are_read_anew_by_every_call(muon):
    g = torch.ones(1000, device="cuda")
    group = muon.GradGroup([g])
    a = group.norm()
    g.mul_(3.0)
    b = group.norm()
    g.zero_()
    assert abs(float(b) - 3 * float(a)) <= 8 * U * float(b) and float(group.norm()) == 0.0


def test_refusals_on_the_gpu(muon):
    a, b = torch.ones(16, device="cuda"), torch.ones(16, device="cuda")
    for call in (lambda: muon.grad_norm([a.double()]), lambda: muon.grad_norm([torch.ones(8, 8, device="cuda").t()]),
                 lambda: muon.grad_norm([a.cpu()]), lambda: muon.clip_grads([a], 1.0, out=[]),
                 lambda: muon.clip_grads([a], 1.0, out=[b[:8]]), lambda: muon.clip_grads([a, a], 1.0),
                 lambda: muon.clip_grads([a, b], 1.0, out=[b, a]), lambda: muon.clip_grads([a], 1.0, out=[a.view(torch.int32)]),
                 lambda: muon.adamw_step([a], [b], [a], [b], 1, 1e-3, grad_scale=torch.ones(2, device="cuda")),
                 lambda: muon.momentum_normalize([a.view(4, 4)], []),
                 lambda: muon.momentum_normalize([a.view(4, 4)], [b.view(2, 8)]),
                 lambda: muon.step([a.view(4, 4)], [b.view(4, 4)], [a.view(4, 4)], 0.1, grad_scale=0.5)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: muon.grad_norm([a], 3.0), lambda: muon.clip_grads([a], -1.0),
                 lambda: muon.clip_grads([a], float("nan")), lambda: muon.clip_scale([a], 1.0, eps=-1.0)):
        with pytest.raises(muon.MuonError):
            call()
    assert float(muon.grad_norm([a, a])) == pytest.approx(math.sqrt(32))   # only read: twice is twice
    assert torch.equal(a, torch.ones(16, device="cuda"))


# ---------------------------------------------------------------- streams and graphs

def test_two_streams_at_once(muon):
    """Calls of one group on two streams, neither waiting for the other."""
    gs, _ = _grads([3_000_001, 400_000], [torch.float32, torch.bfloat16], seed=50)
    group = muon.GradGroup(gs)
    want = group.norm()
    want1 = group.norm(1.0)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(40):
        got.append((group.norm(stream=s[0]), want))
        got.append((group.norm(1.0, stream=s[1].cuda_stream), want1))    # a raw handle too
        with torch.cuda.stream(s[k % 2]):
            got.append((group.clip_scale(0.5)[0], want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    with torch.cuda.stream(s[0]):
        assert torch.equal(group.norm(stream=0), want)                  # the default stream by its handle


def test_two_graphs_of_one_group(muon):
    """Two captures of one group replayed together on two streams, on new
    values, and the results of an eager call in between."""
    gs, _ = _grads([1_000_003, 70_000], [torch.float32], seed=51)
    outs = [torch.empty_like(g) for g in gs]
    outs2 = [torch.empty_like(g) for g in gs]
    ga, gb = muon.GradGroup(gs, out=outs), muon.GradGroup(gs, out=outs2)
    ga.clip(0.5), gb.clip(0.125)
    torch.cuda.synchronize()
    A, B = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(A):
        na = ga.clip(0.5)
    with torch.cuda.graph(B):
        nb = gb.clip(0.125)
    s = [torch.cuda.Stream() for _ in range(2)]
    for k in range(5):
        for g in gs:
            g.mul_(1.5)
        torch.cuda.synchronize()
        with torch.cuda.stream(s[0]):
            A.replay()
        with torch.cuda.stream(s[1]):
            B.replay()
        norm, sa = ga.clip_scale(0.5)
        _, sb = gb.clip_scale(0.125)
        torch.cuda.synchronize()
        assert torch.equal(na, norm) and torch.equal(nb, norm)
        for g, a, b in zip(gs, outs, outs2):
            assert torch.equal(a, g * sa) and torch.equal(b, g * sb)
    del A, B


def test_scales_dropped_while_a_side_stream_still_reads_them(muon):
    """Each round's scale is computed on the current stream, read by steps on a
    side stream behind a long queue, and dropped at once; so are X0s."""
    side = torch.cuda.Stream()
    rng = np.random.default_rng(55)
    shape = (512, 512)
    G = [torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()]
    P, B = [torch.zeros(shape, device="cuda")], [torch.zeros(shape, device="cuda")]
    X0 = [torch.zeros(shape, device="cuda")]
    flat = [torch.zeros(512 * 512, device="cuda") for _ in range(3)]
    adamw = muon.AdamWGroup([flat[0]], [G[0].view(-1)], [flat[1]], [flat[2]], lr=1e-3)
    torch.cuda.synchronize()
    busy = torch.empty(1 << 28, device="cuda")
    bounds = [3.0 * (k + 1) for k in range(12)]
    kept = []
    with torch.cuda.stream(side):
        for _ in range(6):
            busy.fill_(1.0)
    for k, bound in enumerate(bounds):
        scale = muon.clip_scale(G, bound)[1]
        side.wait_stream(torch.cuda.current_stream())
        muon.step(P, G, B, lr=0.02, stream=side, grad_scale=scale)
        adamw.step(k + 1, stream=side, grad_scale=scale)
        kept.append(muon.momentum_normalize(G, X0, stream=side, grad_scale=scale)[0])
        del scale
        junk = [torch.full((), -1.0, device="cuda") for _ in range(8)]   # takes freed places
        del junk
    norms = [muon.grad_norm(G, stream=side) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    got = [t.clone() for t in P + B + X0 + flat + kept]
    assert all(torch.equal(n, norms[0]) for n in norms)
    for t in P + B + X0 + flat:
        t.zero_()
    want_kept = []
    for k, bound in enumerate(bounds):
        scale = muon.clip_scale(G, bound)[1]
        muon.step(P, G, B, lr=0.02, grad_scale=scale)
        adamw.step(k + 1, grad_scale=scale)
        want_kept.append(muon.momentum_normalize(G, X0, grad_scale=scale)[0])
    for a, b in zip(got, P + B + X0 + flat + want_kept):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- the scaled steps

def _dev(xs):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


@pytest.mark.parametrize("scale", [0.0, 1.0, 0.37, 3.0e-5])
def test_adamw_takes_the_scale(muon, scale):
    wl = ADAMW_WORKLOADS["adamw_ragged"]
    st = AdamWStream(wl, seed=60)
    params, us, vs = st.init()
    grads = st.next_grads()
    decay = [t.decay for t in wl.tensors]
    kw = dict(lr=wl.lr, betas=(wl.beta1, wl.beta2), eps=wl.eps, weight_decay=wl.weight_decay, decay=decay)
    s = torch.tensor(scale, device="cuda")
    G = _dev(grads)
    a, b, c = ([_dev(params), _dev(us), _dev(vs)] for _ in range(3))
    muon.adamw_step(a[0], G, a[1], a[2], wl.step, grad_scale=s, **kw)
    muon.adamw_step(b[0], [g * s for g in G], b[1], b[2], wl.step, **kw)
    muon.AdamWGroup(c[0], G, c[1], c[2], **kw).step(wl.step, grad_scale=s)
    for x, y, z in zip(sum(a, []), sum(b, []), sum(c, [])):
        assert torch.equal(x, y) and torch.equal(x, z)
    for g, h in zip(G, grads):
        assert np.array_equal(g.cpu().numpy(), h)                    # the gradients stay as they were


def test_adamw_scaled_against_the_oracle(muon):
    """The plain step's bounds doubled: g' = fp32(s g) adds one rounding u of
    the gradient's terms to m' (4u), two to v' (6u)."""
    rng = np.random.default_rng(61)
    sizes = [1, 5, 2049, 40000]
    p, g, m = ([rng.standard_normal(n).astype(np.float32) for n in sizes] for _ in range(3))
    v = [(rng.standard_normal(n) ** 2).astype(np.float32) for n in sizes]
    s = np.float32(0.2718)
    P, G, M, V = (_dev(x) for x in (p, g, m, v))
    muon.adamw_step(P, G, M, V, 5, 1e-3, betas=(0.9, 0.99), weight_decay=0.0, grad_scale=torch.tensor(s, device="cuda"))
    gs = [x.astype(np.float64) * float(s) for x in g]
    want = adamw_step_ref(p, gs, m, v, 5, 1e-3, 0.9, 0.99, 1e-8, 0.0)
    for i in range(len(sizes)):
        bounds = _bounds(p[i], gs[i], m[i], v[i], 5, 1e-3, 0.9, 0.99, 1e-8, 0.0)
        for got, ref, bound in zip((P[i], M[i], V[i]), (w[i] for w in want), bounds):
            assert np.all(np.abs(got.cpu().numpy() - ref.astype(np.float64)) <= 2 * bound)


@pytest.mark.parametrize("offs", [(0, 0, 0, 0), (1, 1, 1, 1), (3, 3, 3, 3), (0, 1, 0, 0), (2, 1, 3, 0)],
                         ids=["aligned", "off1", "off3", "grad_off", "all_differ"])
def test_adamw_at_every_alignment(muon, offs):
    """Views equally far past a 16-byte boundary take vectors, others single
    elements; both give the aligned tensors' bits and touch nothing outside."""
    rng = np.random.default_rng(67)
    sizes = [1, 2, 3, 4, 5, 7, 8, 2044, 2045, 2047, 2048, 2049, 2051, 4096, 10001]
    decay = [i % 2 == 0 for i in range(len(sizes))]
    host = [[rng.standard_normal(n).astype(np.float32) for n in sizes] for _ in range(4)]
    host[3] = [np.abs(x) for x in host[3]]
    s = torch.tensor(0.7, device="cuda")
    want = [_dev(x) for x in host]
    muon.adamw_step(*want, 3, 1e-2, decay=decay, grad_scale=s)
    views, bases = [], []
    for rows, off in zip(host, offs):
        views.append([])
        for x in rows:
            base = torch.full((x.size + 16,), 7.0, device="cuda")
            base[off:off + x.size] = torch.from_numpy(x).cuda()
            views[-1].append(base[off:off + x.size])
            bases.append((base, off, x.size))
    muon.adamw_step(*views, 3, 1e-2, decay=decay, grad_scale=s)
    for a, b in zip(sum(want, []), sum(views, [])):
        assert torch.equal(a, b)
    _guards_hold(bases)


SHAPES = [(256, 256), (129, 257), (300, 7), (7, 300), (1, 1), (1000, 96), (64, 4)]


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("scale", [1.0, 0.37])
def test_first_kernel_takes_the_scale(muon, scale, nesterov):
    rng = np.random.default_rng(62)
    g = [rng.standard_normal(x).astype(np.float32) for x in SHAPES]
    b = [(rng.standard_normal(x) * 0.1).astype(np.float32) for x in SHAPES]
    s = torch.tensor(scale, device="cuda")
    G, B1, B2 = _dev(g), _dev(b), _dev(b)
    x1 = muon.momentum_normalize(G, B1, 0.95, nesterov, grad_scale=s)
    x2 = muon.momentum_normalize([t * s for t in G], B2, 0.95, nesterov)
    for a, c in zip(list(x1) + B1, list(x2) + B2):
        assert torch.equal(a, c)
    for i in range(len(SHAPES)):
        gd = g[i].astype(np.float64) * float(np.float32(scale))
        new = 0.95 * b[i].astype(np.float64) + gd
        # beta as fp32, the product's and the fma's roundings
        tol = 2 * U * (0.95 * np.abs(b[i])) + 2 * U * np.abs(gd) + 2.0 ** -126
        assert np.all(np.abs(B1[i].cpu().numpy() - new) <= tol)
        u = gd + 0.95 * new if nesterov else new
        x = u / (np.linalg.norm(u) + 1e-7)
        x = x.T if x.shape[0] > x.shape[1] else x
        # bf16's half step 2^-9 of the value's binade, 2^-8 of the value at most; u's roundings are absolute
        # in the size of its terms, a few u
        terms = (np.abs(gd) * 1.95 + np.abs(b[i])) / (np.linalg.norm(u) + 1e-7)
        terms = terms.T if terms.shape[0] > terms.shape[1] else terms
        assert np.all(np.abs(x1[i].float().cpu().numpy() - x) <= 2.0 ** -8 * np.abs(x) + 8 * U * terms)


@pytest.mark.parametrize("steps", [0, 1, 5])
@pytest.mark.parametrize("many", [False, True], ids=["chain", "phases"])
def test_muon_step_takes_the_scale(muon, steps, many):
    """The chain launch, the per-phase launches and the update without
    iterations: bit for bit the step on scaled gradients."""
    rng = np.random.default_rng(63)
    shapes = [(768, 768)] * 20 if many else SHAPES
    p, g, b = ([rng.standard_normal(x).astype(np.float32) for x in shapes] for _ in range(3))
    s = torch.tensor([0.61], device="cuda")
    G, P1, P2, B1, B2 = _dev(g), _dev(p), _dev(p), _dev(b), _dev(b)
    muon.step(P1, G, B1, lr=0.02, ns_steps=steps, grad_scale=s)
    muon.step(P2, [t * s for t in G], B2, lr=0.02, ns_steps=steps)
    for x, y in zip(P1 + B1, P2 + B2):
        assert torch.equal(x, y)


def test_mirrored_and_nd_steps_take_the_scale(muon):
    rng = np.random.default_rng(64)
    shape = (64, 16, 3, 4)
    mk = lambda: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()  # noqa: E731
    p, g, b = mk(), mk(), mk()
    q, c, far = p.clone(), b.clone(), torch.empty(64, 192, device="cuda")
    s = torch.tensor(0.3, device="cuda")
    muon.step([p], [g], [b], lr=0.1, reshape_nd=True, mirrors=[[far]], grad_scale=s)
    muon.step([q], [g * s], [c], lr=0.1, reshape_nd=True)
    assert torch.equal(p, q) and torch.equal(b, c) and torch.equal(far.view(shape), p)


def test_nan_scale_spoils_the_step_and_no_gradient(muon):
    rng = np.random.default_rng(65)
    g = _dev([rng.standard_normal((40, 40)).astype(np.float32)])[0]
    p, b = torch.ones_like(g), torch.zeros_like(g)
    keep = g.clone()
    muon.step([p], [g], [b], lr=0.1, grad_scale=torch.tensor(float("nan"), device="cuda"))
    assert bool(torch.isnan(p).all()) and bool(torch.isnan(b).all()) and torch.equal(g, keep)


def test_sharded_step_takes_the_scale(muon):
    """One process: the owned matrices are all of them."""
    from newton_schulz_norm_b200.sharded import ShardedMuon
    rng = np.random.default_rng(68)
    shapes = [(96, 64), (64, 200)]
    p, g = ([rng.standard_normal(x).astype(np.float32) for x in shapes] for _ in range(2))
    sm = ShardedMuon(shapes)
    for v, x in zip(sm.params, p):
        v.copy_(torch.from_numpy(x))
    G, P, B = _dev(g), _dev(p), [torch.zeros(x, device="cuda") for x in shapes]
    norm, scale = muon.clip_scale(G, 1.0)
    sm.step(G, lr=0.02, grad_scale=scale)
    muon.step(P, G, B, lr=0.02, grad_scale=scale)
    for a, b in zip(list(sm.params) + [sm.bufs[0], sm.bufs[1]], P + B):
        assert torch.equal(a, b)


def test_captured_step_reads_the_scale_anew(muon):
    wl = WORKLOADS["gpt2_block"]
    st = WorkloadStream(wl, seed=66)
    params, bufs = st.init()
    P1, B1, P2, B2 = _dev(params), _dev(bufs), _dev(params), _dev(bufs)
    G = _dev(st.next_grads())
    s = torch.tensor(0.5, device="cuda")
    graph = muon.capture_step(P1, G, B1, lr=wl.lr, grad_scale=s)
    muon.step(P2, G, B2, lr=wl.lr, grad_scale=s)
    for x in (0.25, 2.0):
        s.fill_(x)
        graph.replay()
        muon.step(P2, G, B2, lr=wl.lr, grad_scale=s)
    torch.cuda.synchronize()
    for a, b in zip(P1 + B1, P2 + B2):
        assert torch.equal(a, b)
    del graph


# ---------------------------------------------------------------- together, as a training loop calls them

def test_a_clipped_training_step_against_the_oracle(muon):
    """One norm over the Muon and the AdamW gradients, one scale into both
    steps, three steps, each from the oracle's state."""
    wl, aw = WORKLOADS["gpt2_block"], ADAMW_WORKLOADS["adamw_ragged"]
    st, ast = WorkloadStream(wl, seed=70), AdamWStream(aw, seed=71)
    p, b = st.init()
    q, u, v = ast.init()
    decay = [t.decay for t in aw.tensors]
    P, B, Q, UU, V = (_dev(x) for x in (p, b, q, u, v))
    G = [torch.empty_like(x) for x in P]
    H = [torch.empty_like(x) for x in Q]
    clip = muon.GradGroup(G + H)
    adamw = muon.AdamWGroup(Q, H, UU, V, lr=aw.lr, betas=(aw.beta1, aw.beta2), eps=aw.eps,
                            weight_decay=aw.weight_decay, decay=decay)
    for k in range(3):
        g, h = st.next_grads(), ast.next_grads()
        for d, x in zip(G + H, g + h):
            d.copy_(torch.from_numpy(x))
        norm, scale = clip.clip_scale(1.0)
        muon.step(P, G, B, lr=wl.lr, grad_scale=scale)
        adamw.step(aw.step + k, grad_scale=scale)
        torch.cuda.synchronize()
        want, _ = _norm_ok(norm, G + H, 2.0)
        s = _scale64(want, 1.0, 1e-6)
        g64 = [x.astype(np.float64) * s for x in g]
        h64 = [x.astype(np.float64) * s for x in h]
        p_old = p
        # the plain step's bounds, doubled for the roundings of s and of s g
        bounds = [_bounds(q[i], h64[i], u[i], v[i], aw.step + k, aw.lr, aw.beta1, aw.beta2, aw.eps,
                          aw.weight_decay if decay[i] else 0.0) for i in range(len(q))]
        p, b = muon_step_ref(p, [x.astype(np.float32) for x in g64], b, lr=wl.lr, beta=wl.beta,
                             nesterov=wl.nesterov, ns_steps=wl.ns_steps)
        q, u, v = adamw_step_ref(q, h64, u, v, aw.step + k, aw.lr, aw.beta1, aw.beta2, aw.eps,
                                 aw.weight_decay, decay)
        for i in range(len(P)):
            assert rel_fro(P[i].cpu().numpy() - p_old[i], p[i].astype(np.float64) - p_old[i]) <= (1e-2 if k == 0 else 2e-2)
            assert np.max(np.abs(B[i].cpu().numpy() - b[i])) <= 1e-6 * np.max(np.abs(b[i]))
        for i in range(len(Q)):
            for got, ref, bound in zip((Q[i], UU[i], V[i]), (q[i], u[i], v[i]), bounds[i]):
                assert np.all(np.abs(got.cpu().numpy() - ref.astype(np.float64)) <= 2 * bound)
        for d, x in zip(P + B + Q + UU + V, p + b + q + u + v):
            d.copy_(torch.from_numpy(x))


def test_a_captured_clipped_step_is_the_eager_one(muon):
    """bf16 gradients clipped into fp32 ones, both steps, in one graph."""
    wl, aw = WORKLOADS["gpt2_block"], ADAMW_WORKLOADS["adamw_ragged"]
    st, ast = WorkloadStream(wl, seed=72), AdamWStream(aw, seed=73)
    p, b = st.init()
    q, u, v = ast.init()
    rounds = [st.next_grads() + ast.next_grads() for _ in range(4)]

    def make():
        state = [_dev(x) for x in (p, b, q, u, v)]
        raw = [torch.empty(x.shape, dtype=torch.bfloat16, device="cuda") for x in state[0] + state[2]]
        f32 = [torch.empty(x.shape, device="cuda") for x in state[0] + state[2]]
        group = muon.GradGroup(raw, out=f32)
        n = len(p)
        adamw = muon.AdamWGroup(state[2], f32[n:], state[3], state[4], lr=aw.lr)

        def one():
            norm = group.clip(1.0)
            muon.step(state[0], f32[:n], state[1], lr=wl.lr)
            adamw.step(7)
            return norm

        return state, raw, one

    def load(raw, gs):
        for d, x in zip(raw, gs):
            d.copy_(torch.from_numpy(x))

    s1, raw1, one1 = make()
    s2, raw2, one2 = make()
    eager = []
    for gs in rounds:
        load(raw1, gs)
        eager.append(one1())
    load(raw2, rounds[0])
    assert torch.equal(one2(), eager[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = one2()
    for gs, want in zip(rounds[1:], eager[1:]):
        load(raw2, gs)
        graph.replay()
        assert torch.equal(norm, want)
    torch.cuda.synchronize()
    for x, y in zip(sum(s1, []), sum(s2, [])):
        assert torch.equal(x, y)
    del graph


def test_scaled_norm_and_cast_match_the_stage_oracle(muon):
    """momentum_ref and normalize_ref on scaled gradients, as the plain first
    kernel is checked: at most a bf16 step from the oracle's X0."""
    rng = np.random.default_rng(74)
    g = rng.standard_normal((200, 640)).astype(np.float32)
    b = (rng.standard_normal((200, 640)) * 0.1).astype(np.float32)
    s = np.float32(0.125)                                            # a power of two: s g is exact
    B = _dev([b])
    x = muon.momentum_normalize(_dev([g]), B, grad_scale=torch.tensor(s, device="cuda"))[0]
    new, u = momentum_ref(g * s, b, 0.95, True)
    want = orient(normalize_ref(u))[0]
    got = x.float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 1e-9)
    assert np.max(np.abs(B[0].cpu().numpy() - new)) <= 1e-6 * np.max(np.abs(new))


def test_profiler_counts_the_launches(muon):
    """One launch for a short list; the norm's two, or its first and the
    scaling, for a long one."""
    for n, norms, scales in ((100_000, 1, 1), (3_000_000, 3, 1)):
        g = torch.ones(n, device="cuda")
        group = muon.GradGroup([g], out=[torch.empty_like(g)])
        muon.profile_begin()
        group.norm()
        group.clip(1.0)
        prof = muon.profile_end()
        assert prof["grad_norm"][1] == norms and prof["grad_scale"][1] == scales


def test_around_the_border_of_the_two_forms(muon):
    """32 chunks of 32 KB: the longest list of one cluster, and one element more;
    32 and 33 small tensors, then the borders of the three sizes of table."""
    n = 32 * 8192
    for sizes in ([n], [n + 1], [n - 1], [n - 8192, 8192], [n - 8192, 8193], [5] * 32, [5] * 33, [5] * 64, [5] * 65,
                  [5] * 256, [5] * 257, [5] * 512, [5] * 513, [0] * 9 + [n], [0] * 600 + [n, n]):
        gs, bases = _grads(sizes, [torch.float32], seed=80)
        outs, obases = _grads(sizes, [torch.bfloat16], seed=81, offs=[8])
        for p in (1.0, 2.0, INF):
            _norm_ok(muon.grad_norm(gs, p), gs, p)
        _check_clip(muon, gs, 1.0, outs=outs)
        _check_clip(muon, gs, 1.0)
        _guards_hold(bases)
        _guards_hold(obases)
