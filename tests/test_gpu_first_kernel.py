"""The first kernel (momentum, norm, bf16 cast) at entries and shapes where its
paths differ: rows that are 16-byte aligned or not, whole tiles and ragged ones.

Tolerances: u is computed here in the kernel's own fp32 operations; the norm is
a sum of fp64 squares (or of four fp32 ones, 2^-22 of the sum at most, where
those stay in fp32), and X0 is rounded once to bf16: half a step, 2^-8 of the
value, and the norm's error beside it.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8
NORM_ERR = 2.0 ** -22


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


def _x0_ok(x0, u):
    u64 = u.double().cpu().numpy()
    want = u64 / (np.sqrt(np.sum(u64 * u64)) + 1e-7)
    if want.shape[0] > want.shape[1]:
        want = want.T
    got = x0.double().cpu().numpy()
    assert got.shape == want.shape
    # below bf16's smallest normal a rounding is half the smallest subnormal
    bound = (HALF_STEP + 2 * NORM_ERR) * np.abs(want) + 2.0 ** -134
    assert bool((np.abs(got - want) <= bound).all())


def _wide(shape, low, high, seed):
    """Signs and magnitudes between 10^low and 10^high."""
    rng = np.random.default_rng(seed)
    x = rng.choice([-1.0, 1.0], shape) * 10.0 ** rng.uniform(low, high, shape)
    return torch.from_numpy(x.astype(np.float32)).cuda()


@pytest.mark.parametrize("c", [64, 68, 67])
@pytest.mark.parametrize("r", [64, 70, 3])
def test_entries_whose_squares_leave_fp32(muon, r, c):
    """The norm of finite entries is finite, wherever the row boundaries lie."""
    for low, high in ((20.0, 20.0), (15.0, 37.0), (18.5, 19.5)):
        g = _wide((r, c), low, high, seed=r * c)
        buf = torch.zeros_like(g)
        (x0,) = muon.momentum_normalize([g], [buf], beta=0.5, nesterov=False)
        assert torch.equal(buf, g)
        _x0_ok(x0, g)
        out = muon.orthogonalize(g, ns_steps=0)
        _x0_ok(out if r <= c else out.t(), g)
        ld = (max(r, c) + 7) // 8 * 8
        raw = torch.zeros((min(r, c), ld), dtype=torch.bfloat16, device="cuda")
        buf2 = torch.zeros_like(g)
        assert muon.momentum_normalize_noalloc([g], [buf2], [raw], beta=0.5, nesterov=False) == 0
        assert torch.equal(raw[:, :max(r, c)], x0) and torch.equal(buf2, g)


@pytest.mark.parametrize("c", [64, 68, 67])
def test_an_infinite_entry_is_not_hidden(muon, c):
    g = torch.ones((64, c), device="cuda")
    g[5, 7] = float("-inf")
    (x0,) = muon.momentum_normalize([g], [torch.zeros_like(g)], nesterov=False)
    bad = torch.isnan(x0)
    assert bool(bad[5, 7]) and int(bad.sum()) == 1 and int((x0[~bad] != 0).sum()) == 0


SHAPES = [(1, 4), (4, 1), (3, 60), (60, 3), (64, 60), (65, 64), (64, 68), (63, 100), (100, 63), (130, 132),
          (1000, 100), (100, 1000), (256, 60), (20, 1004), (129, 127), (67, 65)]


@pytest.mark.parametrize("rule", ["plain", "momentum", "nesterov"])
def test_every_kind_of_tile(muon, rule):
    """Whole tiles, edge tiles of aligned rows, and unaligned rows, each stored
    as it is or transposed; nothing beside the matrices is written."""
    rng = np.random.default_rng(5)
    gs, bufs, bases = [], [], []
    for r, c in SHAPES:
        gs.append(torch.from_numpy(rng.standard_normal((r, c)).astype(np.float32)).cuda())
        base = torch.full((r * c + 64,), 7.0, device="cuda")
        bases.append(base)
        bufs.append(base[32:32 + r * c].view(r, c))
        bufs[-1].copy_(torch.from_numpy(rng.standard_normal((r, c)).astype(np.float32)))
    old = [b.double() for b in bufs]
    if rule == "plain":
        outs = [muon.orthogonalize(g, ns_steps=0) for g in gs]
        for g, o in zip(gs, outs):
            _x0_ok(o if g.shape[0] <= g.shape[1] else o.t(), g)
        return
    x0s = muon.momentum_normalize(gs, bufs, beta=0.5, nesterov=rule == "nesterov")
    for g, b, o, base, x0 in zip(gs, bufs, old, bases, x0s):
        # half of an fp32 number plus another is exact in fp64: one rounding
        assert torch.equal(b, (0.5 * o + g.double()).float())
        assert bool((base[:32] == 7.0).all()) and bool((base[32 + b.numel():] == 7.0).all())
        _x0_ok(x0, (0.5 * b.double() + g.double()).float() if rule == "nesterov" else b)


def test_edge_tiles_of_aligned_rows_keep_their_vectors(muon):
    """200000 x 60 has no whole tile, 200000 x 64 nothing else.  With vectors in
    both, the first has 0.94 of the bytes and takes the same time; with single
    elements it takes 1.35 of it."""
    sets = {c: [[torch.randn(200000, c, device="cuda") for _ in range(2)] for _ in range(2)] for c in (60, 64)}

    def once(c):
        muon.profile_begin()
        for i in range(10):
            g, b = sets[c][i % 2]
            muon.momentum_normalize([g], [b])
        ms, n = muon.profile_end()["momentum_norm_cast"]
        assert n == 10
        return ms

    once(60), once(64)
    ratios = sorted(once(60) / once(64) for _ in range(9))
    assert ratios[4] < 1.2, ratios
