"""Rules of the gradient scale at the ends of its range, in each form: one
cluster, two launches, several tables."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
LISTS = {"cluster": [5000], "two launches": [400000, 7], "tables": [300] * 700}


@pytest.fixture(scope="module")
def muon():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from newton_schulz_norm_b200 import build
    build.build()
    import newton_schulz_norm_b200 as m
    yield m
    assert m.status() == 0


@pytest.mark.parametrize("p", [1.0, 2.0, INF])
@pytest.mark.parametrize("sizes", list(LISTS.values()), ids=list(LISTS))
def test_an_infinite_bound(muon, sizes, p):
    """s = 1 for a finite and an infinite norm, NaN for a NaN one."""
    for bad, want in ((1.0, 1.0), (INF, 1.0), (-INF, 1.0), (NAN, NAN)):
        grads = [torch.full((n,), 0.5, device="cuda") for n in sizes]
        grads[-1][3] = bad
        before = [g.clone() for g in grads]
        norm, scale = muon.clip_scale(grads, INF, p)
        outs = [torch.full_like(g, 7.0) for g in grads]
        got = [muon.clip_grads(grads, INF, p, out=outs), muon.clip_grads(grads, INF, p)]
        for n in [norm, *got]:
            assert math.isnan(float(n)) if math.isnan(bad) else \
                (math.isinf(float(n)) if math.isinf(bad) else math.isfinite(float(n)))
        if math.isnan(want):
            assert math.isnan(float(scale))
            assert all(bool(torch.isnan(t).all()) for t in grads + outs)
        else:
            assert float(scale) == want
            assert all(torch.equal(t, b) for t, b in zip(grads + outs, before + before))
