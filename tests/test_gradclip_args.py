"""Gradient norm and clipping: what the C entry points and the binding refuse
before any GPU work, and the host-side rules (no GPU needed)."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
INF = float("inf")


@pytest.fixture(scope="module")
def muon():
    from newton_schulz_norm_b200 import build
    build.build()
    import newton_schulz_norm_b200 as m
    m.library()
    return m


def _args(n=1, ptr=64, dtype=0, numel=10):
    return ((P * max(n, 1))(*[P(ptr)] * max(n, 1)), (ctypes.c_ubyte * max(n, 1))(*[dtype] * max(n, 1)),
            (ctypes.c_int64 * max(n, 1))(*[numel] * max(n, 1)))


def _norm(lib, args=None, n=1, p=2.0, max_norm=1.0, eps=1e-6, norm=64, scale=None, work=64, bytes_=1 << 20):
    g, t, ne = args or _args()
    return lib.muon_grad_norm(g, t, ne, n, p, max_norm, eps, P(norm), P(scale), P(work), bytes_, None)


def _clip(lib, args=None, outs=None, out_types=None, n=1, **kw):
    g, t, ne = args or _args()
    o = (P * 1)(P(128)) if outs is None else outs
    ot = (ctypes.c_ubyte * 1)(0) if out_types is None else out_types
    return lib.muon_clip_grads(g, t, ne, n, o, ot, kw.get("p", 2.0), kw.get("max_norm", 1.0),
                               kw.get("eps", 1e-6), P(64), None, P(64), kw.get("bytes_", 1 << 20), None)


@pytest.mark.parametrize("call", [_norm, _clip])
def test_refusals_of_the_c_entry_points(muon, call):
    lib = muon.library()
    assert call(lib, n=-1) == -1
    assert call(lib, p=3.0) == -1 and call(lib, p=0.0) == -1 and call(lib, p=float("nan")) == -1
    assert call(lib, p=-INF) == -1
    assert call(lib, max_norm=-1.0) == -1 and call(lib, max_norm=float("nan")) == -1
    assert call(lib, eps=-1e-6) == -1 and call(lib, eps=INF) == -1 and call(lib, eps=float("nan")) == -1
    assert call(lib, args=_args(dtype=3)) == -1
    assert call(lib, args=_args(numel=-1)) == -1
    assert call(lib, args=_args(numel=(1 << 40) + 1)) == -1
    assert call(lib, args=_args(ptr=None)) == -1
    assert call(lib, args=_args(ptr=66)) == -2                       # not a float address
    assert call(lib, args=_args(ptr=65, dtype=1)) == -2              # not a bf16 address
    assert call(lib, args=_args(numel=1 << 20), bytes_=8) == -1      # workspace too small
    g, t, ne = _args()
    assert lib.muon_grad_norm(None, t, ne, 1, 2.0, 1.0, 0.0, P(64), None, P(64), 1 << 20, None) == -1
    assert lib.muon_grad_norm(g, None, ne, 1, 2.0, 1.0, 0.0, P(64), None, P(64), 1 << 20, None) == -1
    assert lib.muon_grad_norm(g, t, None, 1, 2.0, 1.0, 0.0, P(64), None, P(64), 1 << 20, None) == -1


def test_refusals_of_results_and_outputs(muon):
    lib = muon.library()
    assert _norm(lib, norm=None) == -1 and _norm(lib, args=_args(numel=1 << 20), work=None) == -1
    assert _norm(lib, norm=66) == -2 and _norm(lib, scale=66) == -2 and _norm(lib, work=68) == -2
    assert _clip(lib, outs=(P * 1)(P(None))) == -1
    assert _clip(lib, outs=(P * 1)(P(130))) == -2
    assert _clip(lib, out_types=(ctypes.c_ubyte * 1)(7)) == -1
    assert _clip(lib, outs=(P * 1)(P(64)), out_types=(ctypes.c_ubyte * 1)(1)) == -1   # in place, another type


def test_refusals_of_the_scaled_steps(muon):
    lib = muon.library()
    arr = (P * 1)(P(16))
    sh = (ctypes.c_int64 * 2)(4, 8)
    ne = (ctypes.c_int64 * 1)(8)
    ld = (ctypes.c_int64 * 1)(8)
    assert lib.muon_step_scaled(arr, arr, arr, sh, 1, 0.1, 0.9, 1, 5, None, None, 0, P(66), None) == -2
    assert lib.muon_step_scaled(arr, arr, arr, sh, -1, 0.1, 0.9, 1, 5, None, None, 0, P(64), None) == -1
    assert lib.muon_step_scaled(None, None, None, None, 0, 0.1, 0.9, 1, 5, None, None, 0, P(64), None) == 0
    assert lib.muon_adamw_step_scaled(arr, arr, arr, arr, ne, None, 1, 1, 1e-3, 0.9, 0.999, 1e-8, 0.0,
                                      P(66), None) == -2
    assert lib.muon_adamw_step_scaled(arr, arr, arr, arr, ne, None, 1, 0, 1e-3, 0.9, 0.999, 1e-8, 0.0,
                                      P(64), None) == -1
    assert lib.muon_momentum_normalize_scaled(arr, arr, arr, ld, sh, 1, 0.9, 1, P(66), None) == -2
    assert lib.muon_momentum_normalize_scaled(None, None, None, None, None, 0, 0.9, 1, P(64), None) == 0


def test_workspace_bytes_counts_the_launches(muon):
    lib = muon.library()

    def ask(numels, dtypes=None):
        n = len(numels)
        t = (ctypes.c_ubyte * max(n, 1))(*(dtypes or [0] * n))
        return lib.muon_grad_workspace_bytes(t, (ctypes.c_int64 * max(n, 1))(*numels), n)

    one = ask([1 << 24])
    assert one > 0 and one % 8 == 0
    assert ask([]) == 0 and ask([0, 0]) == 0 and ask([10]) == 0      # one cluster needs none
    assert ask([7] * 32) == 0 and ask([7] * 33) == one
    assert ask([7] * 512) == one and ask([7] * 513) == 2 * one
    assert ask([0] * 100 + [7] * 512) == one                         # empty tensors take no place
    assert ask([1 << 40] * 9) == 2 * one                             # chunk count of one launch
    assert ask([-1]) == -1 and ask([5], [3]) == -1 and ask([(1 << 40) + 1]) == -1


def test_binding_refuses_tensors_off_the_gpu(muon):
    g = torch.zeros(8)
    for call in (lambda: muon.grad_norm([g]), lambda: muon.clip_scale([g], 1.0),
                 lambda: muon.clip_grads([g], 1.0), lambda: muon.GradGroup([g]),
                 lambda: muon.GradGroup(["no tensor"])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        muon.GradGroup([], out=[g])
    for bad in (1.0, g, torch.zeros(2)):
        with pytest.raises(ValueError):
            muon._scale_ptr(bad)


def test_which_outputs_may_be_written(muon):
    """The overlap rule, on host tensors: only their addresses count."""
    ok = muon.GradGroup._disjoint
    base = torch.zeros(64)
    a, b, c = base[:10], base[10:20], base[40:50]
    assert ok([a, b], [a, b])                                        # in place
    assert ok([a], [b]) and ok([a, b], [c, b])
    assert not ok([a, a], [a, a])                                    # one tensor twice
    assert not ok([a, b], [c, c])                                    # one output twice
    assert not ok([a, b], [base[5:15], c])                           # an output over another gradient
    assert not ok([a, b], [b, a])                                    # swapped
    assert not ok([a], [base[1:11]])                                 # shifted by one
    assert not ok([base[:32]], [base[8:24].view(torch.int32)])       # inside it
    assert ok([a, base[:0]], [a, base[3:3]])                         # empty ones never overlap
    assert not ok([a], [a.view(torch.int32)])                        # same place, another type
    big, inside = base[:40], base[4:6]
    assert not ok([inside, b], [big, c])
    assert not ok([base[60:], base[50:60], a], [big, base[50:60], a])     # a long one over a later one


def test_sharded_step_passes_the_scale_on():
    """ShardedMuon.step hands grad_scale to its step function, and only then."""
    from newton_schulz_norm_b200.sharded import ShardedMuon
    seen = []
    sm = ShardedMuon([(4, 8), (8, 4)], device="cpu", step_fn=lambda p, g, b, **kw: seen.append(kw))
    grads = [torch.zeros(4, 8), torch.zeros(8, 4)]
    scale = torch.tensor(0.5)
    sm.step(grads, lr=0.1, grad_scale=scale)
    sm.step(grads, lr=0.1)
    assert seen[0]["grad_scale"] is scale and "grad_scale" not in seen[1]


def test_another_device_than_the_current_one_is_refused(muon, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    muon._check_device(0, "grads")
    with pytest.raises(ValueError, match="cuda:1"):
        muon._check_device(1, "grads")

    class OnDevice1(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    t = torch.zeros(4, 4).as_subclass(OnDevice1)
    with pytest.raises(ValueError, match="cuda:1"):
        muon._check_mat(t, "grad")
    with pytest.raises(ValueError, match="cuda:1"):
        muon.step([t], [t], [t], 0.1)
    with pytest.raises(ValueError, match="cuda:1"):
        muon.momentum_normalize([t], [t])
    with pytest.raises(ValueError, match="cuda:1"):
        muon.adamw_step([t], [t], [t], [t], 1, 1e-3)
    with pytest.raises(ValueError, match="cuda:1"):
        muon.AdamWGroup([t], [t], [t], [t], lr=1e-3).step(1)
    with pytest.raises(ValueError, match="cuda:1"):
        muon._scale_ptr(torch.zeros(()).as_subclass(OnDevice1))
