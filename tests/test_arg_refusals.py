"""What the binding refuses before it asks for a GPU (none is needed here)."""
import pytest
import torch


@pytest.fixture(scope="module")
def muon():
    from newton_schulz_norm_b200 import build
    build.build()
    import newton_schulz_norm_b200 as m
    m.library()
    return m


def _calls(muon, t):
    return {
        "step": lambda: muon.step([t], [t], [t], 0.1),
        "step nd": lambda: muon.step([t], [t], [t], 0.1, reshape_nd=True),
        "capture_step": lambda: muon.capture_step([t], [t], [t], 0.1),
        "adamw_step": lambda: muon.adamw_step([t], [t], [t], [t], 1, 1e-3),
        "AdamWGroup": lambda: muon.AdamWGroup([t], [t], [t], [t], lr=1e-3),
        "momentum_normalize": lambda: muon.momentum_normalize([t], [t]),
        "orthogonalize": lambda: muon.orthogonalize(t),
        "GradGroup": lambda: muon.GradGroup([t]),
    }


@pytest.mark.parametrize("call", list(_calls(None, None)))
def test_tensors_off_the_gpu_are_a_value_error(muon, call):
    """With a GPU and without one."""
    with pytest.raises(ValueError, match="CUDA tensor"):
        _calls(muon, torch.zeros(4, 4))[call]()
    for other in ("no tensor", None):
        if call != "step nd":      # that one asks for the rank first
            with pytest.raises(ValueError):
                _calls(muon, other)[call]()


def test_views_of_dicts_are_lists_too(muon, monkeypatch):
    """Whatever has a length and can be walked again (a dict's values)."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    class OnDevice0(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

    named = {k: torch.zeros(4, 4).as_subclass(OnDevice0) for k in "ab"}
    values = named.values()
    group = muon.AdamWGroup(values, values, values, values, lr=1e-3)
    assert group._n == 2 and [group._p[i] for i in range(2)] == [t.data_ptr() for t in values]
    off = {"a": torch.zeros(4, 4)}.values()
    for call in (lambda: muon.AdamWGroup(off, off, off, off, lr=1e-3), lambda: muon.step(off, off, off, 0.1),
                 lambda: muon.adamw_step(off, off, off, off, 1, 1e-3),
                 lambda: muon.momentum_normalize(off, off), lambda: muon.GradGroup(off)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_a_tensor_is_asked_few_things(muon, monkeypatch):
    """The checks of a long list take longer than its kernels: five questions
    about a vector, six about a matrix (its rank too), and two for the address and
    the length."""
    asked = {}

    class OnDevice0(torch.Tensor):
        def __getattribute__(self, name):
            if not name.startswith("_"):
                key = torch.Tensor.data_ptr(self)
                asked[key] = asked.get(key, 0) + 1
            return 0 if name == "device" else torch.Tensor.__getattribute__(self, name)

        def get_device(self):
            return 0

        is_cuda = True

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(muon, "library", lambda: Lib())
    monkeypatch.setattr(muon, "_stream_ptr", lambda stream: 0)
    lists = [[torch.zeros(4, 4).as_subclass(OnDevice0) for _ in range(3)] for _ in range(4)]
    muon.adamw_step(*lists, 1, 1e-3)
    counts = [[asked[torch.Tensor.data_ptr(t)] for t in ts[1:]] for ts in lists]
    assert max(counts[0]) <= 6 and max(max(c) for c in counts[1:]) <= 5, counts
    asked.clear()
    muon.step(*lists[:3], 0.1)
    counts = [[asked[torch.Tensor.data_ptr(t)] for t in ts[1:]] for ts in lists[:3]]
    assert max(max(c) for c in counts) <= 6, counts
