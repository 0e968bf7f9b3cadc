"""What every call of the binding does on the host besides its own checks: the GPUs
are counted once a process, and a GPU that is not the only one is made current."""
import contextlib

import pytest
import torch

import __graft_entry__  # noqa: F401
import confidence_scheduled_ragged_amd as dspark
from test_forward_host import forward_args, on_gpu
from test_tree_host import calls, no_device, placed  # noqa: F401


def entries():
    """(entry, its tensors by name, other arguments) of all that go through one launch."""
    old = [(fn, {k: v for k, v in a.items() if isinstance(v, torch.Tensor)},
            {k: v for k, v in a.items() if not isinstance(v, torch.Tensor)})
           for fn, a in forward_args()[:2]]
    return old + calls()


@pytest.fixture
def counted(monkeypatch):
    """The calls of torch.cuda.device_count, which says 1 or what `counted` is told."""
    asked, gpus = [], [1]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: asked.append(1) or gpus[0])
    dspark._gpus.cache_clear()
    yield asked, gpus
    dspark._gpus.cache_clear()


def test_gpus_are_counted_once(no_device, counted):  # noqa: F811
    asked, _ = counted
    for _ in range(3):
        for fn, tensors, rest in entries():
            fn(**placed(tensors, lambda k, j: 0), **rest)
    assert len(no_device) == 3 * len(entries())
    assert len(asked) == 1


@pytest.mark.parametrize("i", range(len(entries())))
@pytest.mark.parametrize("gpu,gpus,current", [(0, 1, []), (0, 2, [0]), (1, 2, [1]), (3, 8, [3])])
def test_the_gpu_of_the_tensors_is_current(no_device, counted, monkeypatch, i, gpu, gpus,  # noqa: F811
                                           current):
    within = []

    @contextlib.contextmanager
    def device(index):
        within.append(index)
        yield
    monkeypatch.setattr(torch.cuda, "device", device)
    counted[1][0] = gpus
    fn, tensors, rest = entries()[i]
    fn(**placed(tensors, lambda k, j: gpu), **rest)
    assert within == current
    (name, args), = no_device
    assert name == fn.__name__ and args[-1] == 1000 + gpu


def test_a_workspace_is_cleared_on_its_own_gpu(no_device, counted, monkeypatch):  # noqa: F811
    within = []

    @contextlib.contextmanager
    def device(index):
        within.append(index)
        yield
    monkeypatch.setattr(torch.cuda, "device", device)
    dspark.dspark_workspace_init(on_gpu(torch.zeros(64, dtype=torch.uint8), 2))
    assert within == [2] and no_device[0][1][1:] == (64, 1002)
