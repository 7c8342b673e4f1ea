"""HybridMuonAdamW with 8-bit moments: a refused step changes nothing, whichever group it is refused for."""
import pytest
import torch

from tests.gpu_common import DEV, build_lib
from tests.test_gpu_optimizer8 import bits, give_grads, model, optimizer

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    return build_lib()


def everything(opt):
    held = [p for g in opt.param_groups for p in g["params"]]
    return [bits(x).clone() for p in held for x in (p.detach(), *opt.state[p].values())]


@pytest.mark.parametrize("group,key,bad", [(1, "lr", NAN), (1, "eps", NAN), (1, "betas", (-0.5, 0.95)), (1, "betas", (0.9, 0.99)),
                                           (2, "lr", NAN), (2, "betas", (0.9, 1.0))])
def test_of_hyperparameters(L, group, key, bad):
    groups, other = model(4), model(4)
    opt, same = optimizer(groups, 8), optimizer(other, 8)
    for o, g in ((opt, groups), (same, other)):
        give_grads(g, 1)
        o.step()
    give_grads(groups, 2), give_grads(other, 2)
    before, steps = everything(opt), [g.get("step") for g in opt.param_groups]
    good = opt.param_groups[group][key]
    opt.param_groups[group][key] = bad
    with pytest.raises((ValueError, L.MuonError)):
        opt.step()
    torch.cuda.synchronize()
    assert steps == [g.get("step") for g in opt.param_groups]
    for x, y in zip(before, everything(opt)):
        assert torch.equal(x, y)
    opt.param_groups[group][key] = good           # and the step is then the one that it would have been
    opt.step(), same.step()
    torch.cuda.synchronize()
    for x, y in zip(everything(opt), everything(same)):
        assert torch.equal(x, y)


def test_of_an_empty_parameter(L):
    groups = model(5)
    groups[1].append(torch.empty((0, 96), dtype=torch.bfloat16, device=DEV))
    opt = optimizer(groups, 8)
    give_grads(groups, 1)
    before = everything(opt)
    with pytest.raises(L.MuonError):
        opt.step()
    torch.cuda.synchronize()
    for x, y in zip(before, everything(opt)):
        assert torch.equal(x, y)


def test_of_another_current_device(L, monkeypatch):
    groups = model(6)
    opt = optimizer(groups, 8)
    give_grads(groups, 1)
    before = everything(opt)
    monkeypatch.setattr(L, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        opt.step()
    torch.cuda.synchronize()
    for x, y in zip(before, everything(opt)):
        assert torch.equal(x, y)
