"""adamw8_check_grouped without a GPU: what adamw8_step_grouped refuses, it refuses, and it takes what that takes."""
import pytest

from adamw_hybrid_optimizer_gb300 import libmuon as L
from tests.test_more_operators_host import BF, F, FAKE, NAN, _tensor, built  # noqa: F401


def check(*ts, n=None):
    arr = (L.adamw8_tensor * max(len(ts), 1))(*ts)
    return L.lib().adamw8_check_grouped(arr, len(ts) if n is None else n)


def test_it_takes_what_the_step_takes():
    for t in (_tensor(), _tensor(m=FAKE + 1, r=FAKE + 3), _tensor(pdt=F, gdt=F), _tensor(master=FAKE), _tensor(n=1)):
        assert check(t) == L.MUON_OK and check(_tensor(), t) == L.MUON_OK


def test_it_refuses_what_the_step_refuses():
    good = _tensor()
    assert L.lib().adamw8_check_grouped(None, 1) == L.MUON_ERR_INVALID_ARG
    assert check(good, n=0) == L.MUON_ERR_INVALID_ARG and check(good, n=(1 << 20) + 1) == L.MUON_ERR_INVALID_ARG
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(r=None), dict(scales=None), dict(hp=False), dict(n=0)):
        assert check(good, _tensor(**kw)) == L.MUON_ERR_INVALID_ARG, kw
    assert check(good, _tensor(n=1 << 41)) == L.MUON_ERR_SHAPE
    assert check(good, _tensor(pdt=2)) == L.MUON_ERR_DTYPE and check(good, _tensor(master=FAKE, pdt=F)) == L.MUON_ERR_DTYPE
    for kw in (dict(param=FAKE + 1), dict(grad=FAKE + 2, gdt=F), dict(scales=FAKE + 4), dict(master=FAKE + 2, pdt=BF)):
        assert check(good, _tensor(**kw)) == L.MUON_ERR_ALIGNMENT, kw
    for hp in ((1e-3, 1.0, 0.95, 1e-8, 0.1, 1), (1e-3, 0.9, 0.95, 1e-8, 0.1, 0), (NAN, 0.9, 0.95, 1e-8, 0.1, 1)):
        assert check(good, _tensor(hp=L.make_adamw_hparams(*hp))) == L.MUON_ERR_INVALID_ARG


def test_the_binding_raises(monkeypatch):
    arr = (L.adamw8_tensor * 2)(_tensor(), _tensor(n=0))
    arr.device = 0
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    with pytest.raises(L.MuonError):
        L.adamw8_check_grouped(arr)
    monkeypatch.setattr(L, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        L.adamw8_check_grouped(arr)


def test_the_binding_takes_an_array_that_the_caller_has_filled():
    """As adamw_step_grouped's does: not every array comes from make_adamw8_tensors."""
    L.adamw8_check_grouped((L.adamw8_tensor * 2)(_tensor(), _tensor(gdt=F)))
    with pytest.raises(L.MuonError):
        L.adamw8_step_grouped((L.adamw8_tensor * 1)(_tensor(n=0)), stream=0)
