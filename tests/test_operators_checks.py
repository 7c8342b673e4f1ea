"""Checks of the operators' arguments that keep a call from overwriting what it still reads, or from handing the GPU memory
that is not its own. They return before anything touches CUDA."""
import pytest

from adamw_hybrid_optimizer_gb300 import libmuon as L

A, B, C = 1 << 20, 1 << 21, 1 << 22     # three buffers that share nothing
BF, F = L.MUON_BF16, L.MUON_F32
D = 8


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def ln_fwd(x=A, xdt=F, ldx=D, y=B, ydt=F, ldy=D, N=4):
    return L.lib().layernorm_forward(x, xdt, ldx, None, None, F, y, ydt, ldy, None, None, N, D, 1e-5, None)


def ln_bwd(dy=A, ydt=F, lddy=D, x=B, xdt=F, ldx=D, dx=C, lddx=D, N=4):
    return L.lib().layernorm_backward(dy, ydt, lddy, x, xdt, ldx, None, F, A, A, dx, lddx, None, None, F, 0, N, D, None, 0,
                                      None)


def accepted(status):     # past the checks: the call ran, or found no GPU to run on
    return status in (L.MUON_ERR_CUDA, L.MUON_ERR_UNSUPPORTED_DEVICE)


def test_layernorm_in_place_needs_one_dtype_and_pitch():
    """A row written at another place than it was read from lies over rows that are still to be read."""
    assert ln_fwd(y=A, ydt=BF) == L.MUON_ERR_INVALID_ARG
    assert ln_fwd(y=A, xdt=BF) == L.MUON_ERR_INVALID_ARG
    assert ln_fwd(y=A, ldy=16) == L.MUON_ERR_INVALID_ARG
    assert ln_fwd(y=A, ldx=16) == L.MUON_ERR_INVALID_ARG
    assert ln_fwd(y=A, ydt=BF, N=1) == L.MUON_ERR_INVALID_ARG
    # dx in the place of dy, and of x
    assert ln_bwd(dx=A, ydt=BF) == L.MUON_ERR_INVALID_ARG
    assert ln_bwd(dx=A, xdt=BF) == L.MUON_ERR_INVALID_ARG
    assert ln_bwd(dx=A, lddx=16) == L.MUON_ERR_INVALID_ARG
    assert ln_bwd(dx=A, lddy=16) == L.MUON_ERR_INVALID_ARG
    assert ln_bwd(dx=B, lddx=16) == L.MUON_ERR_INVALID_ARG
    assert ln_bwd(dx=B, ldx=16) == L.MUON_ERR_INVALID_ARG


def test_layernorm_in_place_as_documented_is_no_error():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the calls would run")
    for st in (ln_fwd(y=A), ln_fwd(y=A, ldx=16, ldy=16), ln_fwd(y=A, xdt=BF, ydt=BF), ln_bwd(dx=A), ln_bwd(dx=B),
               ln_bwd(dx=A, lddx=16, lddy=16), ln_bwd(dx=B, lddx=16, ldx=16, ydt=BF), ln_bwd(dx=A, xdt=BF, ydt=BF),
               ln_fwd(y=A, ldy=16, N=1), ln_bwd(dx=A, lddx=16, N=1),       # a single row has no pitch
               ln_fwd(xdt=BF, ldy=16), ln_bwd(ydt=BF, lddx=16)):           # elsewhere: anything goes
        assert accepted(st)


def test_layernorm_without_rows_has_nothing_in_place():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the calls would run")
    assert accepted(ln_fwd(x=None, y=None, ydt=BF, N=0))
    assert accepted(ln_fwd(y=A, ydt=BF, N=0))


class OnDevice:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, *shape, dtype, is_cuda=True, contiguous=True, at=A):
        self.shape, self.dtype, self.is_cuda, self._contiguous, self._at = shape, dtype, is_cuda, contiguous, at

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return self._contiguous

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self._at


@pytest.fixture
def calls(monkeypatch):
    """Notes what would reach the library, and calls nothing."""
    class Recorder:
        def __init__(self):
            self.made = []

        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return getattr(real, name)
            return lambda *args: self.made.append((name, args)) or L.MUON_OK

    real, rec = L.lib(), Recorder()
    monkeypatch.setattr(L, "lib", lambda: rec)
    return rec.made


def backward_calls(ws, n=40, V=30):
    import torch
    f, i = torch.float32, torch.int64
    t = lambda *shape: OnDevice(*shape, dtype=f)  # noqa: E731
    return {"embedding_backward": lambda: L.embedding_backward(OnDevice(n, dtype=i), t(n, D), t(V, D), ws, stream=0),
            "layernorm_backward": lambda: L.layernorm_backward(t(n, D), t(n, D), t(D), t(n), t(n), t(n, D), t(D), t(D), ws,
                                                               stream=0)}


@pytest.mark.parametrize("name", ["embedding_backward", "layernorm_backward"])
def test_workspace_is_device_memory_without_gaps(calls, name):
    """The kernels write to it: an address of the host is not theirs, and an expanded tensor has fewer bytes than elements."""
    import torch
    u8 = torch.uint8
    for ws in (OnDevice(1 << 20, dtype=u8, is_cuda=False), OnDevice(1 << 20, dtype=u8, contiguous=False)):
        with pytest.raises(ValueError):
            backward_calls(ws)[name]()
    assert calls == []
    backward_calls(OnDevice(1 << 20, dtype=u8, at=C))[name]()
    backward_calls(OnDevice(1 << 18, dtype=torch.float32, at=C))[name]()
    for made, args in calls:
        assert made == name and (C, 1 << 20) in zip(args, args[1:])
    assert len(calls) == 2
    del calls[:]
    backward_calls(None)[name]()      # the call itself says whether it needs one
    assert (None, 0) in zip(calls[0][1], calls[0][1][1:])
