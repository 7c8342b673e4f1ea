"""The operators on more than one device of a process, without a GPU: the library's objects linked over a stand-in for the
CUDA runtime (tests/fake_cudart.cpp) that keeps function attributes per device, as the runtime does."""
import ctypes
import os
import subprocess

import pytest

from adamw_hybrid_optimizer_gb300 import _build
from adamw_hybrid_optimizer_gb300 import libmuon as L

FAKE = 1 << 20


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    _build.build()
    objs = [os.path.join(_build.BUILD, os.path.basename(s) + ".o") for s in _build._sources()]
    if not all(os.path.exists(o) and os.path.getmtime(o) >= os.path.getmtime(s)
               for o, s in zip(objs, _build._sources())):
        _build.build(force=True)
    here = os.path.dirname(os.path.abspath(__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    out = str(tmp_path_factory.mktemp("fake") / "libmuon_fake.so")
    # -Bsymbolic: the stand-in's functions, whatever runtime the process has loaded
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", cuda, os.path.join(here, "fake_cudart.cpp"), *objs,
                    "-Wl,-Bsymbolic", "-o", out], check=True)
    return out


@pytest.fixture
def fake(objects, tmp_path):
    """A copy of the library of its own, so that no other test has set anything on its devices."""
    path = str(tmp_path / "libmuon_fake.so")
    with open(objects, "rb") as src, open(path, "wb") as dst:
        dst.write(src.read())
    lib = ctypes.CDLL(path)
    for name, (res, args) in L.SIGNATURES.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


BF, F = L.MUON_BF16, L.MUON_F32


def embed_fwd(lib, D=1001, n=5000, V=900):
    return lib.embedding_forward(FAKE, L.MUON_I32, FAKE, F, D, FAKE, F, D, n, V, D, 1.0, None)


def embed_bwd(lib, n, D=768, V=900):
    nb = lib.embedding_workspace_bytes(n, V, D)
    return lib.embedding_backward(FAKE, L.MUON_I32, FAKE, BF, D, FAKE, F, D, n, V, D, 1.0, -1, 0, FAKE, nb, None)


def ln_fwd(lib, D, dt=BF, N=4000):
    return lib.layernorm_forward(FAKE, dt, D, FAKE, FAKE, dt, FAKE, dt, D, FAKE, FAKE, N, D, 1e-5, None)


def ln_bwd(lib, D, dt=BF, N=4000):
    nb = lib.layernorm_workspace_bytes(N, D)
    return lib.layernorm_backward(FAKE, dt, D, FAKE, dt, D, FAKE, dt, FAKE, FAKE, FAKE, D, FAKE, FAKE, F, 0, N, D, FAKE, nb,
                                  None)


def distill(lib, N=64, V=50304, K=16):
    return lib.distill_forward_backward(FAKE, BF, V, FAKE, L.MUON_I32, FAKE, BF, None, 1.0, FAKE, FAKE, FAKE, BF, V, N, V, K,
                                        1.0, None)


CALLS = {
    "lookup of odd rows": embed_fwd,
    "gradient, one block sorts": lambda lib: embed_bwd(lib, 500),
    "gradient, sixteen blocks sort": lambda lib: embed_bwd(lib, 100000),
    "gradient of odd rows": lambda lib: embed_bwd(lib, 100000, 771),
    "gradient, long sort": lambda lib: embed_bwd(lib, 200000),
    "layer norm": lambda lib: ln_fwd(lib, 4096),
    "layer norm, fp32": lambda lib: ln_fwd(lib, 4096, F),
    "layer norm, wide": lambda lib: ln_fwd(lib, 16384),
    "layer norm, odd": lambda lib: ln_fwd(lib, 8191),
    "layer norm gradients": lambda lib: ln_bwd(lib, 4096),
    "layer norm gradients, fp32": lambda lib: ln_bwd(lib, 4096, F),
    "layer norm gradients, wide": lambda lib: ln_bwd(lib, 16384),
    "layer norm gradients, odd": lambda lib: ln_bwd(lib, 771),
    "distillation": distill,
}


@pytest.mark.parametrize("name", CALLS)
def test_every_device_of_a_process(fake, name):
    for device in (0, 1, 0, 5, 1):
        fake.fake_use_device(device)
        before = fake.fake_launches()
        assert CALLS[name](fake) == L.MUON_OK, device
        assert fake.fake_launches() > before


@pytest.mark.parametrize("name", [n for n in CALLS if n not in ("distillation",)])
def test_a_failure_is_not_kept(fake, name):
    fake.fake_fail_attributes(1)
    assert CALLS[name](fake) == L.MUON_ERR_CUDA
    fake.fake_fail_attributes(0)
    assert CALLS[name](fake) == L.MUON_OK
    assert CALLS[name](fake) == L.MUON_OK
