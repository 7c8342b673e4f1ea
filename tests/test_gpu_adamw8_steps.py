"""adamw8_step_grouped over many steps: what the held moments do as steps add up."""
import numpy as np
import pytest
import torch

from oracle import adamw8 as o8
from tests.gpu_common import DEV, build_lib, f64
from tests.test_gpu_adamw8 import HP, State, step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return build_lib()


@pytest.mark.parametrize("x", [1e-17, 1e-18, 1e-19, 3e-20, 2e-21])
@pytest.mark.parametrize("off", [0, 1])
def test_small_roots_decay(L, x, off):
    """One gradient of x and then none, with an eps below all roots. A block's largest root is held to fp32, so its square, v,
    follows beta2 v from step to step: an fma of relative 2e-6, and the last bit of fp32's subnormal numbers, 2^-149, once for
    the gradient's square (two roundings) and once for the sum. The others lie within half a step of a code. The weights then
    get m / r, off by half of v's relative error."""
    hp = dict(HP, eps=float(np.float32(1e-37)), weight_decay=0.0)
    st = State(700, "f32", "f32", zero=True, seed=3, off=off)
    st.g.copy_(torch.linspace(0.5, 1.0, st.n) * x)
    for t in range(1, 21):
        p0, g, m0, r0 = st.values()
        step(L, [st], t, hp=hp)
        p, m, r = o8.update(p0, g, m0, r0, t, **hp)
        got_p, _, _, got_r = st.values()
        err = 2e-6 + 2 * 2.0 ** -149 / r ** 2                         # of v
        for a in range(0, st.n, o8.BLOCK):
            own = slice(a, min(st.n, a + o8.BLOCK))
            i = a + int(np.argmax(r[own]))
            assert abs(got_r[i] ** 2 - r[i] ** 2) <= err[i] * r[i] ** 2
        assert np.all(got_r > 0)
        assert np.all(np.abs(got_r - r) <= r * (2.0 ** -4 * (1 + err) + err))
        assert np.all(np.abs(got_p - p) <= (2e-6 + err) * np.abs(p - p0) + 2.0 ** -23 * np.abs(p0))
        st.g.zero_()
