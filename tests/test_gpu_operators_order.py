"""The table gradient's sums, bit for bit, in the order that include/libmuon.h documents."""
import numpy as np
import pytest
import torch

from tests.gpu_common import DEV, build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return build_lib()


def added_in_the_documented_order(ids, dout, V):
    """dout's rows summed as include/libmuon.h says, in fp32."""
    n, D = dout.shape
    group = 16 if -(-n // 16) * -(-D // 256) <= 3648 else 32
    order = np.argsort(np.where((ids < 0) | (ids >= V), V, ids), kind="stable")
    keys = ids[order]
    out = np.zeros((V, D), np.float32)

    def add(rows):
        s = np.zeros(D, np.float32)
        for r in rows:
            s = s + r
        return s

    for v in range(V):
        at = np.flatnonzero(keys == v)
        if not len(at):
            continue
        a, b = int(at[0]), int(at[-1]) + 1
        first = a // group
        if b <= (first + 2) * group:
            out[v] = add(dout[order[a:b]])
            continue
        parts = [add(dout[order[max(a, c * group):min(b, (c + 1) * group)]]) for c in range(first, (b - 1) // group + 1)]
        out[v] = add([add(parts[w::8]) for w in range(8)])
    return out


@pytest.mark.parametrize("n,V,D", [(900, 5, 40), (4097, 9, 300), (3000, 700, 24), (16000, 30, 1030), (5000, 40, 771),
                                   (60000, 90, 260)])
def test_embedding_gradient_is_added_in_the_documented_order(L, n, V, D):
    """Bit for bit: groups of 16 and of 32 sorted positions, runs within one, over two, over many and over more than eight
    times eight of them, with ids that name no row behind them."""
    u = torch.rand(n, generator=torch.Generator().manual_seed(11))
    ids = (u * u * (V + 1)).long()                    # V itself names no row
    dout = torch.randn((n, D), generator=torch.Generator().manual_seed(12))
    g = torch.full((V, D), float("nan"), device=DEV)
    ws = torch.full((L.embedding_workspace_bytes(n, V, D),), 0xCD, dtype=torch.uint8, device=DEV)
    L.embedding_backward(ids.to(DEV), dout.to(DEV), g, ws)
    assert np.array_equal(g.cpu().numpy(), added_in_the_documented_order(ids.numpy(), dout.numpy(), V))
