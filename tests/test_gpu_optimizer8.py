"""HybridMuonAdamW with AdamW moments in 8 bits: the step is adamw8_step_grouped's, beside Muon and 32-bit groups; state size,
saving and resuming."""
import pytest
import torch

from tests.gpu_common import DEV, build_lib

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    return build_lib()


def model(seed, dt=BF):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s: (torch.randn(s, generator=gen) * 1e-2).to(dt).to(DEV)  # noqa: E731
    return [mk(192, 320), mk(320, 192)], [mk(1001, 96), mk(999, 96)], [mk(96), mk(97)]


def give_grads(groups, step):
    gen = torch.Generator().manual_seed(50 + step)
    for ps in groups:
        for p in ps:
            p.grad = (torch.randn(p.shape, generator=gen) * 1e-3).to(p.dtype).to(DEV)


def optimizer(groups, bits, **kw):
    from adamw_hybrid_optimizer_gb300 import HybridMuonAdamW
    hidden, big, small = groups
    return HybridMuonAdamW([{"params": hidden, "kind": "muon"},
                            {"params": big, "kind": "adamw", "lr": 1e-3, "state_bits": bits, **kw},
                            {"params": small, "kind": "adamw", "lr": 2e-3, "weight_decay": 0.0}])


def bits(t):
    return t.contiguous().view(torch.uint8)


def test_the_step_is_the_call_and_other_groups_are_as_without(L):
    a, b, c = model(0), model(0), model(0)
    oa, ob = optimizer(a, 8), optimizer(b, 32)
    codes = lambda p: torch.zeros(p.shape, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # noqa: E731
    own = [(codes(p), codes(p), torch.zeros(((p.numel() + 255) // 256, 2), device=DEV)) for p in c[1]]
    for step in (1, 2, 3):
        for g in (a, b, c):
            give_grads(g, step)
        oa.step()
        ob.step()
        hp = L.make_adamw_hparams(1e-3, 0.9, 0.95, 1e-8, 0.1, step)
        L.adamw8_step_grouped(L.make_adamw8_tensors([(p, p.grad, *s, hp) for p, s in zip(c[1], own)]))
    torch.cuda.synchronize()
    for p, q in zip(a[0] + a[2], b[0] + b[2]):
        assert torch.equal(p, q)
    for p, q, (m, r, s) in zip(a[1], c[1], own):
        assert torch.equal(p, q)
        st = oa.state[p]
        assert torch.equal(bits(st["exp_avg"]), bits(m)) and torch.equal(bits(st["exp_avg_sq"]), bits(r))
        assert torch.equal(st["scales"], s)
    # three steps from the same start stay near those with fp32 moments: every weight has moved by less than 3 lr (1 + wd)
    for p, q in zip(a[1], b[1]):
        assert (p.float() - q.float()).abs().max() <= 2 * 3 * 1e-3 * 1.1 + 2 ** -8 * p.float().abs().max()


def test_state_takes_two_bytes_and_a_sixteenth(L):
    groups = model(1)
    opt = optimizer(groups, 8)
    n = sum(p.numel() for p in groups[1])
    held = sum(t.numel() * t.element_size() for p in groups[1] for t in opt.state[p].values())
    assert 2 * n + n / 32 <= held <= 2 * n + n / 32 + 16 * len(groups[1])


@pytest.mark.parametrize("kw", [{}, {"master_weights": True}, {"is_adamw": False}])
def test_resume_is_bit_for_bit_the_uninterrupted_run(L, kw):
    whole, first = model(2), model(2)
    ow, of = optimizer(whole, 8, **kw), optimizer(first, 8, **kw)
    for step in (1, 2):
        give_grads(whole, step), give_grads(first, step)
        ow.step(), of.step()
    saved = of.state_dict()
    second = [[p.detach().clone() for p in ps] for ps in first]
    os = optimizer(second, 8, **kw)
    os.load_state_dict(saved)
    for step in (3, 4):
        give_grads(whole, step), give_grads(second, step)
        ow.step(), os.step()
    torch.cuda.synchronize()
    for ps, qs in zip(whole, second):
        for p, q in zip(ps, qs):
            assert torch.equal(p, q)
            for k in ow.state[p]:
                assert torch.equal(bits(ow.state[p][k]), bits(os.state[q][k]))


def test_refusals(L):
    from adamw_hybrid_optimizer_gb300 import HybridMuonAdamW
    groups = model(3)
    with pytest.raises(ValueError, match="state_bits"):
        optimizer(groups, 16)
    o8, o32 = optimizer(groups, 8), optimizer(groups, 32)
    for a, b in ((o8, o32), (o32, o8)):
        before = {k: v.clone() for k, v in a.state[groups[1][0]].items()}
        with pytest.raises(ValueError, match="8 bits"):
            a.load_state_dict(b.state_dict())
        for k, v in before.items():
            assert torch.equal(bits(v), bits(a.state[groups[1][0]][k]))
    with pytest.raises(ValueError):
        HybridMuonAdamW([{"params": [torch.zeros(8)], "kind": "adamw", "state_bits": 8}])


def test_only_8_bit_tensors(L):
    """No Muon group and no 32-bit tensor."""
    from adamw_hybrid_optimizer_gb300 import HybridMuonAdamW
    p = torch.ones(700, dtype=F, device=DEV)
    opt = HybridMuonAdamW([{"params": [p], "kind": "adamw", "lr": 0.5, "weight_decay": 0.0, "state_bits": 8}])
    p.grad = torch.full_like(p, 3.0)
    opt.step()
    torch.cuda.synchronize()
    # the first step is lr towards the gradient's sign
    assert (p - 0.5).abs().max() <= 1e-5
