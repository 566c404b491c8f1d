"""Argument checks of the training-step entry points (CPU: every refusal comes before any
device call; nothing to do is no error)."""
import ctypes

import pytest

hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
FAKE = 1 << 32   # device addresses are not touched by the checks


def policy(**kw):
    f = dict(rows=4, vocab=10, ld_logits=10, ld_dlogits=10, logits=FAKE, dlogits=FAKE + 4096, label=FAKE, weight=FAKE,
             advantage=FAKE, old_logp=FAKE, ref_logp=FAKE, logp=FAKE, stats=FAKE, dtype=hm.F32, clip_low=0.2,
             clip_high=0.2, kl_coef=0.0, temperature=1.0, grad_scale=1.0)
    return hm.himuon_policy(**(f | kw))


def refused(fn, *args):
    with pytest.raises(hm.HiMuonError) as e:
        fn(*args)
    assert e.value.status == -1 and str(e.value)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 41), dict(vocab=0), dict(vocab=1 << 31), dict(ld_logits=9), dict(ld_dlogits=9),
    dict(dtype=5), dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_high=float("inf")), dict(clip_high=float("nan")),
    dict(kl_coef=float("inf")), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
    dict(grad_scale=float("nan")), dict(dlogits=FAKE, ld_dlogits=11)])
def test_policy_refuses(kw):
    refused(hm.himuon_policy_workspace, policy(**kw))
    refused(hm.himuon_policy_loss, policy(**kw), FAKE, 1 << 20, 0)


@pytest.mark.parametrize("name", ["logits", "label", "weight", "advantage", "logp", "stats"])
def test_policy_refuses_null(name):
    refused(hm.himuon_policy_loss, policy(**{name: None}), FAKE, 1 << 20, 0)


def test_policy_refuses_a_short_or_misaligned_workspace():
    n = hm.himuon_policy_workspace(policy())
    assert n > 0
    refused(hm.himuon_policy_loss, policy(), FAKE, n - 1, 0)
    refused(hm.himuon_policy_loss, policy(), FAKE + 4, n, 0)
    refused(hm.himuon_policy_loss, policy(), 0, n, 0)


def tensors(*kw):
    f = dict(n=8, weight=FAKE, grad=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE, weight_decay=0.0)
    return (hm.himuon_adamw_tensor * len(kw))(*(hm.himuon_adamw_tensor(**(f | k)) for k in kw))


def config(**kw):
    return hm.himuon_adamw_config(**(dict(weight_dtype=hm.F32, grad_dtype=hm.F32, state_bits=8, beta1=0.9, beta2=0.999,
                                          eps=1e-8) | kw))


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=1 << 41), dict(weight=None), dict(grad=None), dict(m=None), dict(v=None),
                                dict(m_scale=None), dict(v_scale=None), dict(weight_decay=float("nan"))])
def test_adamw_refuses_tensors(kw):
    refused(hm.himuon_adamw_step, tensors({}, kw), config(), 1, 0.1, 0, None, 0, 0)


@pytest.mark.parametrize("kw", [dict(weight_dtype=2), dict(grad_dtype=-1), dict(state_bits=16), dict(beta1=1.0),
                                dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=0.0), dict(eps=float("inf"))])
def test_adamw_refuses_configs(kw):
    refused(hm.himuon_adamw_step, tensors({}), config(**kw), 1, 0.1, 0, None, 0, 0)


def test_adamw_refuses_steps():
    refused(hm.himuon_adamw_step, tensors({}), config(), 0, 0.1, 0, None, 0, 0)
    refused(hm.himuon_adamw_step, tensors({}), config(), 1, float("inf"), 0, None, 0, 0)
    refused(hm.himuon_adamw_step, tensors(dict(n=1 << 40), dict(n=1)), config(), 1, 0.1, 0, None, 0, 0)


def test_adamw_nothing_to_do():
    hm.himuon_adamw_step(tensors(), config(), 1, 0.1, 0, None, 0, 0)
    hm.himuon_adamw_step(tensors(dict(n=0, weight=None, grad=None, m=None, v=None)), config(), 1, 0.1, 0, None, 0, 0)


def test_grad_norm_refuses():
    n = hm.himuon_grad_norm_workspace(3)
    assert n > 0 and hm.himuon_grad_norm_workspace(0) > 0
    refused(hm.himuon_grad_norm_workspace, -1)
    g = lambda *x: (hm.himuon_grad * len(x))(*(hm.himuon_grad(*y) for y in x))  # noqa: E731
    ok = g((4, FAKE))
    for args in [(g((-1, FAKE)), hm.F32, 1.0, FAKE, FAKE, n), (g((4, None)), hm.F32, 1.0, FAKE, FAKE, n),
                 (ok, 2, 1.0, FAKE, FAKE, n), (ok, hm.F32, -1.0, FAKE, FAKE, n), (ok, hm.F32, float("nan"), FAKE, FAKE, n),
                 (ok, hm.F32, 1.0, 0, FAKE, n), (ok, hm.F32, 1.0, FAKE, FAKE, 8), (ok, hm.F32, 1.0, FAKE, FAKE + 4, n),
                 (ok, hm.F32, 1.0, FAKE, 0, n), (g((1 << 40, FAKE), (1, FAKE)), hm.F32, 1.0, FAKE, FAKE, n)]:
        refused(hm.himuon_grad_norm, *args, 0)


def test_structures_have_the_headers_sizes():
    """The layouts that the C header declares on this ABI (natural alignment)."""
    assert ctypes.sizeof(hm.himuon_policy) == 4 * 8 + 9 * 8 + 8 + 5 * 8
    assert ctypes.sizeof(hm.himuon_grad) == 16
    assert ctypes.sizeof(hm.himuon_adamw_tensor) == 64
    assert ctypes.sizeof(hm.himuon_adamw_config) == 16 + 24


def test_adamw_table_refuses():
    many = tensors(*[{}] * 100)
    n = hm.himuon_adamw_table_size(many, config())
    assert n > 0 and hm.himuon_adamw_table_size(tensors({}), config()) == 0
    host = (ctypes.c_uint64 * (n // 8 + 1))()
    at = ctypes.addressof(host)
    hm.himuon_adamw_table(many, config(), at, n)
    refused(hm.himuon_adamw_table, many, config(), at, n - 1)
    refused(hm.himuon_adamw_table, many, config(), at + 4, n)
    refused(hm.himuon_adamw_table, many, config(), 0, n)
    refused(hm.himuon_adamw_table, tensors(dict(m=None)), config(), at, n)
    refused(hm.himuon_adamw_table_size, tensors(dict(n=-1)), config())
    refused(hm.himuon_adamw_step, many, config(), 1, 0.1, 0, None, FAKE + 8, 0)


def test_wrappers_refuse_host_tensors():
    import torch
    from tiled_newton_schulz_tile_amd.adamw import AdamW, GradNorm, adamw_state
    from tiled_newton_schulz_tile_amd.optim import AdamWOptimizer
    from tiled_newton_schulz_tile_amd.policy import policy_loss
    x = torch.zeros(8)
    for call in (lambda: AdamW([(x, x, *adamw_state(x))]), lambda: GradNorm([x]), lambda: AdamW([]), lambda: GradNorm([]),
                 lambda: AdamWOptimizer([torch.nn.Parameter(x)]),
                 lambda: policy_loss(torch.zeros(2, 4), torch.zeros(2, dtype=torch.int64), x[:2], x[:2])):
        with pytest.raises(ValueError):
            call()


def test_adamw_moments_decode_the_8_bit_states():
    import torch
    from oracle import training
    from tiled_newton_schulz_tile_amd.adamw import adamw_moments, adamw_state
    m, r, ms, rs = adamw_state(torch.zeros(300, 2), 8)
    assert m.dtype == torch.float8_e4m3fn and m.shape == (300, 2) and ms.numel() == 3
    g = torch.Generator().manual_seed(0)
    code = torch.randint(0, 127, (600,), generator=g).to(torch.uint8)
    m.view(torch.uint8).view(-1).copy_(code)
    r.view(torch.uint8).view(-1).copy_(code.flip(0))
    ms.copy_(torch.rand(3, generator=g))
    rs.copy_(torch.rand(3, generator=g))
    got = adamw_moments((m, r, ms, rs))
    for x, c, s, square in ((got[0], code, ms, False), (got[1], code.flip(0), rs, True)):
        want = training.unpack8(c.numpy(), s.double().numpy())
        want = torch.from_numpy(want ** 2 if square else want).view(300, 2)
        assert torch.allclose(x.double(), want, rtol=2.0 ** -22, atol=0)
