"""Argument checks of the distillation entry points (CPU: every refusal comes before any device
call)."""
import ctypes

import pytest

hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
FAKE = 1 << 32   # device addresses are not touched by the checks


def refused(fn, *args):
    with pytest.raises(hm.HiMuonError) as e:
        fn(*args)
    assert e.value.status == -1 and str(e.value)


def distill(**kw):
    f = dict(rows=4, vocab=1 << 12, ld_logits=1 << 12, ld_dlogits=1 << 12, ld_top=5, logits=FAKE, dlogits=FAKE + (1 << 20),
             value=FAKE, index=FAKE, rest=FAKE, weight=FAKE, kl=FAKE, loss=FAKE, k=5, dtype=hm.F32, value_dtype=hm.BF16,
             temperature=1.0, grad_scale=1.0)
    return hm.himuon_distill(**(f | kw))


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 41), dict(vocab=0), dict(vocab=(1 << 20) + 1, ld_logits=1 << 21, ld_dlogits=1 << 21),
    dict(ld_logits=4095), dict(ld_dlogits=4095), dict(ld_top=4), dict(k=0), dict(k=-1), dict(k=1025, ld_top=2000),
    dict(dtype=5), dict(value_dtype=-1), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
    dict(temperature=2.0 ** 21), dict(grad_scale=float("inf")), dict(dlogits=FAKE, ld_dlogits=4097), dict(ld_logits=1 << 41),
    dict(ld_top=1 << 41)])
def test_distill_refuses(kw):
    refused(hm.himuon_distill_workspace, distill(**kw))
    refused(hm.himuon_distill_loss, distill(**kw), FAKE, 1 << 20, 0)


@pytest.mark.parametrize("name", ["logits", "value", "index", "weight", "kl", "loss"])
def test_distill_refuses_null(name):
    refused(hm.himuon_distill_loss, distill(**{name: None}), FAKE, 1 << 20, 0)


def test_distill_refuses_a_short_or_misaligned_workspace():
    few = distill(vocab=1 << 16, ld_logits=1 << 16, ld_dlogits=1 << 16)   # rows that are cut into spans
    n = hm.himuon_distill_workspace(few)
    assert n > 0 and hm.himuon_distill_workspace(distill(rows=1000)) == 0
    refused(hm.himuon_distill_loss, few, FAKE, n - 1, 0)
    refused(hm.himuon_distill_loss, few, FAKE + 4, n, 0)
    refused(hm.himuon_distill_loss, few, 0, n, 0)


def test_structure_has_the_headers_size():
    """The layout that the C header declares on this ABI (natural alignment)."""
    assert ctypes.sizeof(hm.himuon_distill) == 5 * 8 + 8 * 8 + 4 * 4 + 2 * 8


def test_wrapper_refuses_host_tensors():
    import torch
    from tiled_newton_schulz_tile_amd.distill import distill_loss
    with pytest.raises(ValueError):
        distill_loss(torch.zeros(2, 4), torch.zeros(2, 1), torch.zeros(2, 1, dtype=torch.int64), torch.zeros(2))
