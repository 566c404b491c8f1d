"""Argument checks of the sampling and top-logits entry points (CPU: every refusal comes before any
device call)."""
import ctypes

import pytest

hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
FAKE = 1 << 32   # device addresses are not touched by the checks


def refused(fn, *args):
    with pytest.raises(hm.HiMuonError) as e:
        fn(*args)
    assert e.value.status == -1 and str(e.value)


def sampling(**kw):
    f = dict(rows=4, vocab=1 << 12, ld_logits=1 << 12, logits=FAKE, uniform=FAKE, token=FAKE, logp=FAKE, kept=FAKE,
             dtype=hm.BF16, top_k=0, temperature=1.0, top_p=1.0, min_p=0.0)
    return hm.himuon_sampling(**(f | kw))


def top(**kw):
    f = dict(rows=4, vocab=1 << 12, ld_logits=1 << 12, ld_top=9, logits=FAKE, value=FAKE, index=FAKE, rest=FAKE, k=9,
             dtype=hm.F32, temperature=1.0)
    return hm.himuon_top(**(f | kw))


ROWS = [dict(rows=-1), dict(rows=1 << 41), dict(vocab=0), dict(vocab=(1 << 20) + 1, ld_logits=1 << 21), dict(ld_logits=4095),
        dict(ld_logits=1 << 41), dict(dtype=2), dict(temperature=-1.0), dict(temperature=float("nan")),
        dict(temperature=2.0 ** -21), dict(temperature=2.0 ** 21)]


@pytest.mark.parametrize("kw", ROWS + [dict(top_p=float("nan")), dict(min_p=float("nan"))])
def test_sample_refuses(kw):
    refused(hm.himuon_sample_workspace, sampling(**kw))
    refused(hm.himuon_sample, sampling(**kw), FAKE, 1 << 30, 0)


@pytest.mark.parametrize("kw", ROWS + [dict(temperature=0.0), dict(k=0), dict(k=1025, ld_top=1025), dict(vocab=8, k=9),
                                       dict(ld_top=8), dict(ld_top=1 << 41)])
def test_top_refuses(kw):
    refused(hm.himuon_top_workspace, top(**kw))
    refused(hm.himuon_top_logits, top(**kw), FAKE, 1 << 30, 0)


@pytest.mark.parametrize("name", ["logits", "uniform", "token", "logp", "kept"])
def test_sample_refuses_null(name):
    refused(hm.himuon_sample, sampling(**{name: None}), FAKE, 1 << 30, 0)


@pytest.mark.parametrize("name", ["logits", "value", "index", "rest"])
def test_top_refuses_null(name):
    refused(hm.himuon_top_logits, top(**{name: None}), FAKE, 1 << 30, 0)


@pytest.mark.parametrize("query,call,args", [(hm.himuon_sample_workspace, hm.himuon_sample, sampling()),
                                             (hm.himuon_top_workspace, hm.himuon_top_logits, top())])
def test_a_short_or_misaligned_workspace_is_refused(query, call, args):
    n = query(args)
    if n:   # (without a need there is nothing to refuse)
        refused(call, args, FAKE, n - 1, 0)
        refused(call, args, FAKE + 4, n, 0)
        refused(call, args, 0, n, 0)


def test_nothing_to_do():
    hm.himuon_sample(sampling(rows=0, logits=None, uniform=None, token=None, logp=None, kept=None), 0, 0, 0)
    hm.himuon_top_logits(top(rows=0, logits=None, value=None, index=None, rest=None), 0, 0, 0)


def test_structures_have_the_headers_sizes():
    """The layouts that the C header declares on this ABI (natural alignment)."""
    assert ctypes.sizeof(hm.himuon_sampling) == 3 * 8 + 9 * 8 + 2 * 4 + 3 * 8
    assert ctypes.sizeof(hm.himuon_top) == 4 * 8 + 4 * 8 + 2 * 4 + 8


def test_wrappers_refuse_host_tensors():
    import torch
    from tiled_newton_schulz_tile_amd.distill import top_logits
    from tiled_newton_schulz_tile_amd.sampling import sample
    with pytest.raises(ValueError):
        sample(torch.zeros(2, 4), torch.zeros(2))
    with pytest.raises(ValueError):
        top_logits(torch.zeros(2, 4), 1)
