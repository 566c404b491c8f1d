"""Where himuon_sample's borders hang on more than ordinary rows show (MI355X only): logits so large that
their powers have no common scale, equal logits with borders that fall between two of them exactly, min_p near
one, and tokens too improbable to be taken."""
import math

import numpy as np
import pytest
import torch

from test_gpu_select import check_sample

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.sampling import sample  # noqa: E402

DEV = "cuda"
INF = float("inf")
# rows and tokens (fp32) for every number of waves a row, where the sweep's stretches have more than one turn
SIZES = [(3, 40003), (300, 9001), (1100, 9001), (2100, 9001), (4200, 9001)]


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def some_of(N):
    return sorted({0, 1, 2, N // 2, N - 2, N - 1})


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("least,most,T", [(1e13, 2e13, 1.0), ("min", -1e30, 1.0), (-2e13, -1e13, 1.0), (9e5, 1e6, 2.0 ** -20)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_huge_logits(N, V, least, most, T, dtype):
    """Two values further apart than any power reaches, the larger one at the row's end only: the smaller one has no
    probability, wherever it is read first."""
    _need_gpu()
    logits = torch.full((N, V), torch.finfo(dtype).min if least == "min" else least, dtype=dtype, device=DEV)
    logits[0::2, [V - 5, V - 2]] = most
    logits[1::2, V - 700:] = most
    uniform = torch.rand(N, generator=torch.Generator().manual_seed(V)).to(DEV)
    uniform[2] = 0.0
    for kw in (dict(), dict(top_p=0.9013), dict(top_k=5), dict(top_k=400), dict(min_p=0.1),
               dict(top_k=300, top_p=0.613, min_p=0.3)):
        kw = dict(temperature=T, **kw)
        got = sample(logits, uniform, **kw)
        some = some_of(N)
        assert check_sample(logits[some], uniform[some], [x[some] for x in got], **kw) == len(some)
        assert (got.token >= V - 700).all()


@pytest.mark.parametrize("N,V", [(3, 40960), (300, 9216), (1100, 9216), (2100, 9216), (4200, 9216), (4200, 512), (300, 512)])
@pytest.mark.parametrize("value,T", [(0.0, 1.0), (3.671875, 0.3), (-1e30, 1.0), (17.5, 1e4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_logits_part_exactly(N, V, value, T, dtype):
    """Of n equal logits, every sum of powers is a whole number: top_p keeps its share of them to the token, and a
    uniform on a border takes the token behind it.  A second row in four has masked tokens of no probability (-inf), a
    third one of so little (1e-130) that they do not move a sum in 64 bits, behind the equal ones."""
    _need_gpu()
    logits = torch.full((N, V), value, dtype=dtype, device=DEV)
    half = V // 2
    logits[1::4, :half] = -INF
    if value > -1e29:
        logits[2::4, half:] = value - 300 * T
    first, count = torch.zeros(N, dtype=torch.int64), torch.full((N,), V)
    first[1::4] = count[1::4] = half
    if value > -1e29:
        count[2::4] = half
    uniform = (torch.arange(N) * 37 % 128).float() / 128
    for kw, share in ((dict(), 1.0), (dict(top_p=0.5), 0.5), (dict(top_p=0.75), 0.75), (dict(top_k=half), None),
                      (dict(top_k=V // 4, top_p=0.5), None), (dict(min_p=1.0), 1.0), (dict(top_p=0.25, min_p=0.9), 0.25)):
        n = (count * share).long() if share else torch.full((N,), half if len(kw) == 1 else V // 8)
        got = sample(logits, uniform.to(DEV), temperature=T, **kw)
        want = first + (uniform.double() * n).long()
        assert torch.equal(got.token.cpu(), want), (kw, (got.token.cpu() != want).nonzero()[:3])
        assert torch.equal(got.kept.cpu(), (n.double() / count).float()), kw
        assert ((got.logp.cpu().double() + count.double().log()).abs() <= 2.0 ** -23 * count.double().log()).all()


@pytest.mark.parametrize("N,V", [(3, 100003), (3, 600), (300, 600), (4200, 600)])
@pytest.mark.parametrize("scale,min_p,T", [(1e-8, 0.99999999, 1.0), (2.5, 0.999992, 2.0 ** 20), (2.5, 1 - 1e-7, 2.0 ** 20),
                                           (2.5, 0.9999, 1e5), (1.0, 0.999, 2.0 ** -20), (1.0, 0.999, 1.0)])
def test_min_p_near_one(N, V, scale, min_p, T):
    """Edges a small part of T below a largest logit of 0 or near it."""
    _need_gpu()
    g = torch.Generator().manual_seed(V)
    z = torch.randn(N, V, generator=g) * scale
    z = torch.where(torch.arange(N)[:, None] % 2 == 0, z - z.amax(1, keepdim=True), z)
    logits, uniform = z.to(DEV), torch.rand(N, generator=g).to(DEV)
    got = sample(logits, uniform, temperature=T, min_p=min_p)
    some = some_of(N)
    assert check_sample(logits[some], uniform[some], [x[some] for x in got], temperature=T, min_p=min_p) == len(some)


@pytest.mark.parametrize("N", [1, 300, 4200])
@pytest.mark.parametrize("T", [2.0 ** -20, 1.0, 700.0, 2.0 ** 20])
def test_min_p_keeps_the_logit_at_its_edge(N, T):
    """The first fp32 number from T log(min_p) on is kept and the one below it is not, also with top_k."""
    _need_gpu()
    for min_p in (1 - 2.9e-8, 1 - 1e-6, 0.999, 0.9, 0.5, 0.3, 1e-3):
        edge = T * math.log(min_p)
        on = np.float32(edge)
        on = on if float(on) >= edge else np.nextafter(on, np.float32(0))
        below = np.nextafter(on, np.float32(-np.inf))
        z = torch.full((N, 500), -60 * T)
        z[:, 7], z[:, 100], z[:, 300] = 0.0, float(below), float(on)
        logits, uniform = z.to(DEV), torch.full((N,), 0.9, device=DEV)
        for more in (dict(), dict(top_k=40)):
            got = sample(logits, uniform, temperature=T, min_p=min_p, **more)
            p, q = math.exp(float(on) / T), math.exp(float(below) / T)
            token = 7 if float(np.float32(0.9)) * (1 + p) < 1 else 300   # (the first one's power is 1)
            assert (got.token == token).all(), (min_p, more)
            assert ((got.kept.double() - (1 + p) / (1 + p + q)).abs() <= 2.0 ** -21).all(), (min_p, more)


@pytest.mark.parametrize("N,V", [(3, 40003), (2100, 9001), (4200, 9001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_uniform_of_zero_takes_a_token_that_can_be_taken(N, V, dtype):
    """Not one of -inf, nor one of about 2^-1000 of the largest's probability, also where such ones are all that a wave
    reads at first."""
    _need_gpu()
    for far in (-700.0, -720.0, -740.0, -5000.0):
        logits = torch.full((N, V), far, dtype=dtype, device=DEV)
        logits[:, 0] = -INF
        logits[:, V - 300:] = 0.0
        logits[1::2, 5] = far + 12
        got = sample(logits, torch.zeros(N, device=DEV))
        assert (got.token == V - 300).all(), far
        assert ((got.logp + math.log(300)).abs() <= 2.0 ** -20).all() and (got.kept == 1).all()
