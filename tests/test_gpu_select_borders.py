"""Where himuon_sample's borders hang on more than ordinary rows show (MI355X only): logits so large that
their powers have no common scale."""
import pytest
import torch

from test_gpu_select import check_sample

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.sampling import sample  # noqa: E402

DEV = "cuda"
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
