"""Calls of the training step's operators at the edges of what their documentation allows
(MI355X only): gradients in the place of the logits for many blocks a row."""
import pytest
import torch

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.policy import policy_loss  # noqa: E402

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def policy_inputs(N, V, dtype, seed, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    logits = (2.5 * rand(N, V + pad)).to(dtype)[:, :V]
    label = torch.randint(0, V, (N,), device=DEV, generator=g)
    label[:5] = torch.tensor([0, V - 1, V // 8 * 8 - 1, min(V - 1, V // 8 * 8), V // 2], device=DEV)
    lp = torch.log_softmax(logits.double(), 1).gather(1, label[:, None])[:, 0].float()
    weight = torch.rand(N, device=DEV, generator=g) + 0.1
    weight[::7] = 0
    return logits, (label, weight, rand(N), lp + 0.2 * rand(N), lp + 0.2 * rand(N))


@pytest.mark.parametrize("N,V", [(6, 150001), (64, 4099), (65, 50257), (100, 32003), (128, 16391), (128, 128256),
                                 (128, 150001)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_policy_few_rows_in_place_equal_their_own_buffer(N, V, dtype):
    """Rows that are cut into spans, as many blocks as the chip holds at once and more, labels in every place: a
    gradient written over the logits has the bits of one with a buffer of its own, and so have the terms and sums."""
    _need_gpu()
    logits, rest = policy_inputs(N, V, dtype, N + V, pad=3)
    kw = dict(clip=(0.2, 0.28), kl_coef=0.1, temperature=0.9)
    want = policy_loss(logits, *rest, **kw)
    z = logits.clone()
    got = policy_loss(z, *rest, dlogits=z, **kw)
    assert torch.equal(got.logp, want.logp) and torch.equal(got.stats, want.stats)
    assert torch.equal(z, want.dlogits)
