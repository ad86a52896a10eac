"""The projection's operators at the edges: values that are not finite, empty
batches, the tails of the activations, the largest sizes.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import binding, linear, linear_backward  # noqa: E402

DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def rand(seed, *shape, sd=1.0, dtype=torch.float32):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=DEV) * sd).to(dtype)


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_nan_passes_every_activation(act, dtype):
    """A row of x that holds NaN gives a row of NaN, forward and backward (dx
    of that row, and every weight gradient: its rows sum over all of them)."""
    for M, N, K in ((3, 40, 64), (40, 300, 200)):
        x, w, b = rand(1, M, K, dtype=dtype), rand(2, N, K, sd=0.1, dtype=dtype), rand(3, N, dtype=dtype)
        dy = rand(4, M, N, dtype=dtype)
        pre = torch.empty(M, N, device=DEV)
        clean = linear(x, w, bias=b, act=act)
        x[1, 5] = math.nan
        y = linear(x, w, bias=b, act=act, pre=pre)
        rest = [i for i in range(M) if i != 1]
        assert torch.isnan(y[1]).all() and torch.equal(y[rest], clean[rest])
        if act == "none":
            continue
        dx, dw, db = linear_backward(dy, x, w, act=act, pre=pre)
        assert torch.isnan(dx[1]).all() and torch.isfinite(dx[rest]).all()
        assert torch.isnan(dw).all() and torch.isnan(db).all()
