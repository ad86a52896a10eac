"""Sums over rows that a gradient makes: values for which a lost share or a
careless order shows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import binding, norm_backward  # noqa: E402

from layers import DEV, U32, say, within  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,C", [(512, 1001), (333, 900), (500, 250), (512, 3000)])
def test_small_terms_behind_large_ones_of_few_rows(M, C):
    """Eight rows of 1, one for each thread of a channel, then rows of a little
    under half a step of 1, each of which is lost where it is added to a 1 by
    itself.  With four sums to each of eight threads or more, of which the joins
    are at most 2 and 12, that is M / 32 + 14 roundings at most."""
    say(f"[case] sums of {M} x {C}")
    dy = torch.full((M, C), 0.99 * 2.0 ** -24, device=DEV)
    dy[:8] = 1.0
    x = torch.ones((M, C), device=DEV)
    stat = torch.tensor([0.0, 1.0], device=DEV).expand(M, 2).contiguous()
    _, dw, db = norm_backward(dy, x, stat, kind="rms", need=("dweight", "dbias"))
    want = dy.double().sum(0)
    tol = (M / 32 + 14) * U32 * want
    within(dw, want, tol, "dweight")
    within(db, want, tol, "dbias")
