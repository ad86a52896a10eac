"""recurrence() and its gradient: the states' gradient in the place of its
input."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from semi_ar_drafter_amd import binding, recurrence, recurrence_backward  # noqa: E402

import test_recurrence_gpu as forms  # noqa: E402
from layers import DEV, IDS, TYPES, say  # noqa: E402

KINDS = ["sigmoid", "decay"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def backward(x, gate, kind, offsets, h0, dh, dlast, states, dh0):
    """dspark_recurrence_backward itself, whose dh0 may be dlast: (dx, dgate)."""
    lib, (T, C), S = binding.load(), x.shape, len(dlast)
    dt = binding.DSPARK_BF16 if x.dtype == torch.bfloat16 else binding.DSPARK_F32
    k = binding.GATES[kind]
    need = binding._bytes("recurrence_backward", T, S, C, dt, k)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    dx, dg = torch.zeros_like(x), torch.zeros_like(gate)
    binding._check(lib.dspark_recurrence_backward(
        T, S, C, dt, k, offsets.data_ptr(), dh.data_ptr(), x.data_ptr(), gate.data_ptr(), h0.data_ptr(), dlast.data_ptr(),
        states.data_ptr(), dx.data_ptr(), dg.data_ptr(), dh0.data_ptr(), ws.data_ptr() if need else None, need,
        torch.cuda.current_stream().cuda_stream))
    return dx, dg


# sequences of two rows over the border of two blocks of 16: the first is one
# wave's last row, the second another wave's (or another tile's) first
ACROSS = [15, 2] + [62, 2] * 60 + [45]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths,C", [(ACROSS, 130), (ACROSS, 2050), ([17] * 40, 384), ([3, 0, 2000, 1, 900], 257),
                                       ([5] * 300, 130), ([1] * 33, 3)])
def test_gradient_of_the_states_in_place(lengths, C, kind, dtype):
    say(f"[case] states in place {len(lengths)} sequences C={C} {kind} {dtype}")
    x, gate, h0, offsets, dh, dlast = forms.inputs(lengths, C, dtype, kind)
    states = forms.kept(x.shape[0], C)
    recurrence(x, gate, kind, offsets=offsets, h0=h0, states=states)
    want = recurrence_backward(dh, x, gate, states, kind, offsets=offsets, h0=h0, dlast=dlast)
    p = forms.Plain(lengths, x, gate, kind, h0, dh, dlast) if C < 2000 else None
    for turn in range(3):
        place = dlast.clone()
        dx, dg = backward(x, gate, kind, offsets, h0, dh, place, states, place)
        assert torch.equal(place, want[2]) and torch.equal(dx, want[0]) and torch.equal(dg, want[1]), turn
    if p is not None:
        forms.within(place.cpu(), p.dh0, p.dh0_tol, "dh0")
