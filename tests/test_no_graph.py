"""Operators that record nothing for autograd refuse what autograd would lose,
forward-mode tangents as well as gradients."""
import pytest

torch = pytest.importorskip("torch")

from torch.autograd import forward_ad  # noqa: E402

from semi_ar_drafter_amd import (binding, gated_linear, gated_linear_backward, linear, linear_backward,  # noqa: E402
                                 markov_loss, markov_loss_backward, norm, norm_backward, recurrence,
                                 recurrence_backward)


def test_gradients_and_tangents():
    x, y = torch.ones(3), torch.ones(3, requires_grad=True)
    binding._no_graph("f", x, None, x)
    with pytest.raises(RuntimeError, match="f.. records no graph"):
        binding._no_graph("f", x, y)
    with torch.no_grad():
        binding._no_graph("f", x, y)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones(3))
        binding._no_graph("f", x, None, x.clone())
        for mode in (torch.no_grad, torch.enable_grad):
            with mode(), pytest.raises(RuntimeError, match="f.. carries no tangents"):
                binding._no_graph("f", None, x, dual)
            with mode():
                binding._no_graph("f", dual.detach())
    binding._no_graph("f", x)


@pytest.mark.gpu
def test_every_operator_refuses_a_tangent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = "cuda:0"
    rand = lambda *sh: torch.randn(sh, device=dev)  # noqa: E731
    x, w, v, pre, pair = rand(6, 8), rand(8, 8), rand(8), rand(6, 8), rand(2, 6, 8)
    states, h0, stat, row = rand(1, 8), rand(1, 8), rand(6, 2), rand(6)
    label = torch.zeros(6, dtype=torch.int32, device=dev)
    calls = [(lambda a, b, c: linear(a, b, c), (x, w, v)),
             (lambda a, b, c, d: linear_backward(a, b, c, act="silu", pre=d), (x, x, w, pre)),
             (lambda a, b, c: norm(a, b, c), (x, v, v)),
             (lambda a, b: norm(a, residual=b), (x, x)),
             (lambda a, b, c, d, e: norm_backward(a, b, c, d, dsum=e), (x, x, stat, v, x)),
             (lambda a, b, c: recurrence(a, b, h0=c), (x, x, h0)),
             (lambda a, b, c, d, e, f: recurrence_backward(a, b, c, d, h0=e, dlast=f), (x, x, x, states, h0, h0)),
             (lambda a, b, c, d, e: gated_linear(a, b, c, d, e), (x, w, w, v, v)),
             (lambda a, b, c, d, e: gated_linear_backward(a, b, c, d, e), (x, x, w, w, pair)),
             (lambda a, b: markov_loss(label, h=a, Wo=b), (x, w)),
             (lambda a, b, c, d: markov_loss_backward(a, b, label, h=c, Wo=d, need=("dh",)), (row, row, x, w))]
    for call, args in calls:
        call(*args)
        with torch.no_grad(), forward_ad.dual_level():
            call(*args)
            for i, t in enumerate(args):
                some = list(args)
                some[i] = forward_ad.make_dual(t, torch.ones_like(t))
                with pytest.raises(RuntimeError, match="tangents"):
                    call(*some)
                some[i] = some[i].detach()
                call(*some)
    torch.cuda.synchronize()
