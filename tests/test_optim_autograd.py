"""The step is an in-place change that autograd can see (no GPU needed: the library is a
stand-in)."""
import pytest

torch = pytest.importorskip("torch")

from test_optim_outputs import library, make  # noqa: E402, F401


@pytest.mark.parametrize("as_given", [lambda p: p, lambda p: p.detach(), lambda p: p.view(-1)])
def test_tensors_saved_before_a_step_are_stale(library, as_given):  # noqa: F811
    p = torch.ones(2, 3, requires_grad=True)
    opt = make(library, [as_given(p)])
    before = p._version
    y = (p * p).sum()
    opt.grad_norm([torch.ones(6)])
    assert p._version == before  # nothing changed
    opt.step([torch.ones(6)])
    assert p._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    (p * p).sum().backward()  # after the step, as ever


def test_master_weights_and_inference_tensors(library):  # noqa: F811
    w = torch.ones(3)
    opt = make(library, [torch.ones(3, dtype=torch.bfloat16)], master=[w])
    opt.step([torch.ones(3, dtype=torch.bfloat16)])
    assert w._version == 1
    with torch.inference_mode():
        p = torch.ones(3)
    make(library, [p]).step([torch.ones(3)])  # they keep no count
