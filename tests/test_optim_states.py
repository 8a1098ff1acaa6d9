"""optim.AdamW.load_state on the host (no GPU needed: the library is a stand-in)."""
import pytest

torch = pytest.importorskip("torch")

from test_optim_outputs import library, make  # noqa: E402, F401


def params(kinds=("bf16", "fp32", "bf16")):
    types = {"bf16": torch.bfloat16, "fp32": torch.float32}
    gen = torch.Generator().manual_seed(1)
    return [torch.randn(3, 4 + i, generator=gen).to(types[k]) for i, k in enumerate(kinds)]


def content(opt):
    return [t.clone() for t in [opt.m, opt.v, *opt.params, *(w for w in opt.master if w is not None)]]


def trained(library, **kw):
    """An optimiser that looks as after some steps."""
    opt = make(library, params(), **kw)
    gen = torch.Generator().manual_seed(2)
    for t in (opt.m, opt.v):
        t.copy_(torch.rand(t.shape, generator=gen))
    for p, w in zip(opt.params, opt.master):
        if w is not None:
            w.copy_(torch.randn(w.shape, generator=gen))
            p.copy_(w)
    return opt


@pytest.mark.parametrize("state", ["full", "8bit"])
def test_master_weights_come_with_the_states(library, state):  # noqa: F811
    old, new = trained(library, master=True, state=state), make(library, params(), master=True, state=state)
    new.load_state(old.state_dict())
    for a, b in zip(content(old), content(new)):
        assert torch.equal(a.float(), b.float())
    for p, w in zip(new.params, new.master):
        assert w is None or torch.equal(p, w.to(p.dtype))
    assert library.calls[-1][0] == "qml_opt_set_step"


def test_a_state_that_does_not_fit_is_refused_and_changes_nothing(library):  # noqa: F811
    saved = trained(library, master=True).state_dict()
    w = saved["master"]
    new = make(library, params(), master=True)
    before = content(new)
    for bad in (dict(master=w[:2]), dict(master=[w[0], None, None]), dict(master=[w[0], w[0], w[2]]),
                dict(master=[w[0][:1, :1], None, w[2]]), dict(master=[w[0], None, w[2].double()]),
                dict(master=[w[0], None, torch.zeros(4, 4)]), dict(m=saved["m"][:256]), dict(v=saved["v"].double()),
                dict(m_scale=torch.zeros(3)), dict(step=-1),
                dict(master=make(library, params()).state_dict()["master"])):  # of a handle without master weights
        with pytest.raises(ValueError):
            new.load_state(saved | bad)
        assert all(torch.equal(a, b) for a, b in zip(before, content(new))), bad
    with pytest.raises(ValueError):
        make(library, params()).load_state(saved)  # master weights for a handle without
    new.load_state({k: saved[k] for k in ("step", "m", "v")})  # the states alone
    assert torch.equal(new.m, saved["m"]) and all(torch.equal(a, b) for a, b in zip(before[2:], content(new)[2:]))


def test_parameters_that_require_gradients_take_loaded_weights(library):  # noqa: F811
    old = trained(library, master=True)
    new = make(library, [p.requires_grad_() for p in params()], master=[None, None, torch.zeros(3, 6)])
    saved = old.state_dict()
    saved["master"][0] = None
    new.load_state(saved)
    assert torch.equal(new.params[2], saved["master"][2].to(torch.bfloat16))
