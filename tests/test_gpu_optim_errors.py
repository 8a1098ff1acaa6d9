"""What the optimiser's and the 8-bit slots' entry points return when something else has
failed before them on the host."""
import contextlib
import ctypes

import pytest

from test_gpu_optim import bits, make, optim, qml, same

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def an_error_left_behind():
    """The runtime as another caller's failed call leaves it: no such device."""
    runtime = ctypes.CDLL("libcudart.so.12")
    assert runtime.cudaSetDevice(99) == 101
    try:
        yield
    finally:
        runtime.cudaGetLastError()


@pytest.mark.parametrize("sizes", [[300], [70_000, 300], [3] * 500])
@pytest.mark.parametrize("state", ["full", "8bit"])
def test_an_error_of_someone_else_is_not_the_steps(sizes, state):
    runs = []
    for left in (False, True):
        params, grads = make(sizes, "fp32", "fp32", 50)
        opt = optim().AdamW(params, state=state)
        for call in (lambda: opt.step(grads), lambda: opt.step(grads, max_norm=1.0), lambda: opt.grad_norm(grads),
                     lambda: setattr(opt, "step_count", 7), lambda: opt.step(grads)):
            with an_error_left_behind() if left else contextlib.nullcontext():
                call()
        assert opt.step_count == 8
        runs.append(bits(params + [opt.m, opt.v]))
    assert same(*runs)


@pytest.mark.parametrize("n", [3, 13])
def test_an_error_of_someone_else_is_not_the_slots(n):
    ctx = qml().Context(n, 3, 2, ckpt_block=1, storage="int8")
    psi = torch.randn(2, 1 << n, 2, device="cuda")
    out = torch.empty_like(psi)
    with an_error_left_behind():
        ctx.ckpt_save(0, psi)
    with an_error_left_behind():
        ctx.ckpt_restore(0, out)
    assert float((out - psi).abs().max()) <= float(psi.abs().max()) / 64
    ctx.sync()


def test_a_device_that_is_not_there_is_refused_before_anything_is_written():
    lib, q = qml().load_library(), qml()
    p = torch.zeros(3, 256, device="cuda")
    t = (q._OptTensor * 1)(q._OptTensor(p[0].data_ptr(), None, p[1].data_ptr(), p[2].data_ptr(), None, None, 256, 0, 0,
                                        1.0, 0.0))
    cfg, h = q._OptConfig(0, 0.9, 0.999, 1e-8, 0), ctypes.c_void_p()
    assert lib.qml_opt_create(ctypes.byref(cfg), 1, t, 63, ctypes.byref(h)) == 0
    nbytes = lib.qml_opt_workspace_bytes(h)
    ws = torch.full((nbytes + 256,), 5, dtype=torch.uint8, device="cuda")
    at = ctypes.c_void_p((ws.data_ptr() + 255) // 256 * 256)
    torch.cuda.synchronize()
    assert lib.qml_opt_set_workspace(h, at, nbytes, None) == 4
    g = (ctypes.c_void_p * 1)(p[0].data_ptr())
    assert lib.qml_opt_step(h, g, 1e-3, None, 1.0, 0.0, None, None) == 3  # there is no workspace
    lib.qml_opt_destroy(h)
    torch.cuda.synchronize()
    assert bool((ws == 5).all())


def test_factors_beyond_the_arithmetics_type_are_refused():
    for dtype, refused in (("fp32", True), ("bf16", True), ("fp64", False)):
        params, grads = make([300], dtype, dtype, 51)
        opt = optim().AdamW(params, weight_decay=0.0)
        before = bits(params + [opt.m, opt.v])
        for kw in (dict(lr=1e39), dict(grad_scale=1e39), dict(grad_scale=-1e39, max_norm=1.0)):
            if not refused:
                opt.step(grads, **kw)
                continue
            with pytest.raises(qml().QmlError) as e:
                opt.step(grads, **kw)
            assert e.value.code == 1
        assert opt.step_count == (0 if refused else 3)
        assert same(before, bits(params + [opt.m, opt.v])) == refused
        assert bool(torch.isfinite(params[0]).all())
