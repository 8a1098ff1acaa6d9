"""The optimiser's outputs and temporaries under captured graphs and other streams."""
import math

import numpy as np
import pytest

from adjoint_gradients_b200.inputs import random_case
from test_gpu_optim import bits, make, optim, qml, same

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [[24], [70_000, 300]])
def test_replays_of_a_step_whose_norm_was_dropped_leave_other_tensors_alone(sizes):
    params, grads = make(sizes, "fp32", "fp32", 30)
    opt = optim().AdamW(params)
    opt.step(grads, max_norm=1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        opt.step(grads, max_norm=1.0)  # the norm is dropped
    for _ in range(40):
        opt.grad_norm(grads)
    others = [torch.full((1,), 7.0, device="cuda") for _ in range(400)]  # whatever small memory is free
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(float(x) == 7.0 for x in others)
    assert opt.step_count == 4


def test_norms_of_another_stream_belong_to_it():
    params, grads = make([70_000], "fp32", "fp32", 31)
    opt = optim().AdamW(params)
    want = math.sqrt(float((grads[0].double() ** 2).sum()))
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):  # an object, a handle
        side.wait_stream(torch.cuda.current_stream())
        for call in (lambda: opt.step(grads, max_norm=1.0, stream=stream), lambda: opt.grad_norm(grads, stream=stream)):
            norm = call()
            side.synchronize()
            assert float(norm) == pytest.approx(want, rel=1e-6)
            at = norm.data_ptr()
            del norm
            torch.cuda.synchronize()
            others = [torch.empty(1, device="cuda") for _ in range(300)]
            assert at not in {x.data_ptr() for x in others}  # not for other streams' tensors
    assert torch.cuda.current_stream() != side


def test_a_captured_norm_is_the_graphs():
    params, grads = make([24, 5003], "fp32", "fp32", 32)
    opt = optim().AdamW(params)
    opt.step(grads, max_norm=1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm = opt.step(grads, max_norm=1.0)
        alone = opt.grad_norm(grads, grad_scale=2.0)
    for k in range(3):
        for g in grads:
            g.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
        assert float(norm) == pytest.approx(want, rel=1e-6) and float(alone) == pytest.approx(2 * want, rel=1e-6)


@pytest.mark.parametrize("n,L,B,handle", [(6, 3, 5, False), (16, 12, 8, False), (16, 12, 8, True)])
def test_training_steps_on_another_stream(n, L, B, handle):
    # the current stream allocates and fills memory while the other one works: nothing of
    # the step may lie in it
    x, theta, y = (torch.from_numpy(a.astype(np.float32)).cuda() for a in random_case(88, B, n, L))
    runs = []
    for other in (False, True):
        ctx = qml().Context(n, L, B, ckpt_block=2)
        th = theta.clone()
        opt = optim().AdamW([th], lr=0.05)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        stream = (side.cuda_stream if handle else side) if other else None
        outs = []
        for _ in range(4):
            outs.append(ctx.train_step(th, x, y, opt, max_norm=0.5, stream=stream))
            if other:
                noise = [torch.full_like(t, math.nan) for t in (ctx.new_state(B), ctx.new_state(B), theta, y, y[:1])
                         for _ in range(3)]
        torch.cuda.synchronize()
        ctx.sync(stream)
        opt.sync(stream)
        runs.append(bits([th, opt.m, opt.v] + [t for o in outs for t in o]))
    assert same(*runs)
    assert len(noise) == 15


def test_reading_the_status_is_the_given_streams_business():
    # on the default stream the clearing of the status word could follow a later call's
    # error on another one; shown by the default stream's work, which nothing waits for
    params, grads = make([24, 5003], "fp32", "fp32", 33)
    opt = optim().AdamW(params)
    ctx = qml().Context(4, 2, 3)
    grads[1][7] = math.nan
    side = torch.cuda.Stream()
    opt.step(grads, max_norm=1.0, stream=side)  # (what the first call sets up waits, too)
    side.synchronize()
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000_000)  # about a second
    busy = torch.cuda.Event()
    busy.record()
    opt.step(grads, max_norm=1.0, stream=side)
    with pytest.raises(qml().QmlError) as e:
        opt.sync(side)
    assert e.value.code == 6
    opt.step(grads, max_norm=1.0, stream=side)
    with pytest.raises(qml().QmlError) as e:
        opt.sync(side)
    opt.sync(side)
    ctx.sync(side)
    with torch.cuda.stream(side):
        assert opt.step_count == 0
    assert not busy.query()
    torch.cuda.synchronize()


def test_the_default_stream_given_while_another_is_current():
    n, L, B = 6, 3, 5
    x, theta, y = (torch.from_numpy(a.astype(np.float32)).cuda() for a in random_case(89, B, n, L))
    torch.cuda.synchronize()
    runs = []
    for stream in (None, 0, torch.cuda.default_stream()):
        ctx = qml().Context(n, L, B, ckpt_block=1)
        th = theta.clone()
        opt = optim().AdamW([th], lr=0.05)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.current_stream() if stream is None else torch.cuda.Stream()):
            outs = [ctx.train_step(th, x, y, opt, max_norm=0.5, stream=stream) for _ in range(3)]
            outs.append((opt.grad_norm([theta], stream=stream),))
            torch.cuda.synchronize()
            runs.append(bits([th, opt.m, opt.v] + [t for o in outs for t in o]))
    assert same(*runs[:2]) and same(*runs[1:])
