"""Context.train_step in the forms that other tests leave out: fp64 contexts, captured
steps, working states and learning rates of the caller's."""
import math
import subprocess
import sys

import numpy as np
import pytest

import oracle
from adjoint_gradients_b200.inputs import random_case
from test_gpu_optim import BETAS, EPS, bits, host, optim, qml, same

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def case(seed, n, L, B, dtype):
    x, theta, y = random_case(seed, B, n, L)
    return x, theta, y, [torch.from_numpy(a).to(dtype).cuda() for a in (x, theta, y)]


def test_fp64_training_steps():
    # the fp64 passes' gradients are within 1e-9 of the oracle's; Adam divides them by
    # their own size, so angles with a small gradient are compared by the step's bound
    n, L, B, lr, clip = 6, 3, 5, 0.05, 0.3
    x, _, y, (xd, th, yd) = case(91, n, L, B, torch.float64)
    ctx = qml().Context(n, L, B, ckpt_block=1, precision="fp64", storage="fp64")
    opt = optim().AdamW([th], lr=lr, betas=BETAS, eps=EPS, weight_decay=0.01)
    m, v = np.zeros(th.shape), np.zeros(th.shape)
    for t in range(1, 5):
        th0 = host(th)
        E, loss, norm = ctx.train_step(th, xd, yd, opt, max_norm=clip)
        Eo = oracle.forward(x, th0)
        go, _ = oracle.adjoint(x, th0, oracle.loss_seed(Eo, y))
        no = math.sqrt(float((go ** 2).sum()))
        np.testing.assert_allclose(host(E), Eo, atol=1e-10)
        assert abs(float(norm) - no) <= 1e-9 * math.sqrt(go.size)
        g = go * min(1.0, clip / no)
        m, v = BETAS[0] * m + (1 - BETAS[0]) * g, BETAS[1] * v + (1 - BETAS[1]) * g * g
        den = np.sqrt(v / (1 - BETAS[1] ** t)) + EPS
        want = th0 * (1 - lr * 0.01) - lr / (1 - BETAS[0] ** t) * m / den
        big = np.abs(g) >= 1e-3
        assert big.sum() > 10
        # an error of 1e-9 in gradients above 1e-3: 1e-6 of a step, twice for m and for v, of up to 7.3 lr
        assert np.all(np.abs(host(th) - want)[big] <= lr * 7.3 * 4e-6)
    ctx.sync()
    opt.sync()


@pytest.mark.parametrize("state,storage", [("full", "fp32"), ("8bit", "int8")])
@pytest.mark.parametrize("n,L,B", [(4, 3, 5), (14, 5, 3)])
def test_captured_training_steps(n, L, B, state, storage):
    runs = []
    for captured in (False, True):
        _, _, _, (x, th, y) = case(92, n, L, B, torch.float32)
        ctx = qml().Context(n, L, B, ckpt_block=1, storage=storage)
        opt = optim().AdamW([th], state=state)
        lr = torch.full((1,), 0.02, device="cuda")
        first = ctx.train_step(th, x, y, opt, max_norm=0.5, lr=lr)
        outs = first
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs = ctx.train_step(th, x, y, opt, max_norm=0.5, lr=lr)
        for k in range(4):
            lr.fill_(0.02 / (k + 1))
            x.mul_(0.9)
            if captured:
                graph.replay()
            else:
                outs = ctx.train_step(th, x, y, opt, max_norm=0.5, lr=lr)
        assert opt.step_count == 5
        ctx.sync()
        opt.sync()
        runs.append(bits([th, opt.m, opt.v, *first, *outs]))
    assert same(*runs)


def test_working_states_of_the_callers():
    n, L, B = 13, 4, 3
    runs = []
    for own in (False, True):
        _, _, _, (x, th, y) = case(93, n, L, B, torch.float32)
        ctx = qml().Context(n, L, B, ckpt_block=2)
        ctx.set_reupload(True)
        opt = optim().AdamW([th])
        kw = dict(psi=ctx.new_state(B), lam=ctx.new_state(B)) if own else {}
        outs = [ctx.train_step(th, x, y, opt, lr=0.01, **kw) for _ in range(3)]
        assert all(norm is None for _, _, norm in outs)
        runs.append(bits([th, opt.m, opt.v] + [t for E, loss, _ in outs for t in (E, loss)]))
    assert same(*runs)


@pytest.mark.parametrize("dtype,state,n", [("float32", "full", 24), ("bfloat16", "8bit", 70_000), ("float64", "full", 300)])
def test_the_first_step_of_a_process_captured(dtype, state, n):
    # nothing of the library has run before the capture
    code = f"""
import torch
from adjoint_gradients_b200 import optim
p, g = torch.zeros({n}, dtype=torch.{dtype}, device="cuda"), torch.ones({n}, dtype=torch.{dtype}, device="cuda")
opt = optim.AdamW([p], lr=0.5, state="{state}", weight_decay=0.0)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    norm = opt.step([g], max_norm=1e9)
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
assert opt.step_count == 2 and abs(float(norm) - {n} ** 0.5) <= 1e-6 * {n} ** 0.5, (opt.step_count, norm)
assert float((p + 1).abs().max()) <= (0.01 if "{dtype}" == "bfloat16" else 1e-6), p
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
