"""Optimiser steps and 8-bit slots whose offsets pass 32 bits."""
import math

import pytest

from test_gpu_optim import optim, qml

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,state", [(torch.bfloat16, "8bit"), (torch.float16, "full")])
def test_a_tensor_of_more_than_2_31_elements(dtype, state):
    n = (1 << 31) + 777
    at = [0, 255, (1 << 31) - 1, 1 << 31, (1 << 31) + 600, n - 1]
    p, g = torch.zeros(n, dtype=dtype, device="cuda"), torch.zeros(n, dtype=dtype, device="cuda")
    g[at] = 1.0
    opt = optim().AdamW([p], lr=0.5, state=state, weight_decay=0.0)
    norm = opt.step([g], max_norm=math.inf)
    assert float(norm) == pytest.approx(math.sqrt(len(at)), rel=1e-6)
    assert p[at].tolist() == [-0.5] * len(at)  # m / sqrt(v) = 1 with the bias corrections
    assert int(torch.count_nonzero(p)) == len(at)
    m = opt.m[:n].view(torch.uint8) if state == "8bit" else opt.m[:n]
    assert int(torch.count_nonzero(m)) == len(at) and bool((m[at] != 0).all())


def test_a_slot_of_more_than_2_31_amplitudes():
    n, B = 26, 33
    ctx = qml().Context(n, 2, B, ckpt_block=1, storage="int8")
    psi = torch.empty(B, 1 << n, 2, device="cuda")
    gen = torch.Generator("cuda").manual_seed(1)
    for b in range(B):
        psi[b].normal_(generator=gen)
    out = torch.full_like(psi, 9.0)
    ctx.ckpt_save(0, psi)
    ctx.ckpt_restore(0, out)
    for b in range(B):
        # half a step of 2^k <= max / 64, a whole one for a block's largest; another
        # amplitude's value would be off by more somewhere
        assert float((out[b] - psi[b]).abs().max()) <= float(psi[b].abs().max()) / 64
    ctx.sync()
