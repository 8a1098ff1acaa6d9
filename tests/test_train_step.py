"""Context.train_step on the host: order, streams, process groups (no GPU needed: the
context's passes are stand-ins)."""
import pytest

torch = pytest.importorskip("torch")

from adjoint_gradients_b200 import qml  # noqa: E402


class Fake(qml.Context):
    """A context whose gradient is theta / 2 + x's mean; `log` holds the calls, each with
    the stream that was current."""

    def __init__(self, log):
        self.device, self.n, self.L, self.f64, self._real_dtype = 0, 2, 1, False, torch.float32
        self.log, self.current = log, None

    def __del__(self):
        pass

    def _note(self, what, stream):
        self.log.append((what, self.current if stream is None else stream))

    def new_state(self, B):
        self._note("new_state", None)
        return torch.zeros(B, 4, 2)

    def forward(self, theta, x, psi=None, expect=None, stream=None):
        psi = self.new_state(x.shape[0]) if psi is None else psi
        self._note("forward", stream)
        return psi, x.mean(1)

    def loss_seed(self, expect, y, stream=None):
        self._note("loss_seed", stream)
        return expect - y, ((expect - y) ** 2).mean().view(1)

    def backward(self, theta, x, psi, lam, dLdE, grad=None, stream=None):
        self._note("backward", stream)
        return theta / 2 + x.mean()


class FakeOpt:
    def __init__(self, ctx, params):
        self.ctx, self.params, self.taken = ctx, params, []

    def step(self, grads, lr=None, max_norm=None, stream=None):
        self.ctx._note("step", stream)
        self.taken += [g.clone() for g in grads]
        return torch.ones(1) if max_norm else None


def case():
    return torch.arange(6.0).view(1, 2, 3), torch.ones(3, 2), torch.zeros(3)


def test_a_step_on_another_stream_allocates_there(monkeypatch):
    # what train_step allocates and drops must belong to the stream that uses it, or the
    # current stream's next tensors take it from under the queued kernels
    log = []
    ctx = Fake(log)
    theta, x, y = case()

    def run_on(stream, device, call):
        ctx.current, before = stream, ctx.current
        out = call()
        ctx.current = before
        return out

    monkeypatch.setattr(qml, "_run_on", run_on, raising=False)
    ctx.train_step(theta, x, y, FakeOpt(ctx, [theta]), max_norm=1.0, stream="side")
    assert [w for w, _ in log] == ["new_state", "forward", "loss_seed", "new_state", "backward", "step"]
    assert {s for _, s in log} == {"side"}
    with pytest.raises(ValueError):
        ctx.train_step(theta, x, y, FakeOpt(ctx, [theta]), stream="side", group=object())


def test_an_optimiser_of_other_parameters_is_refused():
    log = []
    ctx = Fake(log)
    theta, x, y = case()
    for params in ([theta.clone()], [theta, theta.clone()], [theta[:, :1]], [theta.view(-1)[1:]]):
        opt = FakeOpt(ctx, params)
        with pytest.raises(ValueError):
            ctx.train_step(theta, x, y, opt)
        assert not log and not opt.taken  # refused before anything ran
    for same in (theta, theta.view(-1), theta.detach()):
        opt = FakeOpt(ctx, [same])
        E, loss, norm = ctx.train_step(theta, x, y, opt)
        assert norm is None and torch.equal(opt.taken[0], theta / 2 + x.mean())


def _rank(rank, world, port, out):
    import os

    import torch.distributed as dist

    os.environ["MASTER_ADDR"], os.environ["MASTER_PORT"] = "127.0.0.1", str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        log = []
        ctx = Fake(log)
        theta, x, y = case()
        x = x * (rank + 1)
        taken = []
        for group in (dist.group.WORLD, dist.new_group([0, 1]), None):
            opt = FakeOpt(ctx, [theta])
            ctx.train_step(theta, x, y, opt, group=group)
            taken += opt.taken
        torch.save(taken, f"{out}{rank}")
    finally:
        dist.destroy_process_group()


def test_ranks_of_a_group_step_with_the_mean_gradient(tmp_path):
    import torch.multiprocessing as mp

    from test_multiprocess import _free_port

    out = str(tmp_path / "taken")
    mp.start_processes(_rank, args=(2, _free_port(), out), nprocs=2, start_method="spawn")
    theta = case()[0]
    for rank in range(2):
        mean, pair, own = torch.load(f"{out}{rank}")
        # theta / 2 + 1 on rank 0, theta / 2 + 2 on rank 1
        assert torch.equal(mean, theta / 2 + 1.5) and torch.equal(pair, mean)
        assert torch.equal(own, theta / 2 + 1 + rank)  # without a group every rank keeps its own
