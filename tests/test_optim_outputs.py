"""Who owns what an optimiser's call returns (no GPU needed: the library is a stand-in
that records its arguments)."""
import pytest

torch = pytest.importorskip("torch")

from adjoint_gradients_b200 import optim, qml  # noqa: E402


class Library:
    """Accepts every call; `calls` holds their names and arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args):
            self.calls.append((name, args))
            return 0 if name != "qml_opt_workspace_bytes" else 256

        return f


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(qml, "load_library", lambda: lib)
    lib.stream, lib.capturing = 0, False
    monkeypatch.setattr(qml, "_current_stream", lambda device=None: lib.stream)
    monkeypatch.setattr(optim.AdamW, "_check_buffer", lambda self, t, dtype, numel, what: None)
    return lib


def make(library, params, **kw):
    opt = optim.AdamW(params, **kw)
    opt._index = params[0].get_device()
    opt._on_device, opt._capturing = lambda: opt._index, lambda: library.capturing
    return opt


def test_norms_of_captured_calls_have_memory_of_their_own(library):
    # a captured step keeps the address that it was given: memory shared with the norms of
    # eager calls would go to another tensor when those are dropped, under the graph's writes
    p, g = torch.zeros(5), torch.ones(5)
    opt = make(library, [p])
    norms = []
    for k in range(200):
        library.capturing = k % 7 == 1
        norms.append(opt.grad_norm([g]) if k % 2 else opt.step([g], max_norm=1.0))
        assert norms[-1].shape == (1,) and norms[-1].is_contiguous()
        if library.capturing:
            assert norms[-1].untyped_storage().nbytes() == norms[-1].element_size()
    assert len({n.data_ptr() for n in norms}) == len(norms)
    given = [a[6] for name, a in library.calls if name == "qml_opt_step"]
    assert given == [n.data_ptr() for n in norms[::2]]


def test_norms_of_two_streams_share_no_memory(library):
    p, g = torch.zeros(5), torch.ones(5)
    opt = make(library, [p])
    memory = {0: set(), 8: set()}
    for k in range(200):
        library.stream = 8 * (k // 5 % 2)
        norm = opt.grad_norm([g])
        memory[library.stream].add(norm.untyped_storage().data_ptr())
        opt.kept = getattr(opt, "kept", []) + [norm]
    assert not memory[0] & memory[8]
