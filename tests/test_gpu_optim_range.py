"""8-bit optimiser states where one block holds magnitudes that are far apart: what
the codes' definition says must hold to the ends of fp32's range."""
import numpy as np
import pytest

from test_gpu_optim import BETAS, EPS, codes_in_fp32, optim, random_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F = np.float32


def second(g):
    """sqrt((1 - beta2) g^2), the root of a first step's second moment, in fp32."""
    return np.sqrt((g * g) * F(1 - BETAS[1]))


# one launch and the general kernel; whole blocks, and the last one ragged
@pytest.mark.parametrize("n", [256, 300, 65_536, 70_001])
@pytest.mark.parametrize("top,low", [(1e10, -22), (1e19, -22), (1.0, -22), (1e-3, -24)])
def test_a_positive_second_moment_never_becomes_zero(n, top, low):
    # a block's largest fixes the scale; the others go down to where g^2 vanishes in fp32
    rng = np.random.default_rng(n)
    g = (10.0 ** rng.uniform(low, np.log10(top), n)).astype(F) * rng.choice([-1, 1], n).astype(F)
    g[::256] = top
    seed = 5
    opt = optim().AdamW([torch.ones(n, device="cuda")], betas=BETAS, eps=EPS, state="8bit", seed=seed, weight_decay=0.0)
    opt.step([torch.from_numpy(g).cuda()], lr=0.1)
    r = second(g)
    got = opt.v.float().cpu().numpy()[:n]
    assert (r == 0).any() and (r[got == 0] == 0).all(), np.abs(g[(got == 0) & (r > 0)]).max()
    pad = np.zeros(-n % 256, F)
    want, _ = codes_in_fp32(np.concatenate([r, pad]), random_bits(seed, 1, 0, n + len(pad)) >> np.uint32(16), True)
    assert np.array_equal(got, want[:n])


@pytest.mark.parametrize("n", [65_536, 200_001])
def test_a_first_moment_without_a_second_one_is_not_kept(n):
    # g^2 vanishes in fp32 for all but each block's first element.  A first moment that
    # rounds up to a code there would be divided by eps alone at the next step, and at
    # the random number 0 everything positive rounds up.
    seed = 2
    first = np.arange(n) % 256 == 0
    zero = ((random_bits(seed, 1, 0, n) & np.uint32(0xFFFF)) == 0) & ~first
    assert zero.any()
    g = np.where(first, 1.0, 1e-24 * np.where(np.arange(n) % 2, 1, -1)).astype(F)
    assert (second(g)[~first] == 0).all()
    p = torch.ones(n, device="cuda")
    opt = optim().AdamW([p], betas=BETAS, eps=EPS, state="8bit", seed=seed, weight_decay=0.0)
    for _ in range(3):
        opt.step([torch.from_numpy(g).cuda()], lr=0.1)
        m, v = (x.cpu().numpy() for x in opt.moments(0))
        assert (v[~first] == 0).all() and (v[first] > 0).all() and (m[first] > 0).all()
        assert (m[~first] == 0).all(), m[zero]
        # lr m / eps of the moments before rounding: 0.1 * 1e-24 / 1e-8 a step, nothing in fp32
        assert (p.cpu().numpy()[~first] == 1.0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16", "fp64"])
@pytest.mark.parametrize("n", [5000, 65_536, 300_007])
def test_the_norm_whatever_the_gradients_alignment(dtype, n):
    # fp32: of two squares' sum, each of two operations is off by u = 2^-24 of it at most,
    # four exact 16-bit squares' by two sums, so the root by u; then its own rounding, u.
    # The fp64 sums of n terms add n 2^-53 (fp64: each of the squares' roundings among them).
    types = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "fp64": torch.float64}
    gen = torch.Generator("cuda").manual_seed(n)
    x = (torch.randn(n, generator=gen, device="cuda", dtype=torch.float64) * 0.1).to(types[dtype])
    want = float((x.cpu().numpy().astype(np.longdouble) ** 2).sum() ** np.longdouble(0.5)) if dtype in ("fp32", "fp64") \
        else float(x.double().square().sum().sqrt())
    bound = (0 if dtype == "fp64" else 2 * 2.0 ** -24) + (n + 2) * 2.0 ** -53
    for shift in (0, 1, 3):
        buf = torch.empty(n + 8, dtype=types[dtype], device="cuda")
        g = buf[shift:shift + n].copy_(x)
        opt = optim().AdamW([torch.zeros(n, dtype=types[dtype], device="cuda")])
        got = [float(opt.grad_norm([g])), float(opt.step([g], max_norm=1.0)), float(opt.step([g], max_norm=float("inf")))]
        again = [float(opt.grad_norm([g])), float(opt.step([g], max_norm=1.0)), float(opt.step([g], max_norm=float("inf")))]
        assert got == again
        assert all(abs(x - want) <= bound * want for x in got), (shift, got, want)
