"""What s carries on its way out of the rank: all of its 24 bits, whatever the
output's type and however many rows there are."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def rounded(v):
    """To bf16 and back to 64 bits."""
    return torch.from_numpy(v.astype(np.float32)).to(BF16).double().numpy()


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("rows,rank,cols_in,cols_out", [(20, 16, 40, 96), (400, 16, 200, 136), (400, 64, 200, 136), (400, 200, 72, 40),
                                                        (2100, 16, 96, 72), (2100, 12, 96, 136), (2100, 64, 96, 72)])
def test_s_leaves_the_rank_whole(lh, rows, rank, cols_in, cols_out, grad):
    """bf16 throughout, and an output that is what is left of s after its 16 upper
    bits are gone: s0 = x0 + x1 + x2 with x1 and x2 some 2^-9 and 2^-17 of x0, base
    = -bf16(s0), and a second rank that gives v = -bf16(s0 + base); y = base + s0 +
    v = r, some 2^-17 of s0.  All products are exact (the factors are powers of
    two).  Added in fp32 in any order are three terms for s0, off by 2 u s0 (u =
    2^-24; twice that where sums are truncated), and at most three parts of s0 and
    one of v, off by another 3 u (6 u) and 2 u for the sum with base; y's own
    rounding is 2^-8 of r."""
    rng = np.random.default_rng([rows, rank, grad])
    x = np.zeros((rows, cols_in))
    at = rng.choice(cols_in, 4, replace=False)
    x0 = rounded(rng.uniform(1, 2, rows) * 2.0 ** rng.integers(-3, 4, rows)) * rng.choice([-1, 1], rows)
    x1 = rounded(x0 * rng.uniform(0.5, 1, rows) * 2.0 ** -9)
    x2 = rounded(x0 * rng.uniform(0.5, 1, rows) * 2.0 ** -17)
    s0 = x0 + x1 + x2
    base = -rounded(s0)
    v = -rounded(s0 + base)
    r = base + s0 + v
    assert np.median(np.abs(r / s0)) > 2.0 ** -19 and (np.abs(r) <= 2.0 ** -16 * np.abs(s0)).all()
    for c, part in zip(at, (x0, x1, x2, v)):
        x[:, c] = part
    inner, outer = np.zeros((2, rank, cols_in)), np.zeros((2, rank, cols_out))
    k0, k1 = rng.choice(rank, 2, replace=False)
    inner[1, k0, at[:3]], inner[1, k1, at[3]] = 1, 1
    power = 2.0 ** rng.integers(-2, 3, cols_out) * rng.choice([-1, 1], cols_out)
    outer[1, k0], outer[1, k1] = power, power
    outer[0], inner[0] = 3, 5                        # an adapter that no row takes

    def dev(a):
        t = torch.from_numpy(a.astype(np.float32)).to(BF16)
        assert np.array_equal(t.double().numpy(), a)
        return t.to(DEV)

    f = lh.lh_lora_grad if grad else lh.lh_lora
    a, b = (outer, inner) if grad else (inner, outer)
    y = f(dev(x), dev(a), dev(b), base=dev(base[:, None] * power), adapter_ids=torch.ones(1, dtype=torch.int32, device=DEV))
    want = r[:, None] * power
    tol = 2.0 ** -8 * np.abs(want) + 16 * U * np.abs(s0[:, None] * power)
    off = np.abs(y.double().cpu().numpy() - want)
    assert (off <= tol).all(), "%d of %d outside, worst %.3g of its tolerance" % ((off > tol).sum(), off.size, (off / tol).max())
