"""lh_quantize_nvfp4 where its quotients leave the range of reciprocals, and for
what is not a finite number, against the definition in IEEE single precision
(numpy on the CPU, subnormals included) and the max rule's own calls."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float32)
CODES = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][1:127])


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def nearest(v, points):
    """Index of the nearest point (ascending fp64), ties to the even index; no NaN."""
    v = v.astype(np.float64)
    hi = np.clip(np.searchsorted(points, v), 1, len(points) - 1)
    down, up = v - points[hi - 1], points[hi] - v
    return np.where((down < up) | ((down == up) & ((hi - 1) % 2 == 0)), hi - 1, hi)


def definition(x, amax):
    """(code, r, c) of fp32 x [rows, c_in]: t = fl(fl(a / 6) / S_g), s = fl(c S_g), r = E2M1(fl(x / s))."""
    with np.errstate(all="ignore"):
        b = x.reshape(x.shape[0], -1, 16)
        s_g = np.float32(amax) / np.float32(2688)
        a = np.abs(b).max(-1)
        t = (a / np.float32(6)) / s_g if s_g > 0 else np.zeros_like(a)
        code = np.maximum(nearest(np.minimum(t, np.float32(448)), np.concatenate([[0], CODES])), 1)
        c = CODES[code - 1].astype(np.float32)
        s = (c * s_g)[..., None]
        q = np.where(s == 0, np.float32(0), np.abs(b) / s)
        r = GRID[nearest(np.minimum(q, np.float32(6)), GRID.astype(np.float64))] * np.sign(b)
    return code, r, c


def check(lh, x, amax, what, rule=True):
    """x [rows, c_in] on the CPU, amax a float; rule: the max rule's own calls agree as well."""
    xd, ad = x.to(DEV), torch.full((1,), amax, dtype=F32, device=DEV)
    got = {k: v[0].cpu() if v.dim() > 1 else v.cpu()
           for k, v in lh.lh_quantize_nvfp4(xd, ad, packed=True, scale_e4m3=True, global_scale=True).items()}
    code, r, c = definition(x.float().numpy(), amax)
    assert np.array_equal(got["scale_e4m3"].numpy(), code), "%s: codes" % what
    u = (r * c[..., None]).reshape(x.shape)
    assert np.array_equal(got["values"].float().numpy(), u), "%s: values" % what
    assert not torch.signbit(got["values"].float()[torch.from_numpy(u) == 0]).any(), "%s: a negative zero" % what
    if rule:
        idx, _, _ = lh.lh_select_scales(lh.LH_RULE_MAX, xd, None, ad)
        ref = lh.lh_fake_quant_nvfp4(xd, idx, ad, packed=True, scale_e4m3=True, global_scale=True)
        for k in ("packed", "scale_e4m3", "global_scale"):
            assert torch.equal(got[k], ref[k].cpu().view(got[k].shape)), "%s: %s differs from the rule's" % (what, k)


def activations(seed, dt):
    rng = np.random.default_rng(seed)
    x = np.clip(rng.standard_t(3, (20, 208)) / 12, -1, 1) * 1.9   # the largest is below 2
    x[:, 32:64] *= 2.0 ** -7
    x[:, 64:80] *= 2.0 ** -14
    x[rng.random(x.shape) < 0.05] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(dt)


# 2^-100 and 2^100 (times 6 / 2688, or a code) bound the reciprocals; S_g is subnormal below 2^-114, zero below 2^-138
@pytest.mark.parametrize("e", [-149, -145, -139, -137, -130, -126, -115, -112, -110, -100, -95, -90, -80, -1, 60, 88, 100,
                               105, 108, 110, 112, 126, 127])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_amax_of_any_exponent(lh, e, dt):
    print("case 2^%d %s" % (e, dt), flush=True)
    x = (activations([3, e + 200], F32).double() * 2.0 ** e).float().to(dt)
    check(lh, x, x.float().abs().max().item(), "own amax")
    if e > -140:
        check(lh, x, 2.0 ** e, "a power of two")


@pytest.mark.parametrize("dt", [BF16, F32])
def test_zero_amax_with_activations(lh, dt):
    check(lh, activations(5, dt), 0.0, "zero amax")


@pytest.mark.parametrize("amax", [1.0, 2688.0, 2.0 ** -110, 2.0 ** 110])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_infinities_take_the_largest_code(lh, amax, dt):
    x = activations(7, dt) * amax
    x[0, 0], x[3, 17], x[3, 18], x[19, 207] = float("inf"), -float("inf"), float("inf"), -float("inf")
    check(lh, x, amax, "infinities", rule=amax in (1.0, 2688.0))
    got = lh.lh_quantize_nvfp4(x.to(DEV), torch.full((1,), amax, device=DEV))["values"][0].cpu()
    assert [got[i].item() for i in ((0, 0), (3, 17), (3, 18), (19, 207))] == [2688, -2688, 2688, -2688]


@pytest.mark.parametrize("amax", [1.0, 2.0 ** -110, 2.0 ** 110])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_a_nan_stays_in_its_place(lh, amax, dt):
    """It counts for nothing in its block's maximum and leaves as +-6 times the block's scale."""
    x = activations(9, dt) * amax
    places = [(0, 0), (2, 31), (7, 100), (19, 207)]
    without = x.clone()
    for p in places:
        x[p], without[p] = float("nan"), 0.0
    a = torch.full((1,), amax, device=DEV)
    got, ref = (lh.lh_quantize_nvfp4(v.to(DEV), a, packed=True, scale_e4m3=True) for v in (x, without))
    assert torch.equal(got["scale_e4m3"], ref["scale_e4m3"])
    v, w = got["values"][0].float().cpu(), ref["values"][0].float().cpu()
    c = got["scale_e4m3"][0].cpu().view(torch.float8_e4m3fn).float()
    for p in places:
        assert abs(v[p].item()) == 6 * c[p[0], p[1] // 16].item()
        v[p] = 0.0
    assert torch.equal(v, w)


def test_an_amax_that_is_no_number_shows_in_the_global_scale(lh):
    x = activations(11, F32).to(DEV)
    for bad in (float("inf"), float("nan")):
        s = lh.lh_quantize_nvfp4(x, torch.full((1,), bad, device=DEV), global_scale=True)["global_scale"].item()
        assert s == bad or (s != s and bad != bad)
