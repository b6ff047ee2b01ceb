"""lh_quantize_nvfp4: codes, nibbles and S_g bit for bit as the max rule
followed by the fake-quant (both checked against the oracle elsewhere), and
against the definition in 64 bits where the quotients are exact."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def _check(lh, x, amax, what):
    """Every output against lh_select_scales(MAX) + lh_fake_quant_nvfp4, values against codes and nibbles."""
    xc = x.contiguous()
    got = lh.lh_quantize_nvfp4(x, amax, packed=True, scale_e4m3=True, global_scale=True)
    idx, _, _ = lh.lh_select_scales(lh.LH_RULE_MAX, xc, None, amax)
    ref = lh.lh_fake_quant_nvfp4(xc, idx, amax, packed=True, scale_e4m3=True, global_scale=True)
    for k in ("packed", "scale_e4m3", "global_scale"):
        assert torch.equal(got[k], ref[k]), "%s: %s differs" % (what, k)
    # the values are exact: times S_g in fp32 they are r * c * S_g up to the order of two roundings
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    p = got["packed"].cpu()
    r = torch.stack([grid[(p & 15).long()], grid[(p >> 4).long()]], dim=-1).flatten(-2)
    c = got["scale_e4m3"].cpu().view(torch.float8_e4m3fn).double()
    u = r * c.repeat_interleave(16, dim=-1)
    assert got["values"].dtype == x.dtype
    assert torch.equal(got["values"].cpu().double(), u), "%s: values" % what
    for dt in (BF16, F32):
        alone = lh.lh_quantize_nvfp4(x, amax, values=True, values_dtype=dt)["values"]
        assert torch.equal(alone.cpu().double(), u), "%s: values alone, %s" % (what, dt)


@pytest.mark.parametrize("g,rows,c_in", [(1, 1, 16), (1, 1, 4096), (1, 3, 48), (2, 7, 272), (1, 300, 1040), (5, 2, 64),
                                         (70, 1, 32)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_as_max_rule_and_fake_quant(lh, g, rows, c_in, dt):
    print("case g=%d rows=%d c_in=%d %s" % (g, rows, c_in, dt), flush=True)
    rng = np.random.default_rng([g, rows, c_in])
    x = rng.standard_t(3, (g, rows, c_in)) * np.exp(rng.standard_normal((g, 1, c_in)) * 3)
    x[:, :, : c_in // 16 * 4] *= 1e-6          # blocks whose scale is at the smallest codes
    x[rng.random((g, rows, c_in)) < 0.05] = 0.0
    x = torch.from_numpy(x.astype(np.float32)).to(dt).to(DEV)
    _check(lh, x, lh.lh_absmax(x), "own amax")
    # an amax of the calibration: smaller and larger than these activations' own
    _check(lh, x, lh.lh_absmax(x) * 0.01, "saturating")
    _check(lh, x, lh.lh_absmax(x) * 1e4, "small codes")


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("shift", [1, 2, 5])
def test_strides_and_alignment(lh, dt, shift):
    rng = np.random.default_rng(3)
    big = torch.from_numpy(rng.standard_normal((9, 200)).astype(np.float32)).to(dt).to(DEV)
    x = big[1:8, shift:shift + 160]
    _check(lh, x, lh.lh_absmax(x), "shift %d" % shift)


def test_zero_amax_zero_blocks_and_ties(lh):
    x = torch.zeros((2, 4, 32), dtype=F32, device=DEV)
    got = lh.lh_quantize_nvfp4(x, torch.zeros(2, device=DEV), packed=True, scale_e4m3=True, global_scale=True)
    assert bool((got["values"] == 0).all()) and bool((got["packed"] == 0).all())
    assert bool((got["scale_e4m3"] == 1).all()) and bool((got["global_scale"] == 0).all())
    assert not bool(torch.signbit(lh.lh_quantize_nvfp4(-x, torch.ones(2, device=DEV))["values"]).any())
    # S_g = 1, block maximum 6: c = 1, so the values are the cast of x itself; ties go to the even code
    row = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.2]
    want = [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.0, -1.0, -1.0, -2.0, -2.0, -4.0, -4.0, 0.0]
    amax = torch.full((1,), 2688.0, device=DEV)
    for dt in (F32, BF16):
        v = lh.lh_quantize_nvfp4(torch.tensor([row], dtype=dt, device=DEV), amax)["values"]
        assert v.flatten().tolist() == want


def test_tokens_as_groups(lh):
    """One scale per token: the rows given as groups."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy((rng.standard_normal((40, 64)) * np.exp(rng.standard_normal((40, 1)) * 4)).astype(np.float32)).to(DEV)
    rows = x.unsqueeze(1)
    amax = lh.lh_absmax(rows)
    q = lh.lh_quantize_nvfp4(rows, amax, global_scale=True)
    back = (q["values"][:, 0].double() * q["global_scale"].double().unsqueeze(1)).cpu()
    err = (back - x.double().cpu()).abs().view(40, 4, 16).amax(-1)
    # a block scale is within 2^-4 of the wanted one (or half the smallest code), the grid's widest half step is 1 of 6
    top = x.double().cpu().abs().view(40, 4, 16).amax(-1)
    assert bool((err <= top * (1 / 6 + 2 ** -4) * 1.07 + amax.double().cpu().view(40, 1) / 2688 * 2 ** -9 * 6).all())


def test_more_rows_than_a_grid_dimension(lh):
    x = torch.randn((70000, 48), device=DEV).to(BF16)[:, :32]       # strided: rows are not flattened
    _check(lh, x, lh.lh_absmax(x), "70000 strided rows")


def test_refusals(lh):
    x = torch.zeros((4, 64), dtype=BF16, device=DEV)
    amax = torch.ones(1, device=DEV)
    with pytest.raises(lh.LHError):
        lh.lh_quantize_nvfp4(x[:, :24], amax)
    with pytest.raises(ValueError):
        lh.lh_quantize_nvfp4(x, torch.ones(2, device=DEV))
    with pytest.raises(TypeError):
        lh.lh_quantize_nvfp4(x.half(), amax)
    with pytest.raises(ValueError):
        lh.lh_quantize_nvfp4(x.cpu(), amax)
    with pytest.raises(lh.LHError):
        lh.lh_quantize_nvfp4(x, amax, values=False)
    with pytest.raises(ValueError):
        lh.lh_quantize_nvfp4(x, amax, packed=torch.empty((1, 4, 31), dtype=torch.uint8, device=DEV))
