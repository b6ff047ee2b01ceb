"""A product without a workspace takes the kernel that is best without partial
sums, not the tiles that would be best with them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def timed(f, n=50):
    """Microseconds per call, the least of five runs."""
    f()
    best = float("inf")
    for _ in range(5):
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ev[0].record()
        for _ in range(n):
            f()
        ev[1].record()
        torch.cuda.synchronize()
        best = min(best, ev[0].elapsed_time(ev[1]) / n * 1e3)
    return best


def test_few_tokens_of_a_long_sum(lh):
    """32 tokens x (4096 x 17408): with parts some 20 us, in 64 x 256 tiles.
    Those without parts would be 16 workgroups that walk 136 chunks each, some
    seven times that; tiles of 16 x 32 take less than twice."""
    t, c_out, c_in = 32, 4096, 17408
    gen = torch.Generator(device=DEV).manual_seed(1)
    packed = torch.randint(0, 256, (1, c_out, c_in // 2), dtype=torch.uint8, device=DEV, generator=gen)
    codes = torch.randint(0x28, 0x50, (1, c_out, c_in // 16), dtype=torch.uint8, device=DEV, generator=gen)
    s = torch.full((1,), 1e-3, device=DEV)
    x = torch.randn((t, c_in), device=DEV, generator=gen).to(torch.bfloat16)
    y = torch.empty((t, c_out), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(lh.lh_linear_nvfp4_workspace_bytes(t, c_in, c_out), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    parts = timed(lambda: lh.lh_linear_nvfp4(x, packed, codes, s, y=y, workspace=ws))
    alone = timed(lambda: lh.lh_linear_nvfp4(x, packed, codes, s, y=y, workspace=None))
    print("with parts %.1f us, without a workspace %.1f us" % (parts, alone), flush=True)
    assert alone < 4 * parts
