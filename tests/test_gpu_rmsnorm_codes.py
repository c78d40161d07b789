"""The norm's 8-bit output byte by byte: from the stored reciprocal root, each
scale is the fp32 quotient max|y| / 448 and each byte the E4M3 value nearest to
the fp32 quotient y / scale, in every form of access and over every width."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FP16, BF16 = 0, 1
TORCH = {FP16: torch.float16, BF16: torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module")
def zs():
    import zero_mixed_precision_shard_gb300 as pkg
    torch.cuda.set_device(0)
    return pkg


@pytest.fixture(scope="module")
def ctx(zs):
    c = zs.Ctx()
    yield c
    c.close()


def rand(rows, cols, dt, seed, skew=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    base = (torch.randn(rows * cols + skew, device="cuda", generator=g) * scale).to(TORCH[dt])
    return base[skew:].view(rows, cols)


def expected(x, res, w, rstd, group):
    """Codes and scales by IEEE operations on the host, in the definition's order."""
    f = [t.float().cpu().numpy() for t in (x, w, rstd)]
    h = f[0] if res is None else f[0] + res.float().cpu().numpy()
    y = h * f[2][:, None] * f[1]
    rows, cols = y.shape
    group = group or cols
    groups = -(-cols // group)
    wide = np.zeros((rows, groups * group), np.float32)
    wide[:, :cols] = y
    c = np.abs(wide).reshape(rows, groups, group).max(2) / np.float32(448)
    c = np.maximum(c, np.float32(2.0 ** -126))
    q = y / np.repeat(c, group, 1)[:, :cols]
    return torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8), torch.from_numpy(c)


@pytest.mark.parametrize("cols", [7, 64, 255, 768, 1000, 1024, 2047, 4096, 8192, 16_384, 20_001])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("skews", [(0, 0), (1, 1), (1, 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_bytes_and_scales(zs, ctx, cols, group, skews, residual):
    """Without a residual a row's quotients repeat those of its halves, many on
    the midpoints between two bytes."""
    rows, dt = max(9, min(700, 400_000 // cols)), BF16
    x = rand(rows, cols, dt, 1, skews[0])
    res = rand(rows, cols, dt, 2, skews[0]) if residual else None
    w = rand(1, cols, dt, 3)[0] if residual else torch.ones(cols, dtype=TORCH[dt], device="cuda")
    q = torch.zeros(rows * cols + skews[1], dtype=torch.uint8, device="cuda")[skews[1]:]
    scales = torch.zeros(rows, -(-cols // group) if group else 1, device="cuda")
    rstd = torch.zeros(rows, device="cuda")
    zs.zs_rmsnorm(ctx, zs.make_norm_shape(rows, cols, dt, EPS, bits=8, group=group), x, res, w,
                  None, q.view(torch.float8_e4m3fn).view(rows, cols), scales, rstd)
    codes, c = expected(x, res, w, rstd, group)
    assert torch.equal(scales.cpu(), c)
    got = q.view(rows, cols).cpu()
    # (a zero's sign is that of y, which a zero sum of halves may lose)
    assert ((got == codes) | ((got & 0x7F) + (codes & 0x7F) == 0)).all()


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -60, 2.0 ** 60])
@pytest.mark.parametrize("group", [0, 32])
def test_bytes_of_small_and_large_rows(zs, ctx, scale, group):
    rows, cols, dt = 50, 1024, BF16
    x, w = rand(rows, cols, dt, 1), rand(1, cols, dt, 3, 0, scale)[0]
    q = torch.zeros(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    scales, rstd = torch.zeros(rows, cols // group if group else 1, device="cuda"), torch.zeros(rows, device="cuda")
    zs.zs_rmsnorm(ctx, zs.make_norm_shape(rows, cols, dt, EPS, bits=8, group=group), x, None, w,
                  None, q, scales, rstd)
    codes, c = expected(x, None, w, rstd, group)
    assert torch.equal(scales.cpu(), c)
    assert torch.equal(q.view(torch.uint8).cpu(), codes)
