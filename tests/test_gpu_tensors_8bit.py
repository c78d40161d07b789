"""8-bit moments byte by byte: the new moments are bit for bit those of the 32-bit
form from the decoded ones, each byte the nearest to the fp32 quotient by its
block's scale, and the weights as good as the 32-bit form's, over every format,
alignment and divisor."""
import pytest
import torch

from _tensors import BF16, FP16, Tensors, assert_8bit_equals_32bit

pytestmark = pytest.mark.gpu


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


SMALL = [1, 255, 256, 257, 2048, 4099, 70_001, 300_000]


@pytest.mark.parametrize("dt", [FP16, BF16])
@pytest.mark.parametrize("grads", ["half", "fp32"])
@pytest.mark.parametrize("skew", [0, 1])
@pytest.mark.parametrize("div", [1024.0, 3.0])
@pytest.mark.parametrize("max_norm", [0.0, 0.01])
def test_8bit_step_is_the_32bit_one(zs, ctx, dt, grads, skew, div, max_norm):
    """... whatever grad_div is, clipped or not, from aligned arrays or not."""
    made = Tensors(zs, SMALL, dt, 1, seed=int(div), grads=grads, skews=(skew,))
    assert_8bit_equals_32bit(zs, ctx, made, div, max_norm)


@pytest.mark.parametrize("seed", [1, 2])
def test_8bit_step_without_gradients(zs, ctx, seed):
    """Moments that only decay: quotients that fall on the codes' midpoints."""
    made = Tensors(zs, SMALL, BF16, 1, seed=seed)
    for e in made.t:
        e["g"].zero_()
        e["mc"].fill_(2.0 ** -20)
        e["vc"].fill_(2.0 ** -18)
    assert_8bit_equals_32bit(zs, ctx, made, 1.0, 0.0)


@pytest.mark.parametrize("sigma", [0.05, 1e-12])
@pytest.mark.parametrize("div", [1.0, 3.0])
def test_weights_that_start_at_zero(zs, ctx, sigma, div):
    """The weight is the update alone, so all its bits are seen."""
    made = Tensors(zs, [3_000_000, 5000], BF16, 1, seed=9, sigma=sigma)
    for e in made.t:
        e["p"].zero_()
        e["mc"] *= sigma
        e["vc"] *= sigma
    assert_8bit_equals_32bit(zs, ctx, made, div, 0.0)


@pytest.mark.parametrize("c", [2.0 ** -126, 2.0 ** -100, 2.0 ** -60, 2.0 ** 40])
def test_8bit_scales_at_the_ends(zs, ctx, c):
    """Blocks of very small and large moments, without gradients (roots below
    2^-75 have no square in fp32 and are the least code's, or zero, in both)."""
    made = Tensors(zs, [3000, 517], BF16, 1, seed=4)
    for e in made.t:
        e["g"].zero_()
        e["mc"].fill_(c)
        e["vc"].fill_(c)
    assert_8bit_equals_32bit(zs, ctx, made, 1.0, 0.0)
