"""The list's sum of squares and norm over gradients whose squares lie below
fp32's range, down to the least value of each format."""
import pytest
import torch

from _tensors import BF16, HP, Tensors

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


def check_norm(zs, ctx, made, div=3.0):
    """The sum of squares and the norm within 1e-6 of the sum in 64 bits."""
    lst = made.list(ctx)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = torch.zeros(1, dtype=torch.float64, device="cuda")
    zs.zs_tensors_check(lst, div, flag, got)
    want = sum(e["g"].double().square().sum().item() for e in made.t) / div ** 2
    assert flag.item() == 0
    assert abs(got.item() - want) <= 1e-6 * want, (got.item(), want)
    norm = torch.zeros((), device="cuda")
    d = zs.DeviceState(zs.zs_scaler_init(div, 1.0, 1000, 1, False))
    zs.zs_tensors_step_async(lst, 1, 1, zs.make_hparams(*HP), None, 1.0, d, norm)
    # (one more half unit for the rounding to fp32, and its least value's below its normals)
    assert abs(norm.item() - want ** 0.5) <= 1e-6 * want ** 0.5 + 2.0 ** -149
    lst.close()


@pytest.mark.parametrize("value", [1e-17, 1e-19, 1e-20, 1e-22, 1e-25, 1e-30, 1e-38])
@pytest.mark.parametrize("grads", ["half", "fp32"])
@pytest.mark.parametrize("skew", [0, 1])
def test_norm_of_small_values(zs, ctx, value, grads, skew):
    """Squares below fp32's range count: alone, beside larger ones, in every
    place of a batch, and where most gradients are zero."""
    made = Tensors(zs, [40_000, 5, 3000], BF16, 0, seed=2, grads=grads, skews=(skew,), sigma=value)
    made.t[2]["g"][:2900] = 0
    check_norm(zs, ctx, made)
    made.t[0]["g"][::7] *= 1e-3
    made.t[0]["g"][5000:30_000] = 0
    check_norm(zs, ctx, made)
    made.t[2]["g"][2950] = value * 1e6
    check_norm(zs, ctx, made)
    for e in made.t:
        e["g"].zero_()
    made.t[0]["g"][12_345] = value
    check_norm(zs, ctx, made)


def test_norm_of_the_least_values(zs, ctx):
    """fp32's and bf16's own subnormals, and one gradient of each size at once."""
    for grads, least in (("fp32", 2.0 ** -149), ("half", 2.0 ** -133)):
        made = Tensors(zs, [1000], BF16, 0, grads=grads)
        made.t[0]["g"].fill_(least)
        check_norm(zs, ctx, made)
        made.t[0]["g"].copy_(torch.logspace(-44, 30, 1000, base=10.0, dtype=torch.float64))
        check_norm(zs, ctx, made)
        made.t[0]["g"].copy_(torch.logspace(-44, -19, 1000, base=10.0, dtype=torch.float64))
        check_norm(zs, ctx, made)
