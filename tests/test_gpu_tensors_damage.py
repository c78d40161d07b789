"""Values that are not finite among the stored moments, or in gradients that
nobody checked, show in the moments instead of being taken for numbers."""
import numpy as np
import pytest
import torch

from _tensors import BF16, BLOCK, HP, Tensors, decode

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


DAMAGE = [("m", 0x7F), ("m", 0xFF), ("v", 0x7F), ("mc", float("nan")), ("vc", float("nan")),
          ("mc", float("inf")), ("vc", float("inf")), ("p", float("nan"))]


@pytest.mark.parametrize("what,value", DAMAGE)
@pytest.mark.parametrize("skew", [0, 1])
@pytest.mark.parametrize("block", [0, 9, 16])
def test_damaged_moments_show(zs, ctx, what, value, skew, block):
    """A NaN or inf among stored moments makes its block's values NaN, not
    small numbers, and leaves every other block as it would have been."""
    n = 16 * BLOCK + 100
    good = Tensors(zs, [n], BF16, 1, seed=7, skews=(skew,))
    bad = good.clone()
    if skew:
        bad = Tensors(zs, [n], BF16, 1, seed=7, skews=(skew,))
    at = block * BLOCK + 37
    bad.t[0][what][block if what in ("mc", "vc") else at] = value
    hp = zs.make_hparams(*HP)
    for x in (good, bad):
        zs.zs_tensors_step_async(x.list(ctx), 1, 1, hp, None, 0.0,
                                 zs.DeviceState(zs.zs_scaler_init(1.0, 1.0, 9, 1, False), step=5))
    torch.cuda.synchronize()
    g, b = good.t[0], bad.t[0]
    lo, hi = block * BLOCK, min(n, (block + 1) * BLOCK)
    moment = what[0]
    if moment != "p":
        assert torch.isnan(decode(b[moment], b[moment + "c"], n)[lo:hi]).all()
    else:
        assert torch.isnan(b["p"][at])
    for k in ("p", "h", "m", "v"):
        assert torch.equal(b[k][:lo], g[k][:lo]) and torch.equal(b[k][hi:], g[k][hi:]), k
        if k in ("m", "v") and k != moment:
            assert torch.equal(b[k], g[k])
    for k in ("mc", "vc"):
        keep = torch.arange(g[k].numel(), device="cuda") != block
        assert torch.equal(b[k][keep], g[k][keep])


@pytest.mark.parametrize("states", [0, 1])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_gradient_past_the_check_shows(zs, ctx, states, value):
    """The update alone, told that nothing overflowed, takes no NaN or inf for a
    number: the first moment shows it, in both forms, and its neighbours stay."""
    made = Tensors(zs, [2048 + 300], BF16, states, seed=3)
    for at in (5, 2300):
        made.t[0]["g"][at] = value
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    zs.zs_tensors_apply(made.list(ctx), flag, None, 0.0, 1.0, zs.make_hparams(*HP), 3)
    e = made.t[0]
    m = decode(e["m"], e["mc"], 2348) if states else e["m"]
    for at in (5, 2300):
        if np.isnan(value):
            assert torch.isnan(m[at])
        elif states == 0:
            assert torch.isinf(m[at])
        else:  # held to 2^63
            assert m[at] == m.max() and m[at] > 2.0 ** 58
    assert torch.isfinite(m[BLOCK:2048]).all()
