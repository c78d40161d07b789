"""The list step's clipping coefficient and norm are formed as the flat shard's:
the same bits from the same sum of squares, in one call or in two phases."""
import numpy as np
import pytest
import torch

from _tensors import BF16, FP16, HP, Tensors

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


@pytest.mark.parametrize("dt", [FP16, BF16])
def test_clipped_update_equals_the_flat_one(zs, ctx, dt):
    """From one sum of squares both forms take the same coefficient, bit for bit."""
    rng = np.random.default_rng(11)
    hp = zs.make_hparams(*HP)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    made = Tensors(zs, [4096], dt, 0, seed=1)
    flat = made.clone().t[0]
    lst = made.list(ctx)
    start = {k: x.clone() for k, x in made.t[0].items()}
    for i in range(60):
        sumsq = torch.tensor([float(np.exp(rng.uniform(-6, 6)))], dtype=torch.float64, device="cuda")
        limit = float(np.float32(sumsq.sqrt().item() * rng.uniform(0.05, 1.05)))
        for k, x in start.items():
            made.t[0][k].copy_(x)
        w = {k: x.clone() for k, x in flat.items()}
        zs.zs_tensors_apply(lst, flag, sumsq, limit, 7.0, hp, 4)
        zs.zs_apply_clipped(ctx, flag, sumsq, limit, [w["g"]], dt, None, 4096, 7.0, w["p"], w["m"],
                            w["v"], w["h"], hp, 4)
        for k in ("p", "m", "v", "h"):
            assert torch.equal(made.t[0][k], w[k]), (i, k)


@pytest.mark.parametrize("states", [0, 1])
@pytest.mark.parametrize("n,accum,scale", [(3, 1, 1.0), (1, 5, 7.0), (2, 1, 1024.0)])
def test_phases_equal_the_step_for_any_divisor(zs, ctx, states, n, accum, scale):
    for k in range(12):
        a = Tensors(zs, [5000, 33], BF16, states, seed=100 + k)
        b = a.clone()
        hp = zs.make_hparams(*HP)
        norm = torch.zeros((), device="cuda")
        zs.zs_tensors_step_async(a.list(ctx), n, accum, hp, None, 0.2 + 0.01 * k,
                                 zs.DeviceState(zs.zs_scaler_init(scale, 1.0, 9, 1, False), step=6),
                                 norm)
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
        lst = b.list(ctx)
        zs.zs_tensors_check(lst, n * accum * scale, flag, sumsq)
        zs.zs_tensors_apply(lst, flag, sumsq, 0.2 + 0.01 * k, n * accum * scale, hp, 7)
        assert all(torch.equal(x[key], y[key]) for x, y in zip(a.t, b.t) for key in x)
        assert norm.item() == np.float32(np.sqrt(sumsq.item()))
