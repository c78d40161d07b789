"""Long lists, whose chunks have several units: the update refills its ring, the
CTAs of the check pass stride over chunks of both gradient formats, and the
ragged last units of tensors lie between whole ones."""
import pytest
import torch

from _tensors import BF16, FP16, HP, Tensors, assert_8bit_equals_32bit

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


# beyond the length from which chunks have several units: tensors of many
# chunks with ragged last units, and short ones between them
LONG = [6_000_000, 100, 8192 * 3, 5_300_001, 2047, 1, 2_500_033, 8193, 3_000_000]


@pytest.mark.parametrize("dt", [FP16, BF16])
@pytest.mark.parametrize("grads", ["half", "mixed"])
@pytest.mark.parametrize("skews", [(0,), (0, 1, 0, 3)])
def test_long_list_of_32bit_moments(zs, ctx, dt, grads, skews):
    """Bit for bit the flat update (fp32 gradients: as its accumulator), and the norm."""
    made = Tensors(zs, LONG, dt, 0, seed=5, grads=grads, skews=skews)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    hp = zs.make_hparams(*HP)
    want = []
    for e in made.t:
        w = {k: e[k].clone() for k in ("p", "m", "v", "h")}
        half = e["g"].dtype != torch.float32
        g = e["g"].clone()
        zs.zs_apply(ctx, flag, [g] if half else None, dt, None if half else g, g.numel(), 512.0,
                    w["p"], w["m"], w["v"], w["h"], hp, 3)
        want.append(w)
    norm = torch.zeros((), device="cuda")
    d = zs.DeviceState(zs.zs_scaler_init(512.0, 1.0, 1000, 1, True), step=2)
    zs.zs_tensors_step_async(made.list(ctx), 1, 1, hp, None, 0.0, d, norm)
    for e, w in zip(made.t, want):
        for k in w:
            assert torch.equal(w[k], e[k]), (k, e["p"].numel())
    ref = sum(e["g"].double().square().sum().item() for e in made.t) ** 0.5 / 512.0
    assert abs(norm.item() - ref) <= 1e-6 * ref


@pytest.mark.parametrize("dt", [FP16, BF16])
@pytest.mark.parametrize("grads", ["half", "mixed"])
@pytest.mark.parametrize("skews", [(0,), (0, 1, 0, 3)])
def test_long_list_of_8bit_moments(zs, ctx, dt, grads, skews):
    made = Tensors(zs, LONG, dt, 1, seed=6, grads=grads, skews=skews)
    assert_8bit_equals_32bit(zs, ctx, made, 256.0, 0.05)


@pytest.mark.parametrize("states", [0, 1])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_overflow_anywhere_in_a_long_list(zs, ctx, states, bad):
    """One bad gradient, in turn in the first and later units and chunks of a
    CTA of the check pass, in either format: nothing is written."""
    made = Tensors(zs, LONG, BF16, states, seed=8, grads="mixed", skews=(0, 1))
    before = made.clone()
    lst = made.list(ctx)
    d = zs.DeviceState(zs.zs_scaler_init(1.0, 1.0, 1000, 1, False), step=2)
    hp = zs.make_hparams(*HP)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    stride = 4 * sms * 8192  # elements between two chunks of one CTA
    places = [(0, 0), (0, 2048), (0, 8191), (0, 5_999_999), (3, 0), (3, 9000), (3, 5_300_000),
              (0, stride + 4095), (6, 2_500_032), (8, 6000), (8, 2_999_999), (5, 0), (7, 8192)]
    for i, (k, at) in enumerate(places):
        keep = made.t[k]["g"][at].clone()
        made.t[k]["g"][at] = bad
        zs.zs_tensors_step_async(lst, 1, 1, hp, None, 1.0, d)
        made.t[k]["g"][at] = keep
        s = d.read()
        assert (s.overflow, s.step, s.iterations) == (1, 2, i + 1), (k, at)
    for e, b in zip(made.t, before.t):
        assert all(torch.equal(e[key], b[key]) for key in e)
