"""The binding of the list step and the norm refuses tensors that do not hold
what the kernels would read or write, before anything is called: formats,
sizes, contiguity and row strides.  No GPU: nothing here reaches the library."""
import pytest
import torch

EPS = 1e-5


@pytest.fixture(scope="module")
def zs():
    import zero_mixed_precision_shard_gb300 as pkg
    return pkg


class Reached(Exception):
    """The call passed the binding's checks."""


class NoCtx:
    """Stands for a context without a device: the library refuses its null
    handle, which shows that the call got there."""
    handle = None

    def __init__(self):
        self.work_bytes = {}

    def check(self, rc):
        assert rc == -1
        raise Reached


def arrays(n=600, states=0, **other):
    moment = torch.uint8 if states else torch.float32
    a = dict(grad=torch.zeros(n, dtype=torch.float16), master=torch.zeros(n),
             m=torch.zeros(n, dtype=moment), v=torch.zeros(n, dtype=moment),
             half_out=torch.zeros(n, dtype=torch.float16), m_scale=torch.zeros(-(-n // 256)),
             v_scale=torch.zeros(-(-n // 256)))
    return {**a, **other}


BAD_ENTRY = [
    ("grad", torch.zeros(599, dtype=torch.float16)), ("grad", torch.zeros(1200, dtype=torch.float16)[::2]),
    ("grad", torch.zeros(1, dtype=torch.float16).expand(600)), ("master", torch.zeros(600, dtype=torch.float64)),
    ("master", torch.zeros(600, dtype=torch.float16)), ("m", torch.zeros(599)), ("v", torch.zeros(300)),
    ("m", torch.zeros(600, dtype=torch.float16)), ("v", torch.zeros(599, dtype=torch.uint8)),
    ("half_out", torch.zeros(600)), ("half_out", torch.zeros(599, dtype=torch.bfloat16)),
    ("m_scale", torch.zeros(2)), ("v_scale", torch.zeros(2)),
    ("v_scale", torch.zeros(3, dtype=torch.float64)), ("m_scale", torch.zeros(3, dtype=torch.bfloat16)),
]


@pytest.mark.parametrize("name,bad", BAD_ENTRY)
def test_entries_that_do_not_fit(zs, name, bad):
    zs.make_tensor(**arrays())
    zs.make_tensor(**arrays(states=1))
    with pytest.raises(ValueError, match=name):
        zs.make_tensor(**arrays(**{name: bad}, count=600))


def test_entries_with_given_count_and_format(zs):
    assert zs.make_tensor(**arrays(), count=300).count == 300
    with pytest.raises(ValueError, match="grad"):
        zs.make_tensor(**arrays(), grad_dtype=zs.ZS_FP32)
    with pytest.raises(ValueError, match="grad"):
        zs.make_tensor(**arrays(grad=torch.zeros(600)), grad_dtype=zs.ZS_FP16)
    bits = arrays(grad=torch.zeros(600, dtype=torch.int16), half_out=torch.zeros(600, dtype=torch.int16))
    assert zs.make_tensor(**bits, grad_dtype=zs.ZS_BF16).grad_dtype == zs.ZS_BF16
    e = zs.make_tensor(4096, 8192, 1024, 2048, count=3, grad_dtype=zs.ZS_FP16)  # addresses
    assert (e.grad, e.master, e.count) == (4096, 8192, 3)


def test_lists_whose_moments_have_another_format(zs):
    def refused(status, states, dt="fp16", **other):
        with pytest.raises(zs.ZsError) as e:
            zs.TensorList(NoCtx(), [zs.make_tensor(**arrays(**other))], dt, states)
        assert e.value.status == status

    codes = torch.zeros(600, dtype=torch.uint8)
    refused(zs.ZS_ERR_ARG, zs.ZS_STATES_8BIT)
    refused(zs.ZS_ERR_ARG, zs.ZS_STATES_FP32, m=codes, v=codes)
    refused(zs.ZS_ERR_ARG, zs.ZS_STATES_FP32, v=codes)
    refused(zs.ZS_ERR_DTYPE, zs.ZS_STATES_FP32, dt="bf16", grad=torch.zeros(600))
    for states in (0, 1):
        with pytest.raises(Reached):
            zs.TensorList(NoCtx(), [zs.make_tensor(**arrays(states=states))], "fp16", states)


def test_new_gradients_that_do_not_fit(zs):
    lst = object.__new__(zs.TensorList)
    lst.handle, lst.ctx, lst.n = None, NoCtx(), 2
    lst.grads = [(zs.ZS_BF16, 100), (zs.ZS_FP32, 50)]
    half, full = torch.zeros(100, dtype=torch.bfloat16), torch.zeros(50)
    for grads in ([half, full], [half.view(10, 10), full], [None, 4096], [4096, full],
                  zs.pointer_array([half, full])):
        with pytest.raises(Reached):
            zs.zs_tensors_set_grads(lst, grads, stream=0)
    for grads in ([half[:99], full], [half, full[:49]], [full, full], [half, half],
                  [half.to(torch.float16), full], [half.view(10, 10).t(), full],
                  [half, torch.zeros(1).expand(50)]):
        with pytest.raises(ValueError):
            zs.zs_tensors_set_grads(lst, grads, stream=0)


def test_scalars_that_do_not_fit(zs):
    lst = object.__new__(zs.TensorList)
    lst.handle, lst.ctx, lst.n, lst.grads = None, NoCtx(), 0, []
    hp = zs.make_hparams(1e-3)
    flag, total, norm = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.float64), torch.zeros(())

    def calls(flag, total, norm):
        return [lambda: zs.zs_tensors_check(lst, 1.0, flag, total, stream=0),
                lambda: zs.zs_tensors_apply(lst, flag, total, 0.0, 1.0, hp, 1, stream=0),
                lambda: zs.zs_tensors_step_async(lst, 1, 1, hp, None, 0.0, 4096, norm, stream=0)]

    for call in calls(flag, total, norm) + calls(4096, None, None):
        with pytest.raises(Reached):
            call()
    short = torch.zeros(0, dtype=torch.int32)
    for call in (calls(flag, norm, total) + calls(total, total, flag) + calls(norm, total, total) +
                 calls(short, total, norm[None][:0])):
        with pytest.raises(zs.ZsError):
            call()


ROWS, COLS = 6, 40


def forward_args(bits=16, group=0, **other):
    h = dict(x=torch.zeros(ROWS, COLS, dtype=torch.bfloat16), residual=torch.zeros(ROWS, COLS, dtype=torch.bfloat16),
             weight=torch.zeros(COLS, dtype=torch.bfloat16), sum_out=torch.zeros(ROWS, COLS, dtype=torch.bfloat16),
             out=torch.zeros(ROWS, COLS, dtype=torch.float8_e4m3fn if bits == 8 else torch.bfloat16),
             scales=torch.zeros(ROWS, -(-COLS // group) if group else 1) if bits == 8 else None,
             rstd=torch.zeros(ROWS))
    return {**h, **other}


def backward_args(work=4096, **other):
    half = {k: torch.zeros(ROWS, COLS, dtype=torch.bfloat16) for k in ("dy", "h", "dsum", "dx")}
    a = dict(half, rstd=torch.zeros(ROWS), weight=torch.zeros(COLS, dtype=torch.bfloat16),
             dweight=torch.zeros(COLS), work=work)
    return {**a, **other}


def run(zs, args, shape=None, ctx=None, **kw):
    shape = shape or zs.make_norm_shape(ROWS, COLS, "bf16", EPS, **kw)
    call = zs.zs_rmsnorm if "x" in args else zs.zs_rmsnorm_bwd
    call(ctx or NoCtx(), shape, **args, stream=0)


HALF_BAD = [torch.zeros(ROWS, COLS), torch.zeros(ROWS, COLS, dtype=torch.float16),
            torch.zeros(ROWS, COLS - 1, dtype=torch.bfloat16), torch.zeros(COLS, ROWS, dtype=torch.bfloat16).t(),
            torch.zeros((), dtype=torch.bfloat16).expand(ROWS, COLS),
            torch.zeros(1, COLS, dtype=torch.bfloat16).expand(ROWS, COLS),
            torch.zeros(ROWS, 2 * COLS, dtype=torch.bfloat16)[:, :COLS]]


@pytest.mark.parametrize("i", range(len(HALF_BAD)))
def test_norm_rows_that_do_not_fit(zs, i):
    for args in (forward_args(), backward_args()):
        with pytest.raises(Reached):
            run(zs, args)
        for name in args:
            if args[name] is None or isinstance(args[name], int) or args[name].shape != (ROWS, COLS):
                continue
            with pytest.raises(zs.ZsError, match=name) as e:
                run(zs, {**args, name: HALF_BAD[i]})
            assert e.value.status == zs.ZS_ERR_ARG


def test_norm_vectors_that_do_not_fit(zs):
    for bits, group in ((16, 0), (8, 0), (8, 32)):
        with pytest.raises(Reached):
            run(zs, forward_args(bits, group), bits=bits, group=group)
    with pytest.raises(Reached):
        run(zs, forward_args(8, 32, out=torch.zeros(ROWS, COLS, dtype=torch.uint8)), bits=8, group=32)
    bad = [({"weight": torch.zeros(COLS - 1, dtype=torch.bfloat16)}, 16, 0), ({"weight": torch.zeros(COLS)}, 16, 0),
           ({"rstd": torch.zeros(ROWS - 1)}, 16, 0), ({"rstd": torch.zeros(ROWS, dtype=torch.bfloat16)}, 16, 0),
           ({"rstd": torch.zeros(2 * ROWS)[::2]}, 16, 0),
           ({"out": torch.zeros(ROWS, COLS, dtype=torch.float8_e4m3fn)}, 16, 0),
           ({"out": torch.zeros(ROWS, COLS, dtype=torch.bfloat16)}, 8, 0),
           ({"scales": torch.zeros(ROWS - 1)}, 8, 0), ({"scales": torch.zeros(ROWS)}, 8, 32),
           ({"scales": torch.zeros(ROWS, 2, dtype=torch.float16)}, 8, 32)]
    for other, bits, group in bad:
        with pytest.raises(zs.ZsError, match=next(iter(other))):
            run(zs, forward_args(bits, group, **other), bits=bits, group=group)
    for other in ({"dweight": torch.zeros(COLS - 1)}, {"dweight": torch.zeros(COLS, dtype=torch.bfloat16)},
                  {"rstd": torch.zeros(ROWS - 1)}, {"weight": torch.zeros(COLS)}):
        with pytest.raises(zs.ZsError, match=next(iter(other))):
            run(zs, backward_args(**other))


def test_norm_strides_that_do_not_fit(zs):
    """A row stride of the shape's own needs memory that reaches as far, and the
    tensor's own stride where it has these rows."""
    wide = torch.zeros(ROWS, 64, dtype=torch.bfloat16)
    strides = dict(x_stride=64, residual_stride=64, sum_stride=64, out_stride=64, dy_stride=64, dx_stride=64)
    views = {k: wide[:, :COLS] for k in ("x", "residual", "sum_out", "out")}
    with pytest.raises(Reached):
        run(zs, forward_args(**views), **strides)
    with pytest.raises(Reached):  # the last row ends with its elements, at the storage's end
        run(zs, forward_args(x=wide.view(-1)[24:].as_strided((ROWS, COLS), (64, 1))), x_stride=64)
    back = {k: wide[:, :COLS] for k in ("dy", "h", "dsum", "dx")}
    with pytest.raises(Reached):
        run(zs, backward_args(**back), **strides)
    for args, names in ((forward_args(**views), views), (backward_args(**back), back)):
        for name in names:
            for bad in (torch.zeros(ROWS, COLS, dtype=torch.bfloat16), wide[:, 25:][:, :COLS][1:],
                        torch.zeros(ROWS, 80, dtype=torch.bfloat16)[:, :COLS], wide[:, :COLS].float()):
                with pytest.raises(zs.ZsError, match=name):
                    run(zs, {**args, name: bad}, **strides)


def test_workspace_that_does_not_fit(zs):
    ctx = NoCtx()
    ctx.work_bytes[ROWS, COLS] = 320
    with pytest.raises(Reached):
        run(zs, backward_args(work=torch.zeros(320, dtype=torch.uint8)), ctx=ctx)
    with pytest.raises(Reached):
        run(zs, backward_args(work=torch.zeros(80)), ctx=ctx)
    for bad in (torch.zeros(319, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8).expand(320)):
        with pytest.raises(zs.ZsError, match="work"):
            run(zs, backward_args(work=bad), ctx=ctx)


def test_a_shape_that_changes(zs):
    """What its arrays hold goes by the shape as it is at the call."""
    shape = zs.make_norm_shape(ROWS, COLS, "bf16", EPS)
    args = forward_args()
    with pytest.raises(Reached):
        run(zs, args, shape)
    shape.rows = ROWS + 1
    with pytest.raises(zs.ZsError, match="x holds"):
        run(zs, args, shape)
    shape.rows = ROWS - 1
    with pytest.raises(Reached):
        run(zs, args, shape)
    shape.dt = zs.ZS_FP16
    with pytest.raises(zs.ZsError, match="x is"):
        run(zs, args, shape)


def test_objects_with_an_address_alone(zs):
    class Buffer:
        def data_ptr(self):
            return 4096

    with pytest.raises(Reached):
        run(zs, {k: None if t is None else Buffer() for k, t in forward_args().items()})
    with pytest.raises(Reached):
        run(zs, {k: Buffer() for k in backward_args()})
