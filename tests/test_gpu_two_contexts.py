"""Several contexts in one process, as programs with overlapping work have
them: what one context launches leaves the others' calls as they were.  The
pairs are launches of one kernel with different amounts of shared memory, the
larger before and after the smaller."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def zs():
    import zero_mixed_precision_shard_gb300 as pkg
    torch.cuda.set_device(0)
    return pkg


@pytest.fixture
def contexts(zs):
    pair = zs.Ctx(), zs.Ctx()
    yield pair
    for c in pair:
        c.close()


def halves(cols, seed, rows=40):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, cols, device="cuda", generator=g).to(torch.bfloat16)


def gradients(zs, ctx, cols, dsum, stream=None):
    h, dy = halves(cols, 1), halves(cols, 2)
    ds = halves(cols, 3) if dsum else None
    w, rstd = halves(cols, 4, 1)[0], torch.rsqrt(h.float().square().mean(1) + EPS)
    shape = zs.make_norm_shape(len(h), cols, "bf16", EPS)
    work = torch.empty(zs.zs_rmsnorm_bwd_work(ctx, shape), dtype=torch.uint8, device="cuda")
    dx, dw = torch.zeros_like(h), torch.zeros(cols, device="cuda")
    zs.zs_rmsnorm_bwd(ctx, shape, dy, h, rstd, w, ds, dx, dw, work, stream=stream)
    return dx, dw


def forward(zs, ctx, cols, residual, stream=None):
    x, w = halves(cols, 1), halves(cols, 4, 1)[0]
    res = halves(cols, 2) if residual else None
    total, y = torch.zeros_like(x) if residual else None, torch.zeros_like(x)
    zs.zs_rmsnorm(ctx, zs.make_norm_shape(len(x), cols, "bf16", EPS), x, res, w, total, y,
                  stream=stream)
    return (y, total) if residual else (y,)


PAIRS = [
    (gradients, (8192, True), (8192, False)),   # three arrays in the ring, then two
    (gradients, (4096, True), (3584, True)),    # two widths of one kernel
    (gradients, (16_384, True), (8448, True)),
    (forward, (8192, True), (8192, False)),
    (forward, (8192, True), (6144, True)),
    (forward, (16_384, True), (16_384, False)),
    (forward, (16_383, True), (8447, True)),    # rows off the 16-byte boundary
]


@pytest.mark.parametrize("call,large,small", PAIRS)
def test_a_smaller_launch_elsewhere_does_not_bind(zs, contexts, call, large, small):
    a, b = contexts
    first = call(zs, a, *large)
    call(zs, b, *small)
    again = call(zs, a, *large)
    assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_two_threads_with_a_context_each(zs, contexts):
    """Calls of two host threads interleaved at will, each on its own stream."""
    want = [[t.clone() for t in gradients(zs, contexts[0], 8192, dsum)] for dsum in (True, False)]
    torch.cuda.synchronize()
    errors = []

    def work(ctx, k):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for i in range(60):
                    got = gradients(zs, ctx, 8192, (i + k) % 2 == 0)
                    stream.synchronize()
                    for x, y in zip(got, want[(i + k) % 2]):
                        assert torch.equal(x, y)
        except Exception as e:  # noqa: BLE001 (reported by the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c, k)) for k, c in enumerate(contexts)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
