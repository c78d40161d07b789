"""Lists of random tensors made on the GPU, and their 8-bit moments decoded and
encoded by plain operations; shared by the tests of the list step."""
import numpy as np
import torch

FP16, BF16 = 0, 1
TORCH = {FP16: torch.float16, BF16: torch.bfloat16}
BLOCK = 256
HP = (3e-4, 0.9, 0.999, 1e-8, 0.01)


class Tensors:
    """Random tensors of a list, made on the GPU.  grads: "half", "fp32", or
    "mixed" (in turn); skews: elements in front of each tensor's arrays, in turn."""

    def __init__(self, zs, sizes, dt, states, seed=0, grads="half", skews=(0,), sigma=0.05):
        self.zs, self.dt, self.states = zs, dt, states
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.t = []
        for i, n in enumerate(sizes):
            skew = skews[i % len(skews)]

            def put(x):
                base = torch.zeros(len(x) + skew, dtype=x.dtype, device="cuda")
                base[skew:] = x
                return base[skew:]

            def normal(k=n):
                return torch.randn(k, device="cuda", generator=gen)

            fp32 = grads == "fp32" or (grads == "mixed" and i % 2 == 1)
            e = {"g": put((normal() * sigma).to(torch.float32 if fp32 else TORCH[dt])),
                 "p": put(normal() * 0.02), "h": put(torch.zeros(n, dtype=TORCH[dt], device="cuda"))}
            blocks = -(-n // BLOCK)
            if states == 1:
                e["m"] = put((normal().clamp(-3, 3) * 100).to(torch.float8_e4m3fn).view(torch.uint8))
                e["v"] = put(normal().exp().clamp(0.1, 400).to(torch.float8_e4m3fn).view(torch.uint8))
                e["mc"] = put(torch.rand(blocks, device="cuda", generator=gen) * 1e-4)
                e["vc"] = put(torch.rand(blocks, device="cuda", generator=gen) * 1e-4)
            else:
                e["m"], e["v"] = put(normal() * 0.01), put(torch.rand(n, device="cuda", generator=gen) * 1e-3)
            self.t.append(e)

    def entries(self, **kw):
        return [self.zs.make_tensor(e["g"], e["p"], e["m"], e["v"], e["h"], e.get("mc"),
                                    e.get("vc"), **kw) for e in self.t]

    def list(self, ctx):
        return self.zs.TensorList(ctx, self.entries(), self.dt, self.states)

    def clone(self, states=None):
        """A copy; with states=0 of 8-bit tensors, their decoded moments in 32 bits."""
        c = object.__new__(Tensors)
        c.zs, c.dt = self.zs, self.dt
        c.states = self.states if states is None else states
        c.t = [{k: x.clone() for k, x in e.items()} for e in self.t]
        if c.states != self.states:
            for e in c.t:
                n = e["p"].numel()
                r = decode(e["v"], e.pop("vc"), n)
                e["m"], e["v"] = decode(e["m"], e.pop("mc"), n), r * r
        return c


def decode(codes, scales, n):
    """E4M3 bytes times their block's scale, an fp32 product each."""
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(BLOCK)[:n]


def encode(x, root):
    """Bytes and scales of fp32 values, by IEEE divisions on the host."""
    x = x.cpu().numpy()
    n = len(x)
    rows = np.concatenate([x, np.zeros(-n % BLOCK, np.float32)]).reshape(-1, BLOCK)
    c = np.maximum(np.abs(rows).max(1) / np.float32(448), np.float32(2.0 ** -126))
    q = rows / c[:, None]
    if root:
        q = np.where(rows > 0, np.maximum(q, np.float32(2.0 ** -9)), q)
    codes = torch.from_numpy(q.reshape(-1)[:n]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.from_numpy(c)


def equal_bits(a, b):
    """Bit for bit, except that codes of zero of either sign are equal."""
    if a.element_size() == 1:
        a, b = a.cpu(), b.cpu()
        return bool(((a == b) | ((a & 0x7F) + (b & 0x7F) == 0)).all())
    return torch.equal(a.cpu(), b.cpu())


def assert_8bit_equals_32bit(zs, ctx, made, div, max_norm, t=3):
    """One step of the 8-bit list against one of the 32-bit list from its decoded
    moments: the new moments' bytes and scales bit for bit, and the weights within
    the rounding of the update by 32-bit operations, in half units of 2^-24: of
    the update 1 each for m_hat, the root, its bias correction, eps, the quotient and
    the decay's addition (and 2^-4 for what a corrected quotient or root leaves), of
    the decay 1, of the weight 1."""
    wide, start = made.clone(states=0), [e["p"].double() for e in made.t]
    hp = zs.make_hparams(*HP)
    for x in (made, wide):
        lst = x.list(ctx)
        d = zs.DeviceState(zs.zs_scaler_init(div, 1.0, 1000, 1, True), step=t - 1)
        zs.zs_tensors_step_async(lst, 1, 1, hp, None, max_norm, d)
        assert d.read().overflow == 0
        lst.close()
    lr, b1, b2, eps, wd = (float(np.float32(x)) for x in HP)
    for e, w, p0 in zip(made.t, wide.t, start):
        m, v = w["m"].double() / (1 - b1 ** t), w["v"].double() / (1 - b2 ** t)
        u = m / (v.sqrt() + eps)
        want = p0 - lr * (u + wd * p0)
        bound = 2.0 ** -24 * (lr * (6.0625 * u.abs() + wd * p0.abs()) + want.abs()) + 2.0 ** -149
        assert ((e["p"].double() - want).abs() <= bound).all()
        assert torch.equal(e["h"], e["p"].to(e["h"].dtype))
        for key, scale, x in (("m", "mc", w["m"]), ("v", "vc", torch.from_numpy(
                np.sqrt(w["v"].cpu().numpy())))):
            codes, c = encode(x, key == "v")
            assert torch.equal(e[scale].cpu(), c), scale
            assert equal_bits(e[key], codes), key
