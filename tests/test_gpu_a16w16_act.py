"""GPU tests of what the few-token layer on 16-bit experts holds between its two
products: topk_w * act in f32, with f32's bits and f32's range.

The inputs are whole numbers whose sums and products f32 holds exactly, the gates
beyond 88, where silu(g) = g to f32's last bit: the outputs have to be exact.
"""

import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16}


class Layer:
    """x = (1, 64, 0, ...) for every token, so that a row (v % 64, v // 64) of w1 makes v."""

    def __init__(self, n, H, F, E, k, dt, seed=0):
        self.g = torch.Generator()
        self.g.manual_seed(seed)
        self.d = mx.Dims(T=n, T_max=n, H=H, F=F, E=E, k=k, P_total=E, p0=0, P_local=E, R_max=1)
        self.dt = T[dt]
        self.x = torch.zeros(n, H)
        self.x[:, 0], self.x[:, 1] = 1.0, 64.0
        self.logits = torch.zeros(n, E)
        self.w1, self.w2 = torch.zeros(E, 2 * F, H), torch.zeros(E, H, F)

    def make(self, row, v):
        """Row `row` (of all experts, [E, ...]) of w1 makes the whole numbers v."""
        self.w1[:, row, 0], self.w1[:, row, 1] = (v % 64).float(), (v // 64).float()

    def run(self):
        dev = lambda t: t.to(self.dt).cuda()  # noqa: E731
        E = self.d.E
        out = torch.full((self.d.T, self.d.H), 7.0, dtype=self.dt, device="cuda")
        ws = mx.a16w16_workspace(self.d)
        ws.fill_(0xFF)
        mx.moe_forward_a16w16(self.d, dev(self.x), self.logits.cuda(), dev(self.w1), dev(self.w2),
                              torch.ones(E, dtype=torch.int32, device="cuda"),
                              torch.arange(E, dtype=torch.int32, device="cuda"), out, ws)
        torch.cuda.synchronize()
        return out.float().cpu()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,H,F,E,k", [(1, 128, 128, 2, 1), (3, 256, 640, 4, 2), (16, 2176, 256, 3, 1), (20, 256, 512, 4, 2),
                                       (32, 8320, 384, 5, 1), (9, 4224, 2048, 2, 2), (5, 128, 16384, 2, 1)])
def test_bits_of_act(n, H, F, E, k, dt):
    """act of a pair of columns is a * a and (a + 1)(a - 1), up to 24 bits each, and w2
    takes their difference: 1, times 4 for a token of twice the x.  (Equal logits: the
    first k experts, in equal shares.)"""
    print(f"[case] n={n} H={H} F={F} E={E} k={k} {dt}", flush=True)
    c = Layer(n, H, F, E, k, dt, F + n)
    i, j = torch.randperm(F, generator=c.g).view(2, -1)   # the pairs, anywhere in the row
    a = torch.randint(100, 4095, (E, F // 2), generator=c.g)
    c.make(i, a)
    c.make(F + i, a)
    c.make(j, a + 1)
    c.make(F + j, a - 1)
    for h in range(H):
        c.w2[:, h, i[h % (F // 2)]], c.w2[:, h, j[h % (F // 2)]] = 1.0, -1.0
    twice = torch.arange(n) % 2
    c.x *= 2.0 ** twice[:, None]
    got = c.run()
    want = (4.0 ** twice)[:, None].expand(n, H)
    # One expert: every sum is a whole number below 2^24, exact.  Two, in halves: the sums
    # are multiples of 0.5 below 4095^2 < 2^24, where f32's half step is 0.5; an output
    # adds 2 k products in three parts, 6 k additions at most, each off by 0.5, and is
    # then rounded (half a step of bf16 at 7: 2^-6).
    tol = (0.0 if k == 1 else 6 * k * 0.5 + 2.0 ** -6) * want
    assert torch.all((got - want).abs() <= tol), (got - want).abs().max()
    if k == 1:
        assert torch.equal(got, want)


def test_f16_range_of_act():
    """act of 16 million, far past f16's 65504, where the output is an f16 number; and a
    small act beside it in the same 64 columns."""
    for n in (1, 20):
        c = Layer(n, 256, 128, 1, 1, "f16")
        c.make(torch.arange(256), torch.full((1, 256), 4095))
        c.w2[0, :, 0] = 2.0 ** -14
        c.w1[0, 1, :2], c.w1[0, 128 + 1, :2] = torch.tensor([0.0, 2.0]), torch.tensor([2.0 ** -17, 0.0])   # 128 * 2^-17
        c.w2[0, 128:] = 0.0
        c.w2[0, 128:, 1] = 1.0
        got = c.run()
        want = torch.full((n, 256), 4095.0 * 4095.0 * 2.0 ** -14).half().float()
        want[:, 128:] = 2.0 ** -10
        assert torch.equal(got, want), (got, want)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_infinite_act(dt):
    """An infinite act is infinite times w2's sign, and NaN times zero; finite columns
    beside it, and other experts' tokens, do not change."""
    for n in (2, 20):
        c = Layer(n, 128, 256, 2, 1, dt)
        c.make(torch.arange(512), torch.full((2, 512), 100))
        c.logits[:, 0] = torch.arange(n) % 2 * 2.0 - 1.0   # odd tokens: expert 0
        c.w2[:, :, 70], c.w2[:, :, 71] = 1.0, 2.0
        c.w2[0, 1, 70], c.w2[0, 2, 70] = -1.0, 0.0
        clean = c.run()
        assert torch.all(clean[:, 0] == torch.tensor(30000.0).to(c.dt).float())
        c.w1[0, 256 + 70, 0] = float("inf")
        got = c.run()
        assert torch.equal(got[::2], clean[::2])
        assert torch.all(got[1::2, 0] == float("inf")) and torch.all(got[1::2, 1] == -float("inf"))
        assert torch.all(torch.isnan(got[1::2, 2])) and torch.all(got[1::2, 3:] == float("inf"))
