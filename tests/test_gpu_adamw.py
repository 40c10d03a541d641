"""GPU tests of the AdamW step: bit for bit against the formulas evaluated in fp32 with one rounding an operation
(tests/train_ref.py, on the CPU), and against fp64; 8-bit states against their definition."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
F8 = torch.float8_e4m3fn
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.05)
SIZES = [1, 3, 4, 127, 128, 129, 4096, 4097, 5000, 768 * 64, 100_003]


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


def fp32_step(w, g, m, v, step, clip=None, lr=HYPER["lr"]):
    return ref.adamw_fp32(w, g, m, v, step, lr, HYPER["beta1"], HYPER["beta2"], HYPER["eps"], HYPER["weight_decay"], clip)


class Tensors:
    """Parameters of the given sizes: every third bf16 with a master, every third bf16 without."""

    def __init__(self, sizes, bits, seed, offset=0):
        gen = torch.Generator().manual_seed(seed)

        def normal(n, std):
            return torch.randn(n, generator=gen) * std

        def on(t):  # `offset` elements past an aligned address
            buf = torch.zeros(t.numel() + offset, dtype=t.dtype, device=DEV)
            buf[offset:] = t.to(DEV)
            return buf[offset:]

        self.bits, self.sizes = bits, sizes
        self.w = [normal(n, 0.5) for n in sizes]     # on the CPU: what the step starts from
        self.kind = [(torch.float32, False), (BF, True), (BF, False)]
        self.kind = [self.kind[i % 3] for i in range(len(sizes))]
        self.w = [w if k == torch.float32 or master else w.to(k).float() for w, (k, master) in zip(self.w, self.kind)]
        self.params = [on(w.to(k)) for w, (k, _) in zip(self.w, self.kind)]
        self.masters = [on(w) if master else None for w, (_, master) in zip(self.w, self.kind)]
        self.g = [normal(n, 1e-2).to(k).float() for n, (k, _) in zip(sizes, self.kind)]
        self.grads = [on(g.to(k)) for g, (k, _) in zip(self.g, self.kind)]
        self.m, self.v = [normal(n, 1e-2) for n in sizes], [normal(n, 1e-2).square() for n in sizes]
        if bits == 32:
            self.avgs, self.sqs = [on(m) for m in self.m], [on(v) for v in self.v]
            self.scales = {}
        else:
            self.avgs, self.sqs, ms, rs = [], [], [], []
            for i, n in enumerate(sizes):
                held = ref.ceil(n, 128) * 128
                for src, codes, scales in ((self.m[i], self.avgs, ms), (ref.root(self.v[i]), self.sqs, rs)):
                    pad = torch.zeros(held)
                    pad[:n] = src
                    q, s = ref.quantized(pad.view(-1, 128))
                    codes.append(q.to(F8).view(-1).to(DEV))
                    scales.append(s.float().view(-1).to(DEV))
                self.m[i] = (self.avgs[i].cpu().float().view(-1, 128) * ms[i].cpu()[:, None]).view(-1)[:n]
                r = (self.sqs[i].cpu().float().view(-1, 128) * rs[i].cpu()[:, None]).view(-1)[:n]
                self.v[i] = r * r
            self.scales = dict(avg_scales=ms, sq_scales=rs)

    def step(self, gk, step, **kw):
        hyper = dict(HYPER, **{k: kw.pop(k) for k in list(kw) if k in HYPER})
        gk.grkan_adamw_step(self.params, self.grads, self.avgs, self.sqs, step=step, masters=self.masters, **hyper,
                            **self.scales, **kw)

    def compare(self, step, seed=0, clip=None, lr=HYPER["lr"]):
        """Bit for bit against the fp32 formulas; keeps the new values."""
        block = 0
        for i, n in enumerate(self.sizes):
            w, m, v = fp32_step(self.w[i], self.g[i], self.m[i], self.v[i], step, clip, lr)
            kind, master = self.kind[i]
            p = self.params[i].cpu()
            assert torch.equal(p, w.to(kind)), f"parameter {i}"
            if master:
                assert torch.equal(self.masters[i].cpu(), w), f"master {i}"
            self.w[i] = w if master or kind == torch.float32 else p.float()
            if self.bits == 32:
                assert torch.equal(self.avgs[i].cpu(), m) and torch.equal(self.sqs[i].cpu(), v), f"moments {i}"
                self.m[i], self.v[i] = m, v
                continue
            nb = ref.ceil(n, 128)
            r32 = ref.random32(seed, step, block, nb)
            block += nb
            new = []
            for src, codes, scales, r16, root in ((m, self.avgs[i], self.scales["avg_scales"][i], r32 & 0xFFFF, False),
                                                  (ref.root(v), self.sqs[i], self.scales["sq_scales"][i], r32 >> 16, True)):
                pad = torch.zeros(nb * 128)
                pad[:n] = src
                q, s = ref.round_up_sometimes(pad.view(nb, 128), r16, root)
                assert torch.equal(scales.cpu().double(), s), f"scales {i}"
                assert torch.equal(codes.cpu().float().double().view(nb, 128), q), f"codes {i}"
                new.append((q * s[:, None]).float().view(-1)[:n])
            self.m[i], self.v[i] = new[0], new[1] * new[1]


@pytest.mark.parametrize("offset", (0, 1))
@pytest.mark.parametrize("bits", (32, 8))
def test_steps(gk, bits, offset):
    """Three steps of parameters of every size and kind, aligned and not."""
    t = Tensors(SIZES, bits, 1, offset)
    for step in (1, 2, 1000):
        print(f"[adamw] {bits} {offset} {step}", flush=True)
        t.step(gk, step, seed=7)
        t.compare(step, 7)


@pytest.mark.parametrize("bits", (32, 8))
def test_more_tensors_than_a_launch_holds(gk, bits):
    t = Tensors([5, 0, 300, 1, 129] * 40, bits, 2)
    t.step(gk, 3, seed=9)
    t.compare(3, 9)


@pytest.mark.parametrize("bits", (32, 8))
def test_device_scalars_and_graph(gk, bits):
    """step, lr and the gradients' factor read on the device: each replay of a captured step takes them as they are
    then."""
    t = Tensors([300, 5000, 129], bits, 3)
    step = torch.tensor([4], device=DEV)
    lr = torch.tensor([1e-3], device=DEV)
    clip = torch.tensor([0.3], device=DEV)
    lr32 = lambda: float(lr.cpu().double())  # noqa: E731
    t.step(gk, step, lr=lr, grad_scale=clip, seed=5)
    t.compare(4, 5, clip.cpu(), lr32())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.step(gk, step, lr=lr, grad_scale=clip, seed=5)
    for k, rate, c in ((5, 2e-3, 1.5), (6, 5e-4, 0.1), (100, 1e-2, 0.7)):
        step.fill_(k), lr.fill_(rate), clip.fill_(c)
        graph.replay()
        torch.cuda.synchronize()
        t.compare(k, 5, clip.cpu(), lr32())


def test_against_fp64(gk):
    """The formulas in fp64: m within 3 u of its terms, v within 4 u, the weight within 3 u of itself (1 - lr
        weight_decay is rounded, its product with the weight, and the difference) and 16 u of its step."""
    t = Tensors([100_000], 32, 4)
    w, g, m, v = (x[0].double() for x in (t.w, t.g, t.m, t.v))
    t.step(gk, 10)
    m2 = 0.9 * m + 0.1 * g
    v2 = 0.999 * v + 0.001 * g * g
    move = HYPER["lr"] * (m2 / (1 - 0.9 ** 10)) / ((v2 / (1 - 0.999 ** 10)).sqrt() + 1e-8)
    w2 = w * (1 - HYPER["lr"] * 0.05) - move
    u = ref.U
    ref.check("m", t.avgs[0].cpu(), m2, 3 * u * (0.9 * m.abs() + 0.1 * g.abs()))
    ref.check("v", t.sqs[0].cpu(), v2, 4 * u * v2)
    em = 3 * u * (0.9 * m.abs() + 0.1 * g.abs()) / m2.abs().clamp_min(1e-30) * move.abs()
    ref.check("w", t.params[0].cpu(), w2, 3 * u * w.abs() + 16 * u * move.abs() + em)


def test_rounding_has_no_drift(gk):
    """The mean over 4,096 seeds of a moment's 8-bit value is the moment: within 6 of its standard error, a step
    of e4m3 over 2 at most a draw, and the 2^-17 of a step that 16 random bits leave.  A root that is not 0 stays so."""
    n, seeds = 128, 4096
    gen = torch.Generator().manual_seed(5)
    m = torch.randn(n, generator=gen) * 2.0 ** torch.randint(-14, 1, (n,), generator=gen)
    total, least = torch.zeros(n, dtype=torch.float64, device=DEV), []
    p, g = torch.zeros(n, device=DEV), (m / (1 - 0.9)).to(DEV)
    want, _ = fp32_step(torch.zeros(n), g.cpu(), torch.zeros(n), torch.zeros(n), 1)[1:]
    for seed in range(seeds):
        avg, sq, ms, rs = gk.grkan_adamw_state(p, 8)
        gk.grkan_adamw_step([p], [g], [avg], [sq], step=1, lr=0.0, avg_scales=[ms], sq_scales=[rs], seed=seed)
        total += avg.float().double() * ms.double()
        least.append(sq.float().amin())
    scale = float(ms)
    step = ref.binade((want.double().abs() / scale).clamp_min(2.0 ** -6)) / 8 * scale
    ref.check("mean", (total / seeds).cpu(), want.double(), step * (0.5 * 6 / seeds ** 0.5 + 2.0 ** -17))
    assert float(torch.stack(least).min()) > 0


def test_special_values(gk):
    """A NaN or infinite gradient spoils its own value only; in 8 bits it is kept as a NaN, apart from the scale."""
    for bits in (32, 8):
        t = Tensors([256], bits, 6)
        t.grads[0][3], t.grads[0][130] = torch.nan, torch.inf
        t.step(gk, 2)
        p, m = t.params[0].cpu(), t.avgs[0].cpu().float()
        bad = torch.zeros(256, dtype=torch.bool)
        bad[3] = bad[130] = True
        assert p[bad].isnan().all() and p[~bad].isfinite().all() and m[~bad].isfinite().all()
        assert not m[bad].isfinite().any()


def test_optimizer(gk):
    """The optimizer is the step over its parameters, counts steps apart for parameters without a gradient, and
    goes on from a saved state with the same bits."""
    for bits in (32, 8):
        gen = torch.Generator().manual_seed(7)
        shapes = [(40, 30), (129,), (7, 8, 9)]

        def params():
            gen.manual_seed(8)
            return [torch.nn.Parameter(torch.randn(s, generator=gen).to(DEV).to(BF if i == 0 else torch.float32))
                    for i, s in enumerate(shapes)]

        def grads(ps, step):
            gen.manual_seed(100 + step)
            for i, q in enumerate(ps):
                q.grad = torch.randn(q.shape, generator=gen).to(DEV).to(q.dtype)
                if step == 2 and i == 1:
                    q.grad = None

        a, b = params(), params()
        one = gk.GRKANAdamW(a, lr=1e-2, bits=bits, seed=3)
        for step in (1, 2, 3):
            grads(a, step)
            one.step()
        assert [one.state[q]["step"] for q in a] == [3, 2, 3]
        two = gk.GRKANAdamW(b, lr=1e-2, bits=bits, seed=3)
        for step in (1, 2):
            grads(b, step)
            two.step()
        saved = two.state_dict()
        three = gk.GRKANAdamW(b, lr=1e-2, bits=bits, seed=3)
        three.load_state_dict(saved)
        grads(b, 3)
        three.step()
        for p, q in zip(a, b):
            assert torch.equal(p, q)
        # the bf16 parameter is its master's rounded copy
        assert torch.equal(a[0], one.state[a[0]]["master"].to(BF)) and one.state[a[0]]["master"].dtype == torch.float32


def test_optimizer_refuses_a_capture(gk):
    """A captured step would hold its step number: refused before anything is launched or counted."""
    p = torch.nn.Parameter(torch.ones(300, device=DEV))
    p.grad = torch.ones_like(p)
    opt = gk.GRKANAdamW([p])
    opt.step()
    before = p.detach().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captur"):
            opt.step()
    assert opt.state[p]["step"] == 1 and torch.equal(p, before)


def test_optimizer_copies(gk):
    """A copy, and one that takes a saved state, round with the seed of the original."""
    import copy

    def start():
        p = torch.nn.Parameter(torch.linspace(-1.0, 1.0, 1000, device=DEV))
        p.grad = torch.linspace(-0.3, 0.7, 1000, device=DEV)
        return p

    a = start()
    one = gk.GRKANAdamW([a], bits=8, seed=5)
    one.step()
    two = copy.deepcopy(one)
    b, c = two.param_groups[0]["params"][0], start()
    b.grad = a.grad.clone()
    with torch.no_grad():
        c.copy_(a)
    three = gk.GRKANAdamW([c], bits=8)
    three.load_state_dict(one.state_dict())
    for _ in range(3):
        for opt in (one, two, three):
            opt.step()
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("bits", (32, 8))
def test_far_values(gk, bits):
    """A tensor of more than 2^31 values: its last ones as if they were alone."""
    n, last = (1 << 31) + 4096 + 77, 1 << 20 | 77
    p, g = (torch.full((n,), v, device=DEV) for v in (1.0, 0.5))
    gen = torch.Generator().manual_seed(9)
    p[-last:], g[-last:] = (torch.randn(last, generator=gen).to(DEV) for _ in range(2))
    state = gk.grkan_adamw_state(p, bits)
    one = [t[-last:].clone() for t in (p, g)]
    alone = gk.grkan_adamw_state(one[0], bits)
    for (w, grad), (avg, sq, ms, rs) in (((p, g), state), (one, alone)):
        gk.grkan_adamw_step([w], [grad], [avg], [sq], step=1, avg_scales=None if ms is None else [ms],
                            sq_scales=None if rs is None else [rs], **HYPER)
    assert torch.equal(p[-last:], one[0])
    assert int((p[:-last] != p[0]).count_nonzero()) == 0 and float(p[0]) != 1.0
    if bits == 32:
        assert torch.equal(state[0][-last:], alone[0]) and torch.equal(state[1][-last:], alone[1])
