"""The mixture-of-experts layer (w4g128_moe) against its definition in 64
bits, from the canonical codes, scales and minima.

The bound.  One product sum_k x w of depth K = 128 G is built as scale d +
(min - b scale) X per group, d = sum x (b + q), X = sum x, with a bias b of
1024: with B = sum_k |x_k| (|min| + (2 b + 15) scale), the 16 MMAs of a group
err by at most
2 * 24 roundings of that size (a tensor core may truncate: 2^-23 each), the
sum over groups and parts by G + 8 more, so e(K) = (G + 56) 2^-23 B.  x enters
the first product as fp16 scaled by its row's largest value, off by at most
2^-40 of that.  An
activation a = silu(g) u moves by 1.1 |u| e_g + |silu(g)| e_u (|silu'| <= 1.1),
4 fp32 roundings and exp's 2 ulp, and is rounded to 11 bits (2^-11) with at
most 2^-38 of the row's largest besides (twice: where it is stored and where it
is brought to the row's exponent); the down product carries these through |w|
and adds its own e(F); the weights p, from
logits within (D / 8 + 16) 2^-24 sum|x r|, twice that relative plus 2^-20; the
sum over picks 2^-20 relative; the output rounds once, 2^-8.

Picks are integers: a row whose top_k-th and next logit lie closer than their
bounds together may pick either, and is left out."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_g128_gb300 as w  # noqa: E402


def rnd(g, *s):
    return torch.randn(s, generator=g, device="cuda")


class Experts:
    """E seeded matrices: canonical (codes, scales, minima) and their packed bytes, one after another."""

    def __init__(self, E, K, N, g):
        self.E, self.K, self.N = E, K, N
        self.codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (E, K // 8, N), generator=g, device="cuda", dtype=torch.int32)
        self.scales = (torch.rand((E, K // 128, N), generator=g, device="cuda") * 0.018 + 0.002).bfloat16()
        low = -8 * self.scales.float() * (1 + (torch.rand(self.scales.shape, generator=g, device="cuda") * 0.2 - 0.1))
        self.mins = low.bfloat16()
        self.each = w.w4g128_packed_bytes(K, N)
        self.packed = torch.empty(E * self.each, dtype=torch.uint8, device="cuda")
        for e in range(E):
            w.w4g128_pack(self.codes[e], self.scales[e], self.mins[e], K, N, self.packed[e * self.each:], stream=None)

    def matrix(self, e, bias):
        """(w, |min| + (2 bias + 15) scale) [K][N] in 64 bits."""
        shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)[None, :, None]
        q = ((self.codes[e][:, None] >> shift) & 15).reshape(self.K, self.N).double()
        s, m = (t[e].double().repeat_interleave(128, 0) for t in (self.scales, self.mins))
        return m + q * s, m.abs() + (2 * bias + 15) * s


class Layer:
    def __init__(self, M, D, F, E, k, renorm=True, residual=True, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.M, self.D, self.F, self.E, self.k, self.renorm = M, D, F, E, k, renorm
        self.x = rnd(g, M, D).bfloat16()
        self.residual = rnd(g, M, D).bfloat16() if residual else None
        self.router = (rnd(g, E, D) / D ** 0.5).bfloat16()
        self.gate_up, self.down = Experts(E, D, 2 * F, g), Experts(E, F, D, g)

    def args(self, y, x=None, residual=None, M=None):
        x = self.x if x is None else x
        residual = self.residual if residual is None else residual
        return w.MoEArgs(x=x, residual=residual, y=y, router=self.router, gate_up=self.gate_up.packed,
                         down=self.down.packed, M=M or x.shape[0], D=self.D, F=self.F, E=self.E, top_k=self.k,
                         renormalize=int(self.renorm))

    def run(self, x=None, residual=None, in_place=False):
        x = self.x if x is None else x
        residual = self.residual if residual is None else residual
        M = x.shape[0]
        y = residual.clone() if in_place else None
        whole = torch.full((M * self.D + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        if not in_place:
            y = whole[256:256 + M * self.D].view(M, self.D)
        args = self.args(y, x, y if in_place else residual)
        nb = w.w4g128_moe_workspace_bytes(args)
        ws = torch.full((nb + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        w.w4g128_moe(args, ws[4096:], ws_bytes=nb)
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws[4096:]) == 0
        assert (ws[:4096] == 0x5A).all() and (ws[4096 + nb:] == 0x5A).all()
        assert (whole[:256] == 7).all() and (whole[256 + M * self.D:] == 7).all()
        return y

    def reference(self):
        """(y, bound, clear): 64 bits, and the rows whose picks are beyond doubt."""
        x = self.x.double()
        logits = x @ self.router.double().T
        bound = (self.D / 8 + 16) * 2.0 ** -24 * (x.abs() @ self.router.double().abs().T)
        el = bound.max(-1).values
        order = torch.sort(logits, dim=-1, descending=True, stable=True).indices
        clear = torch.ones(self.M, dtype=torch.bool, device="cuda")
        if self.k < self.E:
            s, b = torch.gather(logits, 1, order), torch.gather(bound, 1, order)
            gap, doubt = s[:, self.k - 1] - s[:, self.k], b[:, self.k - 1] + b[:, self.k]
            clear = (gap > doubt) | (doubt == 0)  # (products that are all 0 are exact)
        pick = order[:, :self.k]
        p = torch.gather(torch.softmax(logits, -1), 1, pick)
        if self.renorm:
            p = p / p.sum(-1, keepdim=True)
        ep = 4 * el[:, None] + 2.0 ** -20
        y = torch.zeros((self.M, self.D), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(y)
        eps = lambda K: (K / 128 + 56) * 2.0 ** -23  # noqa: E731
        for e in range(self.E):
            rows, place = torch.nonzero(pick == e, as_tuple=True)
            if not rows.numel():
                continue
            W, B = self.gate_up.matrix(e, 1024)
            h, eh = x[rows] @ W, eps(self.D) * (x[rows].abs() @ B)
            eh = eh + 2.0 ** -40 * x[rows].abs().amax(-1, keepdim=True) * W.abs().sum(0)
            gate, up, eg, eu = h[:, :self.F], h[:, self.F:], eh[:, :self.F], eh[:, self.F:]
            silu = gate * torch.sigmoid(gate)
            act = silu * up
            ea = 1.1 * up.abs() * eg + silu.abs() * eu + 1.1 * eg * eu + (2.0 ** -11 + 2.0 ** -20) * act.abs()
            ea = ea + 2.0 ** -38 * (act.abs() + ea).amax(-1, keepdim=True)
            W, B = self.down.matrix(e, 1024)
            o = act @ W
            eo = ea @ W.abs() + eps(self.F) * ((act.abs() + ea) @ B)
            pe = p[rows, place][:, None]
            y[rows] += pe * o
            tol[rows] += pe * (eo + (ep[rows] + 2.0 ** -20) * o.abs())
        if self.residual is not None:
            y = y + self.residual.double()
        return y, tol * 1.01 + 2.0 ** -8 * y.abs() + 2.0 ** -130, clear

    def check(self, **kw):
        y, tol, clear = self.reference()
        got = self.run(**kw)
        assert clear.sum() >= self.M - max(1, self.M // 8), "the inputs say too little"
        err = (got.double() - y).abs()[clear]
        assert (err <= tol[clear]).all(), float((err / tol[clear]).max())
        return got


SHAPES = [(1, 128, 128, 1, 1), (1, 256, 128, 4, 2), (2, 128, 384, 5, 5), (3, 640, 256, 7, 3), (8, 512, 128, 16, 4),
          (9, 384, 640, 12, 2), (13, 1152, 384, 37, 3), (16, 256, 256, 3, 2), (16, 512, 512, 64, 6), (5, 1280, 1024, 9, 4),
          (16, 128, 128, 512, 16), (1, 2048, 768, 24, 16),
          (16, 2048, 1408, 40, 5), (2, 8192, 128, 2, 1), (3, 128, 8192, 2, 2), (1, 16384, 256, 2, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("renorm,residual", [(True, True), (False, False)])
def test_against_reference(shape, renorm, residual):
    Layer(*shape, renorm=renorm, residual=residual, seed=sum(shape)).check()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(16, 512, 256, 8, 3), (7, 1152, 640, 40, 5), (12, 256, 128, 2, 1), (16, 2048, 384, 40, 5),
                                   (16, 384, 256, 2, 2), (2, 640, 1152, 9, 4)],
                         ids=str)
def test_a_row_alone_gives_the_same_bits(shape):
    layer = Layer(*shape, seed=4)
    y = layer.run()
    for m in range(shape[0]):
        assert torch.equal(layer.run(layer.x[m:m + 1], layer.residual[m:m + 1]), y[m:m + 1]), m
    half = shape[0] // 2
    assert torch.equal(layer.run(layer.x[half:].clone(), layer.residual[half:].clone()), y[half:])
    assert torch.equal(layer.run(), y)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 4096, 256, 12, 6), (2, 4096, 256, 12, 6), (2, 1024, 256, 12, 2),
                                   (1, 65536, 128, 24, 16), (2, 65536, 128, 24, 16)], ids=str)
def test_one_and_two_rows_add_up_in_the_down_projection(shape):
    """Few units and many, up to more than a team adds up at once."""
    layer = Layer(*shape, seed=6)
    y = layer.check()
    for m in range(shape[0]):
        assert torch.equal(layer.run(layer.x[m:m + 1], layer.residual[m:m + 1]), y[m:m + 1]), m


@pytest.mark.gpu
def test_every_row_on_one_expert_and_equal_logits():
    """Equal logits (a router of zeros, with either sign of zero): the lowest experts, at equal weights; 16 rows of
    one expert fill both 8-row operand tiles."""
    layer = Layer(16, 256, 256, 6, 2, seed=1)
    layer.router.zero_()
    layer.router[1] = -0.0
    layer.check()
    layer.router[4, 0] = 1.0  # logit x[0]: expert 4 first or last
    layer.x[:, 0] = torch.where(torch.arange(16, device="cuda") % 2 == 0, 3.0, -3.0).bfloat16()
    layer.check()


@pytest.mark.gpu
def test_residual_in_place():
    layer = Layer(4, 256, 128, 8, 2, seed=2)
    assert torch.equal(layer.check(in_place=True), layer.run())


@pytest.mark.gpu
def test_experts_that_no_row_picks_are_not_read():
    layer = Layer(3, 256, 256, 16, 2, seed=3)
    y = layer.run()
    x = layer.x.double() @ layer.router.double().T
    picked = set(torch.topk(x, 2, dim=-1).indices.flatten().tolist())
    for e in range(16):
        if e not in picked:
            for m in (layer.gate_up, layer.down):
                m.packed[e * m.each:(e + 1) * m.each] = 0xFF  # scales and minima are NaN
    assert torch.equal(layer.run(), y)


@pytest.mark.gpu
def test_non_finite_rows_stay_among_themselves():
    layer = Layer(6, 256, 128, 8, 3, seed=5)
    y = layer.run()
    layer.x[2, 7] = float("nan")
    layer.x[4, 100] = float("inf")
    got = layer.run()
    keep = torch.tensor([0, 1, 3, 5], device="cuda")
    assert torch.equal(got[keep], y[keep])
    assert torch.isnan(got[2]).all()
    layer.x[0].zero_()  # every logit 0, every activation 0
    assert torch.equal(layer.run()[0], layer.residual[0])


@pytest.mark.gpu
def test_largest_logits_and_activations():
    """Far apart logits: weights 1 and 0; gates far below 0: activations of 0."""
    layer = Layer(4, 128, 128, 5, 2, seed=6)
    layer.router[3] = 0
    layer.router[3, 0] = 30000.0
    layer.x[:, 0] = 8.0
    layer.check()


@pytest.mark.gpu
def test_streams_graph_replay_and_reused_workspace():
    layer = Layer(5, 512, 256, 10, 2, seed=7)
    want = layer.run().clone()
    y = torch.zeros_like(want)
    args = layer.args(y)
    ws = torch.empty(w.w4g128_moe_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step = w.MoEStep(args, ws)
        for _ in range(20):  # back to back on one workspace
            step.run()
    s.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.w4g128_moe(args, ws)
        w.w4g128_moe(args, ws)
    for seed in (1, 2):
        layer.x.copy_(torch.randn(layer.x.shape, device="cuda"))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws) == 0
        assert torch.equal(y, layer.run())


@pytest.mark.gpu
def test_two_calls_at_once():
    layers = [Layer(3, 1024, 512, 16, 4, seed=s) for s in (8, 9)]
    want = [m.run().clone() for m in layers]
    ys, steps = [], []
    for m in layers:
        y = torch.zeros_like(want[0])
        a = m.args(y)
        ys.append(y)
        steps.append(w.MoEStep(a, torch.empty(w.w4g128_moe_workspace_bytes(a), dtype=torch.uint8, device="cuda"),
                               stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for s in steps:
            s.run()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])


@pytest.mark.gpu
def test_logits_that_are_not_numbers_rank_last():
    """A router row of NaN: its expert is picked only where no other is left."""
    layer = Layer(2, 128, 128, 4, 2, seed=10)
    layer.router[1] = float("nan")
    layer.router[2] = float("nan")
    got = layer.run()
    layer.router[1] = layer.router[0]
    layer.router[2] = layer.router[0]
    ref = Layer(2, 128, 128, 4, 2, seed=10)
    ref.router[1:3] = -1e30 * torch.sign(ref.x[0].float()).bfloat16()  # far below for row 0
    assert torch.equal(got[0], ref.run()[0])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3, 12])
@pytest.mark.parametrize("orders", [12, 23, 25, 26, 28, 30])
def test_activations_far_below_the_largest_of_their_row(orders, M):
    """Activations `orders` binary orders and more below others of their row, which meet weights of zero.  What an
    activation a may lose besides its 2^-11 is 2^-39 of the row's largest, T, where it is brought to the row's exponent
    (and as much of its tile's, at most 2^-11 of T here, where it is stored): a share 2^-39 T / rms(a) of the small
    ones.  A product with random weights keeps that share, and a share of 2^-11, in the mean over its columns; twice
    that is allowed, and 2^-8 for the output's rounding."""
    layer = Layer(M, 256, 384, 4, 2, residual=False, seed=orders)
    up, down = layer.gate_up, layer.down
    for t in (up.scales, up.mins):
        t[:, :, 384:512] *= 2.0 ** orders  # the up columns of activations 0..127
    for t in (down.scales, down.mins):
        t[:, 0] = 0                        # and the rows of the down matrix that they meet
    for m in (up, down):
        for e in range(m.E):
            w.w4g128_pack(m.codes[e], m.scales[e], m.mins[e], m.K, m.N, m.packed[e * m.each:], stream=None)
    y, _, clear = layer.reference()
    got = layer.check().double()
    W = [up.matrix(e, 0)[0] for e in range(4)]
    for r in range(M):
        if not clear[r]:
            continue
        share = 0.0
        for e in torch.topk(layer.x[r].double() @ layer.router.double().T, 2).indices.tolist():
            h = layer.x[r].double() @ W[e]
            a = h[:384] * torch.sigmoid(h[:384]) * h[384:]
            share = max(share, (2.0 ** -39 * a.abs().max() / a[128:].pow(2).mean().sqrt()).item())
        assert orders < 30 or share > 2.0 ** -9
        assert (got[r] - y[r]).norm() <= (2.0 ** -8 + 2 * (2.0 ** -11 + share)) * y[r].norm(), r


def norm_errors(layer, got):
    """|got - y| / |y| of each row whose picks are beyond doubt, for a layer without residual.  Bound: the output's
    rounding 2^-8; the activations' 2^-11, which a product with random weights passes on in the mean, twice that
    allowed; the three products' fp32 sums, whose terms carry a bias of 1024 (some 224 times the weights), 8 of them
    truncated by 2^-23 in a group: 2^-12 each.  Together below 2^-8 + 2^-9."""
    y, _, clear = layer.reference()
    return ((got.double() - y).norm(dim=1) / y.norm(dim=1))[clear]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("renorm", [True, False])
def test_norm_of_the_error(shape, renorm):
    """The element bounds add up worst cases and grow past |y| with the depth; the norm of a row's error does not."""
    layer = Layer(*shape, renorm=renorm, residual=False, seed=1 + sum(shape))
    assert (norm_errors(layer, layer.run()) <= 2.0 ** -8 + 2.0 ** -9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape,kernel", [((16, 1024, 2048, 64, 8), "gate and up"), ((16, 1152, 2048, 64, 8), "gate and up"),
                                          ((16, 8192, 1024, 64, 8), "down"), ((5, 8192, 1152, 64, 16), "down"),
                                          ((2, 16384, 1024, 40, 16), "down"), ((1, 20480, 1024, 24, 16), "down")], ids=str)
def test_units_drawn_from_the_counter(shape, kernel):
    """More units than the eight that each team knows from the start, and depths of 8 groups and more, where the rest
    are drawn: against the reference, row by row, back to back on one workspace and replayed."""
    M, D, F, E, k = shape
    layer = Layer(*shape, residual=False, seed=12)
    picked = torch.topk(layer.x.double() @ layer.router.double().T, k).indices.unique().numel()
    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    if kernel == "down":  # units of 64 columns, two teams a CTA
        assert F >= 1024 and picked * (D // 64) > 8 * 2 * ctas
    else:                 # of 32 activations, one team
        assert D >= 1024 and picked * (F // 32) > 8 * ctas
    y, tol, clear = layer.reference()  # (at these depths the logits' bound leaves some rows' picks in doubt)
    got = layer.run()
    assert clear.any() and ((got.double() - y).abs() <= tol)[clear].all()
    assert (norm_errors(layer, got) <= 2.0 ** -8 + 2.0 ** -9).all()
    for m in {0, M // 2, M - 1}:
        assert torch.equal(layer.run(layer.x[m:m + 1]), got[m:m + 1]), m
    y = torch.zeros_like(got)
    args = layer.args(y)
    ws = torch.empty(w.w4g128_moe_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    for _ in range(8):
        w.w4g128_moe(args, ws)
    torch.cuda.synchronize()
    assert torch.equal(y, got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.w4g128_moe(args, ws)
        w.w4g128_moe(args, ws)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, got)
