"""The operators of a decode step together, as a program runs them: for each
layer the q, k, v projections (w4g128_decode_step), attention over the paged
cache, the output projection folded into the residual add and RMS norm
(w4g128_gemm_add_rmsnorm) and the mixture of experts; then the lm_head product
and sampling.  The whole step is captured in one CUDA graph.

Every operator's rows are independent of one another, so a verify step of M
rows gives exactly the bits, and draws exactly the tokens, of M one-token steps
from the same cache; and a graph replay gives what the calls give."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_g128_gb300 as w  # noqa: E402

D, HQ, HKV, DIM, F, E, K, V, LAYERS = 512, 8, 2, 64, 256, 12, 3, 2000 // 16 * 16, 2
PAGE, PAGES, MAX_LEN = 16, 40, 320


def packed(K_, N, g, count=1):
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (count, K_ // 8, N), generator=g, device="cuda", dtype=torch.int32)
    scales = (torch.rand((count, K_ // 128, N), generator=g, device="cuda") * 0.018 + 0.002) / K_ ** 0.5 * 8
    mins = (-7.5 * scales).bfloat16()
    each = w.w4g128_packed_bytes(K_, N)
    out = torch.empty(count * each, dtype=torch.uint8, device="cuda")
    for i in range(count):
        w.w4g128_pack(codes[i], scales[i].bfloat16(), mins[i], K_, N, out[i * each:])
    return out


class Model:
    def __init__(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g = g
        n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.embed = n(V, D)
        self.gamma = (1 + 0.1 * torch.randn((LAYERS, D), generator=g, device="cuda")).bfloat16()
        self.router = [(n(E, D).float() / D ** 0.5).bfloat16() for _ in range(LAYERS)]
        self.q, self.kv = ([packed(D, N, g) for _ in range(LAYERS)] for N in (HQ * DIM, 2 * HKV * DIM))
        self.o = [packed(HQ * DIM, D, g) for _ in range(LAYERS)]
        self.gate_up, self.down = ([packed(*s, g, E) for _ in range(LAYERS)] for s in ((D, 2 * F), (F, D)))
        self.head = packed(D, V, g)
        self.k = n(LAYERS, PAGES, PAGE, HKV, DIM)
        self.v = n(LAYERS, PAGES, PAGE, HKV, DIM)
        self.table = torch.randperm(PAGES, generator=g, device="cuda").int()[None, :MAX_LEN // PAGE].contiguous()


class Step:
    """A step of M rows; `run` makes every call on the current stream."""

    def __init__(self, m, M, max_new):
        self.m, self.M = m, M
        b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x, self.qb, self.kvb, self.att = b(M, D), b(M, HQ * DIM), b(M, 2 * HKV * DIM), b(M, HQ * DIM)
        self.h, self.normed, self.logits = b(M, D), b(M, D), b(M, V)
        self.tokens = torch.zeros(M, dtype=torch.int32, device="cuda")
        self.u = torch.zeros(M, device="cuda")
        self.lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        self.temperature = torch.full((M,), 0.8, device="cuda")
        self.top_p = torch.full((M,), 0.9, device="cuda")
        self.attend, self.moe = [], []
        for i in range(LAYERS):
            k = m.k[i]
            self.attend.append(w.AttendArgs(
                q=self.qb, k_new=self.kvb, v_new=self.kvb[:, HKV * DIM:], k_cache=k, v_cache=m.v[i], page_table=m.table,
                row_offsets=self.offsets, lens=self.lens, out=self.att, q_row=HQ * DIM, kv_row=2 * HKV * DIM,
                out_row=HQ * DIM, page_stride=k.stride(0), slot_stride=k.stride(1), head_stride=k.stride(2),
                table_row=m.table.stride(0), rows=M, count=1, q_heads=HQ, kv_heads=HKV, head_dim=DIM, pages=PAGES,
                page_size=PAGE, max_len=MAX_LEN, max_new=max_new, window=0 if i else 100, sinks=0 if i else 4,
                scale=DIM ** -0.5))
            self.moe.append(w.MoEArgs(x=self.normed, residual=self.h, y=self.x, router=m.router[i],
                                      gate_up=m.gate_up[i], down=m.down[i], M=M, D=D, F=F, E=E, top_k=K, renormalize=1))
        self.sample = w.SampleArgs(logits=self.logits, row_stride=V, temperature=self.temperature, top_p=self.top_p,
                                   u=self.u, tokens=self.tokens, rows=M, vocab=V)
        ws = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.proj = [[(m.q[i], self.x, self.qb, D, HQ * DIM), (m.kv[i], self.x, self.kvb, D, 2 * HKV * DIM)]
                     for i in range(LAYERS)]
        self.ws = dict(proj=ws(w.w4g128_decode_step_workspace_bytes(self.proj[0], M)),
                       o=ws(w.w4g128_workspace_bytes(M, HQ * DIM, D)), head=ws(w.w4g128_workspace_bytes(M, D, V)),
                       attend=[ws(w.w4g128_attend_workspace_bytes(a)) for a in self.attend],
                       moe=ws(w.w4g128_moe_workspace_bytes(self.moe[0])))

    def run(self):
        m, s = self.m, self.ws
        for i in range(LAYERS):
            w.w4g128_verify_step(self.proj[i], self.M, s["proj"])
            w.w4g128_attend(self.attend[i], s["attend"][i])
            w.w4g128_gemm_add_rmsnorm(m.o[i], self.att, self.x, m.gamma[i], 1e-6, self.h, self.normed, self.M, HQ * DIM,
                                      D, 1, s["o"])
            w.w4g128_moe(self.moe[i], s["moe"])
        w.w4g128_gemm_verify(m.head, self.x, self.logits, self.M, D, V, s["head"])
        w.w4g128_sample(self.sample)

    def load(self, tokens, length, u):
        self.x.copy_(self.m.embed[torch.tensor(tokens, device="cuda")])
        self.lens.fill_(length)
        self.u.copy_(torch.tensor(u, device="cuda"))

    def check_status(self):
        for ws in (self.ws["proj"], self.ws["o"], self.ws["head"], self.ws["moe"], *self.ws["attend"]):
            assert w.w4g128_workspace_status(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("start,M", [(0, 5), (3, 8), (250, 8), (299, 16), (17, 2)])
def test_a_verify_step_is_its_one_token_steps(start, M):
    model = Model(start)
    rng = np.random.default_rng(M)
    tokens, u = rng.integers(0, V, M).tolist(), rng.random(M).astype(np.float32)
    kc, vc = model.k.clone(), model.v.clone()
    many = Step(model, M, max_new=M)
    many.load(tokens, start + M, u)
    many.run()
    torch.cuda.synchronize()
    many.check_status()
    assert torch.isfinite(many.logits).all() and (many.tokens >= 0).all() and (many.tokens < V).all()
    after = model.k.clone(), model.v.clone()
    assert not torch.equal(after[0], kc)
    model.k.copy_(kc)
    model.v.copy_(vc)
    one = Step(model, 1, max_new=1)
    for i in range(M):
        one.load(tokens[i:i + 1], start + i + 1, u[i:i + 1])
        one.run()
        torch.cuda.synchronize()
        one.check_status()
        assert torch.equal(one.logits[0], many.logits[i]), i
        assert one.tokens[0] == many.tokens[i]
    assert torch.equal(model.k, after[0]) and torch.equal(model.v, after[1])


@pytest.mark.gpu
def test_captured_steps_generate_what_the_calls_generate():
    """Twelve tokens, each fed back, by calls and by replays of one captured step."""
    model = Model(77)
    kc, vc = model.k.clone(), model.v.clone()
    step = Step(model, 1, max_new=1)
    u = np.random.default_rng(0).random(12).astype(np.float32)

    def generate(run):
        model.k.copy_(kc)
        model.v.copy_(vc)
        out, token = [], 5
        for i in range(12):
            step.load([token], 40 + i, u[i:i + 1])
            run()
            torch.cuda.synchronize()
            token = int(step.tokens[0])
            out.append((token, step.logits.clone()))
        step.check_status()
        return out

    plain = generate(step.run)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    replayed = generate(g.replay)
    for (a, x), (b, y) in zip(plain, replayed):
        assert a == b and torch.equal(x, y)
    assert len({t for t, _ in plain}) > 3
