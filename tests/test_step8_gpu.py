"""A decode step over an 8-bit cache, as a program runs it: for each layer the
q, k, v projections (w4g128_decode_step's verify form), rotation and append
(w4g128_append), attention over the 8-bit pages (w4g128_attend8), the output
projection folded into the residual add and RMS norm, and the mixture of
experts; then the lm_head product, penalties and grammar mask over the tokens so
far (w4g128_penalize) and sampling.

With a scale for each position the rows of a step are independent of one
another: a verify step of M rows gives the bits, and draws the tokens, of M
one-token steps.  With larger blocks a step's rows share scales; a graph replay
gives what the calls give in any case."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_g128_gb300 as w  # noqa: E402
from test_step_gpu import D, DIM, E, F, HKV, HQ, K, LAYERS, MAX_LEN, PAGE, PAGES, V, Model  # noqa: E402

KV = HKV * DIM


class Model8(Model):
    def __init__(self, seed, block):
        super().__init__(seed)
        self.block = block
        del self.k, self.v
        shape = (LAYERS, PAGES, PAGE, HKV, DIM)
        self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full((LAYERS, PAGES, HKV, PAGE // block), float("nan"), device="cuda") for _ in range(2))
        self.freqs = 1e4 ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device="cuda") / DIM)
        self.mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, -(-V // 32)), generator=self.g, dtype=torch.int32, device="cuda")

    def state(self):
        return [t.clone() for t in (self.k, self.v, self.ks, self.vs)]

    def restore(self, state):
        for t, s in zip((self.k, self.v, self.ks, self.vs), state):
            t.copy_(s)


class Step:
    """A step of M rows; `run` makes every call on the current stream."""

    def __init__(self, m, M, max_new):
        self.m, self.M = m, M
        b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        i = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        self.x, self.qb, self.kvb, self.att = b(M, D), b(M, HQ * DIM), b(M, 2 * KV), b(M, HQ * DIM)
        self.h, self.normed, self.logits = b(M, D), b(M, D), b(M, V)
        self.tokens, self.u, self.lens = i(M), torch.zeros(M, device="cuda"), i(1)
        self.offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        self.history, self.history_len = i(MAX_LEN), i(M)
        self.full = lambda v: torch.full((M,), v, device="cuda")
        self.append, self.attend, self.moe = [], [], []
        for n in range(LAYERS):
            k, ks = m.k[n], m.ks[n]
            paged = dict(k_cache=k, v_cache=m.v[n], k_scale=ks, v_scale=m.vs[n], page_table=m.table, row_offsets=self.offsets,
                         lens=self.lens, page_stride=k.stride(0), slot_stride=k.stride(1), head_stride=k.stride(2),
                         scale_page=ks.stride(0), scale_head=ks.stride(1), table_row=m.table.stride(0), rows=M, count=1,
                         q_heads=HQ, kv_heads=HKV, head_dim=DIM, pages=PAGES, page_size=PAGE, block=m.block,
                         max_len=MAX_LEN, max_new=max_new, q=self.qb, q_row=HQ * DIM)
            self.append.append(w.AppendArgs(**paged, q_out=self.qb, q_out_row=HQ * DIM, k_new=self.kvb,
                                            v_new=self.kvb[:, KV:], kv_row=2 * KV, freqs=m.freqs, rot_dim=DIM,
                                            interleaved=n % 2))
            self.attend.append(w.Attend8Args(**paged, out=self.att, out_row=HQ * DIM, window=0 if n else 100,
                                             sinks=0 if n else 4, scale=DIM ** -0.5))
            self.moe.append(w.MoEArgs(x=self.normed, residual=self.h, y=self.x, router=m.router[n],
                                      gate_up=m.gate_up[n], down=m.down[n], M=M, D=D, F=F, E=E, top_k=K, renormalize=1))
        self.penalize = w.PenalizeArgs(logits=self.logits, out=self.logits, row_stride=V, out_stride=V, history=self.history,
                                       history_len=self.history_len, repetition=self.full(1.2), presence=self.full(0.5),
                                       frequency=self.full(0.25), mask=m.mask, mask_row=0, rows=M, vocab=V,
                                       history_size=MAX_LEN, bias_size=0)
        self.sample = w.SampleArgs(logits=self.logits, row_stride=V, temperature=self.full(0.8), top_p=self.full(0.9),
                                   u=self.u, tokens=self.tokens, rows=M, vocab=V)
        ws = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.proj = [[(m.q[n], self.x, self.qb, D, HQ * DIM), (m.kv[n], self.x, self.kvb, D, 2 * KV)] for n in range(LAYERS)]
        self.ws = dict(proj=ws(w.w4g128_decode_step_workspace_bytes(self.proj[0], M)),
                       o=ws(w.w4g128_workspace_bytes(M, HQ * DIM, D)), head=ws(w.w4g128_workspace_bytes(M, D, V)),
                       append=[ws(w.w4g128_append_workspace_bytes(a)) for a in self.append],
                       attend=[ws(w.w4g128_attend8_workspace_bytes(a)) for a in self.attend],
                       moe=ws(w.w4g128_moe_workspace_bytes(self.moe[0])))

    def run(self):
        m, s = self.m, self.ws
        for n in range(LAYERS):
            w.w4g128_verify_step(self.proj[n], self.M, s["proj"])
            w.w4g128_append(self.append[n], s["append"][n])
            w.w4g128_attend8(self.attend[n], s["attend"][n])
            w.w4g128_gemm_add_rmsnorm(m.o[n], self.att, self.x, m.gamma[n], 1e-6, self.h, self.normed, self.M, HQ * DIM,
                                      D, 1, s["o"])
            w.w4g128_moe(self.moe[n], s["moe"])
        w.w4g128_gemm_verify(m.head, self.x, self.logits, self.M, D, V, s["head"])
        w.w4g128_penalize(self.penalize)
        w.w4g128_sample(self.sample)

    def load(self, tokens, history, u):
        """tokens: this step's rows; history: every token up to and with the first of them."""
        self.x.copy_(self.m.embed[torch.tensor(tokens, device="cuda")])
        n = len(history)
        self.history[:n + len(tokens) - 1] = torch.tensor(history + tokens[1:], dtype=torch.int32, device="cuda")
        self.history_len.copy_(torch.arange(n, n + len(tokens), dtype=torch.int32))
        self.lens.fill_(n - 1 + len(tokens))
        self.u.copy_(torch.tensor(u, device="cuda"))

    def check_status(self):
        s = self.ws
        for ws in (s["proj"], s["o"], s["head"], s["moe"], *s["append"], *s["attend"]):
            assert w.w4g128_workspace_status(ws) == 0


def prompt(model, n, seed):
    """n tokens, put through the model in steps of up to 16 rows."""
    rng = np.random.default_rng(seed)
    tokens = rng.integers(0, V, n).tolist()
    for at in range(0, n, 16):
        part = tokens[at:at + 16]
        step = Step(model, len(part), max_new=len(part))
        step.load(part, tokens[:at + 1], np.zeros(len(part), np.float32))
        step.run()
        torch.cuda.synchronize()
        step.check_status()
    return tokens


@pytest.mark.gpu
@pytest.mark.parametrize("start,M", [(0, 5), (3, 8), (250, 8), (299, 16), (17, 2)])
def test_a_verify_step_is_its_one_token_steps(start, M):
    model = Model8(start, block=1)
    history = prompt(model, start, M)
    rng = np.random.default_rng(M)
    tokens, u = rng.integers(0, V, M).tolist(), rng.random(M).astype(np.float32)
    before = model.state()
    many = Step(model, M, max_new=M)
    many.load(tokens, history + tokens[:1], u)
    many.run()
    torch.cuda.synchronize()
    many.check_status()
    assert not torch.isnan(many.logits).any() and (many.tokens >= 0).all() and (many.tokens < V).all()
    after = model.state()
    assert not torch.equal(after[0], before[0])
    model.restore(before)
    one = Step(model, 1, max_new=1)
    for i in range(M):
        one.load(tokens[i:i + 1], history + tokens[:i + 1], u[i:i + 1])
        one.run()
        torch.cuda.synchronize()
        one.check_status()
        assert torch.equal(one.logits[0], many.logits[i]), i
        assert one.tokens[0] == many.tokens[i]
    for a, b in zip(model.state(), after):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 16])
def test_captured_steps_generate_what_the_calls_generate(block):
    """Twelve tokens, each fed back, by calls and by replays of one captured step; the grammar allows each of them."""
    model = Model8(77, block)
    start = prompt(model, 40, 1)
    before = model.state()
    step = Step(model, 1, max_new=1)
    u = np.random.default_rng(0).random(12).astype(np.float32)

    def generate(run):
        model.restore(before)
        out, tokens = [], start + [5]
        for i in range(12):
            step.load(tokens[-1:], tokens, u[i:i + 1])
            run()
            torch.cuda.synchronize()
            tokens.append(int(step.tokens[0]))
            out.append((tokens[-1], step.logits.clone()))
        step.check_status()
        return out

    plain = generate(step.run)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    replayed = generate(g.replay)
    for (a, x), (b, y) in zip(plain, replayed):
        assert a == b and torch.equal(x, y)
    words = model.mask[0].tolist()
    assert all(words[t // 32] >> (t % 32) & 1 for t, _ in plain)
    assert len({t for t, _ in plain}) > 3
