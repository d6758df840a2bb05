"""Penalties, biases and masks on logits (w4g128_penalize) against the formulas
in 64 bits.  Each of the six fp32 operations (a division is a product with the
inverse) is off by at most 2^-24 of its result, which is no larger than the sum of
the terms' magnitudes; the output
rounds once, 2^-8 of the value (of 2^-133 at least, bf16's smallest step)."""
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_g128_gb300 as w  # noqa: E402


class Call:
    def __init__(self, rows, vocab, history=50, bias=5, masked=True, seed=0, stride=None, out_stride=None, shift=0,
                 out_shift=0, same=False):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.R, self.V = rows, vocab
        rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
        self.stride, self.out_stride = stride or vocab, out_stride or stride or vocab
        self.whole = torch.full((shift + rows * self.stride + 8,), 3.0, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.as_strided(self.whole, (rows, vocab), (self.stride, 1), shift)
        self.logits.copy_(4 * torch.randn((rows, vocab), generator=g, device="cuda"))
        self.same = same
        self.whole_out = self.whole if same else \
            torch.full((out_shift + rows * self.out_stride + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.out = self.logits if same else torch.as_strided(self.whole_out, (rows, vocab), (self.out_stride, 1), out_shift)
        ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
        lens = [(history * (r + 2)) // (r + 1) if history else 0 for r in range(rows)]
        starts = [sum(lens[:r]) for r in range(rows)]
        self.history = (vocab * rand(sum(lens) + 3) ** 3).int().clamp(max=vocab - 1)
        self.start, self.len = ints(starts, torch.int64), ints(lens)
        self.prompt = ints([n // (2 + r % 3) for r, n in enumerate(lens)])
        r = torch.arange(rows, device="cuda")
        self.repetition = 0.8 + 0.3 * (r % 4).float()
        self.presence = 0.37 * (r % 3).float() - 0.1
        self.frequency = 0.21 * (r % 5).float()
        each = [bias + r % 2 if bias else 0 for r in range(rows)]
        self.bias_at = [sum(each[:r]) for r in range(rows + 1)]
        self.bias_offsets = ints(self.bias_at)
        n = sum(each)
        self.bias_tokens = (vocab * rand(n)).int().clamp(max=vocab - 1)
        self.bias_values = 30 * rand(n) - 15
        self.mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, -(-vocab // 32)), generator=g, dtype=torch.int32,
                                  device="cuda") if masked else None

    def args(self, **kw):
        a = dict(logits=self.logits, out=self.out, row_stride=self.stride,
                 out_stride=self.stride if self.same else self.out_stride, history=self.history,
                 history_start=self.start, history_len=self.len, prompt_len=self.prompt, repetition=self.repetition,
                 presence=self.presence, frequency=self.frequency, bias_tokens=self.bias_tokens,
                 bias_values=self.bias_values, bias_offsets=self.bias_offsets, mask=self.mask,
                 mask_row=self.mask.stride(0) if self.mask is not None else 0, rows=self.R, vocab=self.V,
                 history_size=self.history.numel(), bias_size=self.bias_tokens.numel())
        return w.PenalizeArgs(**{**a, **kw})

    def reference(self, without=()):
        V, out = self.V, self.logits.double()
        listed, added = self.bias_tokens.tolist(), self.bias_values.tolist()
        tol = torch.zeros_like(out)
        for r in range(self.R):
            z = out[r]
            size = z.abs()
            if "history" not in without:
                at = torch.arange(self.history.numel(), device="cuda")
                s = int(self.start[r]) if "history_start" not in without else 0
                n = max(int(self.len[r]), 0)
                prompt = int(self.prompt[r]) if "prompt_len" not in without else 0
                t = self.history.long()
                mine = (at >= s) & (at < s + n) & (t >= 0) & (t < V)
                answer = mine & (at >= s + prompt)
                seen = torch.zeros(V, dtype=torch.bool, device="cuda")
                seen[t[mine]] = True
                count = torch.bincount(t[answer], minlength=V).double()
                rep = float(self.repetition[r]) if "repetition" not in without else 1.0
                z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
                size = torch.maximum(size, z.abs())
                if "frequency" not in without:
                    z = z - float(self.frequency[r]) * count
                    size = size + abs(float(self.frequency[r])) * count
                if "presence" not in without:
                    z = z - float(self.presence[r]) * (count > 0)
                    size = size + abs(float(self.presence[r]))
            if "bias_tokens" not in without:
                last = {}
                for j in range(max(self.bias_at[r], 0), min(self.bias_at[r + 1], self.bias_tokens.numel())):
                    if 0 <= listed[j] < V:
                        last[listed[j]] = added[j]
                if last:
                    t, v = (torch.tensor(list(x), device="cuda") for x in (last.keys(), last.values()))
                    z[t] += v.double()
                    size[t] += v.double().abs()
            if self.mask is not None and "mask" not in without:
                bits = (self.mask[r][:, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
                z = torch.where(bits.flatten()[:V] == 0, -float("inf"), z)
            out[r] = z
            tol[r] = 2.0 ** -8 * z.abs() + 6 * 2.0 ** -24 * size * 1.01 + 2.0 ** -134
        return out, tol

    def check(self, without=(), **kw):
        ref, tol = self.reference(without)
        inputs, outside = self.whole.clone().view(torch.int16), self.whole_out.clone()
        w.w4g128_penalize(self.args(**{n: None for n in without}, **kw))
        torch.cuda.synchronize()
        got = self.out.double()
        fine = torch.isfinite(ref)
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert (got[~fine & ~torch.isnan(ref)] == ref[~fine & ~torch.isnan(ref)]).all()
        assert ((got - ref)[fine].abs() <= tol[fine]).all()
        keep = torch.ones_like(outside, dtype=torch.bool)  # nothing beside the rows is written
        torch.as_strided(keep, self.out.shape, self.out.stride(), self.out.storage_offset()).fill_(False)
        assert torch.equal(self.whole_out[keep], outside[keep])
        if not self.same:
            assert torch.equal(self.whole.view(torch.int16), inputs)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 31, 33, 127, 128, 129, 1000, 4095, 32000, 50261, 131071])
@pytest.mark.parametrize("masked", [False, True])
def test_vocabularies(vocab, masked):
    Call(3, vocab, masked=masked, seed=vocab).check()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab", [(1, 248320), (16, 248320), (2, 524160), (300, 1003), (4096, 40)])
def test_sizes(rows, vocab):
    Call(rows, vocab, history=20 if rows > 100 else 3000, bias=2 if rows > 100 else 200, seed=rows).check()


@pytest.mark.gpu
@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("other", [0, 1, 5])
def test_alignments(shift, other):
    """Rows that start anywhere, in logits and in out, with odd strides."""
    Call(3, 517, stride=517 + other, out_stride=520, shift=shift, out_shift=(shift + other) % 8, seed=shift).check()
    Call(3, 517, stride=528, out_stride=536, shift=shift, out_shift=shift, seed=shift).check()
    Call(2, 517, stride=517 + other, shift=shift, same=True, seed=shift).check()


@pytest.mark.gpu
@pytest.mark.parametrize("without", [("history",), ("bias_tokens",), ("mask",), ("history", "bias_tokens"), ("history_start",),
                                     ("prompt_len",), ("repetition",), ("presence",), ("frequency",),
                                     ("history", "bias_tokens", "mask"), ("repetition", "presence", "frequency")])
def test_parts_left_out(without):
    c = Call(4, 1234, seed=1)
    kw = {}
    if "history" in without:
        kw.update(history_len=None, history_size=0)
    if "bias_tokens" in without:
        kw.update(bias_values=None, bias_offsets=None)
    c.check(without, **kw)


@pytest.mark.gpu
def test_one_mask_for_all_rows():
    c = Call(5, 1000, seed=2)
    c.mask[:] = c.mask[0]
    c.check(mask_row=0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 511, 8191, 8193, 300001])
def test_long_histories(n):
    Call(2, 2049, history=n, seed=n).check()


@pytest.mark.gpu
def test_a_token_repeated_throughout():
    c = Call(2, 3000, history=70000, seed=3)
    c.history.fill_(2999)
    c.check()


@pytest.mark.gpu
def test_tokens_outside_the_vocabulary_are_ignored():
    c = Call(3, 1000, seed=4, bias=20)
    c.history[::3] = torch.tensor([-1, 1000, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda").repeat(200)[:c.history[::3].numel()]
    c.bias_tokens[::4] = 1000
    c.bias_tokens[1::4] = -7
    c.check()


@pytest.mark.gpu
def test_ranges_outside_the_buffers_are_not_read():
    """Histories that begin before or end behind their buffer, lists behind theirs; lengths below 0."""
    c = Call(6, 1000, history=100, seed=5)
    size = c.history.numel()
    c.start[:] = torch.tensor([-30, size - 10, size + 5, -2 ** 63, 2 ** 62, 3], dtype=torch.int64)
    c.len[:] = torch.tensor([100, 100, 7, 9, 9, -4], dtype=torch.int32)
    c.prompt[:] = torch.tensor([50, 4, 1, 1, 1, -1], dtype=torch.int32)
    c.bias_at = [-5, 4, 9, 9, 8, 12, 10 ** 6]
    c.bias_offsets[:] = torch.tensor(c.bias_at, dtype=torch.int32)
    c.check()


@pytest.mark.gpu
def test_list_offsets_of_any_value():
    """Ends far below 0 behind starts above it are empty lists; entries from bias_size on count for nothing."""
    at = [1, -2 ** 31, 3, -1, 2 ** 31 - 1, -2 ** 31 + 1, 4, 2 ** 31 - 1, -2 ** 31, 2, -2 ** 31 + 1]
    c = Call(len(at) - 1, 1000, bias=5, seed=13)
    size = c.bias_tokens.numel()
    tokens = torch.arange(70000, dtype=torch.int32, device="cuda") % 1000  # every token is listed behind bias_size
    values = torch.full((70000,), 1e4, device="cuda")
    tokens[:size], values[:size] = c.bias_tokens, c.bias_values
    c.bias_at = at
    c.bias_offsets[:] = torch.tensor(at, dtype=torch.int32)
    c.check(bias_tokens=tokens, bias_values=values)


@pytest.mark.gpu
def test_the_last_of_a_tokens_biases_counts():
    c = Call(2, 900, bias=400, seed=6)
    c.bias_tokens[:] = c.bias_tokens % 3 + 17  # three neighbours, many times each
    c.check()
    c.bias_tokens.fill_(899)
    c.check()


@pytest.mark.gpu
def test_lists_up_to_their_limit():
    c = Call(1, 70000, bias=65535, seed=7)
    c.bias_tokens[:] = torch.randperm(70000, device="cuda")[:c.bias_tokens.numel()].int()
    c.check()
    more = Call(1, 70000, bias=65600, seed=7, masked=False)
    more.bias_tokens[:] = torch.randperm(70000, device="cuda")[:more.bias_tokens.numel()].int()
    before = int(more.bias_at[1])
    more.bias_at[1] = 65535  # the rest of a longer list is not read
    more.bias_offsets[1] = before
    more.check()


@pytest.mark.gpu
def test_non_finite_logits():
    c = Call(3, 2000, history=4000, seed=8)
    c.logits[:, ::5], c.logits[:, 1::5], c.logits[:, 2::5] = float("inf"), -float("inf"), float("nan")
    c.check()


@pytest.mark.gpu
def test_rows_stand_alone_and_calls_repeat():
    c = Call(9, 50261, history=999, seed=9)
    w.w4g128_penalize(c.args())
    torch.cuda.synchronize()
    all_rows = c.out.clone()
    for r in (0, 4, 8):
        one = lambda t: t[r:r + 1]  # noqa: E731
        out = torch.zeros_like(c.out[r:r + 1])
        w.w4g128_penalize(c.args(logits=c.logits[r:r + 1], out=out, rows=1, history_start=one(c.start), history_len=one(c.len),
                                 prompt_len=one(c.prompt), repetition=one(c.repetition), presence=one(c.presence),
                                 frequency=one(c.frequency), bias_offsets=c.bias_offsets[r:r + 2], mask=c.mask[r:r + 1]))
        torch.cuda.synchronize()
        assert torch.equal(out[0].view(torch.int16), all_rows[r].view(torch.int16))
    for _ in range(5):
        c.out.fill_(0)
        w.w4g128_penalize(c.args())
        torch.cuda.synchronize()
        assert torch.equal(c.out.view(torch.int16), all_rows.view(torch.int16))


@pytest.mark.gpu
def test_streams_graphs_and_two_at_once():
    calls = [Call(4, 20011, history=700, seed=s) for s in (10, 11)]
    want = []
    for c in calls:
        c.check()
        want.append(c.out.clone())
        c.out.fill_(0)
    streams = [torch.cuda.Stream() for _ in calls]
    steps = [w.PenalizeStep(c.args(), stream=s) for c, s in zip(calls, streams)]
    torch.cuda.synchronize()
    for _ in range(10):
        for st in steps:
            st.run()
    torch.cuda.synchronize()
    for c, o in zip(calls, want):
        assert torch.equal(c.out, o)
    c = calls[0]
    args = c.args()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.w4g128_penalize(args)
    for n in (0, 1, 300):
        c.len.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        ref, tol = c.reference()
        fine = torch.isfinite(ref)
        assert ((c.out.double() - ref)[fine].abs() <= tol[fine]).all()


@pytest.mark.gpu
def test_sampled_after_the_mask():
    """A mask that allows one token makes w4g128_sample draw it."""
    c = Call(5, 3001, history=100, seed=12)
    allowed = [0, 31, 32, 1999, 3000]
    c.mask.zero_()
    for r, t in enumerate(allowed):
        bit = 1 << (t % 32)
        c.mask[r, t // 32] = bit - (1 << 32) if bit >= 1 << 31 else bit
    w.w4g128_penalize(c.args())
    tokens = torch.zeros(5, dtype=torch.int32, device="cuda")
    w.w4g128_sample(w.SampleArgs(logits=c.out, row_stride=c.out.stride(0), u=torch.rand(5, device="cuda"), tokens=tokens,
                                 rows=5, vocab=3001))
    torch.cuda.synchronize()
    assert tokens.tolist() == allowed
