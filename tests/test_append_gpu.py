"""Rotated queries, and rotated keys and values appended to a paged cache
(w4g128_append), against the definition in 64 bits.

Bounds: cosine and sine are off by at most 2^-22 (the angle's fp32 argument
2^-25 radians, the functions 2 units of 2^-24, the far position's turns 2^-28),
the two products and their sum by 2^-23 of |a| + |b|: 2^-21 (|a| + |b|) in all,
then one rounding: 2^-8 of the value in bf16, 2^-4 of it (2^-10 scales below the
normal range) as a code.  Values are not computed with: their codes are exact."""
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_g128_gb300 as w  # noqa: E402
from paged_cases import Paged, fresh_scale, to_codes, values  # noqa: E402


class Call(Paged):
    def __init__(self, seqs, rot=None, pairs=0, base=1e4, size=0, **kw):
        super().__init__(seqs, **kw)
        self.rot, self.pairs = self.D if rot is None else rot, pairs
        i = torch.arange(self.rot // 2, dtype=torch.float64, device="cuda")
        self.freqs = base ** (-2 * i / max(self.rot, 1))
        rows = lambda: self.rnd(self.rows, self.Hkv * self.D + self.pad)[:, :self.Hkv * self.D]  # noqa: E731
        self.k_new, self.v_new = rows(), rows()
        if size:  # rows of very different magnitudes
            e = torch.randint(-size, size + 1, (self.rows, 1), generator=self.g, device="cuda")
            self.k_new *= torch.exp2(e.double()).bfloat16()
            self.v_new *= torch.exp2(e.double()).bfloat16()
        self.q_out = torch.full((self.rows, self.Hq * self.D + self.pad), 7.0, dtype=torch.bfloat16, device="cuda")

    def args(self, **kw):
        a = dict(self.common(), q_out=self.q_out, q_out_row=self.q_out.stride(0), k_new=self.k_new, v_new=self.v_new,
                 kv_row=self.k_new.stride(0), freqs=self.freqs if self.rot else None, rot_dim=self.rot,
                 interleaved=self.pairs)
        return w.AppendArgs(**{**a, **kw})

    def run(self, status=0, **kw):
        args = self.args(**kw)
        nb = w.w4g128_append_workspace_bytes(args)
        assert nb > 0
        ws = torch.full((nb,), 0x5A, dtype=torch.uint8, device="cuda")
        w.w4g128_append(args, ws)
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws) == status

    def rotated(self, x, pos):
        """[n][heads][dim] in 64 bits, and |a| + |b| of each value's pair."""
        x = x.double().reshape(pos.numel(), -1, self.D)
        out, size = x.clone(), torch.zeros_like(x)
        h = self.rot // 2
        if h:
            angle = pos.double()[:, None, None] * self.freqs
            c, s = torch.cos(angle), torch.sin(angle)
            ia, ib = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.pairs else (slice(0, h), slice(h, self.rot))
            a, b = x[..., ia], x[..., ib]
            out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
            size[..., ia] = size[..., ib] = a.abs() + b.abs()
        return out, size * 2.0 ** -21

    def check(self, **kw):
        before = {n: getattr(self, n).clone() if getattr(self, n) is not None else None
                  for n in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale")}
        q = self.q.clone()
        self.run(**kw)
        want = {n: t.clone() if t is not None else None for n, t in before.items()}
        near = torch.zeros(before["k_cache"].shape, dtype=torch.bool, device="cuda")  # keys that need not be equal
        for b, (n, new) in enumerate(self.seqs):
            start = max(0, n - new)
            real = n - start if new else 0
            if real <= 0:
                continue
            lo = self.offsets[b] + new - real
            rows = slice(lo, lo + real)
            pos = torch.arange(start, n, device="cuda")
            ids, slot = self.table[b, pos // self.page].long(), pos % self.page
            y, slack = self.rotated(q[rows], pos)
            got = self.q_out[rows, :self.Hq * self.D].reshape(real, self.Hq, self.D).double()
            assert ((got - y).abs() <= 2.0 ** -8 * y.abs() + slack * 1.01).all()
            want["q_out"][rows, :self.Hq * self.D] = self.q_out[rows, :self.Hq * self.D]
            for name, (x, slack) in (("k", self.rotated(self.k_new[rows], pos)),
                                     ("v", (self.v_new[rows].double().reshape(real, self.Hkv, self.D), None))):
                cache, now = want[name + "_cache"], getattr(self, name + "_cache")
                if not self.block:
                    if slack is None:
                        cache[ids, slot] = x.bfloat16()
                    else:
                        got = now[ids, slot].double()
                        same = (got == x) | (torch.isnan(got) & torch.isnan(x))
                        assert (same | ((got - x).abs() <= 2.0 ** -8 * x.abs() + slack * 1.01)).all()
                        near[ids, slot] = True
                    continue
                scales = want[name + "_scale"]
                finite = torch.where(torch.isfinite(x), x, 0.0)
                for p0 in range(start // self.block * self.block, n, self.block):
                    i0, i1 = max(p0 - start, 0), min(p0 + self.block, n) - start
                    page, blk = ids[i0], slot[i0] // self.block
                    top = finite[i0:i1].abs().amax((0, 2))
                    new_scale = fresh_scale(top)
                    held = max(start - p0, 0)
                    if held:
                        was = scales[page, :, blk].double()
                        new_scale = torch.where((was > 0) & (top <= 448 * was), was, new_scale)
                        old = (slot[i0] - held + torch.arange(held, device="cuda")).long()
                        grown = new_scale != was
                        again = to_codes(values(cache[page, old]) * (was / new_scale)[None, :, None])
                        cache[page, old] = torch.where(grown[None, :, None], again, cache[page, old])
                    scales[page, :, blk] = new_scale.float()
                    codes = x[i0:i1] / new_scale[None, :, None]
                    if slack is None:
                        cache[ids[i0:i1], slot[i0:i1]] = to_codes(codes)
                    else:
                        got = values(now[ids[i0:i1], slot[i0:i1]])
                        off = (got - codes).abs()
                        ok = off <= torch.maximum(2.0 ** -4 * codes.abs(), torch.tensor(2.0 ** -10, device="cuda")) + \
                            slack[i0:i1] / new_scale[None, :, None] * 1.01
                        assert (ok | (torch.isnan(got) & ~torch.isfinite(codes))).all()
                        near[ids[i0:i1], slot[i0:i1]] = True
        for n, t in want.items():
            if t is not None:
                now = getattr(self, n)
                same = (now == t) | (torch.isnan(now) & torch.isnan(t)) if now.is_floating_point() else now == t
                if n == "k_cache":
                    same |= near
                assert same.all(), (n, (~same).nonzero()[:5])


SEQS = [(1, 1), (2, 2), (15, 3), (16, 1), (17, 5), (31, 16), (63, 1), (64, 4), (65, 2), (80, 16), (129, 7), (300, 1),
        (5, 0), (0, 0)]
PROMPTS = [(17, 17), (64, 64), (65, 40), (300, 299), (129, 1), (200, 63), (130, 66), (77, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("block", [0, 1, 2, 16])
@pytest.mark.parametrize("seqs", [SEQS, PROMPTS], ids=["few", "prompts"])
def test_lengths(dim, block, seqs):
    Call(seqs, q_heads=6, kv_heads=3, dim=dim, block=block, seed=dim + block, size=3).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,rot", [(64, 0), (64, 16), (64, 48), (128, 32), (128, 112), (256, 64), (256, 240)])
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("seqs", [SEQS, PROMPTS], ids=["few", "prompts"])
def test_rotations(dim, rot, pairs, seqs):
    Call(seqs, dim=dim, rot=rot, pairs=pairs, block=0, seed=rot).check()
    Call(seqs, dim=dim, rot=rot, pairs=pairs, block=4, seed=rot + 1).check()


@pytest.mark.gpu
@pytest.mark.parametrize("block,page", [(0, 48), (16, 48), (32, 32), (64, 64), (64, 192), (8, 1024)])
@pytest.mark.parametrize("seqs", [SEQS, PROMPTS, [(1000, 1000), (2000, 77)]], ids=["few", "prompts", "long"])
def test_pages_and_blocks(block, page, seqs):
    Call(seqs, q_heads=8, kv_heads=2, dim=128, block=block, page=page, seed=block + page, size=5).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(head_major=True), dict(pad=8), dict(pad=64, head_major=True, block=4),
                                dict(max_len=5000, block=0), dict(kv_heads=1, q_heads=16), dict(kv_heads=40, q_heads=40)])
def test_layouts(kw):
    for seqs in (SEQS, PROMPTS):
        Call(seqs, dim=128, seed=3, **kw).check()


@pytest.mark.gpu
def test_more_rows_than_the_length():
    """Rows at negative positions are left as they are."""
    for block in (0, 16):
        Call([(0, 3), (2, 5), (0, 0), (7, 7), (1, 16)], block=block, seed=1).check()
        Call([(0, 30), (2, 50), (70, 90)], block=block, seed=2).check()


@pytest.mark.gpu
@pytest.mark.parametrize("pos", [2 ** 24 - 1, 2 ** 24 - 17, 10 ** 7, 3 * 10 ** 6 + 1])
@pytest.mark.parametrize("base", [1e4, 1e6])
def test_far_positions(pos, base):
    """The angle is as exact at the far end: a product in 32 bits is off by a whole turn there."""
    c = Call([(pos % 64 + 1 + 64, 3)], dim=64, page=64, max_len=2 ** 24, base=base, block=0, seed=5)
    c.seqs = [(pos + 1, 3)]
    c.lens[0] = pos + 1
    c.table[0, (pos - 2) // 64] = 0
    c.table[0, pos // 64] = 1
    c.check()


@pytest.mark.gpu
def test_frequencies_of_any_kind():
    """Negative, zero and large frequencies."""
    c = Call(SEQS, dim=64, seed=6, block=0)
    c.freqs[:8] = torch.tensor([0.0, -1.0, -1e-9, 2 * torch.pi, 100.5, -77.25, torch.pi, 0.25 * torch.pi])
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 4, 16, 64])
@pytest.mark.parametrize("new", [1, 3, 16, 40])
def test_blocks_that_grow(block, new):
    """A sequence that grows by `new` rows at a time, of rising and falling magnitudes: each time as the rule says."""
    c = Call([(150, new)], kv_heads=2, dim=64, page=64, block=block, seed=new, size=9)
    c.k_scale.fill_(float("nan"))  # what a block holds before its first position counts for nothing
    c.v_scale.fill_(float("nan"))
    n, at = 0, 0
    while n < 150:
        step = min(new, 150 - n)
        n += step
        c.seqs, c.offsets = [(n, step)], [0, step]
        c.lens[0], c.offsets_d[1] = n, step
        c.k_new[:] = c.k_new.roll(1, 0)
        c.v_new[:] = (c.v_new.roll(1, 0).float() * (40.0 if at % 5 == 3 else 1 / 16 if at % 5 == 4 else 1.0)).bfloat16()
        c.v_new.clamp_(-1e30, 1e30)
        at += 1
        c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 256])
def test_rows_at_once_are_rows_one_by_one(dim):
    """With a scale of its own a row is what it is alone: queries, codes and scales bit for bit; a bf16 cache too."""
    for block in (0, 1):
        kw = dict(q_heads=4, kv_heads=2, dim=dim, block=block, max_len=100, seed=8, size=4)
        many = Call([(90, 16)], **kw)
        one = Call([(90, 16)], **kw)
        many.run()
        for i in range(16):
            one.lens[0] = 75 + i
            one.offsets_d[:] = torch.tensor([i, i + 1], dtype=torch.int32)
            one.run()
        prompt = Call([(90, 16)], max_new=90, **kw)  # the form for prompts
        prompt.run()
        for other in (one, prompt):
            for n in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale"):
                if getattr(many, n) is not None:
                    assert torch.equal(getattr(many, n), getattr(other, n)), (n, block)


@pytest.mark.gpu
def test_the_same_call_again_changes_nothing():
    for block in (0, 4, 16):
        c = Call(SEQS, block=block, seed=9, size=6)
        c.run()
        now = [t.clone() for t in (c.q_out, c.k_cache, c.v_cache)] + ([c.k_scale.clone(), c.v_scale.clone()] if block else [])
        c.run()
        for a, b in zip(now, [c.q_out, c.k_cache, c.v_cache] + ([c.k_scale, c.v_scale] if block else [])):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_non_finite_values():
    """In a bf16 cache as they are (values), in 8 bits NaN codes that do not touch the scale."""
    for block in (0, 1, 16):
        c = Call([(40, 5), (90, 20)], rot=0, block=block, seed=10)
        for t in (c.k_new, c.v_new):
            t[1, 3], t[2, 64], t[9, :64], t[7, 1] = float("inf"), -float("inf"), float("nan"), float("nan")
        c.check()
        if block:
            assert torch.isfinite(c.v_scale).all() and (c.v_cache.view(torch.uint8) & 0x7F == 0x7F).sum() >= 67


@pytest.mark.gpu
def test_zeros_and_the_smallest_values():
    c = Call([(20, 4), (33, 33)], block=16, seed=11)
    c.k_new.zero_()
    c.v_new[:] = 2.0 ** -130
    c.check()
    c = Call([(4, 4), (33, 33)], block=4, seed=11)
    c.v_new[:] = 3.3e38
    c.check()


@pytest.mark.gpu
def test_queries_in_place_and_none():
    c = Call(SEQS, block=16, seed=12)
    c.run()
    d = Call(SEQS, block=16, seed=12)
    d.run(q_out=d.q, q_out_row=d.q.stride(0))
    live = c.offsets[-1]
    real = torch.cat([torch.arange(c.offsets[b] + max(0, new - n), c.offsets[b + 1]) for b, (n, new) in enumerate(SEQS)])
    assert torch.equal(d.q[real], c.q_out[real]) and torch.equal(d.q[live:], c.q[live:])
    e = Call(SEQS, block=16, seed=12)
    e.run(q=None, q_out=None, q_heads=0)
    for x in (d, e):
        assert torch.equal(x.k_cache, c.k_cache) and torch.equal(x.v_scale, c.v_scale)
    p = Call(PROMPTS, block=0, seed=13)
    r = Call(PROMPTS, block=0, seed=13)
    p.run()
    r.run(q_out=r.q, q_out_row=r.q.stride(0))
    assert torch.equal(r.q[:p.offsets[-1]], p.q_out[:p.offsets[-1]])


@pytest.mark.gpu
def test_values_out_of_range_are_reported_and_left_out():
    for seqs in ([(100, 2), (60, 2), (80, 2)], [(100, 20), (60, 30), (80, 40)]):
        clean = Call(seqs, max_len=112, seed=4)
        clean.run()
        for field, at, wrongs in (("lens", 1, (-1, 113, 2 ** 31 - 1, -2 ** 31)), ("offsets_d", 1, (-1, 2 ** 31 - 1, -2 ** 31)),
                                  ("table", (1, 3), (-1, clean.pages, 2 ** 31 - 1, -2 ** 31))):
            for wrong in wrongs:
                c = Call(seqs, max_len=112, seed=4)
                getattr(c, field)[at] = wrong
                start = [t.clone() for t in (c.k_cache, c.v_cache, c.k_scale, c.v_scale)]
                c.run(status=w.ERR_CACHE)
                a, b = c.offsets[2], c.offsets[3]
                assert torch.equal(c.q_out[a:b], clean.q_out[a:b])  # the last sequence is as it should be
                mine = c.table[1, :4].long() if field != "table" else c.table[1, 3:].long()[:0]
                for t, s, ok in zip((c.k_cache, c.v_cache, c.k_scale, c.v_scale), start,
                                    (clean.k_cache, clean.v_cache, clean.k_scale, clean.v_scale)):
                    assert torch.equal(t[c.table[2, :5].long()], ok[c.table[2, :5].long()])
                    assert torch.equal(t[mine], s[mine])
                if field == "table":
                    assert torch.equal(c.q_out, clean.q_out)
        c = Call(seqs, max_len=112, seed=4)
        c.table[1, 4:] = 10 ** 9  # pages behind the new rows are not looked at
        c.table[1, 0] = -5        # nor those before
        c.run()
        assert torch.equal(c.v_cache, clean.v_cache)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    H, D, page = 8, 128, 64
    c = Call([(200, 3)], q_heads=16, kv_heads=H, dim=D, page=page, block=0, seed=6)
    pages = (1 << 31) // (H * D * page) + 40
    first = pages - c.pages
    d = Call([(200, 3)], q_heads=16, kv_heads=H, dim=D, page=page, block=0, seed=6)
    d.k_cache, d.v_cache = (torch.zeros((pages, page, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    d.table[0, :4] += first
    d.pages = pages
    c.run()
    d.run()
    pos = torch.arange(197, 200, device="cuda")
    for a, b in ((c.k_cache, d.k_cache), (c.v_cache, d.v_cache)):
        assert torch.equal(a[c.table[0, pos // page].long(), pos % page], b[d.table[0, pos // page].long(), pos % page])
        assert not b[:first].any()


@pytest.mark.gpu
def test_many_sequences():
    seqs = [((b * 37) % 100 + 3, b % 4) for b in range(700)]
    Call(seqs, q_heads=2, kv_heads=1, dim=64, seed=14).check()


@pytest.mark.gpu
def test_streams_graphs_and_status_of_replays():
    c = Call([(100, 2), (60, 1)], max_len=112, seed=15)
    twin = Call([(100, 2), (60, 1)], max_len=112, seed=15)
    args = c.args()
    ws = torch.empty(w.w4g128_append_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        w.AppendStep(args, ws).run()
    s.synchronize()
    twin.run()
    assert torch.equal(c.k_cache, twin.k_cache) and torch.equal(c.q_out, twin.q_out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.w4g128_append(args, ws)
    for length, status in ((60, 0), (500, w.ERR_CACHE), (59, 0), (-1, w.ERR_CACHE), (12, 0)):
        c.lens[1] = length
        g.replay()
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws) == status, length
        if status == 0:
            twin.seqs[1] = (length, 1)
            twin.lens[1] = length
            twin.check()
            for n in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale"):
                assert torch.equal(getattr(c, n), getattr(twin, n))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,block", [(64, 0), (128, 0), (256, 0), (128, 1), (64, 16), (256, 4)])
@pytest.mark.parametrize("new", [8, 9, 16])
def test_few_sequences_and_many(dim, block, new):
    """The forms for few rows and for many, on both sides of what chooses them."""
    for count in (1, 7, 9, 10, 11):
        seqs = [((b * 53) % 90 + 1, min((b * 7) % 90 + 1, new)) for b in range(count - 1)] + [(77, new)]
        Call(seqs, dim=dim, block=block, max_len=100, seed=count).check()


@pytest.mark.gpu
def test_sequences_of_a_batch_are_sequences_alone():
    for block in (0, 16):
        seqs = [((b * 37) % 90 + 4, b % 3) for b in range(100)]
        kw = dict(q_heads=4, kv_heads=2, dim=64, block=block, seed=16)
        many, alone = Call(seqs, **kw), Call(seqs, **kw)
        many.run()
        lens, offsets, table = alone.lens, alone.offsets_d, alone.table
        for b in range(len(seqs)):
            alone.seqs, alone.lens, alone.offsets_d, alone.table = [seqs[b]], lens[b:], offsets[b:], table[b:]
            alone.run()
        for n in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale"):
            if getattr(many, n) is not None:
                assert torch.equal(getattr(many, n), getattr(alone, n)), (n, block)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,block", [(64, 0), (128, 0), (256, 16), (128, 64)])
def test_prompts_beside_single_tokens(dim, block):
    """One long prompt among sequences of few rows or none, wherever it stands; and prompts of one length."""
    for at in (0, 7, 39):
        seqs = [(3 + 5 * b, b % 3) for b in range(40)]
        seqs[at] = (900, 850)
        Call(seqs, dim=dim, block=block, page=64, q_heads=6, kv_heads=2, seed=at).check()
    Call([(200, 100), (100, 100), (163, 100)], dim=dim, block=block, page=64, q_heads=6, kv_heads=2, extra_rows=0, seed=17).check()


@pytest.mark.gpu
@pytest.mark.parametrize("block", [0, 16])
def test_any_number_of_rows_allowed(block):
    """max_new at its bound with as many sequences as there may be, and more heads than are worked on at once."""
    seqs = [(b % 7, min(b % 7, b % 4)) for b in range(1024)]
    Call(seqs, dim=256, block=block, q_heads=24, kv_heads=3, max_new=1 << 20, seed=18).check()
    Call([(90, 80)], dim=256, block=block, q_heads=24, kv_heads=3, max_new=1 << 20, seed=19).check()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** 125, 2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 127])
@pytest.mark.parametrize("dim,block,seqs", [(64, 16, SEQS), (128, 64, PROMPTS), (256, 4, PROMPTS)], ids=["few", "prompts", "wide"])
def test_blocks_that_hold_the_largest_scales(scale, dim, block, seqs):
    """A block's scale stays where the new rows fit under it, up to the largest: its inverse is below fp32's normal range."""
    c = Call(seqs, dim=dim, block=block, page=64, seed=20)
    c.k_scale.fill_(scale)
    c.v_scale.fill_(scale)
    c.k_new.mul_(2.0 ** 124).clamp_(-2.0 ** 127, 2.0 ** 127)  # (turned: up to 2^127.5)
    c.v_new.mul_(2.0 ** 124)
    c.check()
    held = [b for b, (n, new) in enumerate(seqs) if new and 0 < (n - new) % block]
    for b in held:
        n, new = seqs[b]
        page, at = c.table[b, (n - new) // 64].long(), (n - new) % 64
        assert (c.v_scale[page, :, at // block] == scale).all()
        assert (c.v_cache[page, at].view(torch.uint8) & 0x7F != 0).any()


@pytest.mark.gpu
@pytest.mark.parametrize("block", [0, 1, 16])
@pytest.mark.parametrize("seqs", [[(9, 3), (40, 2)], [(100, 90), (33, 20)]], ids=["few", "prompts"])
@pytest.mark.parametrize("pairs", [0, 1])
def test_rotations_beyond_the_range_of_fp32(block, seqs, pairs):
    """Pairs of 3e38 turn to up to 4.2e38: infinite in bf16, a NaN code in 8 bits, and no part of a block's magnitude."""
    c = Call(seqs, dim=64, block=block, pairs=pairs, seed=21)
    c.q.fill_(3e38)
    c.k_new.fill_(3e38)
    c.run()
    top = torch.finfo(torch.float32).max
    seen = 0
    for b, (n, new) in enumerate(seqs):
        rows, pos = slice(c.offsets[b], c.offsets[b] + new), torch.arange(n - new, n, device="cuda")
        ids, slot = c.table[b, pos // c.page].long(), pos % c.page
        for x, got in ((c.q, c.q_out[rows, :c.Hq * c.D].reshape(new, c.Hq, c.D)), (c.k_new, c.k_cache[ids, slot])):
            y, slack = c.rotated(x[rows], pos)
            if got.dtype == torch.bfloat16:  # bf16 rounds to infinity from 2^128 (1 - 2^-9) on
                over, clear = y.abs() > 2.0 ** 128 * (1 - 2.0 ** -9), (y.abs() - 2.0 ** 128 * (1 - 2.0 ** -9)).abs() > slack
                assert (torch.isinf(got) == over)[clear].all()
            else:
                over, clear = y.abs() > top, (y.abs() - top).abs() > slack
                assert (torch.isnan(values(got)) == over)[clear].all()
            seen += int((over & clear).sum())
        if block:
            fits = torch.where(y.abs() <= top, y.abs(), 0.0)
            assert torch.isfinite(c.k_scale[ids, :, slot // block]).all()
            assert (448 * c.k_scale[ids, :, slot // block].double() * (1 + 2.0 ** -20) >= fits.amax(-1) - slack.amax(-1)).all()
    assert seen > 100
