"""Attention of new tokens over a paged cache of e4m3 codes (w4g128_attend8)
against the definition in 64 bits, computed row by row from the dense values.

The bound, per element, with A = sum_j softmax_j |v_j| (64 bits): the weights
times the values' scales are rounded to fp16 (2^-11 relative each, or 2^-31 of
the row's largest for what lies below fp16's normal range), the sum of weights
is not, so that error is at most 2^-11 A and 2^-31 sum |code| times the largest
scale; a score's fp32 sum of D products is off by (D + 4) 2^-24 scale sum|q k|,
which moves a weight by that much relative, numerator and denominator; exp2,
log2 and the inverse add 2^-20, the fp32 sums over L positions at most
(L + 64) 2^-24 each; the output rounds once, 2^-8."""
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_g128_gb300 as w  # noqa: E402
from paged_cases import Paged, values  # noqa: E402


class Call(Paged):
    def __init__(self, seqs, window=0, sinks=0, **kw):
        super().__init__(seqs, **kw)
        self.window, self.sinks, self.scale = window, sinks, self.D ** -0.5
        self.out = torch.full((self.rows, self.Hq * self.D + self.pad), 7.0, dtype=torch.bfloat16, device="cuda")

    def args(self, **kw):
        return w.Attend8Args(**{**self.common(), **dict(out=self.out, out_row=self.out.stride(0), window=self.window,
                                                        sinks=self.sinks, scale=self.scale), **kw})

    def run(self, status=0, **kw):
        args = self.args(**kw)
        nb = w.w4g128_attend8_workspace_bytes(args)
        assert nb > 0
        ws = torch.full((nb,), 0x5A, dtype=torch.uint8, device="cuda")
        w.w4g128_attend8(args, ws)
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws) == status
        return self.out[:, :self.Hq * self.D].reshape(self.rows, self.Hq, self.D)

    def dense(self, b):
        """(k, v) [length][head][dim] of sequence b and the values' scales [length][head]."""
        pos = torch.arange(self.seqs[b][0], device="cuda")
        ids, slot = self.table[b, pos // self.page].long(), pos % self.page
        ks, vs = (s[ids, :, slot // self.block].double() for s in (self.k_scale, self.v_scale))
        return values(self.k_cache[ids, slot]) * ks[..., None], values(self.v_cache[ids, slot]) * vs[..., None], vs

    def reference(self):
        """out and its bound, [rows][head][dim] in 64 bits; rows of no sequence: NaN."""
        out = torch.full((self.rows, self.Hq, self.D), float("nan"), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        G = self.Hq // self.Hkv
        for b, (n, new) in enumerate(self.seqs):
            k, v, vs = self.dense(b)
            for i in range(new):
                r, p = self.offsets[b] + i, n - new + i
                pos = torch.arange(max(p + 1, 0), device="cuda")
                if self.window:
                    pos = pos[(p - pos < self.window) | (pos < self.sinks)]
                if pos.numel() == 0:
                    out[r] = 0
                    continue
                q = self.q[r].double().view(self.Hkv, G, self.D)
                kk, vv = k[pos], v[pos]
                a = torch.softmax(torch.einsum("hgd,lhd->hgl", q, kk) * self.scale, -1)
                o = torch.einsum("hgl,lhd->hgd", a, vv)
                A = torch.einsum("hgl,lhd->hgd", a, vv.abs())
                s = (torch.einsum("hgd,lhd->hgl", q.abs(), kk.abs()).amax(-1) * abs(self.scale))[..., None]
                e = 2 * (self.D + 4) * 2.0 ** -24 * s + 2.0 ** -20 + 2 * (pos.numel() + 64) * 2.0 ** -24
                small = 2.0 ** -31 * (vv.abs() / vs[pos][..., None]).sum(0) * vs[pos].amax(0)[:, None]
                out[r] = o.reshape(self.Hq, self.D)
                tol[r] = (2.0 ** -8 * o.abs() + (A + o.abs()) * (2.0 ** -11 + e) * 1.02 + small[:, None]).reshape(self.Hq, self.D)
        return out, tol

    def check(self, **kw):
        ref, tol = self.reference()
        before = [t.clone() for t in (self.k_cache, self.v_cache, self.k_scale, self.v_scale)]
        rest = self.out.clone()
        got = self.run(**kw)
        mine = ~torch.isnan(ref[:, 0, 0])
        err = (got[mine].double() - ref[mine]).abs()
        assert torch.isfinite(got[mine]).all()
        assert (err <= tol[mine]).all(), float((err / tol[mine].clamp(min=1e-30)).max())
        assert torch.equal(got[~mine], rest[:, :self.Hq * self.D].reshape(got.shape)[~mine])
        assert torch.equal(self.out[:, self.Hq * self.D:], rest[:, self.Hq * self.D:])
        for t, b in zip((self.k_cache, self.v_cache, self.k_scale, self.v_scale), before):
            assert torch.equal(t, b)
        return got


LENGTHS = [(1, 1), (2, 2), (15, 3), (16, 1), (17, 5), (31, 16), (63, 1), (64, 4), (65, 2), (80, 16), (129, 7), (300, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv_heads,group,block", [(1, 1, 16), (2, 4, 1), (1, 16, 4), (3, 5, 8)])
def test_lengths(dim, kv_heads, group, block):
    Call(LENGTHS, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, block=block, seed=dim + group).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,n,new,page,block", [(64, 5003, 16, 16, 16), (128, 9001, 8, 64, 64), (256, 4097, 3, 48, 16),
                                                  (128, 70001, 1, 256, 32), (64, 300011, 2, 64, 1)])
def test_long(dim, n, new, page, block):
    Call([(n, new)], q_heads=8, kv_heads=2, dim=dim, page=page, block=block, seed=n).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kv_heads,count", [(1, 1), (1, 2), (5, 1), (7, 3), (8, 2), (11, 2), (4, 20), (64, 5), (256, 3)])
def test_splits(kv_heads, count):
    """From one head on many clusters to many heads on one CTA each."""
    Call([(3001 - 7 * b, 1 + b % 3) for b in range(count)], q_heads=kv_heads, kv_heads=kv_heads, dim=64, seed=kv_heads,
         block=2).check()


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (64, 4), (100, 70), (5000, 4), (1 << 30, 9)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows_and_sinks(window, sinks, dim):
    Call(LENGTHS + [(2000, 9), (1999, 16)], dim=dim, window=window, sinks=sinks, seed=window % 1000 + sinks,
         page=32, block=32).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(head_major=True), dict(pad=8), dict(page=48, pad=64, head_major=True, block=4),
                                dict(max_len=5000), dict(page=1024, block=64), dict(spread=12)])
def test_layouts(kw):
    Call([(333, 4), (20, 1), (1, 1), (150, 16)], q_heads=12, kv_heads=2, dim=128, seed=3, **kw).check()


@pytest.mark.gpu
def test_rows_that_see_nothing():
    for max_len in (16, 1000):
        c = Call([(0, 0), (0, 3), (2, 5), (40 if max_len > 16 else 9, 0), (7, 7), (0, 16)], max_len=max_len, seed=1)
        got = c.check()
        assert torch.equal(got[0:3], torch.zeros_like(got[0:3])) and torch.equal(got[3:6], torch.zeros_like(got[3:6]))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,window,sinks", [(64, 0, 0), (128, 0, 0), (256, 0, 0), (128, 200, 5), (64, 37, 40)])
@pytest.mark.parametrize("count", [1, 4])
def test_a_row_alone_gives_the_same_bits(dim, window, sinks, count):
    """Each new token of a verify step, decoded alone from the same cache, gives its row's bits."""
    seqs = [(1500, 16), (77, 5), (16, 16), (900, 1)][:count]
    kw = dict(q_heads=6, kv_heads=2, dim=dim, window=window, sinks=sinks, max_len=1600, spread=4)
    c = Call(seqs, seed=5, **kw)
    together = c.run().clone()
    for b, (n, new) in enumerate(seqs):
        for i in (0, new // 2, new - 1):
            one = Call([(n - new + i + 1, 1)] + [(0, 0)] * (count - 1), seed=5, **kw)
            one.k_cache, one.v_cache, one.k_scale, one.v_scale, one.pages = c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.pages
            one.table = c.table[b:b + 1].repeat(count, 1)
            r = c.offsets[b] + i
            one.q[0] = c.q[r]
            assert torch.equal(one.run()[0], together[r]), (b, i)
    assert torch.equal(c.run(), together)  # and again: deterministic


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_masked_codes_and_scales_take_no_part(dim):
    """NaN codes and any scales behind a row's own position, before its window, in unused slots and in unseen pages;
    the page ids of unseen pages are out of range."""
    c = Call([(203, 8), (50, 8)], dim=dim, window=40, sinks=3, page=16, block=1, max_len=256, seed=7)
    clean = c.check().clone()
    bad = float("nan")
    pos = torch.arange(3, 203 - 8 - 39, device="cuda")  # before the first row's window
    for cache, scale in ((c.k_cache, c.k_scale), (c.v_cache, c.v_scale)):
        cache[c.table[0, pos // 16].long(), pos % 16] = 0xFF
        scale[c.table[0, pos // 16].long(), :, pos % 16] = bad
        cache[c.table[0, 12].long(), 203 - 192:] = 0x7F  # slots behind the end
        scale[c.table[0, 12].long(), :, 203 - 192:] = float("inf")
        cache[c.table[0, 12].long(), 200 - 192] = 0x7F   # position 200: rows 0..4 of sequence 0 do not see it
        scale[c.table[1, 3].long(), :, 49 - 48] = -float("inf")  # position 49: the last row of sequence 1 alone does
    c.table[0, 1:9] = 10 ** 9          # whole pages that nobody sees
    got = c.run()
    assert torch.equal(got[:5], clean[:5]) and torch.equal(got[8:15], clean[8:15])
    assert torch.isnan(got[5:8]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 256])
def test_window_edges_inside_a_tile_with_nan_codes(dim):
    """A value that the first rows still see and the last rows do not: its columns are NaN, the others as they were."""
    c = Call([(90, 16)], dim=dim, window=30, page=16, max_len=96, seed=9)
    clean = c.run().clone()
    pos = 90 - 16 - 30 + 8  # seen by rows 0..7
    cols = torch.tensor([0, 1, 2, 3, 17, 30, dim - 1], device="cuda")
    c.v_cache[c.table[0, pos // 16].long(), pos % 16, 1, cols] = 0x7F
    got = c.run()
    assert torch.equal(got[8:], clean[8:])
    want = clean[:8].clone()
    want[:, 2:, cols] = float("nan")  # heads 2 and 3 share the key/value head 1
    assert torch.equal(torch.isnan(got[:8]), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got[:8]), torch.nan_to_num(want))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,new", [(64, 3), (128, 1), (128, 16), (256, 16)])
@pytest.mark.parametrize("scores", [lambda p: p / 32, lambda p: p / 2, lambda p: -p / 4, lambda p: 5.5 * (p // 16),
                                    lambda p: 5.0 * (p // 64 % 2), lambda p: 300.0 * (p == 390), lambda p: -1e4 + p / 8],
                         ids=["slow", "fast", "falling", "steps", "to and fro", "a peak", "far below zero"])
def test_scores_that_move_the_maximum(dim, new, scores):
    """Scores rising by less, and by more, than the factor that the kernel lets a row's weights grow to."""
    from paged_cases import fresh_scale, to_codes
    c = Call([(401, new), (64, new)], q_heads=8, kv_heads=2, dim=dim, block=1, seed=new)
    c.scale = 1.0
    c.q[:] = 0
    c.q.view(c.rows, 8, dim)[:, :, 0] = torch.tensor([1.0, 0.5, 1.0, 2.0] * 2, device="cuda").bfloat16()
    for b, (n, _) in enumerate(c.seqs):
        pos = torch.arange(n, device="cuda")
        s = scores(pos.double())
        scale = fresh_scale(s.abs())
        ids = c.table[b, pos // c.page].long()
        c.k_cache[ids, pos % c.page, :, 0] = to_codes(s / scale)[:, None]
        c.k_scale[ids, :, pos % c.page] = scale.float()[:, None]
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("small,large", [(2.0 ** -70, 1.0), (2.0 ** -30, 2.0 ** 30), (1.0, 2.0 ** 100), (0.0, 1.0), (0.3, 0.7),
                                         (2.0 ** -80, 2.0 ** 40), (2.0 ** -79, 2.0 ** -79)])
def test_scales_of_any_size(small, large):
    """Scales that are no powers of two, and neighbours of very different sizes: a value without weight in the sum
    still has its weight in the softmax.  0 counts as 2^-80."""
    c = Call([(200, 3), (31, 1), (1700, 2)], block=4, seed=21)
    pick = torch.rand(c.v_scale.shape, generator=c.g, device="cuda") < 0.5
    c.v_scale[:] = torch.where(pick, small, large) * (1 + torch.rand(c.v_scale.shape, generator=c.g, device="cuda"))
    c.k_scale *= 1.1
    given = c.v_scale.clone()
    c.v_scale.clamp_(min=2.0 ** -80)
    ref, tol = c.reference()
    c.v_scale[:] = given
    got = c.run()
    mine = ~torch.isnan(ref[:, 0, 0])
    assert ((got[mine].double() - ref[mine]).abs() <= tol[mine]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 40])
def test_queries_of_any_size(dim, size):
    """q's row scaled up or down by a power of two and the keys the other way: the same scores, the same bits."""
    c = Call([(300, 4), (40, 16)], dim=dim, seed=22)
    want = c.run().clone()
    c.q *= size
    c.k_scale /= size
    assert torch.equal(c.run(), want)


@pytest.mark.gpu
def test_non_finite_queries_stay_with_their_rows():
    c = Call([(300, 4)], dim=128, seed=23)
    want = c.run().clone()
    c.q[1, 5] = float("nan")
    c.q[2, 130] = float("inf")  # head 1
    got = c.run()
    assert torch.isnan(got[1, 0]).all() and torch.isnan(got[2, 1]).all()
    keep = torch.ones(c.rows, c.Hq, dtype=torch.bool, device="cuda")
    keep[1, 0] = keep[2, 1] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.gpu
def test_values_out_of_range_are_reported_and_left_out():
    for max_len in (112, 40000):
        c = Call([(100, 2), (60, 2), (80, 2)], max_len=max_len, seed=4)
        clean = c.run().clone()

        def again(status=w.ERR_CACHE, **kw):
            c.out.fill_(7.0)
            return c.run(status=status, **kw)

        for wrong in (-1, max_len + 1, 2 ** 31 - 1, -2 ** 31):
            c.lens[1] = wrong
            got = again()
            assert torch.equal(got[:2], clean[:2]) and torch.equal(got[4:6], clean[4:6]) and (got[2:4] == 7).all()
        c.lens[1] = 60
        for wrong in ((0, 2, 1, 6), (0, -1, 4, 6), (0, 2, 4, 2 ** 31 - 1), (0, 2, 4, -2 ** 31)):
            c.offsets_d.copy_(torch.tensor(wrong, dtype=torch.int32))
            got = again()
            if wrong[1] == 2:
                assert torch.equal(got[:2], clean[:2])
        c.offsets_d.copy_(torch.tensor([0, 2, 4, 6], dtype=torch.int32))
        for wrong in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
            keep = c.table[1, 2].item()
            c.table[1, 2] = wrong              # positions 32..47 of sequence 1
            got = again()
            assert torch.equal(got[:2], clean[:2]) and torch.equal(got[4:6], clean[4:6])
            assert torch.isfinite(got[2:4]).all() and not torch.equal(got[2:4], clean[2:4])
            c.table[1, 2] = keep
        assert torch.equal(again(status=0), clean)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Pages whose codes start beyond 2^32, scales beyond 2^31 elements."""
    H, D, page = 8, 128, 64
    pages = (1 << 32) // (H * D * page) + 40
    c = Call([(200, 3)], q_heads=16, kv_heads=H, dim=D, page=page, block=64, seed=6)
    small = c.run().clone()
    first = pages - c.pages
    for name in ("k_cache", "v_cache"):
        t = torch.empty((pages, page, H, D), dtype=torch.uint8, device="cuda")
        t[first:] = getattr(c, name)
        setattr(c, name, t)
    stride = (1 << 31) // first + 8
    for name in ("k_scale", "v_scale"):
        t = torch.empty(pages * stride, dtype=torch.float32, device="cuda").view(pages, stride)[:, :H, None]
        t[first:] = getattr(c, name)
        setattr(c, name, t)
    assert first * stride >= 1 << 31
    c.table[0, :4] += first
    c.pages = pages
    assert torch.equal(c.run(scale_head=1), small)


@pytest.mark.gpu
def test_streams_and_graph_replay_follow_the_lengths():
    c = Call([(500, 2), (300, 1)], q_heads=8, kv_heads=2, dim=128, max_len=512, seed=8)
    want = c.run().clone()
    args = c.args()
    ws = torch.empty(w.w4g128_attend8_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.out.fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        w.Attend8Step(args, ws).run()
    s.synchronize()
    assert torch.equal(c.out.view(c.rows, c.Hq, c.D), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.w4g128_attend8(args, ws)
    for seqs, status in (([(500, 2), (300, 1)], 0), ([(130, 2), (299, 1)], 0), ([(2, 2), (1, 1)], 0),
                         ([(497, 2), (513, 1)], w.ERR_CACHE), ([(497, 2), (64, 1)], 0)):
        c.seqs = seqs
        c.lens.copy_(torch.tensor([n for n, _ in seqs], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws) == status
        if status == 0:
            ref, tol = c.reference()
            got = c.out.view(c.rows, c.Hq, c.D)[:3].double()
            assert ((got - ref[:3]).abs() <= tol[:3]).all()


@pytest.mark.gpu
def test_workspace_is_not_exceeded():
    for seqs, kw in (([(1000, 16), (40, 3)], dict(window=100, sinks=5)), ([(9000, 5)], dict(kv_heads=1))):
        c = Call(seqs, q_heads=8, dim=64, seed=1, **kw)
        args = c.args()
        nb = w.w4g128_attend8_workspace_bytes(args)
        whole = torch.full((nb + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        w.w4g128_attend8(args, whole[4096:], ws_bytes=nb)
        torch.cuda.synchronize()
        assert (whole[:4096] == 0x5A).all() and (whole[4096 + nb:] == 0x5A).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.125, 2.0])
def test_scales(dim, scale):
    """Negative scales prefer the smallest scores, 0 makes every visible position count the same."""
    c = Call([(300, 4), (40, 16)], dim=dim, seed=12, window=150, sinks=2)
    c.scale = scale
    c.check()


@pytest.mark.gpu
def test_two_calls_at_once():
    calls = [Call([(3000, 8)], q_heads=16, kv_heads=4, dim=128, seed=s) for s in (13, 14)]
    want = [c.run().clone() for c in calls]
    steps, streams = [], [torch.cuda.Stream() for _ in calls]
    for c, s in zip(calls, streams):
        c.out.fill_(7.0)
        a = c.args()
        steps.append(w.Attend8Step(a, torch.empty(w.w4g128_attend8_workspace_bytes(a), dtype=torch.uint8, device="cuda"),
                                   stream=s))
    torch.cuda.synchronize()
    for _ in range(10):
        for st in steps:
            st.run()
    torch.cuda.synchronize()
    for c, o in zip(calls, want):
        assert torch.equal(c.out.view(c.rows, c.Hq, c.D)[:8], o[:8])


@pytest.mark.gpu
@pytest.mark.parametrize("dim,n,new,page", [(64, 5003, 16, 16), (256, 4097, 3, 48), (128, 70001, 1, 256), (64, 300011, 2, 64)])
def test_long_norm_of_the_error(dim, n, new, page):
    """Over many positions the element bounds exceed the output, which is a mean of independent values.  The norm of a
    row's error: the output's rounding, 2^-8 of each element, and the weights', 2^-11 each and without relation to the
    values.  A tile left out shows."""
    c = Call([(n, new)], q_heads=8, kv_heads=2, dim=dim, page=page, seed=n + 1)
    ref, _ = c.reference()
    got = c.run()
    ref, got = ref[:new].flatten(1), got[:new].double().flatten(1)
    assert ((got - ref).norm(dim=1) <= (2.0 ** -8 + 2.0 ** -10) * ref.norm(dim=1)).all()


BATCH = [(3000, 16), (1, 1), (0, 0), (5000, 3), (777, 2), (64, 16), (1024, 1), (16, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim,kv_heads,group,block", [(64, 2, 4, 1), (64, 1, 1, 16), (128, 3, 2, 16), (128, 2, 16, 4), (256, 2, 2, 2),
                                                      (256, 1, 16, 16)])
@pytest.mark.parametrize("max_len", [5000, 100000])
def test_batches_of_ragged_sequences(dim, kv_heads, group, block, max_len):
    """More than three sequences: a CTA takes a chunk of positions, which may lie behind the sequence's end."""
    Call(BATCH, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, block=block, max_len=max_len, seed=dim + group).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("max_len,lengths", [(900, (900,)), (500, (200, 333)), (6000, (5000, 9, 3000, 1111, 640))])
def test_a_row_alone_gives_the_same_bits_in_clusters_and_chunks(dim, max_len, lengths):
    kw = dict(q_heads=8, kv_heads=2, dim=dim, max_len=max_len, spread=4)
    seqs = [(n, 1 + 15 * (b % 2 == 0) if n > 16 else 2) for b, n in enumerate(lengths)]
    c = Call(seqs, seed=25, **kw)
    together = c.run().clone()
    for b, (n, new) in enumerate(seqs):
        for i in sorted({0, new // 2, new - 1}):
            one = Call([(n - new + i + 1, 1)] + [(0, 0)] * (len(seqs) - 1), seed=25, **kw)
            one.k_cache, one.v_cache, one.k_scale, one.v_scale, one.pages = c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.pages
            one.table = c.table[b:b + 1].repeat(len(seqs), 1)
            r = c.offsets[b] + i
            one.q[0] = c.q[r]
            assert torch.equal(one.run()[0], together[r]), (b, i)
    assert torch.equal(c.run(), together)


@pytest.mark.gpu
def test_values_out_of_range_in_a_batch():
    c = Call([(2000, 2), (60, 2), (3000, 2), (80, 2), (4000, 2)], max_len=4000, seed=26)
    clean = c.run().clone()
    keep = c.table[2, 100].item()
    for at, wrong in ((1, -1), (1, 4001), (3, 2 ** 31 - 1), (0, -2 ** 31)):
        was = c.lens[at].item()
        c.lens[at] = wrong
        c.out.fill_(7.0)
        got = c.run(status=w.ERR_CACHE)
        for b in range(5):
            rows = slice(2 * b, 2 * b + 2)
            assert (got[rows] == 7).all() if b == at else torch.equal(got[rows], clean[rows])
        c.lens[at] = was
    for wrong in (-1, c.pages):
        c.table[2, 100] = wrong
        c.out.fill_(7.0)
        got = c.run(status=w.ERR_CACHE)
        assert torch.equal(got[:4], clean[:4]) and torch.equal(got[6:10], clean[6:10]) and torch.isfinite(got[4:6]).all()
    c.table[2, 100] = keep
    assert torch.equal(c.run(), clean)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,new", [(64, 4), (128, 4), (128, 16), (256, 1), (256, 8), (256, 10)])
def test_nan_codes_of_few_rows_and_many(dim, new):
    """A NaN code that every row sees makes its column NaN; one that only the last row sees, that row's."""
    c = Call([(200, new), (40, new)], dim=dim, seed=27)
    clean = c.run().clone()
    for pos, seen in ((77, new), (199, 1)):
        page = c.table[0, pos // 16].long()
        cols = torch.tensor([0, 5, 31, 32, dim // 2 - 1, dim // 2, dim - 1], device="cuda")
        was = c.v_cache[page, pos % 16, 1, cols].clone()
        c.v_cache[page, pos % 16, 1, cols] = 0xFF
        want = clean.clone()
        want[new - seen:new, 2:, cols] = float("nan")
        got = c.run()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
        c.v_cache[page, pos % 16, 1, cols] = was


@pytest.mark.gpu
def test_a_wide_batch_of_short_sequences():
    seqs = [((b * 29) % 70, min((b * 29) % 70, b % 3)) for b in range(400)]
    Call(seqs, q_heads=4, kv_heads=2, dim=64, seed=28).check()


@pytest.mark.gpu
def test_graphs_captured_with_one_workspace():
    """Two captured calls that share a workspace, replayed one after the other."""
    calls = [Call([(2500, 3)], q_heads=8, kv_heads=2, dim=128, seed=29), Call([(1900, 16)], q_heads=8, kv_heads=2, dim=128, seed=30,
                                                                               max_len=2500)]
    want = [c.run().clone() for c in calls]
    args = [c.args() for c in calls]
    ws = torch.empty(max(w.w4g128_attend8_workspace_bytes(a) for a in args), dtype=torch.uint8, device="cuda")
    graphs = []
    for a in args:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            w.w4g128_attend8(a, ws)
    for c in calls:
        c.out.fill_(7.0)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, o in zip(calls, want):
        assert torch.equal(c.out.view(c.rows, c.Hq, c.D)[:c.rows - 1], o[:c.rows - 1])


@pytest.mark.gpu
def test_a_batch_far_below_its_longest_length():
    """max_len cuts the sequences into far more chunks than they have."""
    c = Call([(700 + 97 * b, b % 3) for b in range(40)], q_heads=8, kv_heads=4, dim=64, max_len=1 << 18, seed=31)
    # Chunks of at least 1 / 16384 of all positions: 16384 and one more (the last, shorter one) for each of 160 pairs of
    # a sequence and head, each with 2 x 2 rows (heads that share one, new tokens) of 64 sums, a reference and a sum.
    assert w.w4g128_attend8_workspace_bytes(c.args()) <= 256 + (16384 + 160) * 4 * (64 + 2) * 4
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("max_len", [6000, 9600, 100000])
def test_bad_pages_among_many_are_found(max_len):
    """More page ids than one CTA looks over: any of them, and only those that some row sees."""
    seqs = [(2000 + 50 * b, 1) for b in range(60)]
    c = Call(seqs, q_heads=2, kv_heads=1, dim=64, max_len=max_len, seed=32)
    clean = c.run().clone()
    for b in (0, 17, 59):
        last = (seqs[b][0] - 1) // 16
        for at in (0, last // 2, last):
            keep = c.table[b, at].item()
            c.table[b, at] = c.pages
            c.out.fill_(7.0)
            got = c.run(status=w.ERR_CACHE)
            others = torch.arange(60, device="cuda") != b
            assert torch.equal(got[:60][others], clean[:60][others])
            c.table[b, at] = keep
        c.table[b, last + 1] = -1  # behind the end
    assert torch.equal(c.run(), clean)


def scales_far_apart(seqs, kv_heads, dim, block, order, small, large, **kw):
    """Value scales of blocks of `small` and `large`, up to twice that, and codes up to 1."""
    from paged_cases import to_codes
    c = Call(seqs, q_heads=kv_heads, kv_heads=kv_heads, dim=dim, block=block, page=64, seed=33, **kw)
    c.v_cache.copy_(to_codes(2 * torch.rand(c.v_cache.shape, generator=c.g, device="cuda").double() - 1).view(c.v_cache.dtype))
    more = 1 + torch.rand(c.v_scale.shape, generator=c.g, device="cuda")
    c.v_scale.fill_(small)
    for b, (n, _) in enumerate(c.seqs):
        pos = torch.arange(n, device="cuda") // block * block
        pos = pos[{"small first": pos >= n // 2, "large first": pos < n // 2, "in turn": pos // 64 % 2 == 1,
                   "one large": pos == (n - 1) // block * block}[order]]
        c.v_scale[c.table[b, pos // 64].long(), :, pos % 64 // block] = large
    c.v_scale *= more
    return c


def check_scales_far_apart(c):
    """Beside reference()'s bound: score and logarithm of the scale add up to 2^8 at most, an fp32 sum (2^-16) of a logarithm
    good to 2^-22 of its 2^7; a weight is off by as much relative, numerator and denominator."""
    ref, tol = c.reference()
    A = torch.full_like(ref, 0.0)
    for b, (n, new) in enumerate(c.seqs):
        _, v, _ = c.dense(b)
        if new:
            A[c.offsets[b]:c.offsets[b + 1]] = v.abs().amax(0).amax(-1).repeat_interleave(c.Hq // c.Hkv, 0)[None, :, None]
    got = c.run()
    mine = ~torch.isnan(ref[:, 0, 0])
    tol = tol + 2 * (2.0 ** -16 + 2.0 ** -15) * A
    err = (got[mine].double() - ref[mine]).abs()
    assert torch.isfinite(got[mine]).all()
    assert (err <= tol[mine]).all(), float((err / tol[mine].clamp(min=1e-300)).max())
    # and as a whole: the weights' roundings have no relation to one another
    for r in torch.nonzero(mine).flatten().tolist():
        assert (got[r].double() - ref[r]).norm() <= (2.0 ** -8 + 2.0 ** -10) * ref[r].norm(), r


FAR_FORMS = {"one CTA": ([(300, 2), (200, 1), (280, 3)], 128, 64), "cluster": ([(600, 2), (200, 3)], 2, 128),
             "tiles of a group": ([(900, 3), (40, 1)], 64, 64), "second kernel": ([(1700, 2), (31, 1)], 2, 256),
             "chunks": ([(5000, 3), (9, 1), (3000, 16), (1111, 2), (640, 1)], 2, 128)}


@pytest.mark.gpu
@pytest.mark.parametrize("form", FAR_FORMS)
@pytest.mark.parametrize("block", [1, 4, 16, 64])
@pytest.mark.parametrize("order", ["small first", "large first", "in turn", "one large"])
def test_value_scales_far_apart(form, block, order):
    """Weights of values of small scales stay in the sum beside values of scales 2^127 and more times as large, whichever
    comes first, in one group's tiles and in another's, another CTA's or another chunk's."""
    seqs, kv_heads, dim = FAR_FORMS[form]
    for small, large in ((2.0 ** -80, 2.0 ** 47), (2.0 ** -80, 2.0 ** 60), (2.0 ** -40, 2.0 ** 90), (2.0 ** -80, 2.0 ** 124)):
        check_scales_far_apart(scales_far_apart(seqs, kv_heads, dim, block, order, small, large))


@pytest.mark.gpu
@pytest.mark.parametrize("form", FAR_FORMS)
@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("small,large", [(2.0 ** 126, 2.0 ** 126), (2.0 ** 127, 2.0 ** 127), (2.0 ** -80, 2.0 ** 127), (1.0, 2.0 ** 126)])
def test_value_scales_up_to_the_largest(form, block, small, large):
    """Scales whose inverse is below fp32's normal range (codes up to 1/4, so that the outputs are finite)."""
    from paged_cases import to_codes
    seqs, kv_heads, dim = FAR_FORMS[form]
    c = scales_far_apart(seqs, kv_heads, dim, block, "in turn", small, large)
    c.v_cache.copy_(to_codes(values(c.v_cache) / 4).view(c.v_cache.dtype))
    assert torch.isfinite(c.v_scale).all()
    check_scales_far_apart(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("block", [1, 16])
def test_key_scales_up_to_the_largest(dim, block):
    """Keys of zeros with the largest scales beside others: their score is 0 while scale, query and key scale stay within 2^140."""
    c = Call([(300, 3), (1200, 2), (31, 1)], dim=dim, block=block, seed=34)
    c.q.view(c.rows, c.Hq, dim)[:, :, 0] = 2.0 ** 14
    c.scale = 0.5
    c.k_cache[..., 0] = 0
    zero = torch.rand(c.k_scale.shape, generator=c.g, device="cuda") < 0.3
    slots = zero.repeat_interleave(block, 2).transpose(1, 2)  # [page][slot][head]
    c.k_cache[slots] = 0
    c.k_scale[zero] = 2.0 ** 127
    c.check()
