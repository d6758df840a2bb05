"""Attention of new tokens over a paged cache (w4g128_attend) against the
definition in 64 bits, computed sequence by sequence from dense keys and values.

The bound, per element, with A = sum_j softmax_j |v_j| (64 bits): the softmax
weights are rounded to bf16 (2^-8 relative each) and normalised by their
rounded sum, so that error is at most 2^-8 (A + |out|); a score's fp32 sum of
D products is off by (D + 4) 2^-24 scale sum|q k|, which moves a weight by
that much relative, numerator and denominator; exp2 adds 2^-22, the fp32 sums
over L positions at most (L + 64) 2^-24 each; the output rounds once, 2^-8."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_g128_gb300 as w  # noqa: E402


class Call:
    """One set of inputs: ragged sequences over shuffled pages.  seqs: [(length with the new tokens, new tokens)]."""

    def __init__(self, seqs, q_heads=4, kv_heads=2, dim=64, page=16, window=0, sinks=0, max_len=None, max_new=None,
                 head_major=False, pad=0, extra_rows=1, fused=True, seed=0, spare=2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.seqs, self.Hq, self.Hkv, self.D, self.page = seqs, q_heads, kv_heads, dim, page
        self.window, self.sinks, self.fused = window, sinks, fused
        self.max_len = max_len or max(1, max(n for n, _ in seqs))
        self.max_new = max_new or max(1, max(n for _, n in seqs))
        self.rows = sum(n for _, n in seqs) + extra_rows
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.q = rnd(self.rows, q_heads * dim + pad)[:, :q_heads * dim]
        self.k_new = rnd(self.rows, kv_heads * dim + pad)[:, :kv_heads * dim]
        self.v_new = rnd(self.rows, kv_heads * dim + pad)[:, :kv_heads * dim]
        used = [-(-n // page) for n, _ in seqs]
        self.pages = sum(used) + spare
        shape = (self.pages, kv_heads, page, dim) if head_major else (self.pages, page, kv_heads, dim)
        k, v = rnd(*shape), rnd(*shape)
        self.k_cache, self.v_cache = (t.transpose(1, 2) if head_major else t for t in (k, v))  # [page][slot][head][dim]
        width = -(-self.max_len // page)
        order = torch.randperm(self.pages, generator=g, device="cuda").int()
        self.table = torch.full((len(seqs), width + 1), -12345, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.offsets = np.concatenate(([0], np.cumsum([n for _, n in seqs]))).astype(int)
        self.offsets_d = torch.tensor(self.offsets, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor([n for n, _ in seqs], dtype=torch.int32, device="cuda")
        self.out = torch.full((self.rows, q_heads * dim + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        self.scale = dim ** -0.5

    def args(self, **kw):
        k = self.k_cache
        a = dict(q=self.q, k_new=self.k_new if self.fused else None, v_new=self.v_new if self.fused else None,
                 k_cache=k, v_cache=self.v_cache, page_table=self.table, row_offsets=self.offsets_d, lens=self.lens,
                 out=self.out, q_row=self.q.stride(0), kv_row=self.k_new.stride(0), out_row=self.out.stride(0),
                 page_stride=k.stride(0), slot_stride=k.stride(1), head_stride=k.stride(2),
                 table_row=self.table.stride(0), rows=self.rows, count=len(self.seqs), q_heads=self.Hq,
                 kv_heads=self.Hkv, head_dim=self.D, pages=self.pages, page_size=self.page, max_len=self.max_len,
                 max_new=self.max_new, window=self.window, sinks=self.sinks, scale=self.scale)
        a.update(kw)
        return w.AttendArgs(**a)

    def run(self, status=0, **kw):
        args = self.args(**kw)
        nb = w.w4g128_attend_workspace_bytes(args)
        assert nb > 0
        ws = torch.full((nb,), 0x5A, dtype=torch.uint8, device="cuda")
        w.w4g128_attend(args, ws)
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws) == status
        return self.out[:, :self.Hq * self.D].reshape(self.rows, self.Hq, self.D)

    def dense(self, b):
        """(k, v) [length][head][dim] of sequence b, its new rows in place."""
        n, new = self.seqs[b]
        pos = torch.arange(n, device="cuda")
        ids = self.table[b, pos // self.page].long()
        both = []
        for cache, fresh in ((self.k_cache, self.k_new), (self.v_cache, self.v_new)):
            d = cache[ids, pos % self.page].clone()
            if self.fused and new and n:
                real = min(n, new)
                rows = fresh[self.offsets[b] + new - real:self.offsets[b] + new]
                d[n - real:] = rows.reshape(real, self.Hkv, self.D)
            both.append(d)
        return both

    def reference(self):
        """out and its bound, [rows][head][dim] in 64 bits; rows of no sequence: NaN."""
        out = torch.full((self.rows, self.Hq, self.D), float("nan"), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        G = self.Hq // self.Hkv
        for b, (n, new) in enumerate(self.seqs):
            k, v = (t.double() for t in self.dense(b))
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
                e = 2 * (self.D + 4) * 2.0 ** -24 * s + 2.0 ** -21 + 2 * (pos.numel() + 64) * 2.0 ** -24
                out[r] = o.reshape(self.Hq, self.D)
                tol[r] = (2.0 ** -8 * o.abs() + (A + o.abs()) * (2.0 ** -8 + e) * 1.02).reshape(self.Hq, self.D)
        return out, tol

    def check(self, **kw):
        ref, tol = self.reference()
        caches = [(c.clone(), [d.clone() for d in ds]) for c, ds in
                  ((self.k_cache, [self.dense(b)[0] for b in range(len(self.seqs))]),
                   (self.v_cache, [self.dense(b)[1] for b in range(len(self.seqs))]))]
        rest = self.out.clone()
        got = self.run(**kw)
        mine = ~torch.isnan(ref[:, 0, 0])
        err = (got[mine].double() - ref[mine]).abs()
        assert torch.isfinite(got[mine]).all()
        assert (err <= tol[mine]).all(), float((err / tol[mine].clamp(min=1e-30)).max())
        # rows of no sequence and the padding stay
        assert torch.equal(got[~mine], rest[:, :self.Hq * self.D].reshape(got.shape)[~mine])
        assert torch.equal(self.out[:, self.Hq * self.D:], rest[:, self.Hq * self.D:])
        # the caches hold the new rows at their places, and nothing else has changed
        for cache, (before, dense) in zip((self.k_cache, self.v_cache), caches):
            want = before
            for b, (n, new) in enumerate(self.seqs):
                for pos in range(max(0, n - new), n):
                    want[self.table[b, pos // self.page].long(), pos % self.page] = dense[b][pos]
            assert torch.equal(cache, want)
        return got


LENGTHS = [(1, 1), (2, 2), (15, 3), (16, 1), (17, 5), (31, 16), (63, 1), (64, 4), (65, 2), (80, 16), (129, 7), (300, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 4), (1, 16), (3, 5)])
def test_lengths(dim, kv_heads, group):
    Call(LENGTHS, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, seed=dim + group).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,n,new,page", [(64, 5003, 16, 16), (128, 9001, 8, 64), (256, 4097, 3, 48), (128, 70001, 1, 256),
                                            (64, 300011, 2, 64)])
def test_long(dim, n, new, page):
    Call([(n, new)], q_heads=8, kv_heads=2, dim=dim, page=page, seed=n).check()


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (64, 4), (100, 70), (5000, 4), (1 << 30, 9)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows_and_sinks(window, sinks, dim):
    Call(LENGTHS + [(2000, 9), (1999, 16)], dim=dim, window=window, sinks=sinks, seed=window % 1000 + sinks,
         page=32).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(head_major=True), dict(pad=8), dict(page=48, pad=64, head_major=True),
                                dict(fused=False), dict(max_len=5000), dict(page=1024)])
def test_layouts(kw):
    Call([(333, 4), (20, 1), (1, 1), (150, 16)], q_heads=12, kv_heads=2, dim=128, seed=3, **kw).check()


@pytest.mark.gpu
def test_rows_that_see_nothing():
    """Empty sequences, sequences without new tokens, more rows than the length: zeros, and no write to the cache."""
    for max_len in (16, 1000):
        c = Call([(0, 0), (0, 3), (2, 5), (40 if max_len > 16 else 9, 0), (7, 7), (0, 16)], max_len=max_len, seed=1)
        got = c.check()
        assert torch.equal(got[0:3], torch.zeros_like(got[0:3])) and torch.equal(got[3:6], torch.zeros_like(got[3:6]))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,window,sinks", [(64, 0, 0), (128, 0, 0), (256, 0, 0), (128, 200, 5), (64, 37, 40)])
def test_a_row_alone_gives_the_same_bits(dim, window, sinks):
    """Each new token of a verify step, decoded alone with the cache as it stood then, gives its row's bits."""
    seqs = [(1500, 16), (77, 5), (16, 16), (900, 1)]
    kw = dict(q_heads=6, kv_heads=2, dim=dim, window=window, sinks=sinks, max_len=1600)
    c = Call(seqs, seed=5, **kw)
    together = c.run().clone()
    for b, (n, new) in enumerate(seqs):
        for i in (0, new // 2, new - 1):
            one = Call([(n - new + i + 1, 1), (0, 0), (0, 0), (0, 0)], seed=5, **kw)
            one.k_cache, one.v_cache, one.pages = c.k_cache, c.v_cache, c.pages
            one.table = c.table[b:b + 1].repeat(4, 1)
            r = c.offsets[b] + i
            one.q[0], one.k_new[0], one.v_new[0] = c.q[r], c.k_new[r], c.v_new[r]
            assert torch.equal(one.run()[0], together[r]), (b, i)
    assert torch.equal(c.run(), together)  # and again: deterministic


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 48), (256, 64)])
@pytest.mark.parametrize("seqs", [[(4099, 9)], [(4097, 3), (130, 16), (0, 2), (2600, 1)],
                                  [(5000 - 301 * b, (5 * b + 2) % 17) for b in range(16)]], ids=["1", "4", "16"])
def test_many_chunks(seqs, dim, page):
    """Lengths on both sides of 2048 and more chunks than are joined at once, for one sequence, a few and many."""
    kw = dict(q_heads=6, kv_heads=2, dim=dim, page=page, max_len=5040)
    c = Call(seqs, seed=9, **kw)
    together = c.check().clone()
    for b, (n, new) in enumerate(seqs[:4]):
        for i in range(0, new, 4):
            one = Call([(n - new + i + 1, 1)] + [(0, 0)] * (len(seqs) - 1), seed=9, **kw) if n >= new else None
            if one is None:
                continue
            one.k_cache, one.v_cache, one.pages = c.k_cache, c.v_cache, c.pages
            one.table = c.table[b:b + 1].repeat(len(seqs), 1)
            r = c.offsets[b] + i
            one.q[0], one.k_new[0], one.v_new[0] = c.q[r], c.k_new[r], c.v_new[r]
            assert torch.equal(one.run()[0], together[r]), (b, i)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_masked_values_take_no_part(dim, bad):
    """Non-finite keys and values behind a row's own position, before its window, in unused slots and in unseen
    pages; the page ids of unseen pages are out of range."""
    c = Call([(203, 8), (50, 8)], dim=dim, window=40, sinks=3, page=16, max_len=256, seed=7)
    clean = c.check().clone()
    for t in (c.k_new, c.v_new):
        t[5] = bad                     # rows 0..4 of sequence 0 do not see it
    pos = torch.arange(3, 203 - 8 - 39, device="cuda")  # before the first row's window
    for cache in (c.k_cache, c.v_cache):
        cache[c.table[0, pos // 16].long(), pos % 16] = bad
        cache[c.table[0, 12].long(), 203 - 192:] = bad  # slots behind the end
    c.table[0, 1:9] = 10 ** 9          # whole pages that nobody sees
    got = c.run()
    assert torch.equal(got[:5], clean[:5]) and torch.equal(got[8:], clean[8:])
    assert torch.isnan(got[5:8]).any() or not torch.isfinite(got[5:8]).all()


@pytest.mark.gpu
def test_window_edges_inside_a_tile_with_non_finite_values():
    """A value that the first rows still see and the last rows do not."""
    c = Call([(90, 16)], window=30, page=16, max_len=96, seed=9)
    clean = c.run().clone()
    pos = 90 - 16 - 30 + 8  # seen by rows 0..7
    c.v_cache[c.table[0, pos // 16].long(), pos % 16] = float("inf")
    got = c.run()
    assert torch.equal(got[8:], clean[8:])
    assert torch.isinf(got[:8]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,new", [(64, 3), (64, 16), (128, 1), (128, 16), (256, 16)])
@pytest.mark.parametrize("scores", [lambda p: p / 32, lambda p: p / 2, lambda p: -p / 4, lambda p: 5.5 * (p // 16),
                                    lambda p: 5.0 * (p // 64 % 2), lambda p: 300.0 * (p == 390), lambda p: -1e4 + p / 8],
                         ids=["slow", "fast", "falling", "steps", "to and fro", "a peak", "far below zero"])
def test_scores_that_move_the_maximum(dim, new, scores):
    """Scores rising by less, and by more, than the factor that the kernel lets a row's weights grow to."""
    c = Call([(401, new), (64, new)], q_heads=8, kv_heads=2, dim=dim, fused=False, seed=new)
    c.scale = 1.0
    c.q[:] = 0
    c.q.view(c.rows, 8, dim)[:, :, 0] = torch.tensor([1.0, 0.5, 1.0, 2.0] * 2, device="cuda").bfloat16()
    for b, (n, _) in enumerate(c.seqs):
        pos = torch.arange(n, device="cuda")
        c.k_cache[c.table[b, pos // c.page].long(), pos % c.page, :, 0] = scores(pos.double())[:, None].bfloat16()
    c.check()


@pytest.mark.gpu
def test_equal_values_come_through_exactly():
    """The weights add up to 1 as rounded: equal values give that value."""
    c = Call([(1000, 3)], dim=128, seed=2)
    c.v_cache.fill_(1.5)
    c.v_new.fill_(1.5)
    got = c.run()[:3]
    assert (got == 1.5).all()


@pytest.mark.gpu
def test_values_out_of_range_are_reported_and_left_out():
    c = Call([(100, 2), (60, 2), (80, 2)], max_len=112, seed=4)
    clean = c.run().clone()
    kc, vc = c.k_cache.clone(), c.v_cache.clone()

    def again(status=w.ERR_CACHE, **kw):
        c.out.fill_(7.0)
        return c.run(status=status, **kw)

    for wrong in (-1, 113, 2 ** 31 - 1, -2 ** 31):
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
    assert torch.equal(c.k_cache, kc) and torch.equal(c.v_cache, vc)
    for wrong in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        keep = c.table[1, 2].item()
        c.table[1, 2] = wrong              # positions 32..47 of sequence 1
        got = again()
        assert torch.equal(got[:2], clean[:2]) and torch.equal(got[4:6], clean[4:6])
        assert torch.isfinite(got[2:4]).all() and not torch.equal(got[2:4], clean[2:4])
        c.table[1, 2] = keep
        keep = c.table[1, 3].item()
        c.table[1, 3] = wrong              # the page of the new rows: not written
        again()
        c.table[1, 3] = keep
        assert torch.equal(c.k_cache, kc) and torch.equal(c.v_cache, vc)
    assert torch.equal(again(status=0), clean)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Pages whose elements start beyond 2^31 (and bytes beyond 2^32)."""
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (H * D * page) + 40
    c = Call([(200, 3)], q_heads=16, kv_heads=H, dim=D, page=page, seed=6)
    small = c.run().clone()
    big = []
    for cache in (c.k_cache, c.v_cache):
        t = torch.empty((pages, page, H, D), dtype=torch.bfloat16, device="cuda")
        t[pages - c.pages:] = cache
        big.append(t)
    c.k_cache, c.v_cache = big
    c.table[0, :4] += pages - c.pages
    c.pages = pages
    c.k_cache[c.table[0, 3].long(), 5:] = 0
    c.v_cache[c.table[0, 3].long(), 5:] = 0
    assert torch.equal(c.run(), small)
    c.fused = False
    assert torch.equal(c.run(), small)


@pytest.mark.gpu
def test_streams_and_graph_replay_follow_the_lengths():
    c = Call([(500, 2), (300, 1)], q_heads=8, kv_heads=2, dim=128, max_len=512, seed=8)
    want = c.run().clone()
    args = c.args()
    ws = torch.empty(w.w4g128_attend_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.out.fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        w.AttendStep(args, ws).run()
    s.synchronize()
    assert torch.equal(c.out.view(c.rows, c.Hq, c.D), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.w4g128_attend(args, ws)
    for seqs in ([(500, 2), (300, 1)], [(130, 2), (299, 1)], [(2, 2), (1, 1)], [(497, 2), (64, 1)]):
        c.seqs = seqs
        c.lens.copy_(torch.tensor([n for n, _ in seqs], dtype=torch.int32))
        ref, tol = c.reference()
        g.replay()
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws) == 0
        got = c.out.view(c.rows, c.Hq, c.D)[:3].double()
        assert ((got - ref[:3]).abs() <= tol[:3]).all()


@pytest.mark.gpu
def test_workspace_is_not_exceeded():
    c = Call([(1000, 16), (40, 3)], q_heads=8, kv_heads=2, dim=64, window=100, sinks=5, max_len=2000, seed=1)
    args = c.args()
    nb = w.w4g128_attend_workspace_bytes(args)
    whole = torch.full((nb + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    w.w4g128_attend(args, whole[4096:], ws_bytes=nb)
    torch.cuda.synchronize()
    assert (whole[:4096] == 0x5A).all() and (whole[4096 + nb:] == 0x5A).all()


@pytest.mark.gpu
def test_status_of_replayed_calls():
    """A replay with a length out of range reports it, the next good one does not."""
    c = Call([(100, 2), (60, 1)], max_len=112, seed=11)
    want = c.run().clone()
    args = c.args()
    ws = torch.empty(w.w4g128_attend_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.w4g128_attend(args, ws)
    for length, status in ((60, 0), (500, w.ERR_CACHE), (60, 0), (-1, w.ERR_CACHE), (60, 0)):
        c.lens[1] = length
        g.replay()
        torch.cuda.synchronize()
        assert w.w4g128_workspace_status(ws) == status, length
    assert torch.equal(c.out.view(c.rows, c.Hq, c.D), want)


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
        steps.append(w.AttendStep(a, torch.empty(w.w4g128_attend_workspace_bytes(a), dtype=torch.uint8, device="cuda"),
                                  stream=s))
    torch.cuda.synchronize()
    for _ in range(10):
        for st in steps:
            st.run()
    torch.cuda.synchronize()
    for c, o in zip(calls, want):
        assert torch.equal(c.out.view(c.rows, c.Hq, c.D)[:8], o[:8])


@pytest.mark.gpu
def test_pages_shared_by_sequences():
    """Two sequences with a common prefix in the same pages, each with new tokens of its own."""
    c = Call([(70, 3), (68, 1)], page=16, seed=15)
    c.table[1, :4] = c.table[0, :4]  # positions 0..63; both sequences' new tokens lie behind
    c.check()


@pytest.mark.gpu
def test_errors_of_calls_of_one_chunk():
    """Short caches take a single kernel, which reports by itself."""
    c = Call([(40, 2), (30, 1), (0, 0)], max_len=48, seed=16)
    clean = c.check().clone()
    for field, at, wrong in ((c.lens, 1, 49), (c.lens, 1, -7), (c.table, (1, 0), c.pages), (c.table, (1, 1), -1),
                             (c.offsets_d, 2, 1)):
        keep = field[at].item()
        field[at] = wrong
        got = c.run(status=w.ERR_CACHE)
        assert torch.equal(got[:2], clean[:2])
        field[at] = keep
    c.table[1, 2] = -9  # behind the length: not seen
    assert torch.equal(c.run(), clean)


@pytest.mark.gpu
def test_an_error_stays_with_its_call():
    """One workspace for calls of one chunk and of several, in turn: each reports its own errors alone."""
    short = Call([(40, 2), (30, 1)], max_len=48, seed=17)
    split = Call([(700, 2), (300, 1)], max_len=1024, seed=18)
    nb = [w.w4g128_attend_workspace_bytes(c.args()) for c in (short, split)]
    assert nb[0] < nb[1]  # the short one keeps no sums of chunks
    ws = torch.full((nb[1],), 0x5A, dtype=torch.uint8, device="cuda")
    good = [c.run().clone() for c in (short, split)]

    def call(c, field=None, at=None, wrong=None):
        keep = field[at].item() if field is not None else None
        if field is not None:
            field[at] = wrong
        w.w4g128_attend(c.args(), ws)
        torch.cuda.synchronize()
        if field is not None:
            field[at] = keep
        return w.w4g128_workspace_status(ws)

    for c, other in ((short, split), (split, short)):
        for wrong in ((c.lens, 1, c.max_len + 1), (c.lens, 0, -1), (c.offsets_d, 2, 1), (c.table, (0, 1), c.pages)):
            assert call(c, *wrong) == w.ERR_CACHE
            assert call(other) == 0 and call(c) == 0
            assert call(c, *wrong) == w.ERR_CACHE
            assert call(c) == 0 and call(other) == 0
    for c, want in zip((short, split), good):
        assert torch.equal(c.out.view(c.rows, c.Hq, c.D), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,n,new,page", [(64, 5003, 16, 16), (256, 4097, 3, 48), (128, 70001, 1, 256), (64, 300011, 2, 64),
                                            (256, 131072, 1, 32)])
def test_long_norm_of_the_error(dim, n, new, page):
    """Over many positions the element bounds exceed the output, which is a mean of independent values.  The norm of a
    row's error: the output's rounding, 2^-8 of each element; the weights' roundings, at most 2^-8 each and without
    relation to the values, so that they weigh against the output as the weights themselves do: 2^-8.  The fp32 sums
    are thousands of times below.  A chunk or a tile left out shows: 1 / 150 of the positions changes 8%."""
    c = Call([(n, new)], q_heads=8, kv_heads=2, dim=dim, page=page, seed=n + 1)
    ref, _ = c.reference()
    got = c.run()
    ref, got = ref[:new].flatten(1), got[:new].double().flatten(1)
    assert ((got - ref).norm(dim=1) <= 2.0 ** -7 * ref.norm(dim=1)).all()
