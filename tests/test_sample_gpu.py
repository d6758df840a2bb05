"""Token sampling (w4g128_sample) against its definition in exact arithmetic:
the order is sorted out on the host, the weights are numpy's exp in 64 bits,
and the drawn token has to be the reference's unless u lies within 1e-11 of
the total from a border between two tokens (the weights agree to about 1e-13).
The log-probability is within 4 fp32 roundings of the reference: the ratio,
one minus it, the logarithm (at most 2 ulp by CUDA's documentation)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_g128_gb300 as w  # noqa: E402

NEAR = 1e-11
INF = float("inf")


def reference(z, T, k, p, minp, u):
    """(token, log-probability, is u near a border) of one row of float64 logits."""
    ok = np.flatnonzero(~np.isnan(z) & (z > -INF))
    if ok.size == 0:
        return -1, -INF, False
    order = ok[np.lexsort((ok, -z[ok]))]
    zs = z[order]
    greedy = not T > 0
    if zs[0] == INF:
        e = (zs == INF).astype(np.float64)
    else:
        e = np.exp((zs - zs[0]) / (1.0 if greedy else float(T)))
    n = 1 if greedy else (k if 0 < k < e.size else e.size)
    near = False
    if not greedy and p < 1:
        cum = np.cumsum(e[:n])
        goal = float(p) * cum[-1]
        before = cum - e[:n]
        near |= bool(np.any((np.abs(before[1:] - goal) < NEAR * cum[-1]) & (e[1:n] > NEAR * cum[-1])))
        n = max(1, int(np.sum(before < goal)))
    if not greedy and minp > 0:
        n = max(1, min(n, int(np.sum(e >= minp)))) if minp <= 1 else 1
    cum = np.cumsum(e[:n])
    goal = min(max(float(u), 0.0), 1 - 2.0 ** -53) * cum[-1]
    i = min(int(np.sum(cum <= goal)), n - 1)
    near |= bool(np.min(np.abs(cum[:-1] - goal), initial=INF) < NEAR * cum[-1])
    return int(order[i]), float(np.log(e[i] / cum[-1])), near


def draw(logits, T=None, k=None, p=None, minp=None, u=None, stride=None, offset=0, step=False):
    """Tokens and log-probabilities for a [rows][vocab] float array."""
    rows, V = logits.shape
    stride = stride or V
    buf = torch.full((offset + rows * stride,), 7.0, dtype=torch.bfloat16, device="cuda")  # large: a stray read shows
    view = buf[offset:].as_strided((rows, V), (stride, 1))
    view.copy_(torch.from_numpy(np.asarray(logits, dtype=np.float32)))
    dev = lambda v, t: None if v is None else torch.tensor(np.broadcast_to(v, rows).copy(), dtype=t).cuda()  # noqa: E731
    tokens = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), 7.0, device="cuda")
    args = w.SampleArgs(logits=view, row_stride=stride, temperature=dev(T, torch.float32), top_k=dev(k, torch.int32),
                        top_p=dev(p, torch.float32), min_p=dev(minp, torch.float32), u=dev(u, torch.float32),
                        tokens=tokens, logprobs=lp, rows=rows, vocab=V)
    if step:
        w.SampleStep(args).run()
    else:
        w.w4g128_sample(args)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), lp.cpu().numpy(), view.double().cpu().numpy()


def check(logits, T=None, k=None, p=None, minp=None, u=None, **kw):
    tok, lp, z = draw(logits, T, k, p, minp, u, **kw)
    rows = z.shape[0]
    at = lambda v, d, r: d if v is None else float(np.float32(np.broadcast_to(v, rows)[r]))  # noqa: E731
    nears = 0
    for r in range(rows):
        t, l, near = reference(z[r], at(T, 1.0, r), int(at(k, 0, r)), at(p, 1.0, r), at(minp, 0.0, r), at(u, 0, r))
        nears += near
        if near:
            continue
        assert tok[r] == t, (r, tok[r], t)
        assert lp[r] == l or abs(lp[r] - l) <= 4 * 2.0 ** -23 * abs(l) + 1e-45, (r, lp[r], l)
    assert nears <= max(1, rows // 8), "the inputs say too little"
    return tok, lp


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 64, 65, 1000, 32000, 50261, 131071, 248320, w.MAX_VOCAB])
@pytest.mark.parametrize("filters", [dict(), dict(k=20), dict(p=0.9), dict(minp=0.05), dict(k=200, p=0.7, minp=0.02)],
                         ids=["none", "k", "p", "min", "all"])
def test_against_reference(V, filters):
    rng = np.random.default_rng(V)
    rows = 3 if V > 100000 else 6
    check(rng.normal(0, 3, (rows, V)), T=0.8, u=rng.random(rows), **filters)


@pytest.mark.gpu
@pytest.mark.parametrize("stride,offset", [(1000, 0), (1001, 0), (1003, 5), (1024, 1), (1000, 7)])
def test_strides_and_alignments(stride, offset):
    rng = np.random.default_rng(stride + offset)
    check(rng.normal(0, 2, (5, 1000)), T=1.3, p=0.95, u=rng.random(5), stride=stride, offset=offset, step=True)


@pytest.mark.gpu
def test_rows_have_their_own_settings_and_do_not_meet():
    rng = np.random.default_rng(3)
    rows, V = 37, 4099
    z, u = rng.normal(0, 3, (rows, V)), rng.random(rows)
    T = np.where(np.arange(rows) % 5 == 2, 0.0, 0.5 + 0.1 * np.arange(rows))
    k = np.where(np.arange(rows) % 3 == 1, 0, 1 + 7 * np.arange(rows))
    p = np.where(np.arange(rows) % 4 == 3, 1.0, 0.3 + 0.018 * np.arange(rows))
    m = np.where(np.arange(rows) % 2 == 0, 0.0, 0.01 * np.arange(rows))
    tok, lp = check(z, T, k, p, m, u)
    for r in (0, 17, 36):  # a row alone gives the same bits
        t1, l1, _ = draw(z[r:r + 1], T[r], k[r], p[r], m[r], u[r])
        assert t1[0] == tok[r] and l1.view(np.int32)[0] == lp.view(np.int32)[r]


@pytest.mark.gpu
def test_greedy_takes_the_lowest_index_of_equals():
    z = np.zeros((4, 5003))
    z[0, [4999, 17, 3000]] = 5
    z[1] = -3
    z[2, 5002] = 1
    z[3, ::2] = -0.0  # -0 equals +0
    for T in (0.0, -1.0, float("nan")):
        tok, lp, _ = draw(z, T=T, u=0.9)
        assert tok.tolist() == [17, 0, 5002, 0] and np.all(lp == 0)
    tok, _, _ = draw(z, k=1, u=0.99)
    assert tok.tolist() == [17, 0, 5002, 0]


@pytest.mark.gpu
def test_equal_logits_are_drawn_by_index():
    """All equal: the token is floor(u V), with -0 and +0 mixed; top_p keeps the first ceil(p V), top_k the first k."""
    V = 4096
    z = np.zeros((1, V))
    z[0, 1::3] = -0.0
    for u in (0.0, 0.25, 0.5, 1 - 2.0 ** -24):
        assert draw(z, u=u)[0][0] == int(u * V)
        assert draw(z, u=u, p=0.5)[0][0] == int(u * V / 2)
        assert draw(z, u=u, k=100)[0][0] == int(np.float32(u) * 100)
        tok, lp, _ = draw(z, u=u, k=1024, p=0.25)
        assert tok[0] == int(u * 256) and abs(lp[0] + np.log(256)) <= 4 * 2.0 ** -23 * np.log(256)


@pytest.mark.gpu
def test_borders_of_u_and_of_the_filters():
    rng = np.random.default_rng(11)
    z = rng.normal(0, 1, (1, 777))
    first = int(np.argmax(draw(z, u=0.0)[2][0]))
    for u in (0.0, -3.0, float("nan")):
        assert draw(z, u=u)[0][0] == first
    last = draw(z, u=1.0)[0][0]
    assert last == draw(z, u=1 - 2.0 ** -24)[0][0] or draw(z, u=5.0)[0][0] == last
    for p in (0.0, -1.0, 1e-30):
        assert draw(z, u=0.999, p=p)[0][0] == first
    for p in (1.0, 2.0, float("nan")):
        assert draw(z, u=0.7, p=p)[0][0] == draw(z, u=0.7)[0][0]
    for m in (0.0, -1.0, float("nan")):
        assert draw(z, u=0.7, minp=m)[0][0] == draw(z, u=0.7)[0][0]
    assert draw(z, u=0.999, minp=1.0)[0][0] == first and draw(z, u=0.999, minp=7.0)[0][0] == first
    for k in (0, -5, 777, 10 ** 9):
        assert draw(z, u=0.7, k=k)[0][0] == draw(z, u=0.7)[0][0]


@pytest.mark.gpu
def test_forbidden_tokens_infinities_and_nan():
    rng = np.random.default_rng(5)
    z = rng.normal(0, 3, (6, 3001))
    z[0, rng.random(3001) < 0.7] = -INF
    z[1] = -INF                      # nothing allowed
    z[2] = np.nan
    z[3] = -INF
    z[3, 2900] = -3.3e38             # one allowed, the lowest finite values
    z[4, [5, 1700]] = INF            # +inf shares the mass
    z[5, ::2] = np.nan
    z[5, 0] = -np.nan
    u = np.array([0.5, 0.5, 0.5, 0.5, 0.75, 0.3])
    tok, lp = check(z, T=0.7, u=u)
    assert tok.tolist()[1:5] == [-1, -1, 2900, 1700] and lp[1] == -INF and lp[2] == -INF and lp[3] == 0
    check(z, T=0.7, u=u, k=9, p=0.9, minp=0.01)
    assert draw(z, T=0.0, u=u)[0].tolist()[1:5] == [-1, -1, 2900, 5]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1e-42, 1e-4, 0.02, 30.0, 1e6, 3e38])
def test_temperatures(T):
    rng = np.random.default_rng(8)
    z = rng.normal(0, 2, (8, 2000))
    check(z, T=T, u=rng.random(8), p=0.97)


@pytest.mark.gpu
def test_extreme_logits():
    """Every finite bf16 value once: all 65280 bins, differences past the fp32 range, subnormal values."""
    bits = np.arange(65536, dtype=np.uint32)
    vals = (bits << 16).view(np.float32)
    vals = vals[np.isfinite(vals)].astype(np.float64)
    rng = np.random.default_rng(9)
    z = np.stack([rng.permutation(vals), rng.permutation(np.where(np.abs(vals) < 30, vals, 0))])
    check(z, T=1.0, u=np.array([0.3, 0.9]))
    check(z, T=2.0, u=np.array([0.3, 0.9]), k=1000, p=0.8)


@pytest.mark.gpu
def test_draws_follow_the_distribution():
    """A stratified u hits every token as often as its weight says, to one draw."""
    rows, V = 2048, 40
    z = np.tile(np.random.default_rng(2).normal(0, 1, V), (rows, 1))
    tok, _, zz = draw(z, u=(np.arange(rows) + 0.5) / rows)
    e = np.exp(zz[0] - zz[0].max())
    assert np.all(np.abs(np.bincount(tok, minlength=V) - rows * e / e.sum()) <= 1)


@pytest.mark.gpu
def test_null_filters_streams_and_graph_replay():
    rng = np.random.default_rng(4)
    V = 9000
    logits = torch.from_numpy(rng.normal(0, 3, (2, V)).astype(np.float32)).cuda().bfloat16()
    u = torch.tensor([0.2, 0.8], device="cuda")
    tokens = torch.zeros(2, dtype=torch.int32, device="cuda")
    args = w.SampleArgs(logits=logits, row_stride=V, u=u, tokens=tokens, rows=2, vocab=V)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w.SampleStep(args).run()
    s.synchronize()
    for r in range(2):
        t, _, near = reference(logits[r].double().cpu().numpy(), 1.0, 0, 1.0, 0.0, float(u[r]))
        assert near or tokens[r].item() == t
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.w4g128_sample(args)
    for _ in range(3):
        logits.copy_(torch.from_numpy(rng.normal(0, 3, (2, V)).astype(np.float32)))
        u.copy_(torch.from_numpy(rng.random(2).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        for r in range(2):
            t, _, near = reference(logits[r].double().cpu().numpy(), 1.0, 0, 1.0, 0.0, float(u[r]))
            assert near or tokens[r].item() == t


@pytest.mark.gpu
@pytest.mark.parametrize("rows,V", [(1, 262144), (9, 262144), (16, 262144), (24, 50000), (40, 300000), (300, 777),
                                    (w.MAX_SAMPLE_ROWS, 64)])
def test_many_rows(rows, V):
    """More rows than fit on the GPU at once, and every cluster size."""
    rng = np.random.default_rng(rows)
    z = rng.normal(0, 3, (rows, V)).astype(np.float32)
    few = np.arange(rows) if rows <= 64 else np.array([0, 1, rows // 2, rows - 1])
    u = rng.random(rows)
    tok, lp, zz = draw(z, T=0.9, k=50, p=0.9, u=u)
    for r in few:
        t, l, near = reference(zz[r], float(np.float32(0.9)), 50, float(np.float32(0.9)), 0.0, float(np.float32(u[r])))
        assert near or (tok[r] == t and abs(lp[r] - l) <= 4 * 2.0 ** -23 * abs(l) + 1e-45), r


@pytest.mark.gpu
def test_the_cluster_size_changes_no_bit():
    """The same row alone, among 9, 16 and 30: 16, 8, 6 and 4 CTAs."""
    rng = np.random.default_rng(21)
    z = rng.normal(0, 3, (30, 100000))
    u = rng.random(30)
    t30, l30, _ = draw(z, T=1.1, p=0.97, u=u)
    for n in (1, 9, 16):
        t, l, _ = draw(z[:n], T=1.1, p=0.97, u=u[:n])
        assert np.array_equal(t, t30[:n]) and np.array_equal(l.view(np.int32), l30[:n].view(np.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("filters", [dict(), dict(k=3), dict(p=0.8), dict(minp=0.2)], ids=["none", "k", "p", "min"])
def test_u_of_1_and_above_draws_the_last_kept_token(filters):
    """Four tokens of real weight each: the fraction just below 1 falls into the last one that the filters keep."""
    z = np.full((5, 501), -INF)
    z[:, [77, 3, 402, 500]] = [1.0, 0.5, 0.0, -0.5]
    tok, _ = check(z, u=[1.0, 5.0, 1e30, INF, 1 - 2.0 ** -24], **filters)
    assert len(set(tok.tolist())) == 1
    assert tok[0] == {"k": 402, "p": 402, "minp": 500}.get(next(iter(filters), ""), 500)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1.0 + 2.0 ** -23, 7.0, 1e20, 1e31, 1e36, 1e38, 3e38, INF])
def test_logits_over_the_whole_range_at_high_temperatures(T):
    """Differences of logits up to twice the largest float, and temperatures whose reciprocal is subnormal: a quotient
    of the two is an ordinary number."""
    vals = (np.arange(65536, dtype=np.uint32) << 16).view(np.float32)
    vals = vals[np.isfinite(vals)].astype(np.float64)
    rng = np.random.default_rng(10)
    z = np.stack([rng.permutation(vals) for _ in range(8)])
    z[4:] = np.where(np.abs(z[4:]) > 2.0 ** 100, z[4:], -INF)  # mass on the large ones alone
    check(z, T=T, u=rng.random(8))
    check(z, T=T, u=rng.random(8), p=0.7)
