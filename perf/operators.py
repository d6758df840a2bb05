"""Cases of the decode-step operators: the mixture-of-experts layer on packed
int4-g128 experts, attention of a few new tokens over a paged cache, and token
sampling.  For each case: its inputs, the operator in plain torch (`own` false)
or through the library (`own` true), its value in 64 bits, and the bytes and
operations it cannot do without.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 1088  # bytes of one packed (16 columns, 128 rows) block: 1024 of codes, 64 of scales and minima


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # one token through a small layer: the call whose launch and latency count most
        _moe("moe one token small experts", M=1, D=2048, F=768, E=64, k=4, renorm=True, residual=False),
        # one token through a layer of the size of the dense projections elsewhere in this repository
        _moe("moe one token", M=1, D=5120, F=1408, E=64, k=8, renorm=True, residual=True),
        # a 6-token draft and its base, weights of the whole softmax, odd counts of everything
        _moe("moe verify 7 odd sizes", M=7, D=2176, F=896, E=37, k=3, renorm=False, residual=False),
        # the longest verify step: 16 rows that together reach most experts
        _moe("moe verify 16", M=16, D=5120, F=1408, E=96, k=6, renorm=True, residual=True),
        # plain decode of one short sequence: latency
        _attn("attention one token short", count=1, new=1, length=611, q_heads=32, kv_heads=8, dim=128, page=16),
        # the verify step of a 7-token draft far into one sequence
        _attn("attention verify 8 long", count=1, new=8, length=32771, q_heads=32, kv_heads=8, dim=128, page=64),
        # sixteen sequences of all lengths, some with no new token this step
        _attn("attention ragged batch", count=16, new=3, length=9001, q_heads=24, kv_heads=4, dim=64, page=16,
              ragged=True),
        # a sliding window with a few first tokens that stay visible, wide heads, longest draft
        _attn("attention window and sinks", count=2, new=16, length=100003, q_heads=16, kv_heads=4, dim=256, page=32,
              window=4096, sinks=4),
        # one row, a small vocabulary, the usual filters: latency
        _sample("sample one row small", rows=1, vocab=32000, k=50, p=0.9, minp=0.0),
        # one row of the full vocabulary, nucleus alone: the whole distribution counts
        _sample("sample one row nucleus", rows=1, vocab=248320, k=0, p=0.95, minp=0.0),
        # every row of a long verify step with settings of its own
        _sample("sample 16 rows mixed", rows=16, vocab=248320, k=200, p=0.9, minp=0.02, mixed=True),
        # an odd vocabulary with tokens that a grammar forbids, flat temperature
        _sample("sample 7 rows masked", rows=7, vocab=50261, k=0, p=1.0, minp=0.05, masked=True),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    kind = rng.choice(("moe", "attn", "sample"))
    if kind == "moe":
        E = rng.randint(8, 96)
        return _moe(None, M=rng.choice((1, 1, 2, 4, 7, 8, 13, 16)), D=128 * rng.randint(4, 40), F=128 * rng.randint(2, 11), E=E,
                    k=rng.randint(1, min(6, E)), renorm=rng.random() < 0.5, residual=rng.random() < 0.5)
    if kind == "attn":
        kv = rng.choice((1, 2, 4, 8))
        count = rng.choice((1, 1, 2, 3, 7, 16))
        dim = rng.choice((64, 128, 128, 256))
        new, group = rng.choice((1, 1, 2, 5, 8, 16)), rng.choice((1, 2, 4, 6, 8))
        while new * group * kv > 512:
            group //= 2
        cap = min(120000 // count, 25600000 // (count * kv * dim))
        window = rng.choice((0, 0, log(64, 8192)))
        return _attn(None, count=count, new=new, length=log(17, cap),
                     q_heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice((16, 32, 64)),
                     window=window, sinks=rng.choice((0, 4, 16)) if window else 0, ragged=rng.random() < 0.5)
    return _sample(None, rows=rng.randint(1, 16), vocab=log(1000, 248320), k=rng.choice((0, 1, 20, 50, 200)),
                   p=rng.choice((1.0, 0.95, 0.9, 0.5)), minp=rng.choice((0.0, 0.02, 0.1)), mixed=rng.random() < 0.5,
                   masked=rng.random() < 0.3)


def _named(name, case):
    return {**({"name": name} if name else {}), **case}


def _moe(name, M, D, F, E, k, renorm, residual):
    return _named(name, dict(op="moe", M=M, D=D, F=F, E=E, k=k, renorm=renorm, residual=residual))


def _attn(name, count, new, length, q_heads, kv_heads, dim, page, window=0, sinks=0, ragged=False):
    return _named(name, dict(op="attn", count=count, new=new, length=length, q_heads=q_heads, kv_heads=kv_heads,
                             dim=dim, page=page, window=window, sinks=sinks, ragged=ragged))


def _sample(name, rows, vocab, k, p, minp, mixed=False, masked=False):
    return _named(name, dict(op="sample", rows=rows, vocab=vocab, k=k, p=p, minp=minp, mixed=mixed, masked=masked))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"moe": _prepare_moe, "attn": _prepare_attn, "sample": _prepare_sample}[case["op"]](case, g)


def run(state):
    if own:
        return _own(state)
    return {"moe": _plain_moe, "attn": _plain_attn, "sample": _plain_sample}[state["op"]](state)


def work(case):
    return {"moe": _work_moe, "attn": _work_attn, "sample": _work_sample}[case["op"]](case)


def exact(case, seed):
    return {"moe": _exact_moe, "attn": _exact_attn, "sample": _exact_sample}[case["op"]](prepare(case, seed))


def _own(s):
    import int4_weight_only_g128_gb300 as w
    step = s.get("step")
    if step is None:  # a program marshals a step's buffers once and keeps its workspace
        if s["op"] == "moe":
            args = w.MoEArgs(x=s["x"], residual=s["residual"], y=s["y"], router=s["router"], gate_up=s["gate_up"],
                             down=s["down"], M=s["M"], D=s["D"], F=s["F"], E=s["E"], top_k=s["k"],
                             renormalize=s["renorm"])
            step = w.MoEStep(args, _workspace(w.w4g128_moe_workspace_bytes(args)))
        elif s["op"] == "attn":
            k = s["k_cache"]
            args = w.AttendArgs(q=s["q"], k_new=s["k_new"], v_new=s["v_new"], k_cache=k, v_cache=s["v_cache"],
                                page_table=s["table"], row_offsets=s["row_offsets"], lens=s["lens"], out=s["out"],
                                q_row=s["q"].stride(0), kv_row=s["k_new"].stride(0), out_row=s["out"].stride(0),
                                page_stride=k.stride(0), slot_stride=k.stride(1), head_stride=k.stride(2),
                                table_row=s["table"].stride(0), rows=s["q"].shape[0], count=s["lens"].numel(),
                                q_heads=s["q"].shape[1], kv_heads=k.shape[2], head_dim=k.shape[3], pages=k.shape[0],
                                page_size=k.shape[1], max_len=s["max_len"], max_new=s["max_new"],
                                window=s["window"], sinks=s["sinks"], scale=s["scale"])
            step = w.AttendStep(args, _workspace(w.w4g128_attend_workspace_bytes(args)))
        else:
            args = w.SampleArgs(logits=s["logits"], row_stride=s["logits"].stride(0), temperature=s["temperature"],
                                top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], u=s["u"], tokens=s["tokens"],
                                logprobs=s["logprobs"], rows=s["logits"].shape[0], vocab=s["logits"].shape[1])
            step = w.SampleStep(args)
        s["step"] = step
    step.run()
    if s["op"] == "moe":
        return {"y": s["y"]}
    if s["op"] == "attn":
        return {"out": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


def _workspace(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device=DEV)


# ------------------------------------------------ mixture of experts (int4-g128)

def _packed(E, K, N, g):
    """E packed K x N matrices: codes uniform, scales U(0.002, 0.02), minima -8 scale (1 + U(-0.1, 0.1)).  The order
    of uniform codes in a block says nothing, so they are drawn in the packed layout itself: [expert][quad][group]
    [tile of the quad] blocks of 1088 bytes."""
    Q, G, last = -(-N // 64), K // 128, (N // 16 - 1) % 4 + 1
    assert last == 4, "whole quads"
    out = torch.empty((E, Q, G, 4, BLOCK), dtype=torch.uint8, device=DEV)
    codes = torch.randint(-2**31, 2**31 - 1, (E, Q, G, 4, 256), dtype=torch.int32, device=DEV, generator=g)
    out[..., :1024] = codes.view(torch.uint8)
    scale = (torch.rand((E, Q, G, 4, 8, 2), device=DEV, generator=g) * 0.018 + 0.002).bfloat16()
    low = -8 * scale.float() * (1 + (torch.rand(scale.shape, device=DEV, generator=g) * 0.2 - 0.1))
    out[..., 1024:] = torch.stack((scale, low.bfloat16()), -1).view(torch.uint8).flatten(-3)
    return out.view(E, -1)


def _prepare_moe(c, g):
    M, D, F, E = c["M"], c["D"], c["F"], c["E"]
    normal = lambda *n: torch.randn(n, device=DEV, generator=g)  # noqa: E731
    return dict(op="moe", M=M, D=D, F=F, E=E, k=c["k"], renorm=c["renorm"], x=normal(M, D).bfloat16(),
                residual=normal(M, D).bfloat16() if c["residual"] else None,
                router=(normal(E, D) / math.sqrt(D)).bfloat16(), gate_up=_packed(E, D, 2 * F, g),
                down=_packed(E, F, D, g), y=torch.zeros((M, D), dtype=torch.bfloat16, device=DEV))


def _dequantised(packed, K, N):
    """[S][bytes] packed -> [S][K][N] in 32 bits: w = min + code scale."""
    S = packed.shape[0]
    b = packed.view(S, N // 64, K // 128, 4, BLOCK)
    words = b[..., :1024].contiguous().view(torch.int32).view(S, N // 64, K // 128, 4, 2, 8, 4, 4)  # h, r, c, j
    shift = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    q = ((words[..., None] >> shift) & 15).view(S, N // 64, K // 128, 4, 2, 8, 4, 4, 2, 2, 2)  # b, a, e
    # k = 64 h + 16 j + 8 a + 2 c + b, n = 64 quad + 16 tile + 8 e + r
    q = q.permute(0, 2, 4, 7, 9, 6, 8, 1, 3, 10, 5).float().reshape(S, K // 128, 128, N)
    meta = b[..., 1024:].contiguous().view(torch.bfloat16).view(S, N // 64, K // 128, 4, 8, 2, 2)
    meta = meta.permute(0, 2, 1, 3, 5, 4, 6).float().reshape(S, K // 128, 1, N, 2)
    return (meta[..., 1] + q * meta[..., 0]).reshape(S, K, N)


def _plain_moe(s):
    M, D, F, k = s["M"], s["D"], s["F"], s["k"]
    x = s["x"].float()
    logits = (x[:, None, :] * s["router"].float()[None]).sum(-1)
    # the k largest, the lower expert first among equals
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    e = torch.exp(logits - logits.max(-1, keepdim=True).values)
    p = torch.gather(e / e.sum(-1, keepdim=True), 1, order)
    if s["renorm"]:
        p = p / p.sum(-1, keepdim=True)
    pick = order.reshape(-1)
    gu = torch.matmul(x.repeat_interleave(k, 0)[:, None], _dequantised(s["gate_up"][pick], D, 2 * F))[:, 0]
    act = gu[:, :F] / (1 + torch.exp(-gu[:, :F])) * gu[:, F:]
    y = torch.matmul(act[:, None], _dequantised(s["down"][pick], F, D))[:, 0].view(M, k, D)
    y = (y * p[..., None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": s["y"].copy_(y)}


def _matrix64(packed, K, N):
    """One packed matrix -> [K][N] in 64 bits, each code found by its place in the documented layout."""
    k = torch.arange(K, device=DEV)[:, None]
    n = torch.arange(N, device=DEV)[None, :]
    base = ((n // 64) * (K // 128) + k // 128) * (4 * BLOCK) + (n // 16 % 4) * BLOCK
    kk, nn = k % 128, n % 16
    lane = (nn % 8) * 4 + kk % 8 // 2
    word = base + kk // 64 * 512 + lane * 16 + kk // 16 % 4 * 4
    nibble = 4 * (kk % 2) + 2 * (kk // 8 % 2) + nn // 8
    code = (packed[word + nibble // 2].to(torch.int64) >> (nibble % 2 * 4)) & 15
    entry = base + 1024 + nn % 8 * 8 + nn // 8 * 4

    def bf16_at(at):
        bits = packed[at].to(torch.int32) | packed[at + 1].to(torch.int32) << 8
        return (bits << 16).view(torch.float32).double()
    return bf16_at(entry + 2) + code.double() * bf16_at(entry)


def _exact_moe(s):
    M, D, F, k = s["M"], s["D"], s["F"], s["k"]
    x = s["x"].double()
    logits = x @ s["router"].double().T
    y = torch.zeros((M, D), dtype=torch.float64, device=DEV)
    softmax = torch.softmax(logits, -1)
    left, weight = logits.clone(), torch.zeros_like(logits)
    for _ in range(k):  # the largest that is left; argmax of equals by the lowest index
        best = left == left.max(-1, keepdim=True).values
        best &= best.cumsum(-1) == 1
        weight += best * softmax
        left[best] = -math.inf
    if s["renorm"]:
        weight /= weight.sum(-1, keepdim=True)
    for e in range(s["E"]):
        rows = torch.nonzero(weight[:, e])[:, 0]
        if rows.numel():
            h = x[rows] @ _matrix64(s["gate_up"][e], D, 2 * F)
            h = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
            y[rows] += weight[rows, e, None] * (h @ _matrix64(s["down"][e], F, D))
    return {"y": y if s["residual"] is None else y + s["residual"].double()}


def _work_moe(c):
    M, D, F, E, k = (c[n] for n in ("M", "D", "F", "E", "k"))
    distinct = E * (1 - (1 - k / E) ** M)  # experts that M random picks of k reach
    weights = 3 * D * F * 17 / 32
    rows = 2 * M * D * (3 if c["residual"] else 2)
    return {"bytes": distinct * weights + 2 * E * D + rows, "flops": 2 * M * k * 3 * D * F + 2 * M * E * D}


# ------------------------------------- attention of new tokens over a paged cache

def _lengths(c):
    """(length with the new tokens, new tokens) of each sequence."""
    if not c["ragged"]:
        return [(max(c["length"], c["new"]), c["new"])] * c["count"]
    new = [(b * 5 + c["new"]) % (c["new"] + 1) for b in range(c["count"])]  # 0 .. new
    return [(max(n, 1 + c["length"] * (2 * b + 1) // (2 * c["count"])), n) for b, n in enumerate(new)]


def _prepare_attn(c, g):
    both = _lengths(c)
    lens, new = [b[0] for b in both], [b[1] for b in both]
    rows, width = sum(new) + 1, -(-max(lens) // c["page"])  # one row behind the last sequence
    normal = lambda *n: torch.randn(n, device=DEV, generator=g).bfloat16()  # noqa: E731
    used = [-(-n // c["page"]) for n in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, device=DEV, generator=g).int()
    table, at = torch.full((c["count"], width), -1, dtype=torch.int32, device=DEV), 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, c["page"], c["kv_heads"], c["dim"])
    offsets = [sum(new[:b]) for b in range(c["count"] + 1)]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(op="attn", q=normal(rows, c["q_heads"], c["dim"]), k_new=normal(rows, c["kv_heads"], c["dim"]),
                v_new=normal(rows, c["kv_heads"], c["dim"]), k_cache=normal(*shape), v_cache=normal(*shape),
                table=table, lens=ints(lens), row_offsets=ints(offsets),
                out=torch.zeros((rows, c["q_heads"], c["dim"]), dtype=torch.bfloat16, device=DEV),
                window=c["window"], sinks=c["sinks"], scale=c["dim"] ** -0.5, max_new=max(1, max(new)),
                max_len=width * c["page"], longest=max(lens))


def _plain_attn(s):
    q, lens, offsets, table = s["q"], s["lens"].long(), s["row_offsets"].long(), s["table"].long()
    rows, Hq, dim = q.shape
    B, page, Hkv = lens.numel(), s["k_cache"].shape[1], s["k_cache"].shape[2]
    row = torch.arange(rows, device=DEV)
    seq = (row[:, None] >= offsets[None, 1:]).sum(1).clamp(max=B - 1)
    at = lens[seq] - offsets[seq + 1] + row  # this row's position
    real = row < offsets[-1]
    # the new keys and values go to their pages (rows behind the last sequence go nowhere)
    spot = table[seq, (at // page).clamp(0, table.shape[1] - 1)] * page + at % page
    spot = torch.where(real, spot, spot[0])
    for cache, fresh in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])):
        flat = cache.view(-1, Hkv, dim)
        flat[spot] = torch.where(real[:, None, None], fresh, fresh[:1])
    n = torch.arange(s["max_new"], device=DEV)
    mine = (offsets[:-1, None] + n).clamp(max=rows - 1)  # [B][new]
    L = torch.arange(s["longest"], device=DEV)
    spots = table[:, L // page].clamp(min=0) * page + L % page
    K = s["k_cache"].view(-1, Hkv, dim)[spots].float()
    V = s["v_cache"].view(-1, Hkv, dim)[spots].float()
    qs = q[mine].float().view(B, -1, Hkv, Hq // Hkv, dim).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, dim)
    score = torch.matmul(qs, K.permute(0, 2, 3, 1)) * s["scale"]  # [B][Hkv][G new][L]
    pos = (lens - (offsets[1:] - offsets[:-1]))[:, None] + n
    seen = L <= pos[..., None]
    if s["window"]:
        seen = seen & ((pos[..., None] - L < s["window"]) | (L < s["sinks"]))
    score = score.view(B, Hkv, Hq // Hkv, -1, L.numel()).masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(score - score.max(-1, keepdim=True).values)
    o = torch.matmul(e.view(B, Hkv, -1, L.numel()), V.transpose(1, 2)).view(B, Hkv, Hq // Hkv, -1, dim)
    o = (o / e.sum(-1, keepdim=True)).permute(0, 3, 1, 2, 4).reshape(B, -1, Hq, dim)
    o = o[seq, (row - offsets[seq]).clamp(0, s["max_new"] - 1)]
    s["out"].copy_(torch.where(real[:, None, None], o, s["out"].float()))
    return {"out": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _exact_attn(s):
    """Sequence by sequence and row by row, from the cache with the new rows in it; None for the caches, which are copies."""
    Hq, dim = s["q"].shape[1:]
    _, page, Hkv, _ = s["k_cache"].shape
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    offsets = s["row_offsets"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        first, last = offsets[b], offsets[b + 1]
        old = n - (last - first)
        ids = s["table"][b, :-(-n // page)].long()
        flat = [torch.cat((c[ids].flatten(0, 1)[:old], f[first:last])) for c, f in
                ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"]))]
        for r in range(first, last):
            p = old + r - first
            lo = max(0, p - s["window"] + 1) if s["window"] else 0
            at = torch.cat((torch.arange(0, min(lo, s["sinks"])), torch.arange(lo, p + 1))).to(DEV)
            K, V = (f[at].double() for f in flat)
            q = s["q"][r].double().view(Hkv, -1, dim)
            a = torch.softmax(torch.einsum("hgd,lhd->hgl", q, K) * s["scale"], -1)
            out[r] = torch.einsum("hgl,lhd->hgd", a, V).reshape(Hq, dim)
    return {"out": out, "k_cache": None, "v_cache": None}


def _work_attn(c):
    rows = pairs = cached = 0
    for n, new in _lengths(c):
        rows += new
        pos = range(n - new, n)
        low = [max(0, p - c["window"] + 1) if c["window"] else 0 for p in pos]
        pairs += sum(p + 1 - lo + min(lo, c["sinks"]) for p, lo in zip(pos, low))
        cached += n - new - low[0] + min(low[0], c["sinks"]) if new else 0
    row = 2 * c["dim"]
    return {"bytes": row * (2 * c["kv_heads"] * (cached + 2 * rows) + 2 * c["q_heads"] * rows),
            "flops": 4 * c["dim"] * c["q_heads"] * pairs}


# ----------------------------------------------------------------- sampling

def _prepare_sample(c, g):
    R, V = c["rows"], c["vocab"]
    logits = (3 * torch.randn((R, V), device=DEV, generator=g)).bfloat16()
    if c["masked"]:  # what a grammar forbids
        logits[torch.rand((R, V), device=DEV, generator=g) < 0.3] = -math.inf
    full = lambda v, t: torch.full((R,), v, dtype=t, device=DEV)  # noqa: E731
    s = dict(op="sample", logits=logits, temperature=full(0.8, torch.float32), top_k=full(c["k"], torch.int32),
             top_p=full(c["p"], torch.float32), min_p=full(c["minp"], torch.float32),
             u=torch.rand((R,), device=DEV, generator=g), tokens=full(-2, torch.int32),
             logprobs=full(0.0, torch.float32))
    if c["mixed"]:  # rows of different requests: greedy, unfiltered, and others
        row = torch.arange(R, device=DEV)
        s["temperature"] = torch.where(row % 5 == 3, 0.0, 0.6 + 0.05 * row).float()
        s["top_k"] = torch.where(row % 4 == 1, 0, c["k"]).int()
        s["top_p"] = torch.where(row % 3 == 2, 1.0, s["top_p"]).float()
        s["min_p"] = torch.where(row % 4 == 2, 0.0, s["min_p"]).float()
    return s


def _plain_sample(s):
    """In 64 bits: a token's place in the cumulative sum depends on the last bits of the sum."""
    z = s["logits"].double()
    V = z.shape[1]
    z, index = torch.sort(z, dim=1, descending=True, stable=True)
    T = s["temperature"].double()[:, None]
    greedy = T <= 0
    e = torch.exp((z - z[:, :1]) / torch.where(greedy, 1.0, T))
    rank = torch.arange(V, device=DEV)[None]
    k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
    k = torch.where(greedy, 1, k)
    e = torch.where(rank < k, e, 0.0)
    cum = e.cumsum(1)
    p = s["top_p"].double()[:, None]
    e = torch.where((p >= 1) | (rank == 0) | (cum - e < p * cum[:, -1:]), e, 0.0)
    e = torch.where((rank == 0) | (e >= s["min_p"].double()[:, None]), e, 0.0)
    cum = e.cumsum(1)
    at = (cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(1, keepdim=True)
    at = torch.minimum(at, (e > 0).sum(1, keepdim=True) - 1)
    s["tokens"].copy_(torch.gather(index, 1, at)[:, 0])
    s["logprobs"].copy_(torch.log(torch.gather(e, 1, at) / cum[:, -1:])[:, 0])
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


def _exact_sample(s):
    """Row by row; weights of each distinct value, then the place within the equal values."""
    tokens, logprobs = [], []
    for r in range(s["logits"].shape[0]):
        z, T = s["logits"][r].double(), float(s["temperature"][r])
        k, p, least = int(s["top_k"][r]), float(s["top_p"][r]), float(s["min_p"][r])
        value, count = torch.unique(z, return_counts=True)  # ascending
        value, count = value.flip(0), count.flip(0)
        alive = value > -math.inf
        value, count = value[alive], count[alive]
        k = 1 if T <= 0 else k if k > 0 else z.numel()
        weight = torch.exp((value - value[0]) / (T if T > 0 else 1.0))
        before = count.cumsum(0) - count
        count = torch.minimum(count, (k - before).clamp(min=0))
        if p < 1:
            mass = weight * count
            below = mass.cumsum(0) - mass
            room = torch.ceil((p * mass.sum() - below) / weight).clamp(min=0)  # tokens whose sum before them is below p
            room[0] = room[0].clamp(min=1)
            count = torch.minimum(count, room.long())
        if least > 0:
            low = weight < least
            low[0] = False
            count = torch.where(low, 0, count)
        mass = weight * count
        cum = mass.cumsum(0)
        goal = float(s["u"][r]) * cum[-1]
        i = min(int((cum <= goal).sum()), int(count.nonzero().max()))
        j = min(int((goal - (cum[i] - mass[i])) / weight[i]), int(count[i]) - 1)
        tokens.append(int(torch.nonzero(z == value[i])[j, 0]))
        logprobs.append(float(torch.log(weight[i] / cum[-1])))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32),
            "logprobs": torch.tensor(logprobs, dtype=torch.float64)}


def _work_sample(c):
    return {"bytes": c["rows"] * (2 * c["vocab"] + 28), "flops": 4 * c["rows"] * c["vocab"]}
