"""Cases of three operators of a decode, verify or prompt step: new keys and
values rotated and appended to a paged cache (bf16, or 8 bits with a scale for
each block of positions and head), attention over the 8-bit cache, and
penalties, biases and grammar masks on logits.  For each case: its inputs, the
operator in plain torch (`own` false) or through the library (`own` true), its
value in 64 bits, and the bytes and operations it cannot do without.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TOP = 448.0  # the largest e4m3 value
LOWEST = -100  # the smallest scale's exponent


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token of one short sequence, rotated and put into a bf16 cache: latency
        _append("append one token", count=1, new=1, length=611, q_heads=32, kv_heads=8, dim=128, rot=128, page=16),
        # a step of sixteen sequences of all lengths with up to three tokens each, into 8 bits, blocks part full
        _append("append ragged batch 8 bits", count=16, new=3, length=9001, q_heads=24, kv_heads=4, dim=64, rot=64,
                page=16, block=16, ragged=True),
        # a long prompt behind a cached prefix, into 8 bits
        _append("append prompt 8 bits", count=1, new=8191, length=12005, q_heads=32, kv_heads=8, dim=128, rot=128,
                page=64, block=64),
        # two prompts far into their sequences, wide heads of which a quarter is rotated in neighbouring pairs
        _append("append prompts pairs", count=2, new=2049, length=100003, q_heads=16, kv_heads=4, dim=256, rot=64,
                page=32, pairs=True),
        # plain decode of one short sequence from 8 bits: latency
        _attn("attention 8 bits short", count=1, new=1, length=611, q_heads=32, kv_heads=8, dim=128, page=16, block=16),
        # the verify step of a 7-token draft far into one sequence
        _attn("attention 8 bits verify 8", count=1, new=8, length=32771, q_heads=32, kv_heads=8, dim=128, page=64,
              block=64),
        # sixteen sequences of all lengths, some with no new token this step, a scale for each position
        _attn("attention 8 bits ragged", count=16, new=3, length=9001, q_heads=24, kv_heads=4, dim=64, page=16, block=1,
              ragged=True),
        # a sliding window with a few first tokens that stay visible, wide heads, longest draft, slots of a head together
        _attn("attention 8 bits window", count=2, new=16, length=100003, q_heads=16, kv_heads=4, dim=256, page=32,
              block=32, window=4096, sinks=4, heads_first=True),
        # one row of a small vocabulary after a short answer: latency
        _logits("penalties one row small", rows=1, vocab=32000, history=613, bias=8, masked=False),
        # one row of the full vocabulary under a grammar, a long conversation behind it
        _logits("penalties one row grammar", rows=1, vocab=248320, history=32771, bias=0, masked=True),
        # every row of a long verify step: one history, of which each row has one token more
        _logits("penalties 16 rows", rows=16, vocab=248320, history=4099, bias=300, masked=True, shared=True),
        # rows of different requests, an odd vocabulary
        _logits("penalties 7 rows odd", rows=7, vocab=50261, history=1537, bias=5, masked=True),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    kind = rng.choice(("append", "attn", "logits"))
    if kind == "logits":
        rows = rng.randint(1, 16)
        return _logits(None, rows=rows, vocab=log(1000, 248320), history=rng.choice((0, 1, log(2, 40000))),
                       bias=rng.choice((0, 1, 17, 300)), masked=rng.random() < 0.6, shared=rng.random() < 0.5)
    kv, dim, page = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 128, 256)), rng.choice((16, 32, 64))
    block = rng.choice([b for b in (1, 4, 16, 32, 64) if b <= page])
    group = rng.choice((1, 2, 4, 6, 8))
    if kind == "append":
        count = rng.choice((1, 1, 2, 5, 16))
        most = 33_000_000 // (count * kv * (group + 2) * dim)
        new = rng.choice((1, 1, 2, 8, log(17, min(8191, most))))
        return _append(None, count=count, new=new, length=new + log(1, 100000 // count), q_heads=kv * group, kv_heads=kv,
                       dim=dim, rot=rng.choice((dim, dim, dim // 2, dim // 4)), page=page,
                       block=rng.choice((0, block, block)), pairs=rng.random() < 0.3, ragged=rng.random() < 0.5)
    count = rng.choice((1, 1, 2, 3, 7, 16))
    new = rng.choice((1, 1, 2, 5, 8, 16))
    while new * group * kv > 512:
        group = max(1, group // 2)
        new = new // 2 if group == 1 else new
    cap = min(120000 // count, 25600000 // (count * kv * dim))
    window = rng.choice((0, 0, log(64, 8192)))
    return _attn(None, count=count, new=new, length=log(17, cap), q_heads=kv * group, kv_heads=kv, dim=dim, page=page,
                 block=block, window=window, sinks=rng.choice((0, 4, 16)) if window else 0, ragged=rng.random() < 0.5,
                 heads_first=rng.random() < 0.5)


def _named(name, case):
    return {**({"name": name} if name else {}), **case}


def _append(name, count, new, length, q_heads, kv_heads, dim, rot, page, block=0, pairs=False, ragged=False):
    """block 0: a bf16 cache; rot: values of a head that are rotated, pairs: neighbours of each other."""
    return _named(name, dict(op="append", count=count, new=new, length=length, q_heads=q_heads, kv_heads=kv_heads,
                             dim=dim, rot=rot, page=page, block=block, pairs=pairs, ragged=ragged))


def _attn(name, count, new, length, q_heads, kv_heads, dim, page, block, window=0, sinks=0, ragged=False,
          heads_first=False):
    return _named(name, dict(op="attn", count=count, new=new, length=length, q_heads=q_heads, kv_heads=kv_heads,
                             dim=dim, page=page, block=block, window=window, sinks=sinks, ragged=ragged,
                             heads_first=heads_first))


def _logits(name, rows, vocab, history, bias, masked, shared=False):
    return _named(name, dict(op="logits", rows=rows, vocab=vocab, history=history, bias=bias, masked=masked, shared=shared))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"append": _prepare_append, "attn": _prepare_attn, "logits": _prepare_logits}[case["op"]](case, g)


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attn": _plain_attn, "logits": _plain_logits}[state["op"]](state)


def work(case):
    return {"append": _work_append, "attn": _work_attn, "logits": _work_logits}[case["op"]](case)


def exact(case, seed):
    return {"append": _exact_append, "attn": _exact_attn, "logits": _exact_logits}[case["op"]](prepare(case, seed))


def _own(s):
    import int4_weight_only_g128_gb300 as w
    step = s.get("step")
    if step is None:  # a program marshals a step's buffers once and keeps its workspace
        if s["op"] == "logits":
            step = w.PenalizeStep(w.PenalizeArgs(
                logits=s["logits"], out=s["out"], row_stride=s["logits"].stride(0), out_stride=s["out"].stride(0),
                history=s["history"], history_start=s["history_start"], history_len=s["history_len"],
                prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                frequency=s["frequency"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"],
                bias_offsets=s["bias_offsets"], mask=s["mask"], mask_row=0 if s["mask"] is None else s["mask"].stride(0),
                rows=s["logits"].shape[0], vocab=s["logits"].shape[1], history_size=s["history"].numel(),
                bias_size=s["bias_tokens"].numel()))
        else:
            k, ks = s["k_cache"], s["k_scale"]
            common = dict(q=s["q"], k_cache=k, v_cache=s["v_cache"], page_table=s["table"], row_offsets=s["row_offsets"],
                          lens=s["lens"], q_row=s["q"].stride(0), table_row=s["table"].stride(0), rows=s["q"].shape[0],
                          count=s["lens"].numel(), q_heads=s["q"].shape[1], kv_heads=s["kv_heads"], head_dim=s["dim"],
                          page_stride=k.stride(0), slot_stride=k.stride(1), head_stride=k.stride(2),
                          pages=k.shape[0], page_size=k.shape[1], max_len=s["max_len"], max_new=s["max_new"],
                          k_scale=ks, v_scale=s["v_scale"], block=s["block"])
            if ks is not None:
                common.update(scale_page=ks.stride(0), scale_head=ks.stride(1))
            if s["op"] == "attn":
                args = w.Attend8Args(**common, out=s["out"], out_row=s["out"].stride(0), window=s["window"],
                                     sinks=s["sinks"], scale=s["scale"])
                step = w.Attend8Step(args, _workspace(w.w4g128_attend8_workspace_bytes(args)))
            else:
                args = w.AppendArgs(**common, q_out=s["q_out"], q_out_row=s["q_out"].stride(0), k_new=s["k_new"],
                                    v_new=s["v_new"], kv_row=s["k_new"].stride(0), freqs=s["freqs"], rot_dim=s["rot"],
                                    interleaved=s["pairs"])
                step = w.AppendStep(args, _workspace(w.w4g128_append_workspace_bytes(args)))
        s["step"] = step
    step.run()
    return _outputs(s)


def _outputs(s):
    if s["op"] == "logits":
        return {"out": s["out"]}
    if s["op"] == "attn":
        return {"out": s["out"]}
    # (codes are returned as the e4m3 tensors that they are, the scales beside them)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"],
            **({"k_scale": s["k_scale"], "v_scale": s["v_scale"]} if s["block"] else {})}


def _workspace(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------- both cache operators

def _lengths(c):
    """(length with the new tokens, new tokens) of each sequence."""
    if not c["ragged"]:
        return [(max(c["length"], c["new"]), c["new"])] * c["count"]
    new = [(b * 5 + c["new"]) % (c["new"] + 1) for b in range(c["count"])]  # 0 .. new
    return [(max(n, 1 + c["length"] * (2 * b + 1) // (2 * c["count"])), n) for b, n in enumerate(new)]


def _batch(c, g):
    """Rows, pages and lengths of the sequences, and caches of what they hold so far."""
    both = _lengths(c)
    lens, new = [b[0] for b in both], [b[1] for b in both]
    width = -(-max(lens) // c["page"])
    used = [-(-n // c["page"]) for n in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, device=DEV, generator=g).int()
    table, at = torch.full((c["count"], width), -1, dtype=torch.int32, device=DEV), 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    offsets = [sum(new[:b]) for b in range(c["count"] + 1)]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = dict(op=c["op"], table=table, lens=ints(lens), row_offsets=ints(offsets), rows=sum(new) + 1,  # one row behind the last
             max_new=max(1, max(new)), max_len=width * c["page"], longest=max(lens), dim=c["dim"], kv_heads=c["kv_heads"],
             block=c["block"], k_scale=None, v_scale=None)
    for n in ("k", "v"):
        s[n + "_cache"], s[n + "_scale"] = _cache(c, pages, g)
    return s


def _cache(c, pages, g):
    """Keys or values of every slot; in 8 bits each block's magnitude is its own."""
    H, page, dim, block = c["kv_heads"], c["page"], c["dim"], c["block"]
    x = torch.randn((pages, H, page, dim), device=DEV, generator=g, dtype=torch.float16)
    if not block:
        return x.transpose(1, 2).bfloat16().contiguous(), None
    size = 2.0 ** torch.randint(-3, 2, (pages, H, page // block), device=DEV, generator=g)
    top = x.view(pages, H, page // block, -1).abs().amax(-1).float() * size
    scale = torch.exp2(torch.floor(torch.log2(top)) - 5)
    codes = x.view(pages, H, page // block, -1) * (size / scale)[..., None].half()
    codes = codes.to(E4M3).view(pages, H, page, dim)
    codes = codes.view(torch.uint8).transpose(1, 2)
    return (codes if c.get("heads_first") else codes.contiguous()).view(E4M3), scale


def _places(s):
    """Of each row: its sequence, position, slot in the flat cache and whether it belongs to a sequence."""
    lens, offsets, table = s["lens"].long(), s["row_offsets"].long(), s["table"].long()
    page = s["k_cache"].shape[1]
    row = torch.arange(s["rows"], device=DEV)
    seq = (row[:, None] >= offsets[None, 1:]).sum(1).clamp(max=lens.numel() - 1)
    at = lens[seq] - offsets[seq + 1] + row
    spot = table[seq, (at // page).clamp(0, table.shape[1] - 1)] * page + at % page
    return seq, at, spot, row < offsets[-1]


# ---------------------------------------------------------------- rotate and append

def _prepare_append(c, g):
    s = _batch(c, g)
    normal = lambda *n: torch.randn(n, device=DEV, generator=g).bfloat16()  # noqa: E731
    # one projection's output holds the keys and the values of a row side by side; some rows are larger than what is cached
    kv = torch.randn((s["rows"], 2, c["kv_heads"], c["dim"]), device=DEV, generator=g)
    kv = (kv * 2.0 ** torch.randint(-2, 7, (s["rows"], 2, c["kv_heads"], 1), device=DEV, generator=g)).bfloat16()
    i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
    return dict(s, q=normal(s["rows"], c["q_heads"], c["dim"]), k_new=kv[:, 0], v_new=kv[:, 1],
                q_out=torch.zeros((s["rows"], c["q_heads"], c["dim"]), dtype=torch.bfloat16, device=DEV),
                freqs=1e6 ** (-2 * i / c["rot"]), rot=c["rot"], pairs=int(c["pairs"]))


def _rotated(x, cos, sin, rot, pairs):
    x = x.float()
    first, rest = x[..., :rot], x[..., rot:]
    a, b = (first[..., 0::2], first[..., 1::2]) if pairs else (first[..., :rot // 2], first[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    first = torch.stack((u, v), -1).flatten(-2) if pairs else torch.cat((u, v), -1)
    return torch.cat((first, rest), -1)


def _plain_append(s):
    seq, at, spot, real = _places(s)
    angle = at.double()[:, None, None] * s["freqs"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotated(s["q"], cos, sin, s["rot"], s["pairs"])
    s["q_out"].copy_(torch.where(real[:, None, None], q, s["q_out"].float()))
    k = _rotated(s["k_new"], cos, sin, s["rot"], s["pairs"])
    for n, x in (("k", k), ("v", s["v_new"].float())):
        _put(s, s[n + "_cache"], s[n + "_scale"], x, seq, at, spot, real)
    return _outputs(s)


def _put(s, cache, scale, x, seq, at, spot, real):
    H, dim, page, block = s["kv_heads"], s["dim"], cache.shape[1], s["block"]
    spot, x = spot[real], x[real]
    if not block:
        cache.view(-1, H, dim)[spot] = x.bfloat16()
        return
    codes = cache.view(torch.uint8)
    # a block's scale: what it has stays if the new rows fit under it
    of_block = spot // block
    top = torch.zeros((cache.shape[0] * page // block, H), device=DEV)
    top.index_reduce_(0, of_block, x.abs().amax(-1), "amax")
    flat = scale.transpose(1, 2).reshape(-1, H)
    fresh = torch.exp2((torch.floor(torch.log2(top)) - 5).clamp(min=LOWEST))
    start = (s["lens"] - (s["row_offsets"][1:] - s["row_offsets"][:-1])).long()
    some = s["row_offsets"][1:] > s["row_offsets"][:-1]
    table = s["table"].long()
    b = torch.arange(start.numel(), device=DEV)
    page_at = table[b, (start // page).clamp(max=table.shape[1] - 1)]
    begun = torch.where(some, page_at * page + start % page, 0) // block  # the block in which a sequence goes on
    filled = torch.zeros(top.shape[0], device=DEV).index_add_(0, begun, torch.where(some, start % block, 0).float())
    held = filled > 0
    touched = torch.zeros(top.shape[0], device=DEV).index_fill_(0, of_block, 1) > 0
    new = torch.where(held[:, None] & (top <= TOP * flat), flat, fresh)
    new = torch.where(touched[:, None], new, flat)
    # what such blocks hold already (the slots before the new rows), in the new scale
    slots = begun[:, None] * block + torch.arange(block, device=DEV)
    grows = (held[:, None] & (new > flat))[begun][:, None] & (slots % block < filled[begun][:, None])[..., None]
    old = codes[slots // page, slots % page]
    again = (old.view(E4M3).float() * (flat / new)[begun][:, None, :, None]).to(E4M3).view(torch.uint8)
    codes[slots // page, slots % page] = torch.where(grows[..., None], again, old)
    codes[spot // page, spot % page] = (x / new[of_block][..., None]).to(E4M3).view(torch.uint8)
    scale.copy_(new.view(cache.shape[0], page // block, H).transpose(1, 2))


def _to_e4m3_64(x):
    """The e4m3 value next to x (to even), in 64 bits: steps of 2^-9 below 2^-6, of an eighth of the power of two above."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    """Sequence by sequence, blocks of each by reshaping."""
    lens, offsets, page, block = s["lens"].tolist(), s["row_offsets"].tolist(), s["k_cache"].shape[1], s["block"]
    H, dim, rot = s["kv_heads"], s["dim"], s["rot"]
    q_out = s["q_out"].double()
    caches = {n: s[n + "_cache"].double() for n in ("k", "v")}
    scales = {n: s[n + "_scale"].double() for n in ("k", "v")} if block else {}
    for b, n in enumerate(lens):
        lo, hi = offsets[b], offsets[b + 1]
        if lo == hi:
            continue
        start = n - (hi - lo)
        pos = torch.arange(start, n, device=DEV)
        angle = pos.double()[:, None] * s["freqs"]
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]

        def rotated(x):
            x = x.double().clone()
            a, b_ = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["pairs"] else (x[..., :rot // 2], x[..., rot // 2:rot])
            z = torch.complex(a, b_) * turn
            a.copy_(z.real)
            b_.copy_(z.imag)
            return x
        q_out[lo:hi] = rotated(s["q"][lo:hi])
        ids = s["table"][b].long()
        for name, x in (("k", rotated(s["k_new"][lo:hi])), ("v", s["v_new"][lo:hi].double())):
            cache = caches[name]
            if not block:
                cache[ids[pos // page], pos % page] = x
                continue
            first = start // block * block  # the blocks from here on, whole
            every = torch.arange(first, -(-n // block) * block, device=DEV)
            blocks = torch.zeros((every.numel(), H, dim), dtype=torch.float64, device=DEV)
            blocks[start - first:n - first] = x
            blocks = blocks.view(-1, block, H, dim)
            top = blocks.abs().amax((1, 3))
            at = torch.arange(first, n, block, device=DEV)
            into = (ids[at // page, None], torch.arange(H, device=DEV)[None], (at % page // block)[:, None])
            new = torch.exp2((torch.floor(torch.log2(top)) - 5).clamp(min=LOWEST))
            if start > first:
                was = scales[name][ids[first // page], :, first % page // block]
                new[0] = torch.where(top[0] <= TOP * was, was, new[0])
                slot = torch.arange(first, start, device=DEV) % page
                held = cache[ids[first // page], slot]
                cache[ids[first // page], slot] = _to_e4m3_64(held * (was / new[0])[:, None])
            scales[name][into] = new
            codes = _to_e4m3_64(blocks / new[:, None, :, None]).view(-1, H, dim)[start - first:n - first]
            cache[ids[pos // page], pos % page] = codes
    return {"q": q_out, "k_cache": caches["k"], "v_cache": caches["v"],
            **({"k_scale": scales["k"], "v_scale": scales["v"]} if block else {})}


def _work_append(c):
    rows = sum(n for _, n in _lengths(c))
    kv, width = 2 * c["kv_heads"] * c["dim"], 1 if c["block"] else 2
    scales = 8 * c["kv_heads"] * sum(-(-n // c["block"]) + 1 for _, n in _lengths(c) if n) if c["block"] else 0
    return {"bytes": rows * (4 * c["q_heads"] * c["dim"] + kv * (2 + width)) + scales,
            "flops": rows * (3 * (c["q_heads"] + c["kv_heads"]) * c["rot"] + 2 * kv)}


# ---------------------------------------------------------------- attention over 8 bits

def _prepare_attn(c, g):
    s = _batch(c, g)
    normal = lambda *n: torch.randn(n, device=DEV, generator=g).bfloat16()  # noqa: E731
    return dict(s, q=normal(s["rows"], c["q_heads"], c["dim"]),
                out=torch.zeros((s["rows"], c["q_heads"], c["dim"]), dtype=torch.bfloat16, device=DEV),
                window=c["window"], sinks=c["sinks"], scale=c["dim"] ** -0.5)


def _values(cache, scale, ids, slot, block):
    """[...][heads][dim] of the slots: codes times their blocks' scales."""
    return cache.view(torch.uint8)[ids, slot].view(E4M3).float() * scale.transpose(1, 2)[ids, slot // block][..., None]


def _plain_attn(s):
    q, lens, offsets, table = s["q"], s["lens"].long(), s["row_offsets"].long(), s["table"].long()
    rows, Hq, dim = q.shape
    B, page, Hkv = lens.numel(), s["k_cache"].shape[1], s["kv_heads"]
    seq, _, _, real = _places(s)
    n = torch.arange(s["max_new"], device=DEV)
    mine = (offsets[:-1, None] + n).clamp(max=rows - 1)  # [B][new]
    L = torch.arange(s["longest"], device=DEV)
    ids, slot = table[:, L // page].clamp(min=0), (L % page).expand(B, -1)
    K = _values(s["k_cache"], s["k_scale"], ids, slot, s["block"])
    V = _values(s["v_cache"], s["v_scale"], ids, slot, s["block"])
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
    row = torch.arange(rows, device=DEV)
    o = o[seq, (row - offsets[seq]).clamp(0, s["max_new"] - 1)]
    s["out"].copy_(torch.where(real[:, None, None], o, s["out"].float()))
    return _outputs(s)


def _exact_attn(s):
    """Sequence by sequence and row by row."""
    Hq, dim = s["q"].shape[1:]
    page, Hkv, block = s["k_cache"].shape[1], s["kv_heads"], s["block"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    offsets = s["row_offsets"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        first, last = offsets[b], offsets[b + 1]
        for r in range(first, last):
            p = n - last + r
            lo = max(0, p - s["window"] + 1) if s["window"] else 0
            at = torch.cat((torch.arange(0, min(lo, s["sinks"])), torch.arange(lo, p + 1))).to(DEV)
            ids = s["table"][b].long()[at // page]
            K, V = (s[x + "_cache"].view(torch.uint8)[ids, at % page].view(E4M3).double() *
                    s[x + "_scale"][ids, :, at % page // block].double()[..., None] for x in ("k", "v"))
            q = s["q"][r].double().view(Hkv, -1, dim)
            a = torch.softmax(torch.einsum("hgd,lhd->hgl", q, K) * s["scale"], -1)
            out[r] = torch.einsum("hgl,lhd->hgd", a, V).reshape(Hq, dim)
    return {"out": out}


def _work_attn(c):
    rows = pairs = cached = 0
    for n, new in _lengths(c):
        rows += new
        pos = range(n - new, n)
        low = [max(0, p - c["window"] + 1) if c["window"] else 0 for p in pos]
        pairs += sum(p + 1 - lo + min(lo, c["sinks"]) for p, lo in zip(pos, low))
        cached += n - low[0] + min(low[0], c["sinks"]) if new else 0
    return {"bytes": 2 * c["kv_heads"] * cached * (c["dim"] + 4 / c["block"]) + 4 * c["dim"] * c["q_heads"] * rows,
            "flops": 4 * c["dim"] * c["q_heads"] * pairs}


# ---------------------------------------------------------------- penalties, biases and masks

def _prepare_logits(c, g):
    R, V, n, nb = c["rows"], c["vocab"], c["history"], c["bias"]
    rand = lambda *shape: torch.rand(shape, device=DEV, generator=g)  # noqa: E731
    # a row's history: the same as the row's before and one token more, or its own; a few words come often
    history = (V * rand(n + R if c["shared"] else n * R) ** 4).int().clamp(max=V - 1)
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device=DEV)  # noqa: E731
    lens = [(n + r if n else 0) if c["shared"] else n - (r * 389) % max(1, n) for r in range(R)]
    each = [nb if r % 3 != 1 else nb // 2 for r in range(R)]
    at = [sum(each[:r]) for r in range(R + 1)]
    mask = None
    if c["masked"]:
        bits = torch.randint(-2**31, 2**31 - 1, (R, -(-V // 32)), dtype=torch.int32, device=DEV, generator=g)
        mask = bits & torch.randint(-2**31, 2**31 - 1, bits.shape, dtype=torch.int32, device=DEV, generator=g)
    row = torch.arange(1, R + 1, device=DEV)  # rows with settings of their own, some without one or the other
    # a list names no token twice: the tokens of a row are apart by at least one
    place = torch.tensor([i - at[r] for r in range(R) for i in range(at[r], at[r + 1])], device=DEV)
    spread = torch.tensor([max(1, V // max(1, each[r])) for r in range(R) for _ in range(each[r])], device=DEV)
    bias_tokens = (place * spread).int() if nb else ints([])
    return dict(op="logits", logits=(3 * torch.randn((R, V), device=DEV, generator=g)).bfloat16(),
                out=torch.zeros((R, V), dtype=torch.bfloat16, device=DEV), history=history,
                history_start=ints([0 if c["shared"] else r * n for r in range(R)], torch.int64), history_len=ints(lens),
                prompt_len=ints([m // 3 for m in lens]),
                repetition=(1.0 + 0.05 * (row % 4)).float(), presence=(0.25 * (row % 3)).float(),
                frequency=(0.125 * (row % 5)).float(), bias_tokens=bias_tokens,
                bias_values=20 * rand(bias_tokens.numel()) - 10, bias_offsets=ints(at), mask=mask)


def _plain_logits(s):
    R, V = s["logits"].shape
    z = s["logits"].float()
    at = torch.arange(s["history"].numel(), device=DEV)
    begin = s["history_start"][:, None]
    inside = (at >= begin) & (at < begin + s["history_len"][:, None])
    written = inside & (at >= begin + s["prompt_len"][:, None])
    token = s["history"].long().expand(R, -1)
    count = torch.zeros((R, V), device=DEV).scatter_add_(1, token, written.float())
    seen = torch.zeros((R, V), device=DEV).scatter_add_(1, token, inside.float()) > 0
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][:, None] * count
    z = z - s["presence"][:, None] * (count > 0)
    if s["bias_tokens"].numel():
        i = torch.arange(s["bias_tokens"].numel(), device=DEV)
        row = (i[:, None] >= s["bias_offsets"][None, 1:]).sum(1)
        z[row, s["bias_tokens"].long()] += s["bias_values"]
    if s["mask"] is not None:
        t = torch.arange(V, device=DEV)
        z = z.masked_fill(((s["mask"][:, t // 32] >> (t % 32).int()) & 1) == 0, -math.inf)
    s["out"].copy_(z)
    return _outputs(s)


def _exact_logits(s):
    """Row by row."""
    out = s["logits"].double()
    at = s["bias_offsets"].tolist()
    for r in range(out.shape[0]):
        V, z = out.shape[1], out[r]
        begin = int(s["history_start"][r])
        tokens = s["history"][begin:begin + int(s["history_len"][r])].long()
        rep = s["repetition"][r].double()
        t = torch.unique(tokens)
        z[t] = torch.where(z[t] > 0, z[t] / rep, z[t] * rep)
        count = torch.bincount(tokens[int(s["prompt_len"][r]):], minlength=V).double()
        z -= s["frequency"][r].double() * count + s["presence"][r].double() * (count > 0)
        z[s["bias_tokens"][at[r]:at[r + 1]].long()] += s["bias_values"][at[r]:at[r + 1]].double()
        if s["mask"] is not None:
            bits = (s["mask"][r][:, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
            z[bits.flatten()[:V] == 0] = -math.inf
    return {"out": out}


def _work_logits(c):
    each = 4 * c["vocab"] + (c["vocab"] / 8 if c["masked"] else 0) + 8 * c["bias"]
    return {"bytes": c["rows"] * each + 4 * (c["history"] + 1) * (1 if c["shared"] else c["rows"]),
            "flops": 6 * c["rows"] * c["vocab"]}
