"""Ragged sequences over the shuffled pages of an 8-bit or bf16 cache, for the
tests of the operators on it: layouts, and the format's rules restated in plain
torch (scales and codes of a block, 64 bits)."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def fresh_scale(top):
    """The scale of a block of magnitude top: 2^max(floor(log2 top) - 5, -100)."""
    e = torch.frexp(top.double())[1] - 1  # floor(log2 top) above 0
    return torch.where(top > 0, torch.exp2((e - 5).clamp(min=-100).double()), torch.full_like(top.double(), 2.0 ** -100))


def to_codes(x):
    """e4m3 codes (uint8) of 64-bit values up to 448: to nearest, ties to even; NaN for what is not finite."""
    finite = torch.isfinite(x)
    y = torch.where(finite, x, 0.0)
    step = torch.exp2((torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 1 - 3).double())
    y = (torch.round(y / step) * step).float().to(E4M3)  # (the value is representable: this conversion is exact)
    y = torch.where(torch.signbit(x) & (y.float() == 0), torch.full_like(y.float(), -0.0).to(E4M3).float(), y.float()).to(E4M3)
    return torch.where(finite, y.view(torch.uint8), torch.full_like(y.view(torch.uint8), 0x7F))


def values(codes):
    return codes.view(E4M3).double()


class Paged:
    """seqs: [(length with the new tokens, new tokens)]; block 0: a bf16 cache."""

    def __init__(self, seqs, q_heads=4, kv_heads=2, dim=64, page=16, block=16, max_len=None, max_new=None,
                 head_major=False, pad=0, extra_rows=1, seed=0, spare=2, spread=1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.seqs, self.Hq, self.Hkv, self.D, self.page, self.block = g, seqs, q_heads, kv_heads, dim, page, block
        self.max_len = max_len or max(1, max(n for n, _ in seqs))
        self.max_new = max_new or max(1, max(n for _, n in seqs))
        self.rows = sum(n for _, n in seqs) + extra_rows
        self.pad = pad
        self.q = self.rnd(self.rows, q_heads * dim + pad)[:, :q_heads * dim]
        used = [-(-n // page) for n, _ in seqs]
        self.pages = sum(used) + spare
        k, v = (self.rnd(self.pages, kv_heads, page, dim) for _ in range(2))
        self.k_scale = self.v_scale = None
        if block:
            both = []
            for x in (k, v):
                x = x.double().view(self.pages, kv_heads, page // block, block * dim)
                x = x * torch.exp2(torch.randint(-3 * spread, 3 * spread + 1, x.shape[:3], device="cuda", generator=g).double())[..., None]
                scale = fresh_scale(x.abs().amax(-1))
                both.append((to_codes(x / scale[..., None]).view(self.pages, kv_heads, page, dim), scale.float()))
            (k, self.k_scale), (v, self.v_scale) = both
        if head_major:
            self.k_cache, self.v_cache = k.transpose(1, 2), v.transpose(1, 2)  # [page][slot][head][dim]
        else:
            self.k_cache, self.v_cache = k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
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

    def rnd(self, *s):
        return torch.randn(s, generator=self.g, device="cuda").bfloat16()

    def common(self):
        k = self.k_cache
        a = dict(q=self.q, k_cache=k, v_cache=self.v_cache, page_table=self.table, row_offsets=self.offsets_d,
                 lens=self.lens, q_row=self.q.stride(0), page_stride=k.stride(0), slot_stride=k.stride(1),
                 head_stride=k.stride(2), table_row=self.table.stride(0), rows=self.rows, count=len(self.seqs),
                 q_heads=self.Hq, kv_heads=self.Hkv, head_dim=self.D, pages=self.pages, page_size=self.page,
                 block=self.block, max_len=self.max_len, max_new=self.max_new)
        if self.block:
            s = self.k_scale
            a.update(k_scale=s, v_scale=self.v_scale, scale_page=s.stride(0), scale_head=s.stride(1))
        return a
