"""A cache of codes as the library defines it, in plain torch on the CPU."""
from __future__ import annotations

import torch

GROUP = 64


def quantise(x, bits):
    """Codes (one a byte), scales and biases of float32 values [..., d], by the definition's float32 operations."""
    top = 2 ** bits - 1
    x = torch.where(torch.isnan(x), torch.zeros(()), x.float()).clamp(-65280.0, 65280.0)
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    bias, scale = lo.half(), ((hi - lo) / top).half()
    s = scale.float()
    inverse = torch.where(s > 0, 1.0 / torch.where(s > 0, s, torch.ones(())), torch.zeros(()))
    code = torch.round((g - bias.float()) * inverse).clamp(0, top).to(torch.uint8)
    return code.flatten(-2), torch.cat((scale, bias), -1)


def values(code, affine):
    """s c + b in float64, of unpacked codes."""
    a = affine.double()
    return (code.unflatten(-1, (-1, GROUP)).double() * a[..., :1] + a[..., 1:]).flatten(-2)


def pack(code, bits):
    return code if bits == 8 else code[..., 0::2] | code[..., 1::2] << 4


def unpack(packed, bits):
    return packed if bits == 8 else torch.stack((packed & 15, packed >> 4), -1).flatten(-2)


class Pool:
    """A cache of codes on the device. Pages are shuffled, slots and pages that no sequence uses hold any codes with scales and
    biases of NaN, unused entries of the page table are out of range. `parts`: keys and values of each sequence as
    (codes, affine), [len, heads, d]."""

    def __init__(self, lengths, heads, page, d, bits, gen, layout="hnd", spare=3, size=1.0, extra=1):
        self.lengths, self.heads, self.page, self.d, self.bits = lengths, heads, page, d, bits
        used = [max(0, -(-n // page)) for n in lengths]
        self.max_pages, self.pages = max(1, max(used)) + extra, sum(used) + spare
        order = torch.randperm(self.pages, generator=gen)
        self.table = torch.full((len(lengths), self.max_pages), -7, dtype=torch.int32)
        if extra:
            self.table[:, -1] = 1 << 30
        w = d * bits // 8
        shape = (self.pages, heads, page) if layout == "hnd" else (self.pages, page, heads)
        self.k, self.v = (torch.randint(256, (*shape, w), generator=gen, dtype=torch.uint8) for _ in range(2))
        self.ka, self.va = (torch.full((*shape, d // GROUP, 2), float("nan"), dtype=torch.float16) for _ in range(2))
        if layout != "hnd":
            self.k, self.v, self.ka, self.va = (t.transpose(1, 2) for t in (self.k, self.v, self.ka, self.va))
        self.own, self.parts, at = [], [], 0
        for i, n in enumerate(lengths):
            own = order[at:at + used[i]]
            at += used[i]
            self.table[i, :used[i]] = own.int()
            self.own.append(own)
            j = torch.arange(max(n, 0))
            sides = []
            for code, affine in ((self.k, self.ka), (self.v, self.va)):
                c, a = quantise(size * torch.randn((max(n, 0), heads, d), generator=gen), bits)
                code[own[j // page], :, j % page] = pack(c, bits)
                affine[own[j // page], :, j % page] = a
                sides.append((c, a))
            self.parts.append(sides)

    def place(self, seq, j):
        return self.own[seq][j // self.page], j % self.page

    def device(self, q):
        """The library's cache, and the page table."""
        self.cache = q.QuantKVCache(*(t.cuda() for t in (self.k, self.v, self.ka, self.va)), self.bits)
        return self.cache, self.table.cuda()

    def back(self):
        """Unpacked codes, scales and biases of keys and values on the device, at the CPU."""
        c = self.cache
        return [(unpack(code.cpu(), self.bits), affine.cpu()) for code, affine in ((c.k, c.k_affine), (c.v, c.v_affine))]
