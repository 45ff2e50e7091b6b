"""A 4-bit cache on the GPU, and its layout byte by byte from include/moe.h."""
from __future__ import annotations

import numpy as np
import torch

import bit_moe_decode_02_gb300 as moe
from ops_testlib import Cache, i32

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def places(blk, D):
    """For K and V each: byte and nibble of token t's value d, byte of its scale; arrays [blk][D]."""
    t, d = np.meshgrid(np.arange(blk), np.arange(D), indexing="ij")
    u, g, e, r = t % 32, d // 32, d % 32 // 8, d % 8
    codes = blk * D // 2
    k = (t * (D // 2) + d // 2, d % 2, codes + t // 32 * D + ((2 * (u // 8) + u % 2) * (D // 32) + g) * 4 + u // 2 % 4)
    v = (((t // 32 * (D // 32) + g) * 8 + r) * 64 + u // 8 * 16 + 4 * e + u % 8 // 2, u % 2, codes + (t // 32 * (D // 32) + g) * 32 + u)
    return k, v


def quantise(x):
    """Values [..., D] (float64) -> codes and scale bytes [..., D / 32], from the definition."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    fin = np.where(np.isfinite(g), np.abs(g), 0.0)
    a = fin.max(-1)
    byte = np.zeros(a.shape, np.int64)
    for s in range(1, 255):                                  # smallest 2^(s - 127) with a <= 6 of it
        byte = np.where((byte == 0) & (a >= 2.0 ** -100) & (a <= 6.0 * 2.0 ** (s - 127)), s, byte)
    y = np.where(np.isnan(g), 0.0, g) / np.power(2.0, np.where(byte == 0, 0, byte - 127))[..., None]
    m = np.minimum(np.abs(y), 6.0)
    hi = np.minimum(np.searchsorted(E2M1, m), 7)             # first magnitude >= m
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - E2M1[lo], E2M1[hi] - m
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(byte[..., None] == 0, 0, c + np.where(np.signbit(y), 8, 0))
    return c.reshape(x.shape), byte


class Cache4(Cache):
    """As Cache, in MXFP4."""

    def __init__(self, kv_lens, H, D, blk, seed=0, spare=2, num_blocks=None):
        self.H, self.D, self.blk, self.fmt = H, D, blk, moe.MOE_KV_MXFP4
        self.lens = list(kv_lens)
        rng = np.random.default_rng(seed)
        need = [-(-n // blk) for n in self.lens]
        nb = num_blocks or sum(need) + spare
        order = rng.permutation(nb)[:sum(need)] if nb < 1 << 20 else np.arange(nb - sum(need), nb)
        self.table = np.full((len(need), max(need + [1]) + 1), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.codes = torch.zeros(nb, H, 2, blk * D * 17 // 32, dtype=torch.uint8, device="cuda")
        self.desc = moe.moe_kv_cache_of(self.codes, None, blk, D, moe.MOE_KV_MXFP4)
        self.dtable = i32(self.table.tolist())
        self.where = [[torch.from_numpy(x).cuda() for x in p] for p in places(blk, D)]

    def fill(self, seed=0, spread=3, centre=125, poison=False, zeros=0.02):
        """Random codes, scale bytes around `centre`, some groups of zeros; poison: tokens past a sequence's end have the largest
        codes and scales."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.codes.copy_(torch.randint(0, 256, self.codes.shape, dtype=torch.uint8, generator=g, device="cuda"))
        n = self.blk * self.D // 2
        z = self.codes[..., n:]
        s = torch.randint(centre - spread, centre + 1, z.shape, dtype=torch.uint8, generator=g, device="cuda")
        z.copy_(torch.where(torch.rand(z.shape, generator=g, device="cuda") < zeros, 0, s))
        # a group whose byte is 0 holds zeros
        for i in (0, 1):
            code, scale = self.unpacked(slice(None), i)
            self.repack(slice(None), i, torch.where(scale == 0, 0, code), scale)
        if poison:
            for b, t in enumerate(self.lens):
                if t % self.blk:
                    pid = int(self.table[b, t // self.blk])
                    for i in (0, 1):
                        code, scale = self.unpacked(pid, i)
                        code[:, t % self.blk:], scale[:, t % self.blk:] = 7, 254
                        self.repack(pid, i, code, scale)
        return self

    def unpacked(self, ids, i):
        """Codes and scale bytes of the blocks' values, [..., H, blk, D] each (the group's byte for every value)."""
        at, nib, z = self.where[i]
        rec = self.codes[ids][..., i, :]
        return rec[..., at].int() >> (4 * nib) & 15, rec[..., z].int()

    def repack(self, ids, i, code, scale):
        at, nib, z = self.where[i]
        rec = torch.zeros_like(self.codes[ids][..., i, :])
        for half in (0, 1):
            rec[..., at[nib == half]] |= (code[..., nib == half] << (4 * half)).to(torch.uint8)
        rec[..., z.flatten()] = scale.flatten(-2).to(torch.uint8)
        self.codes[ids, :, i] = rec

    def values(self, b, length):
        blk, D, H = self.blk, self.D, self.H
        ids = torch.from_numpy(self.table[b, :-(-length // blk)].astype(np.int64)).cuda()
        lut = torch.tensor(list(E2M1) + list(-E2M1), dtype=torch.float64, device="cuda")
        out = []
        for i in (0, 1):
            code, scale = self.unpacked(ids, i)
            v = lut[code.long()] * torch.where(scale == 0, 0.0, (scale.long() + 896 << 52).view(torch.float64))
            out.append(v.permute(0, 2, 1, 3).reshape(-1, H, D)[:length])
        return out
