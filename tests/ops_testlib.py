"""Plain forms, in 64 bits, of the operators around the expert block, and what
their tests share.  Written from the definitions in include/moe.h."""
from __future__ import annotations

import math

import numpy as np
import torch

import bit_moe_decode_02_gb300 as moe
from bit_moe_decode_02_gb300 import build_ext

_handle = None


def handle() -> int:
    """One handle for all tests."""
    global _handle
    if _handle is None:
        build_ext.build()
        _handle = moe.moe_ops_create()
    return _handle


def ok(o) -> None:
    assert moe.moe_ops_get_status(o) == 0, moe.moe_last_error()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# E4M3 magnitudes of the codes 0..126 (127 is NaN)
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def decode(codes: np.ndarray, fmt: int) -> np.ndarray:
    if fmt == moe.MOE_KV_INT8:
        return codes.view(np.int8).astype(np.float64)
    mag = np.append(E4M3, np.nan)[codes & 127]
    return np.where(codes >= 128, -mag, mag)


def encode(y: np.ndarray, fmt: int) -> np.ndarray:
    """fp32 values in units of the scale -> codes: nearest, ties to even, saturating, NaN -> 0."""
    y = np.where(np.isnan(y), 0.0, y.astype(np.float64))
    if fmt == moe.MOE_KV_INT8:
        return np.rint(np.clip(y, -127, 127)).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(y), 448.0)
    hi = np.minimum(np.searchsorted(E4M3, a), 126)          # first magnitude >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def block_scale(values: np.ndarray, fmt: int) -> np.float32:
    fin = np.abs(values[np.isfinite(values)])
    a = np.float32(max(float(fin.max()) if fin.size else 0.0, 2.0 ** -100))
    if fmt == moe.MOE_KV_INT8:
        return np.float32(a / np.float32(127))
    e = -120
    while float(a) > 448.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def half_ulp_bf16(x):
    """What one rounding to bf16 (8 significant bits) may cost."""
    return torch.pow(2.0, torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -126))) - 8)


class Cache:
    """A cache on the GPU, its descriptor, and a block table dealt at random."""

    def __init__(self, kv_lens, H, D, blk, fmt, seed=0, spare=2, num_blocks=None):
        self.H, self.D, self.blk, self.fmt = H, D, blk, fmt
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
        self.codes = torch.zeros(nb, H, 2, blk * D, dtype=torch.uint8, device="cuda")
        self.scales = torch.zeros(nb, H, 2, dtype=torch.float32, device="cuda")
        self.desc = moe.moe_kv_cache_of(self.codes, self.scales, blk, D, fmt)
        self.dtable = i32(self.table.tolist())

    def batch(self, new, kv_len):
        cu = np.concatenate(([0], np.cumsum(new))).tolist()
        return moe.moe_kv_batch_of(i32(cu), i32(list(kv_len)), self.dtable, int(cu[-1]))

    def fill(self, seed=0, sigma=1.0, poison=False):
        """Random codes and scales everywhere; poison: tokens past a sequence's end decode to the largest values."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        c = torch.randint(0, 256, self.codes.shape, dtype=torch.uint8, generator=g, device="cuda")
        if self.fmt == moe.MOE_KV_E4M3:
            # exponents around the middle of the format, as data scaled to its maximum has
            c = (c & 0x87) | (torch.randint(6, 15, c.shape, dtype=torch.uint8, generator=g, device="cuda") << 3)
            self.scales.copy_(torch.pow(2.0, torch.randint(-9, -5, self.scales.shape, generator=g, device="cuda").float()) * sigma)
        else:
            c = torch.where(c == 128, 129, c)
            self.scales.copy_((0.5 + torch.rand(self.scales.shape, generator=g, device="cuda")) * (sigma / 60))
        self.codes.copy_(c)
        if poison:
            for b, n in enumerate(self.lens):
                if n % self.blk:
                    t = self.codes[int(self.table[b, n // self.blk])]
                    t[:, 0].view(self.H, self.blk, self.D)[:, n % self.blk:] = 0x7e
                    t[:, 1].view(self.H, self.D, self.blk)[:, :, n % self.blk:] = 0x7e
        return self

    def values(self, b, length):
        """Keys and values of sequence b in float64, [length, H, D] each, on the GPU."""
        blk, D, H = self.blk, self.D, self.H
        ids = torch.from_numpy(self.table[b, :-(-length // blk)].astype(np.int64)).cuda()
        lut = torch.from_numpy(decode(np.arange(256, dtype=np.uint8), self.fmt)).cuda()
        v = lut[self.codes[ids].long()] * self.scales[ids].double()[..., None]
        k = v[:, :, 0].reshape(-1, H, blk, D).permute(0, 2, 1, 3).reshape(-1, H, D)[:length]
        w = v[:, :, 1].reshape(-1, H, D, blk).permute(0, 3, 1, 2).reshape(-1, H, D)[:length]
        return k, w


def attention(cache: Cache, new, kv_len, q, scale, window=0, sinks=None, least=2.0 ** -24):
    """(out, lse, bound) in float64.  bound: what an f16 probability, fp32 scores and one rounding to bf16 may cost; `least`:
    what a key's probability may lose below f16's normal numbers."""
    outs, lses, bounds, at = [], [], [], 0
    Hq = q.shape[1]
    G = Hq // cache.H
    for b, (n, t) in enumerate(zip(new, kv_len)):
        if n == 0:
            continue
        k, v = cache.values(b, t)
        k, v = (x.repeat_interleave(G, 1).permute(1, 0, 2) for x in (k, v))         # [Hq, t, D]
        qq = q[at:at + n].double().permute(1, 0, 2)
        s = qq @ k.transpose(1, 2) * scale
        mag = qq.abs() @ k.abs().transpose(1, 2) * abs(scale)
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        j = torch.arange(t, device="cuda")[None]
        see = (j <= pos) & ((j > pos - window) if window else (j >= 0))
        s = torch.where(see, s, -math.inf)
        mag = torch.where(see, mag, 0.0)
        m = s.amax(-1, keepdim=True)
        if sinks is not None:
            m = torch.maximum(m, sinks.double()[:, None, None])
        e = torch.exp(s - m)
        l = e.sum(-1, keepdim=True)
        if sinks is not None:
            l = l + torch.exp(sinks.double()[:, None, None] - m)
        p = e / l
        o = p @ v
        # a score is a sum of at most 128 fp32 products and their scaling: 2^-22 of its magnitudes' sum covers it, and as
        # much again the exponential's argument; p rounded to f16: 2^-11 of it, or 2^-25 where it is subnormal
        ds = mag.amax(-1, keepdim=True) * 2.0 ** -20
        bound = half_ulp_bf16(o) * 1.01 + (2.0 ** -10.5 + 2 * ds) * (p @ v.abs()) + (see.double() @ v.abs()) * least / l
        outs.append(o.permute(1, 0, 2))
        lses.append((m + l.log())[..., 0].permute(1, 0))
        bounds.append((bound + 1e-30).permute(1, 0, 2))
        at += n
    return torch.cat(outs), torch.cat(lses), torch.cat(bounds)
