"""Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) in whole-number torch
arithmetic, and dropout's mask from it: what the library's masks are checked with."""
import math

import torch

LOW = 0xFFFFFFFF


def philox(counter, key):
    """The four 32-bit words (int64 tensors) of a counter of four and a key of two."""
    c0, c1, c2, c3 = counter
    k0, k1 = key
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64 bits, wrapping
        c0, c1, c2, c3 = (b >> 32 & LOW) ^ c1 ^ k0, b & LOW, (a >> 32 & LOW) ^ c3 ^ k1, a & LOW
        k0, k1 = k0 + 0x9E3779B9 & LOW, k1 + 0xBB67AE85 & LOW
    return c0, c1, c2, c3


def keep_mask(T, d, p, seed, step, site, device="cuda"):
    """[T, d] truth values: kept."""
    c = torch.arange(-(-d // 8), dtype=torch.int64, device=device).expand(T, -1)
    r = torch.arange(T, dtype=torch.int64, device=device)[:, None].expand_as(c)
    words = philox((c, r, torch.full_like(c, site), torch.full_like(c, step & LOW)),
                   (seed & LOW, seed >> 32 & LOW))
    numbers = torch.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], 2)
    return numbers.reshape(T, -1)[:, :d] >= math.floor(p * 65536 + 0.5)


def factor(T, d, p, seed, step, site, device="cuda"):
    """The same as factors 0 and 1 / (1 - p), p in steps of 2^-16, in 64 bits."""
    t = math.floor(p * 65536 + 0.5)
    if t == 0:
        return torch.ones(T, d, dtype=torch.float64, device=device)
    scale = 65536 / (65536 - t) if t < 65536 else 0.0
    return keep_mask(T, d, p, seed, step, site, device).double() * scale
