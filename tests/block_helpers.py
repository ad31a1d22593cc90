"""The block operators' plain counterparts for the tests: the dropout mask from
the generator's definition, in Python integers or int64 tensors."""
import torch

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85
LOW = 0xFFFFFFFF


def philox(counter, key):
    """Philox4x32-10 of Python integers (Salmon et al., SC 2011)."""
    a, b, c, d = counter
    k0, k1 = key
    for _ in range(10):
        p, q = M0 * a, M1 * c
        a, b, c, d = (q >> 32) ^ b ^ k0, q & LOW, (p >> 32) ^ d ^ k1, p & LOW
        k0, k1 = (k0 + W0) & LOW, (k1 + W1) & LOW
    return a, b, c, d


def limit(p):
    return int(p * 65536 + 0.5)


def scale(p):
    return 65536 / (65536 - limit(p)) if limit(p) < 65536 else 0.0


def keep(rows, cols, p, seed, site, step, device="cuda"):
    """Truth values rows x cols, by int64 tensors whose products wrap."""
    n = -(-cols // 8)
    unit = torch.arange(rows * n, dtype=torch.int64, device=device)
    a, b = unit & LOW, unit >> 32
    c, d = torch.full_like(unit, site), torch.full_like(unit, step & LOW)
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        x, y = a * M0, c * M1
        a, b, c, d = (y >> 32 & LOW) ^ b ^ k0, y & LOW, (x >> 32 & LOW) ^ d ^ k1, x & LOW
        k0, k1 = (k0 + W0) & LOW, (k1 + W1) & LOW
    half = torch.stack([v >> s & 0xFFFF for v in (a, b, c, d) for s in (0, 16)], 1)
    return half.reshape(rows, n * 8)[:, :cols] >= limit(p)
