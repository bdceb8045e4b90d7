"""The 4-bit cache by its definition, bit by bit, for the tests (not a test module)."""
import numpy as np
import torch

BF = torch.bfloat16
TINY = 2.0 ** -90


def quantise(x):
    """bf16 [..., d] -> (codes 0 .. 15, scales fp64 [..., d / 32], values fp64), in 64 bits."""
    x = x.double().unflatten(-1, (-1, 32))
    ok = torch.isfinite(x).all(-1, keepdim=True)
    y = torch.where(ok, x, torch.zeros_like(x))
    m = torch.where(y.amax(-1, keepdim=True) >= -y.amin(-1, keepdim=True), y.amax(-1, keepdim=True),
                    y.amin(-1, keepdim=True))
    s = torch.where(m.abs() < TINY, torch.zeros_like(m), -m / 8)
    c = torch.where(s == 0, torch.zeros_like(y), torch.round(y / torch.where(s == 0, torch.ones_like(s), s)))
    c = c.clamp(-8, 7)
    s = torch.where(ok, s, torch.full_like(s, float("nan")))
    return (c + 8).flatten(-2).to(torch.uint8), s.squeeze(-1), (s * c).flatten(-2)


def places(d):
    """(byte, bit) of each of a code's four bits from a unit's start: K and V, [4, 16, d]."""
    j, c = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    w = j // 8 * (d // 32) + c // 32
    out = []
    for v in (False, True):
        lane = (c % 32 // 4 * 4 + j % 8 // 2) if v else (j % 8 * 4 + c % 32 // 8)
        nib = (c % 4 + 4 * (j % 2)) if v else (c % 8 // 2 + 4 * (c % 2))
        at = (8 * d if v else 0) + w // 4 * 512 + lane * 16 + w % 4 * 4
        bit = np.stack([(4 * nib + i + (0 if v else 3)) % 32 for i in range(4)])
        out.append((at + bit // 8, bit % 8))
    return out


def store(cache, k, v, slot):
    """Rows into a numpy uint8 cache [pages, h, U, 18 d] (None leaves a part out)."""
    pages, h, U, b = cache.shape
    d = b // 18
    where = places(d)
    for i, r in enumerate(slot):
        if r < 0 or r >= pages * U * 16:
            continue
        page, u, j = r // (16 * U), r % (16 * U) // 16, r % 16
        for part, x in enumerate((k, v)):
            if x is None:
                continue
            code, s, _ = quantise(x[i])
            byte, bit = where[part]
            for hh in range(h):
                unit = cache[page, hh, u]
                for e in range(4):
                    np.bitwise_and.at(unit, byte[e, j], (~(1 << bit[e, j])).astype(np.uint8))
                    np.bitwise_or.at(unit, byte[e, j], ((code[hh].numpy() >> e & 1) << bit[e, j]).astype(np.uint8))
                at = 16 * d + (j * (d // 16) + part * (d // 32)) * 2
                unit[at:at + d // 16] = s[hh].to(BF).view(torch.uint8).numpy()


def load(cache, rows):
    """K and V values fp64 [n, h, d] of cache rows (a torch uint8 cache)."""
    pages, h, U, b = cache.shape
    d = b // 18
    c = cache.cpu().numpy()
    rows = np.asarray(rows)
    page, u, j = rows // (16 * U), rows % (16 * U) // 16, rows % 16
    units = c[page, :, u]                                                   # [n, h, 18 d]
    out = []
    for part, (byte, bit) in enumerate(places(d)):
        code = 0
        for e in range(4):
            got = np.take_along_axis(units, np.broadcast_to(byte[e][j][:, None], (len(rows), h, d)), 2)
            code = code + ((got >> bit[e][j][:, None]) & 1).astype(np.int64) * 2 ** e
        at = 16 * d + (j[:, None] * (d // 16) + part * (d // 32)) * 2 + np.arange(d // 16)
        sc = np.take_along_axis(units, np.broadcast_to(at[:, None], (len(rows), h, d // 16)), 2)
        sc = torch.from_numpy(np.ascontiguousarray(sc)).view(BF).double()   # [n, h, d / 32]
        val = torch.from_numpy(code - 8).double().unflatten(-1, (-1, 32)) * sc[..., None]
        out.append(val.flatten(-2))
    return out
