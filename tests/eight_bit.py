"""Float64 forms of the 8-bit decode-step operators, for their tests (CPU torch)."""

import math

import torch

FP8 = torch.float8_e4m3fn


def rms_norm(x, w, eps, residual=None):
    """(h, y, scale) with h rounded to x's dtype as the operator defines it."""
    h = x.cpu()
    if residual is not None:
        h = (x.cpu().double() + residual.cpu().double()).to(x.dtype)
    hd = h.double()
    y = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + eps) * w.cpu().double()
    return h, y, y.abs().amax(1) / 127


def pow2_scale(v):
    """The smallest power of two s >= 2^-126 with v <= 448 s (0 for 0)."""
    if v == 0:
        return 0.0
    e = -126
    while v > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def to_codes(x):
    """e4m3 codes of float64 values: nearest even, infinities to +-448, NaN kept. The
    values of the tests are exact in float32, so torch's own rounding is the only one."""
    return x.clamp(-448, 448).float().to(FP8)


def kv_append(codes, scales, new, table, start, count=None, rows=None):
    """The append of one of k / v on CPU clones; returns (codes, scales)."""
    codes, scales = codes.cpu().clone(), scales.cpu().clone()
    new, table = new.cpu().double(), table.cpu().tolist()
    P, page = codes.shape[0], codes.shape[2]
    B, T = new.shape[:2]
    n = T if rows is None else rows.shape[1]
    nan = torch.full(new.shape[2:], math.nan, dtype=torch.float64)
    for b in range(B):
        s0 = int(start[b])
        c = n if count is None else max(0, min(n, int(count[b])))
        if s0 < 0 or s0 > len(table[b]) * page:
            continue
        by_page = {}
        for j in range(c):
            r = j if rows is None else int(rows[b, j])
            by_page.setdefault((s0 + j) // page, []).append(
                ((s0 + j) % page, new[b, r] if 0 <= r < T else nan))
        for p, toks in by_page.items():
            if p >= len(table[b]) or not 0 <= table[b][p] < P:
                continue
            pid, first = table[b][p], toks[0][0]
            for h in range(codes.shape[1]):
                vals = torch.stack([t[1][h] for t in toks])
                fin = vals[torch.isfinite(vals)].abs()
                old = float(scales[pid, h]) if first > 0 else 0.0
                now = max(old, pow2_scale(float(fin.max()) if fin.numel() else 0.0))
                if now > old:
                    kept = codes[pid, h, :first].double() * (old / now)
                    codes[pid, h, :first] = to_codes(kept)
                for slot, v in toks:
                    codes[pid, h, slot] = to_codes(v[h] / (now if now > 0 else 1.0))
                scales[pid, h] = now
    return codes, scales


def same_codes(a, b):
    """Equal bytes, all NaN codes alike."""
    a, b = a.cpu(), b.cpu()
    na, nb = torch.isnan(a.float()), torch.isnan(b.float())
    return torch.equal(na, nb) and torch.equal(a.view(torch.uint8)[~na], b.view(torch.uint8)[~nb])
