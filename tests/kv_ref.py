"""Plain implementations of the paged-cache operators, on the CPU in whole
numbers and 64-bit floats, and how far the kernels may be from them."""
import math

import numpy as np
import torch

# largest relative error of one rounding to nearest
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def pages_of(n, page):
    return -(-n // page)


def grow(lengths, n_new, page, free, cursor, table, n_tokens):
    """(table, lengths, cursor, token_ptr, slots, positions, status) after a growth."""
    R, width = table.shape
    table = table.copy()
    cursor = min(max(cursor, 0), len(free))
    bad = [r for r in range(R)
           if lengths[r] < 0 or n_new[r] < 0 or lengths[r] + n_new[r] > width * page]
    new = [0 if r in bad else n_new[r] for r in range(R)]
    ptr = [0]
    for r in range(R):
        ptr.append(ptr[-1] + new[r])
    slots, positions = [-1] * n_tokens, [-1] * n_tokens
    need = [0 if r in bad else pages_of(lengths[r] + new[r], page) - pages_of(lengths[r], page)
            for r in range(R)]
    status = (0, 0)
    if bad:
        status = (2, bad[0])
    elif ptr[-1] > n_tokens:
        status = (3, ptr[-1])
    elif sum(need) > len(free) - cursor:
        status = (1, sum(need) - (len(free) - cursor))
    if status[0]:
        return table, list(lengths), cursor, ptr, slots, positions, status
    for r in range(R):
        held = pages_of(lengths[r], page)
        for j in range(need[r]):
            table[r, held + j] = free[cursor]
            cursor += 1
        for i in range(new[r]):
            pos = lengths[r] + i
            positions[ptr[r] + i] = pos
            slot = int(table[r, pos // page]) * page + pos % page
            slots[ptr[r] + i] = slot if 0 <= slot < 2 ** 31 else -1
    return (table, [a + b for a, b in zip(lengths, new)], cursor, ptr, slots, positions, status)


def shrink(lengths, keep, page, free, cursor, table):
    """(free, lengths, cursor, status) after pages went back."""
    R, width = table.shape
    free = list(free)
    cursor = min(max(cursor, 0), len(free))
    bad = [r for r in range(R)
           if keep[r] < 0 or keep[r] > lengths[r] or lengths[r] > width * page]
    gone = [0 if r in bad else pages_of(lengths[r], page) - pages_of(keep[r], page)
            for r in range(R)]
    if bad:
        return free, list(lengths), cursor, (2, bad[0])
    if sum(gone) > cursor:
        return free, list(lengths), cursor, (1, sum(gone) - cursor)
    at = cursor - sum(gone)
    for r in range(R):
        for j in range(gone[r]):
            free[at] = int(table[r, pages_of(keep[r], page) + j])
            at += 1
    return free, list(keep), cursor - sum(gone), (0, 0)


def e4m3_values():
    """The 127 finite non-negative values of the 8-bit type, by their bits."""
    out = []
    for b in range(127):
        e, m = b >> 3, b & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def to_e4m3(x):
    """uint8 codes of float32 x: nearest, ties to the even code, saturating, NaN 0x7f."""
    x = np.asarray(x, dtype=np.float32)
    vals = e4m3_values()
    a = np.minimum(np.abs(x.astype(np.float64)), 448.0)
    a = np.where(np.isnan(a), 0.0, a)
    hi = np.searchsorted(vals, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - vals[lo], vals[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(vals[hi] == a, hi, code).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), (code & 0x80) | 0x7f, code).astype(np.uint8)


def visible(n, window, sinks):
    return [t for t in range(n) if not window or t >= n - window or t < sinks]


def attend(q, k, v, table, lengths, scale, window=0, sinks=0, k_scale=None, v_scale=None):
    """out, lse and the bounds of their errors, all float64; q [R, Hq, D], k and v
    [pages, page, H, D], table and lengths whole numbers, all on the CPU."""
    R, Hq, D = q.shape
    n_pages, P, H, _ = k.shape
    G = Hq // H
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    lse_tol = torch.zeros_like(lse)
    width = table.shape[1]
    # rounding of the weights before the second product: 16-bit types carry them in two
    # parts; an 8-bit cache's in one of 11 bits when the output has no more than 8
    u_p = {torch.float32: 2.0 ** -23}.get(k.dtype, 2.0 ** -16)
    if k.dtype == torch.float8_e4m3fn and q.dtype == torch.bfloat16:
        u_p = 2.0 ** -11
    tiny = 0.0 if k.dtype == torch.float32 else 2.0 ** -24     # weights below 16-bit range
    for r in range(R):
        n = min(max(int(lengths[r]), 0), width * P)
        see = [t for t in visible(n, window, sinks) if 0 <= int(table[r, t // P]) < n_pages]
        if not see:
            continue
        t = torch.tensor(see)
        page = table[r].long()[t // P]
        raw_k = (k.view(torch.uint8) if k.dtype == torch.float8_e4m3fn else k)[page, t % P]
        raw_v = (v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v)[page, t % P]
        kk = raw_k.contiguous().view(k.dtype).double()
        vv = raw_v.contiguous().view(v.dtype).double()
        if k_scale is not None:
            kk = kk * k_scale.double()[None, :, None]
        if v_scale is not None:
            vv = vv * v_scale.double()[None, :, None]
        for h in range(Hq):
            kh, vh, qh = kk[:, h // G], vv[:, h // G], q[r, h].double()
            s = scale * (kh @ qh)
            size = abs(scale) * float((kh.abs() @ qh.abs()).max())
            m = s.max()
            p = torch.exp(s - m)
            total = p.sum()
            out[r, h] = (p @ vh) / total
            lse[r, h] = m + torch.log(total)
            # scores: D products and sums in 32 bits, then scaled, the maximum taken off and
            # raised; sums over tokens in blocks of at least 32
            eps = 2 * (D + 16) * 2.0 ** -24 * size + (len(see) / 32 + 96) * 2.0 ** -24
            spread = (p @ vh.abs()) / total
            tol[r, h] = (ROUND[q.dtype] * out[r, h].abs() + (2 * eps + u_p) * spread
                         + tiny * vh.abs().sum(0) / total)
            if q.dtype == torch.float16:
                tol[r, h] += 2.0 ** -25       # results below 16-bit range
            lse_tol[r, h] = eps + 2.0 ** -22 * (abs(float(lse[r, h])) + abs(float(m)))
    return out, lse, tol, lse_tol


def worst(got, ref, tol):
    """Largest error in units of its bound; infinities and NaN have to agree."""
    got, ref = got.double().cpu(), ref.double()
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    err = torch.where(same, 0.0, (got - ref).abs() / tol.clamp(min=1e-300))
    err = torch.where(torch.isnan(err), math.inf, err)
    return float(err.max()) if err.numel() else 0.0
