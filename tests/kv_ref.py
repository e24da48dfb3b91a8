"""Plain 64-bit forms of the 4-bit cache's operations (test infrastructure): the
quantiser, the pool's byte layout place by place, attention, and the page operations
as loops over Python lists."""
import math

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(x):
    """float array [..., dim] -> codes [..., dim], scale bytes [..., dim / 32]: the smallest
    power of two for which no element exceeds 6; the nearest level, a tie to the even code."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    fine = np.isfinite(top)
    byte = np.zeros(top.shape, np.int64)
    pos = fine & (top > 0)
    e = np.ceil(np.log2(np.where(pos, top, 1.0) / 6))
    e = np.where(np.where(pos, top, 1.0) > 6 * 2.0 ** e, e + 1, e)       # guards log2's rounding
    e = np.where(np.where(pos, top, 1.0) <= 6 * 2.0 ** (e - 1), e - 1, e)
    byte[pos] = np.clip(e[pos] + 127, 1, 254).astype(np.int64)
    byte[~fine] = 255
    y = np.where((pos)[..., None], np.abs(np.where(np.isfinite(b), b, 0)), 0) * 2.0 ** (127.0 - byte)[..., None]
    d = np.abs(y[..., None] - LEVELS)
    near = d.min(-1, keepdims=True)
    odd = np.arange(8) % 2
    code = np.where(d == near, odd, 9).argmin(-1)  # among the nearest levels the even code
    code = np.where((byte == 0)[..., None] | (byte == 255)[..., None], 0, code + 8 * np.signbit(b))
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def values(codes, byte):
    """codes and scale bytes -> float64 (NaN where the byte is 255)."""
    v = np.where(codes & 8, -1.0, 1.0) * LEVELS[codes & 7]
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return (v.reshape(*byte.shape, 32) * s[..., None]).reshape(codes.shape)


def stored(x):
    return values(*quantise(x))


def unit_bytes(kc, ks, vc, vs):
    """The 17 dim bytes of one unit from its [16, dim] codes and [16, dim / 32] scale bytes."""
    dim = kc.shape[1]
    nb, out = dim // 32, np.zeros(17 * dim, np.uint8)
    for t in range(16):
        for d in range(dim):
            i, lane = 2 * (d // 32) + t // 8, (t % 8) * 4 + d % 32 // 8
            out[(i // 4) * 512 + lane * 16 + (i % 4) * 4 + d % 8 // 2] |= kc[t, d] << (4 * (d % 2))
            i, lane = d // 16, (d % 8) * 4 + t % 8 // 2
            out[8 * dim + (i // 4) * 512 + lane * 16 + (i % 4) * 4 + d % 16 // 8 + 2 * (t // 8)] |= vc[t, d] << (4 * (t % 2))
        for b in range(nb):
            out[16 * dim + t * nb + b] = ks[t, b]
            out[16 * dim + dim // 2 + ((t % 8 // 2 * nb + b) * 2 + t // 8) * 2 + t % 2] = vs[t, b]
    return out


class Attended:
    """attend(): outputs, log-sums and what their error bounds are made of."""


def attend(q, k, v, first, scale=None, window=0, sinks=0):
    """One sequence: q [m, heads, dim] at positions first.., k and v [tokens, kv heads, dim]
    (float64 tensors).  Returns out, lse, and per element sum p |v| and the largest
    scale * sum |q k| (the accumulation's magnitude)."""
    m, heads, dim = q.shape
    n, kvh = k.shape[0], k.shape[1]
    scale = dim ** -0.5 if scale is None else scale
    r = Attended()
    r.out, r.mag = torch.zeros_like(q), torch.zeros_like(q)
    r.lse = torch.full((m, heads), -math.inf, dtype=torch.float64, device=q.device)
    r.acc = torch.zeros((m, heads), dtype=torch.float64, device=q.device)
    pos = torch.arange(first, first + m, device=q.device)[:, None]
    t = torch.arange(n, device=q.device)[None]
    see = t <= pos
    if window:
        see &= (t > pos - window) | (t < sinks)
    r.vmax = float(torch.nan_to_num(v).abs().max()) if n else 0.0
    for h in range(heads):
        kh, vh = k[:, h // (heads // kvh)], v[:, h // (heads // kvh)]
        s = (q[:, h] @ kh.T * scale).masked_fill(~see, -math.inf) if n else torch.zeros((m, 0), dtype=q.dtype, device=q.device)
        if not n:
            continue
        top = s.amax(-1, keepdim=True)
        top = torch.where(torch.isneginf(top), torch.zeros_like(top), top)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        w = torch.where(total == 0, torch.zeros_like(p), p / total)
        # a token that a row does not see adds nothing, whatever it holds
        live = see & (w != 0) | torch.isnan(w)
        for c in range(0, m, 64):
            wc = torch.where(live[c:c + 64], w[c:c + 64], torch.zeros_like(w[c:c + 64]))
            if torch.isnan(vh).any():
                r.out[c:c + 64, h] = torch.einsum("mt,mtd->md", wc, torch.where(live[c:c + 64, :, None], vh[None], torch.zeros_like(vh[None])))
            else:
                r.out[c:c + 64, h] = wc @ vh
            r.mag[c:c + 64, h] = torch.nan_to_num(wc) @ torch.nan_to_num(vh).abs()
        r.lse[:, h] = torch.where(total[:, 0] == 0, torch.full_like(total[:, 0], -math.inf), top[:, 0] + torch.log(total[:, 0]))
        r.acc[:, h] = (q[:, h].abs() @ torch.nan_to_num(kh).abs().T * scale).masked_fill(~see, 0).amax(-1)
    return r


def bounds(r, n, out_type, q_terms_error=0.0):
    """Largest errors of out and lse, derived from the kernels' roundings:
    scores: FP32 accumulation of exact products, dim <= 256 of them in steps of at most 16
      with a last place of 2^-23 of the running magnitude each way: 2^-19 * acc covers it
      (and q_terms_error * acc where q itself is rounded);
    weights: FP16 (2^-11 relative), the exponential 2^-21; below 2^-30 of the largest a
      weight may vanish, and a value whose scale is below 2^-14 of its block's largest;
    output: one rounding to its type."""
    eps_s = r.acc * (2.0 ** -19 + q_terms_error) + 2.0 ** -20
    eps_out = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -22}[out_type]
    out = r.mag * (2.0 ** -11 + 2 * eps_s[..., None] + 2.0 ** -19) + (n * 2.0 ** -29 + 2.0 ** -14) * r.vmax + r.out.abs() * eps_out
    lse = eps_s + 2.0 ** -21 * r.lse.abs().nan_to_num(posinf=0, neginf=0) + 2.0 ** -20
    return out, lse


def fork(page, n_pages, table, lens, refs, parents, grow, width):
    """The page rules as loops: new table, lens, refs and (source, destination, units) copies."""
    refs = list(refs)
    first = {}
    for i, p in enumerate(parents):
        if p >= 0 and p not in first:
            first[p] = i
    for s, n in enumerate(lens):
        if s not in first:
            for k in range(-(-max(n, 0) // page)):
                refs[table[s][k]] -= 1
    rows, want, copies = [], [], []
    for i, p in enumerate(parents):
        n = max(lens[p], 0) if p >= 0 else 0
        whole, rest = divmod(n, page)
        kept = list(table[p][:whole + (1 if rest and first[p] == i else 0)]) if p >= 0 else []
        if p >= 0 and first[p] != i:
            for x in kept:
                refs[x] += 1
        need = -(-(n + grow[i]) // page) if p >= 0 else 0
        rows.append(kept)
        want.append(need - len(kept) if need <= width else None)
    free = [x for x in range(n_pages) if refs[x] == 0]
    at, out_lens, dropped = 0, [], []
    for i, p in enumerate(parents):
        n = max(lens[p], 0) if p >= 0 else 0
        w = want[i]
        if w is None or (w and at + w > len(free)):
            at += w or 0
            out_lens.append(-1)
            dropped += rows[i]
            rows[i] = []
            continue
        new = free[at:at + w]
        at += w
        if p >= 0 and n % page and first[p] != i:
            copies.append((table[p][n // page], new[0], -(-(n % page) // 16)))
        for x in new:
            refs[x] = 1
        rows[i] = rows[i] + new
        out_lens.append(n + grow[i] if p >= 0 else 0)
    for x in dropped:
        refs[x] -= 1
    return [r + [-1] * (width - len(r)) for r in rows], out_lens, refs, copies


def compact(table, refs):
    live = [p for p, r in enumerate(refs) if r > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    to = {p: p for p in live if p < n}
    moves = list(zip([p for p in live if p >= n], holes))
    to.update(moves)
    out = [[to.get(p, -1) if 0 <= p < len(refs) else p for p in row] for row in table]
    new_refs = [0] * len(refs)
    for p in live:
        new_refs[to[p]] = refs[p]
    return out, new_refs, [to.get(p, -1) for p in range(len(refs))], moves
