"""Operators of a paged key/value cache held in 4 bits: what is measured of them.

The cache stores keys and values as microscaled 4-bit floating point: blocks of 32
channels of one token and head share a power-of-two scale (E8M0 byte, value
2^(byte - 127)), elements are E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives).
The scale is the smallest power of two for which no element exceeds 6; elements are
rounded to nearest, ties to the even code.  Pages of `page` tokens hold all layers;
sequences reach their pages through a table.

  append   new keys and values are quantised into the cache's pages (and read back:
           what is held in 4 bits is returned as the values it stands for)
  attend   attention of the sequences' newest tokens over the cache: grouped query
           heads, causal, optionally a sliding window with a few first tokens that
           stay visible
  fork     sequences continue others (beams, drafts, samples): whole pages are shared,
           a partly filled page is copied, room for new tokens is taken from the free
           pages, pages that nobody holds any longer become free
  compact  the pages in use move to the lowest numbers

A pool is a uint8 tensor [pages, layers, heads, page / 16, 17 * dim]: a unit of 16
tokens of one head is 8 * dim bytes of key codes, 8 * dim of value codes, dim / 2 of
key scales and dim / 2 of value scales; _pack and _unpack give the order inside each.
"""
import random

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- the cases
def listed():
    # q heads / kv heads / dim of 32 / 8 / 128 and 64 / 8 / 128: the k and v projections of this
    # repository's two layer shapes have 1024 rows, their q projections 4096 and 8192
    return [
        # a conversation's first answer token: latency of a call is all there is
        {"name": "attend_first", "op": "attend", "seqs": 1, "lo": 17, "hi": 17, "new_lo": 1, "new_hi": 1, "qh": 32,
         "kvh": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0, "type": "bf16", "out": "bf16", "mix": 1},
        # one step of a full serving batch with conversations of all lengths; queries as the GEMV leaves them
        {"name": "attend_batch", "op": "attend", "seqs": 64, "lo": 1, "hi": 8192, "new_lo": 1, "new_hi": 1, "qh": 32,
         "kvh": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0, "type": "fp32", "out": "bf16", "mix": 2},
        # one token over a book-length context
        {"name": "attend_long", "op": "attend", "seqs": 1, "lo": 400003, "hi": 400003, "new_lo": 1, "new_hi": 1,
         "qh": 32, "kvh": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0, "type": "bf16", "out": "bf16", "mix": 3},
        # drafted tokens checked together, in long streams that keep a window and the first tokens
        {"name": "attend_drafts", "op": "attend", "seqs": 16, "lo": 9000, "hi": 40000, "new_lo": 1, "new_hi": 5,
         "qh": 64, "kvh": 8, "dim": 128, "page": 32, "window": 4096, "sinks": 4, "type": "fp16", "out": "fp16",
         "mix": 4},
        # a small model without shared heads, short pages
        {"name": "attend_unshared", "op": "attend", "seqs": 32, "lo": 1, "hi": 2500, "new_lo": 1, "new_hi": 1,
         "qh": 16, "kvh": 16, "dim": 64, "page": 16, "window": 0, "sinks": 0, "type": "fp16", "out": "fp16", "mix": 5},
        # chunks of two long prompts over what is cached of them
        {"name": "attend_prompt", "op": "attend", "seqs": 2, "lo": 7001, "hi": 13000, "new_lo": 2999, "new_hi": 5003,
         "qh": 32, "kvh": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0, "type": "bf16", "out": "bf16", "mix": 6},
        # one step's keys and values of a full batch, as the GEMV leaves them
        {"name": "append_step", "op": "append", "seqs": 64, "lo": 1, "hi": 8192, "new_lo": 1, "new_hi": 1, "kvh": 8,
         "dim": 128, "page": 64, "type": "fp32", "mix": 7},
        # whole prompts
        {"name": "append_prompts", "op": "append", "seqs": 5, "lo": 6001, "hi": 20000, "new_lo": 2001, "new_hi": 6000,
         "kvh": 8, "dim": 128, "page": 64, "type": "bf16", "mix": 8},
        # a step of beam search: eight beams take new parents
        {"name": "fork_beams", "op": "fork", "seqs": 8, "to": 8, "lo": 700, "hi": 1200, "grow": 1, "layers": 32,
         "kvh": 8, "dim": 128, "page": 64, "spare": 24, "mix": 9},
        # many samples from a few prompts
        {"name": "fork_samples", "op": "fork", "seqs": 6, "to": 64, "lo": 1001, "hi": 3000, "grow": 70, "layers": 32,
         "kvh": 8, "dim": 128, "page": 64, "spare": 150, "mix": 10},
        # the holes that a few ended conversations left
        {"name": "compact_small", "op": "compact", "seqs": 5, "lo": 100, "hi": 600, "layers": 4, "kvh": 8, "dim": 128,
         "page": 32, "free": 0.2, "mix": 11},
        # a pool that was mostly freed
        {"name": "compact_large", "op": "compact", "seqs": 24, "lo": 100, "hi": 1500, "layers": 32, "kvh": 8,
         "dim": 128, "page": 64, "free": 0.5, "mix": 12},
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(a * (b / a) ** rng.random()))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "append", "fork", "compact"))
    c = {"op": op, "mix": rng.randrange(1 << 20), "page": rng.choice((16, 32, 64, 128))}
    heads = rng.choice(((32, 8, 128), (64, 8, 128), (16, 16, 64), (24, 8, 64), (8, 1, 128), (12, 4, 192), (16, 2, 256)))
    if op == "attend":
        c.update(zip(("qh", "kvh", "dim"), heads))
        c["type"] = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        c["out"] = "fp16" if c["type"] == "fp16" else "bf16"
        kind = rng.choice(("step", "step", "drafts", "prompt"))
        if kind == "prompt":
            c["seqs"] = rng.randint(1, 3)
            c["new_hi"] = _log(rng, 40, 3000 // c["seqs"])
            c["new_lo"] = rng.randint(1, c["new_hi"])
            c["hi"] = _log(rng, c["new_hi"], 9000)
        else:
            c["seqs"] = _log(rng, 1, 64)
            c["new_lo"], c["new_hi"] = 1, 1 if kind == "step" else rng.randint(2, 9)
            c["hi"] = _log(rng, 16, min(200000, 250000 // c["seqs"]))
        c["lo"] = rng.choice((1, max(1, c["hi"] // 2), c["hi"]))
        c["window"] = rng.choice((0, 0, 128, _log(rng, 16, 8000)))
        c["sinks"] = rng.choice((0, 1, 4, 20)) if c["window"] else 0
    elif op == "append":
        c.update(zip(("kvh", "dim"), heads[1:]))
        c["type"] = rng.choice(("bf16", "fp16", "fp32"))
        c["seqs"] = _log(rng, 1, 64)
        c["new_hi"] = rng.choice((1, _log(rng, 1, 24000 // c["seqs"])))
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["hi"] = c["new_hi"] + _log(rng, 1, 4000)
        c["lo"] = rng.randint(1, c["hi"])
    else:
        c.update(zip(("kvh", "dim"), rng.choice(((8, 128), (8, 64), (4, 192), (1, 256)))))
        c["layers"] = _log(rng, 1, 32)
        c["seqs"] = _log(rng, 1, 20)
        c["hi"] = _log(rng, 5, 1500)
        c["lo"] = rng.randint(1, c["hi"])
        if op == "fork":
            c["to"] = _log(rng, 1, 48)
            c["grow"] = rng.choice((0, 1, rng.randint(1, 60)))
            c["spare"] = c["to"] * (1 + -(-c["grow"] // c["page"]))
        else:
            c["free"] = rng.choice((0.05, 0.3, 0.6))
    return c


def _lens(case):
    """Tokens in the cache after the new ones, and new tokens, of each sequence (from the case alone)."""
    r = random.Random(case["mix"])
    lens = [_log(r, case["lo"], case["hi"]) for _ in range(case["seqs"])]
    new = [min(n, r.randint(case.get("new_lo", 1), case.get("new_hi", 1))) for n in lens]
    return lens, new


def _unit(case):
    return 17 * case["dim"]


# ---------------------------------------------------------------- the pool's bytes
def _unpack(units, dim):
    """[..., 17 dim] bytes -> key codes, key scales, value codes, value scales ([..., 16, dim], [..., 16, dim / 32])."""
    lead, half, nb = units.shape[:-1], 8 * dim, dim // 32

    def codes(x):
        return torch.stack((x & 15, x >> 4), -1)

    def order(x, shape, perm, out):
        n = len(lead)
        return x.reshape(*lead, *shape).permute(*range(n), *(n + p for p in perm)).reshape(*lead, *out)

    # key codes: [dim / 64][token % 8][channel / 8 % 4][channel / 32 % 2][token / 8][channel / 2 % 4], low nibble first
    k = order(codes(units[..., :half]), (dim // 64, 8, 4, 2, 2, 4, 2), (4, 1, 0, 3, 2, 5, 6), (16, dim))
    # value codes: [dim / 64][channel % 8][token / 2 % 4][channel / 16 % 4][token / 8][channel / 8 % 2], even token low
    v = order(codes(units[..., half:2 * half]), (dim // 64, 8, 4, 4, 2, 2, 2), (4, 2, 6, 0, 3, 5, 1), (16, dim))
    ks = units[..., 2 * half:2 * half + dim // 2].reshape(*lead, 16, nb)
    # value scales: [token / 2 % 4][channel / 32][token / 8][token % 2]
    vs = order(units[..., 2 * half + dim // 2:], (4, nb, 2, 2), (2, 0, 3, 1), (16, nb))
    return k, ks, v, vs


def _pack(k, ks, v, vs):
    """The inverse of _unpack."""
    lead, dim, nb = k.shape[:-2], k.shape[-1], ks.shape[-1]
    n = len(lead)

    def order(x, shape, perm):
        return x.reshape(*lead, *shape).permute(*range(n), *(n + p for p in perm))

    def join(x):
        return (x[..., 0] | (x[..., 1] << 4)).reshape(*lead, 8 * dim)

    kc = join(order(k, (2, 8, dim // 64, 2, 4, 4, 2), (2, 1, 4, 3, 0, 5, 6)))
    vc = join(order(v, (2, 4, 2, dim // 64, 4, 2, 8), (3, 6, 1, 4, 0, 5, 2)))
    vb = order(vs, (2, 4, 2, nb), (1, 3, 0, 2)).reshape(*lead, 16 * nb)
    return torch.cat((kc, vc, ks.reshape(*lead, 16 * nb), vb), -1)


def _quantise(x):
    """float [..., dim] -> E2M1 codes [..., dim] and E8M0 bytes [..., dim / 32] (uint8)."""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1)
    m, e = torch.frexp(top)
    byte = torch.where(m <= 0.75, e + 124, e + 125).clamp(1, 254)  # top = m 2^e <= 6 * 2^(byte - 127)
    byte = torch.where(top == 0, torch.zeros_like(byte), byte)
    byte = torch.where(torch.isfinite(top), byte, torch.full_like(byte, 255))
    y = torch.ldexp(b.abs(), (127 - byte)[..., None])
    # the midpoints between neighbouring levels; a tie goes to the even code
    code = ((y > 0.25).byte() + (y >= 0.75).byte() + (y > 1.25).byte() + (y >= 1.75).byte() + (y > 2.5).byte()
            + (y >= 3.5).byte() + (y > 5.0).byte())
    code = torch.where(((byte == 0) | (byte == 255))[..., None], torch.zeros_like(code), code | (torch.signbit(b).byte() << 3))
    return code.reshape(x.shape), byte.to(torch.uint8)


def _values(codes, scales):
    """E2M1 codes and E8M0 bytes -> float32 values."""
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float32, device=codes.device)
    # (2^-127 and a scale of 255, neither of which the quantiser gives to a finite block, are left out)
    s = torch.exp2(scales.float() - 127.0)
    return (lut[codes.int()].reshape(*scales.shape, 32) * s[..., None]).reshape(codes.shape)


# ---------------------------------------------------------------- what a program has in hand
def _cuda(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _starts(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def _pages(case, lens, seed, more=0):
    """Pages of each sequence in a shuffled pool: a host table with -1 past the end, and the pool's page count."""
    need = [-(-n // case["page"]) for n in lens]
    total = sum(need) + more
    ids = list(range(total))
    random.Random(seed).shuffle(ids)
    width, at, table = max(need) + 1, 0, []
    for n in need:
        table.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    return table, total, ids[at:]


def _tensors(case, seed):
    """Keys and values [tokens of all sequences, heads, dim], with louder channels and quiet first values, and queries."""
    lens, new = _lens(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n, h, d, t = sum(lens), case["kvh"], case["dim"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    loud = torch.exp(0.5 * normal(h, d))
    k = (normal(n, h, d) * loud).to(t)
    v = normal(n, h, d)
    first = _cuda(_starts(lens)[:-1], torch.int64)
    v[first] *= 0.02
    q = None
    if "qh" in case:
        # scores of a standard deviation of about 2 after the 1 / sqrt(dim)
        q = (normal(sum(new), h, case["qh"] // h, d) * (2.0 / loud[:, None])).reshape(sum(new), case["qh"], d).to(t)
    return k, v.to(t), q


def _fill(case, pool, table, lens, k, v):
    """Quantised keys and values of whole sequences into layer 0 of the pool."""
    page, h, d = case["page"], case["kvh"], case["dim"]
    where = []  # row of each pool token; unfilled places take a row of zeros
    n = sum(lens)
    starts = _starts(lens)
    ids = [p for row in table for p in row if p >= 0]
    for i, row in enumerate(table):
        held = sum(p >= 0 for p in row)
        where += list(range(starts[i], starts[i] + lens[i])) + [n] * (held * page - lens[i])
    at = _cuda(where, torch.int64)

    def laid(x):
        c, s = _quantise(x)
        c, s = (torch.cat((y, torch.zeros_like(y[:1])))[at].reshape(len(ids), page // 16, 16, h, -1) for y in (c, s))
        return c.transpose(2, 3).transpose(1, 2), s.transpose(2, 3).transpose(1, 2)  # [pages, heads, units, 16, .]

    pool[_cuda(ids, torch.int64), 0] = _pack(*laid(k), *laid(v))


def prepare(case, seed):
    op = case["op"]
    s = {"case": case}
    if op in ("attend", "append"):
        lens, new = _lens(case)
        table, total, _ = _pages(case, lens, seed)
        layers = 1
        s["pool"] = torch.zeros(total, 1, case["kvh"], case["page"] // 16, _unit(case), dtype=torch.uint8, device="cuda")
        k, v, q = _tensors(case, seed)
        s["table"], s["lens"], s["starts"] = _cuda(table), _cuda(lens), _cuda(_starts(new))
        s["max_new"], s["max_len"], s["rows"] = max(new), max(lens), sum(new)
        if op == "attend":
            _fill(case, s["pool"], table, lens, k, v)
            s["q"] = q
            s["out"] = torch.empty(q.shape, dtype=TYPES[case["out"]], device="cuda")
            s["lse"] = torch.empty(q.shape[:2], device="cuda")
        else:
            # the new tokens are each sequence's last; what was there before is zeros here
            ends = _starts(lens)
            rows = _cuda([ends[i + 1] - new[i] + j for i in range(len(lens)) for j in range(new[i])], torch.int64)
            s["k"], s["v"] = k[rows], v[rows]
            s["k_out"] = torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda")
            s["v_out"] = torch.empty_like(s["k_out"])
    else:
        layers = case["layers"]
        lens, _ = _lens(case)
        r = random.Random(seed + 1)
        if op == "fork":
            table, total, _ = _pages(case, lens, seed, case["spare"])
            parents, grow = _family(case)
            width = max(len(table[0]), max(-(-(lens[p] + g) // case["page"]) for p, g in zip(parents, grow) if p >= 0) if max(parents) >= 0 else 1)
            table = [row + [-1] * (width - len(row)) for row in table]
            refs = [0] * total
            s["parents"], s["grow"] = _cuda(parents), _cuda(grow)
            out = (case["to"], width)
        else:
            held = sum(-(-n // case["page"]) for n in lens)
            table, total, _ = _pages(case, lens, seed, int(held * case["free"] / (1 - case["free"])) + 1)
            # a few sequences share their first pages
            for i in range(1, len(table), 3):
                n = min(sum(p >= 0 for p in table[i]), sum(p >= 0 for p in table[i - 1])) // 2
                table[i][:n] = table[i - 1][:n]
            refs = [0] * total
            out = (len(table), len(table[0]))
        for row in table:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        s["table"], s["lens"], s["refs"] = _cuda(table), _cuda(lens), _cuda(refs)
        s["table_out"] = torch.empty(out, dtype=torch.int32, device="cuda")
        s["lens_out"], s["refs_out"] = torch.empty(out[0], dtype=torch.int32, device="cuda"), torch.empty_like(s["refs"])
        s["map"] = torch.empty_like(s["refs"])
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        s["pool"] = torch.randint(0, 256, (total, layers, case["kvh"], case["page"] // 16, _unit(case)), generator=g,
                                  dtype=torch.uint8, device="cuda")
    if own:
        import lossless_entropy_coded_gb300 as ec
        s["cache"] = ec.kv_cache(layers, s["pool"].shape[0], case["kvh"], case["dim"], case["page"], pool=s["pool"])
        s["seqs"] = ec.kv_seqs(s["table"], s["lens"])
        if op == "attend":
            s["work"] = torch.empty(ec.kv_attend_work_bytes(s["cache"], case["seqs"], s["rows"], case["qh"], s["max_new"],
                                                            s["max_len"], window=case["window"], sinks=case["sinks"]),
                                    dtype=torch.uint8, device="cuda")
        elif op in ("fork", "compact"):
            s["seqs_out"] = ec.kv_seqs(s["table_out"], s["lens_out"])
            s["work"] = torch.empty(ec.kv_pages_work_bytes(s["cache"], case["seqs"], s["table_out"].shape[0]),
                                    dtype=torch.uint8, device="cuda")
    return s


def _family(case):
    """The parent of each new sequence (a few have none) and the tokens that it makes room for."""
    r = random.Random(case["mix"] + 1)
    parents = [r.randrange(case["seqs"]) if r.random() > 0.03 else -1 for _ in range(case["to"])]
    grow = [r.randint(min(1, case["grow"]), case["grow"]) for _ in range(case["to"])]
    return parents, grow


# ---------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_attend(s):
    import lossless_entropy_coded_gb300 as ec
    c = s["case"]
    ec.kv_attend(s["cache"], 0, s["seqs"], s["q"], s["out"], starts=s["starts"], max_new=s["max_new"],
                 max_len=s["max_len"], window=c["window"], sinks=c["sinks"], lse=s["lse"], work=s["work"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    import lossless_entropy_coded_gb300 as ec
    ec.kv_append(s["cache"], 0, s["seqs"], s["k"], s["v"], starts=s["starts"], max_new=s["max_new"])
    ec.kv_read(s["cache"], 0, s["seqs"], s["k_out"], s["v_out"], starts=s["starts"], max_new=s["max_new"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_fork(s):
    import lossless_entropy_coded_gb300 as ec
    ec.kv_fork(s["cache"], s["seqs"], s["refs"], s["seqs_out"], s["refs_out"], parents=s["parents"], grow=s["grow"],
               work=s["work"])
    return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"], "pool": s["pool"]}


def _own_compact(s):
    import lossless_entropy_coded_gb300 as ec
    ec.kv_compact(s["cache"], s["seqs"], s["refs"], s["seqs_out"], s["refs_out"], page_map=s["map"], work=s["work"])
    return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"], "map": s["map"], "pool": s["pool"]}


def _plain_attend(s):
    c = s["case"]
    n, page, h, d = c["seqs"], c["page"], c["kvh"], c["dim"]
    g, m, length = c["qh"] // h, s["max_new"], s["max_len"]
    held = -(-length // page)
    units = s["pool"][s["table"][:, :held].clamp(min=0).long(), 0].transpose(1, 2)  # [seqs, heads, pages, units, bytes]
    kc, ks, vc, vs = (x.reshape(n, h, held * page, -1)[:, :, :length] for x in _unpack(units, d))
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    slot = torch.arange(m, device="cuda")
    row = (starts[:-1, None] + slot).clamp(max=s["rows"] - 1)  # the query of each (sequence, slot); slots past `new` are dropped
    q = s["q"].float()[row].reshape(n, m, h, g, d).permute(0, 2, 3, 1, 4).reshape(n, h, g * m, d)
    score = torch.matmul(q, _values(kc, ks).transpose(2, 3)).mul_(d ** -0.5).reshape(n, h, g, m, length)
    at = (lens - new)[:, None] + slot
    t = torch.arange(length, device="cuda")
    seen = t <= at[:, :, None]
    if c["window"]:
        seen = seen & ((t > at[:, :, None] - c["window"]) | (t < c["sinks"]))
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, h, g * m, length), _values(vc, vs)).reshape(n, h, g, m, d) / total
    keep = slot < new[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(n, m, h * g, d)[keep].to(TYPES[c["out"]])
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(n, m, h * g)[keep]
    return {"out": out, "lse": lse}


def _places(s):
    """Page, head-independent unit and token in the unit of every new row."""
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new, output_size=s["rows"])
    at = torch.arange(s["rows"], device="cuda") - starts[seq + 1] + lens[seq]
    page = s["case"]["page"]
    return s["table"].long()[seq, at // page], at % page // 16, at % 16


def _plain_append(s):
    d = s["case"]["dim"]
    page, unit, tok = _places(s)
    # each unit that a new row falls in is taken apart, filled and put together again
    key = page * (s["case"]["page"] // 16) + unit
    uniq, back = torch.unique(key, return_inverse=True)
    pool = s["pool"][:, 0].transpose(1, 2).reshape(-1, s["case"]["kvh"], _unit(s["case"]))
    parts = [x.clone() for x in _unpack(pool[uniq], d)]  # [units, heads, 16, .]
    for part, new in zip(parts, (*_quantise(s["k"]), *_quantise(s["v"]))):  # the four sections of a unit
        part[back, :, tok] = new
    u = s["case"]["page"] // 16
    s["pool"][uniq // u, 0, :, uniq % u] = _pack(*parts)
    got = _unpack(s["pool"][page, 0, :, unit], d)
    pick = torch.arange(s["rows"], device="cuda")
    kc, ks, vc, vs = (x[pick, :, tok] for x in got)
    return {"k": _values(kc, ks).bfloat16(), "v": _values(vc, vs).bfloat16()}


def _plain_fork(s):
    c = s["case"]
    page, total, to, width = c["page"], s["pool"].shape[0], c["to"], s["table_out"].shape[1]
    table, lens, parents, grow = s["table"].long(), s["lens"].long(), s["parents"].long(), s["grow"].long()
    some, p = parents >= 0, parents.clamp(min=0)
    had = torch.where(some, lens[p], torch.zeros_like(p))
    now = torch.where(some, had + grow, torch.zeros_like(p))
    whole, rest = had // page, had % page
    need = (now + page - 1) // page
    order = torch.arange(to, device="cuda")
    first = torch.full((table.shape[0],), to, device="cuda").scatter_reduce(0, p, torch.where(some, order, to), "amin")
    keeps = some & (first[p] == order) & (rest > 0)  # the first child keeps the partly filled page
    kept = whole + keeps
    col = torch.arange(width, device="cuda")
    shared = torch.where(col < kept[:, None], table[p], torch.full_like(table[p], -1))
    refs = s["refs"].long()
    held = table[(torch.arange(table.shape[1], device="cuda") < ((lens + page - 1) // page)[:, None])]
    refs = refs - torch.bincount(held, minlength=total) + torch.bincount(shared[shared >= 0], minlength=total)
    free = torch.nonzero(refs == 0)[:, 0]
    want = need - kept
    begin = torch.cumsum(want, 0) - want
    fresh = (col >= kept[:, None]) & (col < need[:, None])
    pick = (begin[:, None] + col - kept[:, None])[fresh]
    out = shared
    out[fresh] = free[pick]
    refs[free[pick]] += 1
    copy = torch.nonzero(some & ~keeps & (rest > 0))[:, 0]
    src, dst = table[p[copy], whole[copy]], out[copy, whole[copy]]
    used = torch.arange(page // 16, device="cuda") < ((rest[copy] + 15) // 16)[:, None]
    s["pool"][dst] = torch.where(used[:, None, None, :, None], s["pool"][src], s["pool"][dst])
    return {"table": out.int(), "lens": now.int(), "refs": refs.int(), "pool": s["pool"]}


def _plain_compact(s):
    refs, table = s["refs"].long(), s["table"].long()
    total = refs.shape[0]
    ids = torch.arange(total, device="cuda")
    live = refs > 0
    n = live.sum()
    src, dst = ids[live & (ids >= n)], ids[~live & (ids < n)]
    to = torch.where(live, ids, torch.full_like(ids, -1))
    to[src] = dst
    out = torch.where(table >= 0, to[table.clamp(min=0)], table)
    moved = torch.zeros_like(refs)
    moved[to[live]] = refs[live]
    s["pool"][dst] = s["pool"][src]
    return {"table": out.int(), "lens": s["lens"].clone(), "refs": moved.int(), "map": to.int(), "pool": s["pool"]}


_run_own = {"attend": _own_attend, "append": _own_append, "fork": _own_fork, "compact": _own_compact}
_run_plain = {"attend": _plain_attend, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, d, h = case["op"], case["dim"], case["kvh"]
    lens, new = _lens(case)
    per_token = 2 * h * (d // 2 + d // 32)
    if op == "attend":
        w, k = case["window"], case["sinks"]
        read = pairs = 0
        for n, m in zip(lens, new):
            read += n if not w else min(n, min(n, w + m - 1) + min(k, max(0, n - m + 1 - w)))
            for i in range(m):
                at = n - m + i
                pairs += at + 1 if not w else min(at + 1, w) + min(k, max(0, at + 1 - w))
        rows = sum(new) * case["qh"]
        return {"bytes": read * per_token + rows * (d * (SIZE[case["type"]] + SIZE[case["out"]]) + 4),
                "flops": 4.0 * d * case["qh"] * pairs}
    if op == "append":
        rows = sum(new)
        return {"bytes": rows * (2 * h * d * (SIZE[case["type"]] + 2) + 2 * per_token), "flops": 4.0 * rows * h * d}
    page, layers = case["page"], case["layers"]
    unit = layers * h * _unit(case)
    if op == "fork":
        parents, grow = _family(case)
        seen, bytes_ = set(), 0
        for p in parents:
            if p >= 0:
                if p in seen:
                    bytes_ += 2 * unit * -(-(lens[p] % page) // 16)
                seen.add(p)
                bytes_ += 8 * -(-lens[p] // page)
        return {"bytes": bytes_ + 8 * sum(-(-n // page) for n in lens), "flops": 0}
    held = sum(-(-n // page) for n in lens)
    total = held + int(held * case["free"] / (1 - case["free"])) + 1
    moved = held * (total - held) / total  # about: pages in use past the first `held`, had none been shared
    return {"bytes": 2 * moved * unit * (page // 16) + 8 * (held + total), "flops": 0}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def _stored(x):
    """The values that a cache holds of x [..., dim], from the definition: float64."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2((top / 6).clamp(min=2.0 ** -126))))
    scale = torch.where(top > 6 * scale, 2 * scale, torch.where(top <= 3 * scale, scale / 2, scale))
    y = b / scale.clamp(min=2.0 ** -126)
    # steps of 1/2 below 2, of 1 below 4, of 2 above; torch.round takes ties to the even multiple
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(y / step) * step * scale).reshape(x.shape)


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None  # whole numbers
    lens, new = _lens(case)
    k, v, q = _tensors(case, seed)
    ends = _starts(lens)
    if op == "append":
        rows = torch.cat([torch.arange(ends[i + 1] - new[i], ends[i + 1]) for i in range(len(lens))]).cuda()
        return {"k": _stored(k[rows]), "v": _stored(v[rows])}
    g, scale = case["qh"] // case["kvh"], 1.0 / case["dim"] ** 0.5
    outs, lses, row = [], [], 0
    for i, (n, m) in enumerate(zip(lens, new)):
        ki, vi = _stored(k[ends[i]:ends[i + 1]]), _stored(v[ends[i]:ends[i + 1]])
        o = torch.empty(m, case["qh"], case["dim"], dtype=torch.float64, device=k.device)
        lse = torch.empty(m, case["qh"], dtype=torch.float64, device=k.device)
        pos = torch.arange(n - m, n, device=k.device)[:, None]
        tok = torch.arange(n, device=k.device)[None, :]
        hide = tok > pos
        if case["window"]:
            hide = hide | ((tok <= pos - case["window"]) & (tok >= case["sinks"]))
        for j in range(case["qh"]):
            z = (q[row:row + m, j].double() @ ki[:, j // g].T * scale).masked_fill(hide, float("-inf"))
            lse[:, j] = torch.logsumexp(z, -1)
            o[:, j] = torch.exp(z - lse[:, j, None]) @ vi[:, j // g]
        outs.append(o)
        lses.append(lse)
        row += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
