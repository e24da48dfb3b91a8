"""Rows of one call keep to themselves: what a row does not see, or a neighbour that is
not a number, leaves its output alone, however far apart values, keys and queries lie."""
import math

import pytest
import torch

import kv_ref as R
from test_gpu_kv import BF16, FP16, FP32, Case, ec, starts_of  # noqa: F401 (ec is a fixture)

pytestmark = pytest.mark.gpu


def stored(x):
    return torch.from_numpy(R.stored(x.double().cpu().numpy())).cuda()


def row_bounds(r, q, k, v, first, scale, window, sinks, out_type):
    """Largest errors of attend's out and lse, from the formats, per row, head and block and
    over the tokens that the row sees:
    scores: 2^-19 of sum |q k| (FP32 accumulation, dim <= 256), 2^-22 of it where FP32 queries
      are two FP16 parts, 2^-20 for the exponential's argument;
    weights: FP16, 2^-11 of each, and 2^-22 of the row's largest where they are subnormal: 2^5
      stands for the largest, half of the last place is 2^-25, and a scale may lie 2^8 below
      its block's reference; never more than the weight itself.  A block's magnitude is at most
      twice its largest element;
    output: one rounding."""
    m, heads, dim = q.shape
    n, kvh = k.shape[0], k.shape[1]
    pos = torch.arange(first, first + m, device=q.device)[:, None]
    t = torch.arange(n, device=q.device)[None]
    see = t <= pos
    if window:
        see &= (t > pos - window) | (t < sinks)
    scale = dim ** -0.5 if scale is None else scale
    blocks = torch.nan_to_num(v).abs().reshape(n, kvh, dim // 32, 32).amax(-1)
    eps_s, small = torch.zeros((m, heads), dtype=torch.float64, device=q.device), torch.zeros_like(q)
    for h in range(heads):
        g = h // (heads // kvh)
        s = (q[:, h] @ k[:, g].T * scale).masked_fill(~see, -math.inf)
        p = torch.nan_to_num(torch.exp(s - torch.nan_to_num(s, nan=-math.inf).amax(-1, keepdim=True))) if n else s
        acc = (torch.nan_to_num(q[:, h]).abs() @ torch.nan_to_num(k[:, g]).abs().T * scale).masked_fill(~see, 0)
        if n:
            eps_s[:, h] = acc.amax(-1) * (2.0 ** -19 + 2.0 ** -22) + 2.0 ** -20
        small[:, h] = (p.clamp(max=2.0 ** -22) @ blocks[:, g]).repeat_interleave(32, -1) * 2
    eps_out = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -22}[out_type]
    out = r.mag * (2.0 ** -11 + 2 * eps_s[..., None] + 2.0 ** -19) + small + r.out.abs() * eps_out
    lse = eps_s + 2.0 ** -21 * r.lse.abs().nan_to_num(posinf=0, neginf=0) + 2.0 ** -20
    return out, lse


def check(ec, c, k, v, new, q, out_type=FP32, window=0, sinks=0, scale=None, skip=()):
    """kv_attend against the 64-bit form in every row and head but those of `skip`."""
    out = torch.full(q.shape, 9.0, dtype=out_type, device="cuda")
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    ec.kv_attend(c.cache, c.layer, c.seqs, q, out, starts=starts_of(new), max_new=max(new + [1]), scale=scale or 0.0,
                 window=window, sinks=sinks, lse=lse)
    assert ec.status() == 0
    ks, vs = stored(k), stored(v)
    at = row = 0
    for n, m in zip(c.lens, new):
        n = max(n, 0)
        qd, kd, vd = q[row:row + m].double(), ks[at:at + n], vs[at:at + n]
        r = R.attend(qd, kd, vd, n - m, scale, window, sinks)
        eo, el = row_bounds(r, qd, kd, vd, n - m, scale, window, sinks, out_type)
        o, l = out[row:row + m].double(), lse[row:row + m].double()
        use = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
        for i, h in skip:
            if row <= i < row + m:
                use[i - row, h] = False
        nan = torch.isnan(r.out)
        assert torch.equal(torch.isnan(o)[use], nan[use])
        fine = use[..., None] & ~nan
        worst = ((o - r.out).abs() / eo.clamp(min=1e-300))[fine]
        assert bool(((o - r.out).abs() <= eo)[fine].all()), f"out: {worst.max()} of the bound"
        empty = torch.isneginf(r.lse)
        assert torch.equal(torch.isneginf(l)[use], empty[use])
        fine = use & ~empty & ~torch.isnan(r.lse)
        assert bool(((l - r.lse).abs() <= el)[fine].all()), f"lse: {((l - r.lse).abs() / el)[fine].max()} of the bound"
        at += n
        row += m
    return out, lse


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


SPREADS = [9, 14, 15, 16, 20, 40, 100, -15, -40, -100]
GROUPS = [(2, 1), (4, 1), (80, 1)]   # a few rows, and more than the register form takes


# ------------------------------------------------------------------ values far apart
@pytest.mark.parametrize("qh,kvh", GROUPS)
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("power", SPREADS)
def test_a_later_value_leaves_earlier_rows_alone(ec, qh, kvh, dim, power):
    """Two new tokens: the first sees the first value only, and gives it."""
    c = Case(ec, [2], kvh, dim, 16)
    k = normal(1, 2, kvh, dim)
    v = torch.ones((2, kvh, dim), device="cuda")
    v[1] = 2.0 ** power
    c.fill(k, v)
    q = normal(2, 2, qh, dim)
    check(ec, c, k, v, [2], q)


@pytest.mark.parametrize("qh,kvh", GROUPS)
@pytest.mark.parametrize("power", [12, 20, 60, -20, -60])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_loud_tokens_of_no_weight(ec, qh, kvh, power, dtype):
    """Tokens whose values lie 2^power from the others' and that the queries turn away from."""
    n = 700
    c = Case(ec, [n, 40], kvh, 128, 32)
    k, v = (normal(3, n + 40, kvh, 128) * 0.3).to(dtype).float(), normal(4, n + 40, kvh, 128)
    away = normal(5, kvh, 128)
    away = away / away.norm(dim=-1, keepdim=True) * 128 ** 0.5
    loud = torch.tensor([3, 150, 151, 333, 640, n + 2], device="cuda")
    k[loud] = -away * 12
    v[loud] *= 2.0 ** power
    k, v = k.to(dtype), v.to(dtype)
    c.fill(k, v)
    for new in ([1, 1], [9, 3]):
        q = (away.repeat_interleave(qh // kvh, 0) + 0.5 * normal(6, sum(new), qh, 128)).to(dtype)
        check(ec, c, k, v, new, q)
        check(ec, c, k, v, new, q, window=500, sinks=2)


@pytest.mark.parametrize("qh,kvh,dim", [(4, 1, 128), (8, 4, 64), (3, 1, 192), (2, 2, 256)])
@pytest.mark.parametrize("power", [15, 30, 90])
def test_prompt_with_loud_values(ec, qh, kvh, dim, power):
    """Every row of a prompt against the tokens that it sees; loud values in the middle and at the end."""
    n = 390
    c = Case(ec, [n, 77], kvh, dim, 64)
    k, v = normal(7, n + 77, kvh, dim), normal(8, n + 77, kvh, dim)
    v[200:203] *= 2.0 ** power
    v[n - 1, :, :32] *= 2.0 ** power
    v[n + 30] *= 2.0 ** -power
    c.fill(k, v)
    new = [n, 77]
    q = normal(9, sum(new), qh, dim)
    check(ec, c, k, v, new, q)
    check(ec, c, k, v, new, q.to(BF16), window=50, sinks=1)


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [60, 150]])
def test_values_that_drift(ec, new):
    """Scales that grow and shrink along the sequence, by 2^12 and 2^60 each way."""
    c = Case(ec, [90, 1400], 2, 128, 32)
    k, v = normal(17, 1490, 2, 128) * 0.5, normal(18, 1490, 2, 128)
    t = torch.arange(v.shape[0], device="cuda").float()
    v[:, 0] *= torch.exp2(12 * torch.sin(t / 90))[:, None]
    v[:, 1] *= torch.exp2(60 * torch.sin(t / 200))[:, None]
    v[100:110] = 0
    c.fill(k, v)
    check(ec, c, k, v, new, normal(19, sum(new), 8, 128))


# ------------------------------------------------------------------ keys far apart
@pytest.mark.parametrize("qh,new", [(2, 5), (2, 40), (80, 40)])
@pytest.mark.parametrize("power", [26, 28, 30, 60])
def test_a_later_key_leaves_earlier_rows_alone(ec, qh, new, power):
    c = Case(ec, [40], 1, 128, 16)
    k, v = normal(10, 40, 1, 128), normal(11, 40, 1, 128)
    k[37] *= 2.0 ** power
    c.fill(k, v)
    q = normal(12, new, qh, 128)
    q[-3:] *= 2.0 ** -power
    check(ec, c, k, v, [new], q)


@pytest.mark.parametrize("new", [1, 40])
def test_small_queries_and_large_keys(ec, new):
    """Queries near the smallest numbers and keys near the largest that FP32 scores hold."""
    c = Case(ec, [40], 1, 64, 16)
    k, v = normal(13, 40, 1, 64) * 2.0 ** 104, normal(14, 40, 1, 64)
    c.fill(k, v)
    for power in (-104, -108, -111, -114):
        q = normal(15, new, 2, 64) * 2.0 ** power
        q[..., 4:] = 0
        check(ec, c, k, v, [new], q, scale=2.0 ** -6)


# ------------------------------------------------------------------ neighbours that are no numbers
@pytest.mark.parametrize("qh,kvh", [(8, 4), (8, 2), (8, 1), (80, 1)])
@pytest.mark.parametrize("poison", [math.nan, math.inf])
def test_a_query_of_nan_spoils_its_own_row_only(ec, qh, kvh, poison):
    """Scores and value scales rise along the sequence, so that every row's reference has to move."""
    n = 1200
    c = Case(ec, [n], kvh, 128, 16)
    u = normal(20, 128) * 0.5
    t = torch.arange(n, device="cuda").float()
    k = (u * (t / n * 28 - 14)[:, None])[:, None].repeat(1, kvh, 1).contiguous()
    v = normal(21, n, kvh, 128) * torch.exp2(t / n * 5)[:, None, None]
    c.fill(k, v)
    q = (u * 4 + 0.05 * normal(22, 1, qh, 128))
    for h in range(min(qh, 8)):
        bad = q.clone()
        bad[0, h, 7] = poison
        out, _ = check(ec, c, k, v, [1], bad, skip=[(0, h)])
        assert torch.isnan(out[0, h]).all()


@pytest.mark.parametrize("qh", [1, 2, 48])
def test_a_key_of_nan_spoils_rows_that_see_it(ec, qh):
    n = 1280
    c = Case(ec, [n], 1, 128, 16)
    u = normal(23, 128) * 0.5
    a = torch.full((n,), -1.0, device="cuda")
    a[n - 9] = 3   # outweighs the others; the same place of its unit as the last token
    k = (u * a[:, None])[:, None].contiguous()
    v = normal(24, n, 1, 128)
    k[n - 1] = math.nan
    c.fill(k, v)
    out, _ = check(ec, c, k, v, [2], (u * 4 + 0.05 * normal(25, 2, qh, 128)))
    assert not torch.isnan(out[0]).any() and torch.isnan(out[1]).all()


# ------------------------------------------------------------------ outputs in the queries' place
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens,new", [([700, 90, 5000], [3, 2, 2]), ([700, 90, 5000], [90, 70, 30]), ([400, 90, 130], [90, 70, 30]),
                                      ([10, 40, 3, 17] * 250, [1] * 1000)])
@pytest.mark.parametrize("loud", [0, 8, 60])
def test_outputs_may_replace_the_queries(ec, lens, new, loud, dtype):
    """The same bits as with an output of its own, also where rows are done again."""
    kvh = 8 if len(lens) > 3 else 2
    c = Case(ec, lens, kvh, 128, 32)
    k, v = normal(60, sum(lens), kvh, 128), normal(61, sum(lens), kvh, 128)
    v[2::67] *= 2.0 ** loud
    c.fill(k, v)
    q = normal(62, sum(new), 4 * kvh, 128).to(dtype)
    want = torch.empty_like(q)
    ec.kv_attend(c.cache, 0, c.seqs, q, want, starts=starts_of(new), max_new=max(new))
    if len(lens) == 3:
        check(ec, c, k, v, new, q, dtype)
    for _ in range(5):
        x = q.clone()
        ec.kv_attend(c.cache, 0, c.seqs, x, x, starts=starts_of(new), max_new=max(new))
        assert ec.status() == 0 and torch.equal(x, want)


# ------------------------------------------------------------------ large scores
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("qh,new", [(4, 1), (3, 20), (80, 20), (4, 650)])
@pytest.mark.parametrize("power", [10, 18, 22, 26, 30, 40])
def test_scores_of_any_size(ec, qh, new, power, dtype):
    """One token that outweighs all others that a row sees is what the row gives, however large
    the scores: 2^power times those of the other tests."""
    n = 700
    c = Case(ec, [n], 1, 128, 32)
    u, a = normal(63, 128), 0.05 * normal(64, n)
    a[100], a[690] = 1, 2
    k = (u * a[:, None] * 2.0 ** power)[:, None].to(dtype)
    v = normal(65, n, 1, 128)
    v[690] *= 100   # a scale above the references of the tokens before
    v = v.to(dtype)
    c.fill(k, v)
    q = (u * (0.5 + torch.rand((new, qh, 1), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"))).to(dtype)
    out = torch.empty((new, qh, 128), device="cuda")
    ec.kv_attend(c.cache, 0, c.seqs, q, out, starts=starts_of([new]), max_new=new)
    assert ec.status() == 0
    vs, pos = stored(v), torch.arange(n - new, n, device="cuda")
    for row in range(new):
        if pos[row] >= 100:
            want = vs[690 if pos[row] >= 690 else 100, 0]
            # its weight is 1 but for FP16's 2^-11 and what 699 tokens of weight 0 (2^-22 each at most) leave
            assert bool(((out[row].double() - want).abs() <= want.abs() * 2.0 ** -10 + 1e-12).all()), (row, (out[row].double() - want).abs().max())
