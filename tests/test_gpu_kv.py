"""The 4-bit key/value cache on the GPU against plain 64-bit forms (kv_ref): the bytes
that an append leaves, the values that a read returns, attention over all head layouts,
lengths and masks, and the page operations."""
import random

import numpy as np
import pytest
import torch

import kv_ref as R

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coded_gb300 as ec
    return ec


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(new):
    return i32(np.concatenate([[0], np.cumsum(new)]).tolist())


class Case:
    """Sequences with shuffled pages in a pool that is full of NaN blocks where nothing was written."""

    def __init__(self, ec, lens, kvh, dim, page, seed=0, layers=1, layer=0, spare=2, first_page=0):
        self.ec, self.lens, self.kvh, self.dim, self.page, self.layer = ec, lens, kvh, dim, page, layer
        need = [-(-max(n, 0) // page) for n in lens]
        ids = list(range(sum(need) + spare))
        random.Random(seed).shuffle(ids)
        self.n_pages = len(ids) + first_page
        width = max(need + [0]) + 1
        self.rows, at = [], 0
        for n in need:
            self.rows.append([first_page + p for p in ids[at:at + n]] + [-1] * (width - n))
            at += n
        self.pool = torch.full((self.n_pages, layers, kvh, page // 16, 17 * dim), 255, dtype=torch.uint8, device="cuda")
        self.cache = ec.kv_cache(layers, self.n_pages, kvh, dim, page, pool=self.pool)
        self.table, self.dlens = i32(self.rows).reshape(len(lens), width), i32(lens)
        self.seqs = ec.kv_seqs(self.table, self.dlens)

    def tensors(self, seed, dtype=BF16, rows=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = sum(max(x, 0) for x in self.lens) if rows is None else rows
        x = torch.randn((2, n, self.kvh, self.dim), generator=g, device="cuda")
        return (x * torch.exp2(torch.randint(-3, 4, (2, n, self.kvh, self.dim // 32), generator=g, device="cuda")
                               .float()).repeat_interleave(32, -1)).to(dtype)

    def fill(self, k, v):
        self.ec.kv_append(self.cache, self.layer, self.seqs, k, v, starts=starts_of([max(n, 0) for n in self.lens]),
                          max_new=max(self.lens + [1]))

    def read(self, dtype=FP32, new=None):
        new = [max(n, 0) for n in self.lens] if new is None else new
        out = torch.full((2, sum(new), self.kvh, self.dim), 7.0, dtype=dtype, device="cuda")
        self.ec.kv_read(self.cache, self.layer, self.seqs, out[0], out[1], starts=starts_of(new), max_new=max(new + [1]))
        return out


LENS = [1, 15, 0, 16, 17, 31, 100, -1, 64]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("dim,page,kvh", [(64, 16, 3), (128, 64, 2), (192, 32, 1), (256, 256, 2), (128, 128, 5)])
def test_append_then_read(ec, dim, page, kvh, dtype):
    c = Case(ec, LENS, kvh, dim, page, layers=3, layer=1)
    k, v = c.tensors(1, dtype)
    c.fill(k, v)
    got = c.read()
    assert ec.status() == 0
    for x, y in ((k, got[0]), (v, got[1])):
        assert np.array_equal(y.double().cpu().numpy(), R.stored(x.double().cpu().numpy()))
    assert (c.pool[:, 0] == 255).all() and (c.pool[:, 2] == 255).all()  # other layers are not touched


def test_pool_bytes(ec):
    """The bytes of a unit are where the header says."""
    for dim in (64, 128, 192, 256):
        c = Case(ec, [16], 2, dim, 16)
        k, v = c.tensors(2, FP32)
        c.fill(k, v)
        for h in range(2):
            kq, vq = R.quantise(k[:, h].cpu().numpy()), R.quantise(v[:, h].cpu().numpy())
            got = c.pool[c.rows[0][0], 0, h, 0].cpu().numpy()
            assert np.array_equal(got, R.unit_bytes(*kq, *vq))


@pytest.mark.parametrize("steps", [[1] * 40, [5, 11, 1, 16, 7], [15, 2, 30, 1]])
def test_append_in_steps(ec, steps):
    """Tokens that arrive in pieces share units and bytes with older ones."""
    c = Case(ec, [sum(steps), sum(steps)], 2, 128, 16)
    k, v = c.tensors(3)
    n = sum(steps)
    at = 0
    for s in steps:
        at += s
        c.dlens.copy_(i32([at, at]))
        rows = torch.cat([torch.arange(at - s, at), n + torch.arange(at - s, at)]).cuda()
        ec.kv_append(c.cache, 0, c.seqs, k[rows], v[rows], starts=starts_of([s, s]), max_new=s)
    got = c.read()
    assert ec.status() == 0
    for x, y in ((k, got[0]), (v, got[1])):
        assert np.array_equal(y.double().cpu().numpy(), R.stored(x.double().cpu().numpy()))


def test_append_without_starts(ec):
    c = Case(ec, [1, 20, 33], 2, 64, 32)
    k, v = c.tensors(4, rows=3)
    ec.kv_append(c.cache, 0, c.seqs, k, v)
    out = torch.empty((2, 3, 2, 64), device="cuda")
    ec.kv_read(c.cache, 0, c.seqs, out[0], out[1])
    assert ec.status() == 0
    assert np.array_equal(out[0].double().cpu().numpy(), R.stored(k.double().cpu().numpy()))
    assert np.array_equal(out[1].double().cpu().numpy(), R.stored(v.double().cpu().numpy()))


def test_special_values(ec):
    """Zeros, the levels' midpoints, the smallest and largest numbers, infinities and NaN."""
    c = Case(ec, [16], 1, 64, 16)
    x = torch.zeros((16, 1, 64), device="cuda")
    x[0, 0, :32] = torch.tensor([6, 0.25, -0.75, 1.25, 1.75, -2.5, 3.5, 5] * 4, dtype=FP32)
    x[0, 0, 32:] = -0.0
    x[1, 0, 3] = 3.0
    x[2, 0, 3] = 3.0000002
    x[3, 0, :] = 1e-45
    x[4, 0, :] = 1.1754944e-38
    x[5, 0, :32] = 3.4028234e38
    x[5, 0, 32:] = -1e30
    x[6, 0, 5] = float("inf")
    x[7, 0, 40] = float("nan")
    x[8, 0, :] = torch.linspace(-8, 8, 64)
    x[9, 0, 0], x[9, 0, 1] = 6 * 2.0 ** -126, 2.0 ** -127
    x[10, 0, :] = 1e-38
    c.fill(x, x.flip(0).contiguous())
    got = c.read().cpu().numpy()
    xs = x.cpu().numpy()
    with np.errstate(over="ignore"):  # the largest FP32 number is held as 4 * 2^126, an infinity in FP32
        for w, g in ((xs, got[0]), (xs[::-1], got[1])):
            assert np.array_equal(g, R.stored(np.ascontiguousarray(w)).astype(np.float32), equal_nan=True)
    assert ec.status() == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_strides_and_alignment(ec, dtype):
    """Rows and heads at any stride, in any order, from any element."""
    c = Case(ec, [5, 40], 3, 64, 16)
    k, v = c.tensors(5, dtype)
    wide = torch.empty((3, 45, 2, 67), dtype=dtype, device="cuda")
    ks, vs = wide[:, :, 0, 1:65].transpose(0, 1), wide[:, :, 1, 3:67].transpose(0, 1)
    ks.copy_(k), vs.copy_(v)
    c.fill(ks, vs)
    out = torch.full((2, 45, 3, 69), 5.0, dtype=BF16, device="cuda")
    o = out[..., 1:65]
    ec.kv_read(c.cache, 0, c.seqs, o[0], o[1], starts=starts_of([5, 40]), max_new=40)
    assert ec.status() == 0
    for x, y in ((k, o[0]), (v, o[1])):
        assert np.array_equal(y.double().cpu().numpy(), R.stored(x.double().cpu().numpy()))
    assert (out[..., 0] == 5).all() and (out[..., 65:] == 5).all()


def test_read_a_tail_and_before_the_first_token(ec):
    c = Case(ec, [3, 50], 2, 128, 32)
    k, v = c.tensors(6)
    c.fill(k, v)
    out = c.read(new=[10, 21])
    assert ec.status() == 0
    want = torch.cat([torch.zeros_like(k[:7]), k[:3], k[3 + 29:53]])
    assert np.array_equal(out[0].double().cpu().numpy(), R.stored(want.double().cpu().numpy()))
    only = torch.empty((31, 2, 128), dtype=FP16, device="cuda")
    ec.kv_read(c.cache, 0, c.seqs, None, only, starts=starts_of([10, 21]), max_new=21)
    assert torch.equal(only.float(), out[1].to(FP16).float())


# ------------------------------------------------------------------ attention
def check_attend(ec, c, k, v, new, qh, dtype=BF16, out_type=BF16, window=0, sinks=0, scale=None, seed=9, max_len=0,
                 use_starts=True, q=None):
    """kv_attend of the last `new` tokens of each sequence against the 64-bit form."""
    rows = sum(new)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if q is None:
        q = (torch.randn((rows, qh, c.dim), generator=g, device="cuda") * 1.5).to(dtype)
    out = torch.full((rows, qh, c.dim), 9.0, dtype=out_type, device="cuda")
    lse = torch.full((rows, qh), 9.0, device="cuda")
    ec.kv_attend(c.cache, c.layer, c.seqs, q, out, starts=starts_of(new) if use_starts else None, max_new=max(new + [1]),
                 max_len=max_len, scale=scale or 0.0, window=window, sinks=sinks, lse=lse)
    assert ec.status() == 0
    ks, vs = (torch.from_numpy(R.stored(x.double().cpu().numpy())).cuda() for x in (k, v))
    at = row = 0
    for n, m in zip(c.lens, new):
        n = max(n, 0)
        r = R.attend(q[row:row + m].double(), ks[at:at + n], vs[at:at + n], n - m, scale, window, sinks)
        eo, el = R.bounds(r, n, out_type, 2.0 ** -22 if q.dtype == FP32 else 2.0 ** -28)
        o, l = out[row:row + m].double(), lse[row:row + m].double()
        assert torch.equal(torch.isnan(o), torch.isnan(r.out))
        assert bool(((o - r.out).abs() <= eo)[~torch.isnan(r.out)].all()), f"out: {((o - r.out).abs() / eo).nan_to_num().max()} of the bound"
        empty = torch.isneginf(r.lse)
        assert torch.equal(torch.isneginf(l), empty)
        fine = ~empty & ~torch.isnan(r.lse)
        assert bool(((l - r.lse).abs() <= el)[fine].all()), f"lse: {((l - r.lse).abs() / el)[fine].max()} of the bound"
        at += n
        row += m
    return out, lse


HEADS = [(8, 2, 128), (4, 4, 64), (7, 1, 128), (16, 1, 64), (6, 2, 192), (4, 2, 256), (24, 1, 128)]


@pytest.mark.parametrize("qh,kvh,dim", HEADS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_one_new_token(ec, qh, kvh, dim, dtype):
    c = Case(ec, [1, 2, 15, 16, 17, 0, 100, 257, 530], kvh, dim, 32, layers=2, layer=1)
    k, v = c.tensors(10, dtype)
    c.fill(k, v)
    check_attend(ec, c, k, v, [1] * 9, qh, dtype, FP16 if dtype == FP16 else BF16, use_starts=False)


@pytest.mark.parametrize("page", [16, 64, 256])
def test_long_context_in_shares(ec, page):
    c = Case(ec, [5000, 3, 9001], 2, 128, page)
    k, v = c.tensors(11)
    c.fill(k, v)
    a = check_attend(ec, c, k, v, [1, 1, 1], 8, out_type=FP32)
    b = check_attend(ec, c, k, v, [1, 1, 1], 8, out_type=FP32, max_len=9001)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits every time


@pytest.mark.parametrize("qh,kvh,dim", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (20, 0), (33, 5), (64, 40)])
def test_several_new_tokens_and_windows(ec, qh, kvh, dim, window, sinks):
    c = Case(ec, [40, 7, 300, 65, 1, 0], kvh, dim, 16)
    k, v = c.tensors(12)
    c.fill(k, v)
    check_attend(ec, c, k, v, [5, 7, 9, 0, 1, 2], qh, window=window, sinks=sinks)


@pytest.mark.parametrize("qh,kvh,dim", HEADS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_prompts(ec, qh, kvh, dim, dtype):
    """Whole prompts and chunks: every row sees its own keys."""
    c = Case(ec, [130, 257, 1, 400], kvh, dim, 64)
    k, v = c.tensors(13, dtype)
    c.fill(k, v)
    check_attend(ec, c, k, v, [130, 129, 1, 333], qh, dtype, FP16 if dtype == FP16 else BF16)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("new", [[8, 1, 0, 1, 2], [8, 8, 8, 8, 7], [3, 3, 3, 3, 3], [4, 4, 4, 4, 4], [6, 1, 6, 1, 6], [11, 1, 1, 1, 1]])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_tens_of_rows(ec, dim, new, dtype):
    """Row counts around those where few rows become many, alike and unlike in a batch."""
    c = Case(ec, [900, 15, 0, 1, 333], 1, dim, 32)
    k, v = c.tensors(15, dtype)
    c.fill(k, v)
    check_attend(ec, c, k, v, new, 8, dtype)
    check_attend(ec, c, k, v, new, 8, dtype, window=50, sinks=4)


def test_work_for_many_rows_serves_fewer(ec):
    """A buffer sized for the most rows serves every call of the same bounds with fewer."""
    c = Case(ec, [2000, 1500, 900, 40], 2, 128, 64)
    k, v = c.tensors(16)
    c.fill(k, v)
    most = ec.kv_attend_work_bytes(c.cache, 4, 20, 16, 5, 2000)
    for new in ([5, 5, 5, 5], [5, 1, 1, 1], [1, 0, 0, 5]):
        assert ec.kv_attend_work_bytes(c.cache, 4, sum(new), 16, 5, 2000) <= most
        q = torch.randn((sum(new), 16, 128), device="cuda").to(BF16)
        outs = [torch.empty_like(q) for _ in range(2)]
        ec.kv_attend(c.cache, 0, c.seqs, q, outs[0], starts=starts_of(new), max_new=5, max_len=2000,
                     work=torch.empty(most, dtype=torch.uint8, device="cuda"))
        ec.kv_attend(c.cache, 0, c.seqs, q, outs[1], starts=starts_of(new), max_new=5, max_len=2000)
        assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("window,sinks", [(100, 0), (17, 3), (128, 130), (1, 1)])
@pytest.mark.parametrize("qh,kvh,dim", [(8, 2, 128), (4, 4, 64), (6, 2, 192), (4, 2, 256)])
def test_prompts_with_windows(ec, window, sinks, qh, kvh, dim):
    c = Case(ec, [700, 90, 333], kvh, dim, 32)
    k, v = c.tensors(14)
    c.fill(k, v)
    check_attend(ec, c, k, v, [500, 90, 140], qh, window=window, sinks=sinks)


def test_more_new_rows_than_tokens(ec):
    """Rows before the first token see nothing: zeros and -inf."""
    c = Case(ec, [3, 0, 200], 2, 64, 16)
    k, v = c.tensors(15)
    c.fill(k, v)
    out, lse = check_attend(ec, c, k, v, [5, 4, 210], 4)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all() and (out[5:9] == 0).all() and (out[9:19] == 0).all()


def test_scale_argument_and_large_scores(ec):
    c = Case(ec, [300, 40], 2, 128, 64)
    k, v = c.tensors(16)
    c.fill(k, v)
    check_attend(ec, c, k, v, [1, 2], 8, scale=0.7)
    check_attend(ec, c, k, v, [200, 40], 8, scale=0.7)


@pytest.mark.parametrize("new", [[1, 1], [60, 150]])
def test_scales_far_apart(ec, new):
    """Value scales that grow and shrink along the sequence move the blocks' references."""
    c = Case(ec, [90, 400], 2, 128, 32)
    k, v = c.tensors(17, FP32)
    t = torch.arange(v.shape[0], device="cuda").float()
    v = v * torch.exp2(12 * torch.sin(t / 9))[:, None, None]
    k = k * torch.exp2(3 * torch.sin(t / 5) - 3)[:, None, None]
    v[:4] *= 2.0 ** -30
    v[100:110] = 0
    c.fill(k, v)
    check_attend(ec, c, k, v, new, 8, FP32)
    k[:, 1] *= 2.0 ** -60
    v[:, 1] *= 2.0 ** 90
    c.fill(k, v)
    check_attend(ec, c, k, v, new, 8, FP32)


def test_infinities_and_nan(ec):
    """Masked places may hold anything; what a row sees and weighs makes it NaN."""
    c = Case(ec, [300, 300], 2, 128, 16)
    k, v = c.tensors(18)
    k[5], v[7] = float("inf"), float("nan")   # before sequence 0's window, after its sinks
    k[300 + 299] = float("nan")               # sequence 1's last key: a block of NaN
    v[300 + 100, :, :32] = float("-inf")
    c.fill(k, v)
    a, _ = check_attend(ec, c, k, v, [3, 3], 8, window=100, sinks=4)
    assert not torch.isnan(a[:5]).any() and torch.isnan(a[5]).all()
    b, _ = check_attend(ec, c, k, v, [3, 3], 8)
    assert torch.isnan(b[:3]).all() and torch.isnan(b[3:5, :, :32]).all() and not torch.isnan(b[3:5, :, 32:]).any()
    check_attend(ec, c, k, v, [150, 160], 8, window=100, sinks=4)


def test_queries_of_all_magnitudes(ec):
    c = Case(ec, [200, 70], 2, 128, 64)
    k, v = c.tensors(19)
    c.fill(k, v)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for new in ([1, 2], [200, 70]):
        q = torch.randn((sum(new), 8, 128), generator=g, device="cuda")
        q = (q * torch.exp2(torch.linspace(-40, 6, sum(new), device="cuda"))[:, None, None]).to(BF16)
        q[0, 0] = 0
        check_attend(ec, c, k, v, new, 8, q=q)
        q[0, 3, 4] = float("nan")
        q[1, 2, 5] = float("inf")
        out = torch.empty((sum(new), 8, 128), dtype=BF16, device="cuda")
        ec.kv_attend(c.cache, 0, c.seqs, q, out, starts=starts_of(new), max_new=max(new))
        assert torch.isnan(out[0, 3]).all() and torch.isnan(out[1, 2]).all() and not torch.isnan(out[0, 4]).any()


def test_attend_strides(ec):
    c = Case(ec, [200, 70], 2, 64, 16)
    k, v = c.tensors(20)
    c.fill(k, v)
    for new in ([1, 1], [150, 70]):
        rows = sum(new)
        q = torch.randn((rows, 8, 64), device="cuda").to(BF16)
        want, _ = check_attend(ec, c, k, v, new, 8, q=q)
        wide = torch.empty((8, rows, 77), dtype=BF16, device="cuda")
        qs, os_ = wide[..., 5:69].transpose(0, 1), torch.full((8, rows, 77), 3.0, dtype=BF16, device="cuda")
        qs.copy_(q)
        ec.kv_attend(c.cache, 0, c.seqs, qs, os_[..., 7:71].transpose(0, 1), starts=starts_of(new), max_new=max(new))
        assert ec.status() == 0
        assert torch.equal(os_[..., 7:71].transpose(0, 1), want)
        assert (os_[..., :7] == 3).all() and (os_[..., 71:] == 3).all()


def test_offsets_past_32_bits(ec):
    """Pages that begin more than 4 GB into the pool."""
    page_bytes = 8 * 16 * 17 * 256
    first = (1 << 32) // page_bytes + 3
    ids = first + 6
    pool = torch.empty((ids, 1, 8, 16, 17 * 256), dtype=torch.uint8, device="cuda")
    c = Case(ec, [600, 700], 8, 256, 256, spare=0)
    c.table = c.table + first * (c.table >= 0).int()
    c.rows = c.table.cpu().tolist()
    c.cache = ec.kv_cache(1, ids, 8, 256, 256, pool=pool)
    c.seqs = ec.kv_seqs(c.table, c.dlens)
    k, v = c.tensors(21)
    c.fill(k, v)
    check_attend(ec, c, k, v, [1, 3], 8)
    got = c.read(BF16)
    assert np.array_equal(got[1].double().cpu().numpy(), R.stored(v.double().cpu().numpy()))


def test_other_streams_and_graphs(ec):
    """Calls on a stream of their own, captured and replayed with new contents."""
    c = Case(ec, [500, 33], 2, 128, 64)
    k, v = c.tensors(22)
    q = torch.randn((2, 8, 128), device="cuda").to(BF16)
    out = torch.empty_like(q)
    work = torch.empty(ec.kv_attend_work_bytes(c.cache, 2, 2, 8, 1, 500), dtype=torch.uint8, device="cuda")
    c.fill(k, v)
    want, _ = check_attend(ec, c, k, v, [1, 1], 8, q=q, max_len=500)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ec.kv_attend(c.cache, 0, c.seqs, q, out, max_len=500, work=work, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    last = torch.tensor([499, 532], device="cuda")
    kn, vn = k[last].clone(), v[last].clone()
    with torch.cuda.graph(graph):
        ec.kv_append(c.cache, 0, c.seqs, kn, vn)
        ec.kv_attend(c.cache, 0, c.seqs, q, out, max_len=500, work=work)
    kn.mul_(2), vn.neg_(), out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    k[last], v[last] = kn, vn
    again, _ = check_attend(ec, c, k, v, [1, 1], 8, q=q, max_len=500)
    assert torch.equal(out, again)


def test_inconsistent_tables_are_flagged(ec):
    c = Case(ec, [100, 50], 2, 64, 16)
    k, v = c.tensors(23)
    c.fill(k, v)
    assert ec.status() == 0
    q = torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    out = torch.empty_like(q)

    def flagged(fn):
        fn()
        assert ec.status() == -5 and ec.status() == 0

    good = c.table.clone()
    for bad in (-1, c.n_pages, 1 << 30, -(1 << 31)):
        c.table[0, 2] = bad
        flagged(lambda: ec.kv_attend(c.cache, 0, c.seqs, q, out))
        flagged(lambda: c.fill(k, v))
        flagged(lambda: c.read())
        c.table.copy_(good)
    c.dlens[1] = 1 << 20  # more than the table's row holds
    flagged(lambda: ec.kv_attend(c.cache, 0, c.seqs, q, out))
    c.dlens[1] = 50
    for starts in ([0, 1, 5], [0, -1, 2], [2, 1, 0], [0, 1 << 30, 2]):
        flagged(lambda: ec.kv_attend(c.cache, 0, c.seqs, q, out, starts=i32(starts), max_new=2))
        flagged(lambda: ec.kv_append(c.cache, 0, c.seqs, k[:2], v[:2], starts=i32(starts), max_new=2))
    flagged(lambda: ec.kv_attend(c.cache, 0, c.seqs, q, out, starts=i32([0, 2, 2]), max_new=1))
    c.fill(k, v)
    check_attend(ec, c, k, v, [1, 1], 2)


def test_empty_calls(ec):
    c = Case(ec, [4], 2, 64, 16)
    none = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    seqs = ec.kv_seqs(torch.empty((0, 3), dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"))
    ec.kv_append(c.cache, 0, seqs, none, none)
    ec.kv_read(c.cache, 0, seqs, none, none)
    ec.kv_attend(c.cache, 0, seqs, none, none)
    assert ec.status() == 0


# ------------------------------------------------------------------ pages
def family(rng, n, to, lo=-1):
    return [rng.randint(lo, n - 1) for _ in range(to)]


@pytest.mark.parametrize("seed", range(8))
def test_fork(ec, seed):
    r = random.Random(seed)
    page = r.choice([16, 32, 64])
    n, to = r.randint(1, 9), r.randint(1, 40)
    lens = [r.choice([0, 1, page - 1, page, page + 1, r.randint(0, 5 * page), -1]) for _ in range(n)]
    tight = seed % 2
    c = Case(ec, lens, 2, 64, page, seed, layers=2, spare=r.randint(0, 12) if tight else 4 * to)
    c.pool.random_(0, 256)
    width = max(len(c.rows[0]), 6) if not tight else 5
    if seed == 3:
        parents, to = list(range(n)), n
    else:
        parents = family(r, n, to)
    grow = [r.choice([0, 1, page, r.randint(0, 2 * page)]) for _ in range(to)]
    refs = [0] * c.n_pages
    for row in c.rows:
        for p in row:
            if p >= 0:
                refs[p] += 1
    if c.n_pages > 2:  # a table that is not in this call holds these
        for p in r.sample(range(c.n_pages), 2):
            refs[p] += 1
    drefs, refs_out = i32(refs), torch.full((c.n_pages,), 77, dtype=torch.int32, device="cuda")
    to_seqs = ec.kv_seqs(torch.full((to, width), 55, dtype=torch.int32, device="cuda"), torch.full((to,), 55, dtype=torch.int32, device="cuda"))
    before = c.pool.clone()
    ec.kv_fork(c.cache, c.seqs, drefs, to_seqs, refs_out, parents=None if seed == 3 else i32(parents), grow=i32(grow))
    assert ec.status() == 0
    rows, out_lens, out_refs, copies = R.fork(page, c.n_pages, c.rows, lens, refs, parents, grow, width)
    assert to_seqs.lens.cpu().tolist() == out_lens
    assert to_seqs.table.cpu().tolist() == rows
    assert refs_out.cpu().tolist() == out_refs
    for s, d, u in copies:
        before[d, :, :, :u] = before[s, :, :, :u]
    assert torch.equal(c.pool, before)
    assert drefs.cpu().tolist() == refs


def test_fork_in_a_large_pool(ec):
    """More pages than the counts in shared memory hold; new pages come from far into the pool."""
    c = Case(ec, [40, 90, 7], 1, 64, 16, spare=40000)
    refs = [1] * c.n_pages
    for p in range(30000, c.n_pages, 7):
        refs[p] = 0
    for row in c.rows:
        for p in row:
            if p >= 0:
                refs[p] = 1
    parents, grow = [1, 1, 0, 1, -1], [0, 40, 100, 3, 9]
    to = ec.kv_seqs(torch.zeros((5, 12), dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda"))
    out = torch.empty(c.n_pages, dtype=torch.int32, device="cuda")
    c.pool.random_(0, 256)
    before = c.pool.clone()
    ec.kv_fork(c.cache, c.seqs, i32(refs), to, out, parents=i32(parents), grow=i32(grow))
    assert ec.status() == 0
    rows, lens, new_refs, copies = R.fork(16, c.n_pages, c.rows, c.lens, refs, parents, grow, 12)
    assert to.table.cpu().tolist() == rows and to.lens.cpu().tolist() == lens and out.cpu().tolist() == new_refs
    for s, d, u in copies:
        before[d, :, :, :u] = before[s, :, :, :u]
    assert torch.equal(c.pool, before)


def test_mixed_types(ec):
    """Keys and values of one append have one type; what is read may have two."""
    c = Case(ec, [20], 1, 64, 16)
    k, v = c.tensors(7, BF16)
    for bad in (k.float(), k.to(FP16)):
        with pytest.raises(ec.EcError) as x:
            c.fill(bad, v)
        assert x.value.code == -4
    c.fill(k, v)
    a, b = torch.empty((20, 1, 64), device="cuda"), torch.empty((20, 1, 64), dtype=FP16, device="cuda")
    ec.kv_read(c.cache, 0, c.seqs, a, b, starts=starts_of([20]), max_new=20)
    assert np.array_equal(a.double().cpu().numpy(), R.stored(k.double().cpu().numpy()))
    assert torch.equal(b, c.read()[1].to(FP16))


def test_fork_without_growth_and_to_nothing(ec):
    c = Case(ec, [40, 16], 1, 64, 16, layers=1, spare=5)
    refs = i32([1 if any(p in row for row in c.rows) else 0 for p in range(c.n_pages)])
    out = torch.empty_like(refs)
    none = ec.kv_seqs(torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"))
    ec.kv_fork(c.cache, c.seqs, refs, none, out, parents=torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.sum().item() == 0  # all freed
    same = ec.kv_seqs(torch.empty_like(c.table), torch.empty_like(c.dlens))
    ec.kv_fork(c.cache, c.seqs, refs, same, out)
    assert torch.equal(same.table, c.table) and torch.equal(same.lens, c.dlens) and torch.equal(out, refs)
    assert ec.status() == 0
    ec.kv_fork(c.cache, c.seqs, refs, same, out, parents=i32([0, 7]))
    assert ec.status() == -5  # a parent that is none
    assert same.lens.cpu().tolist() == [40, 0]
    bad = c.table.clone()
    bad[0, 1] = 1 << 20
    ec.kv_fork(c.cache, ec.kv_seqs(bad, c.dlens), refs, same, out, parents=i32([1, 1]))
    assert ec.status() == -5


@pytest.mark.parametrize("seed", range(6))
def test_compact(ec, seed):
    r = random.Random(seed)
    page = r.choice([16, 32, 128])
    lens = [r.randint(0, 6 * page) for _ in range(r.randint(1, 12))]
    c = Case(ec, lens, 3, 64, page, seed, layers=2, spare=r.choice([0, 1, 30, 3000 if seed == 5 else 9]))
    c.pool.random_(0, 256)
    for i in range(1, len(c.rows), 2):  # shared first pages
        n = min(-(-lens[i] // page), -(-lens[i - 1] // page)) // 2
        c.rows[i][:n] = c.rows[i - 1][:n]
    c.table.copy_(i32(c.rows))
    refs = [0] * c.n_pages
    for row in c.rows:
        for p in row:
            if p >= 0:
                refs[p] += 1
    out, refs_out, to_map = (torch.full((n,), 33, dtype=torch.int32, device="cuda") for n in (len(lens), c.n_pages, c.n_pages))
    to = ec.kv_seqs(torch.full_like(c.table, 44), out)
    before = c.pool.clone()
    ec.kv_compact(c.cache, c.seqs, i32(refs), to, refs_out, page_map=to_map if seed % 2 else None)
    assert ec.status() == 0
    rows, new_refs, m, moves = R.compact(c.rows, refs)
    assert to.table.cpu().tolist() == rows and to.lens.cpu().tolist() == lens
    assert refs_out.cpu().tolist() == new_refs
    if seed % 2:
        assert to_map.cpu().tolist() == m
    for s, d in moves:
        before[d] = before[s]
    assert torch.equal(c.pool, before)


def test_beams_decode_as_one_would(ec):
    """Append, attend, fork and compact together: beams over several steps give what
    separate sequences with the same tokens give."""
    r = random.Random(1)
    page, kvh, dim, qh, layers = 16, 2, 64, 4, 2
    n_pages, width, beams = 60, 8, 4
    cache = ec.kv_cache(layers, n_pages, kvh, dim, page)
    cache.pool.fill_(255)
    refs, spare = (torch.zeros(n_pages, dtype=torch.int32, device="cuda") for _ in range(2))
    cur = ec.kv_seqs(torch.full((beams, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(beams, dtype=torch.int32, device="cuda"))
    nxt = ec.kv_seqs(cur.table.clone(), cur.lens.clone())
    text = [[] for _ in range(beams)]  # the (k, v) rows of each beam
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for step in range(40):
        parents = list(range(beams)) if step % 3 else [r.randrange(beams) for _ in range(beams)]
        grow = [r.choice([1, 1, 3]) for _ in range(beams)]
        ec.kv_fork(cache, cur, refs, nxt, spare, parents=i32(parents), grow=i32(grow))
        cur, nxt, refs, spare = nxt, cur, spare, refs
        kv = torch.randn((2, layers, sum(grow), kvh, dim), generator=g, device="cuda")
        q = torch.randn((layers, sum(grow), qh, dim), generator=g, device="cuda")
        text = [list(text[p]) for p in parents]
        at = 0
        for i, m in enumerate(grow):
            text[i] += [kv[:, :, at + j] for j in range(m)]
            at += m
        if step == 20:
            ec.kv_compact(cache, cur, refs, nxt, spare)
            cur, nxt, refs, spare = nxt, cur, spare, refs
        for layer in range(layers):
            ec.kv_append(cache, layer, cur, kv[0, layer], kv[1, layer], starts=starts_of(grow), max_new=3)
            out = torch.empty((sum(grow), qh, dim), device="cuda")
            ec.kv_attend(cache, layer, cur, q[layer], out, starts=starts_of(grow), max_new=3, window=60, sinks=2)
            if step % 8 == 7 or step == 20:
                at = 0
                for i, m in enumerate(grow):
                    t = torch.stack(text[i])[:, :, layer].double().cpu().numpy()
                    ks, vs = (torch.from_numpy(R.stored(t[:, x])).cuda() for x in (0, 1))
                    w = R.attend(q[layer, at:at + m].double(), ks, vs, len(text[i]) - m, None, 60, 2)
                    e, _ = R.bounds(w, len(text[i]), FP32, 2.0 ** -22)
                    assert bool(((out[at:at + m].double() - w.out).abs() <= e).all())
                    at += m
        keep = min(len(t) for t in text)
        assert keep <= width * page
        if keep > 100:
            break
    assert ec.status() == 0
