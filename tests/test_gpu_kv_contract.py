"""What the cache's calls promise about lengths, sizes, windows, buffers and streams."""
import pytest
import torch

import kv_ref as R
from test_gpu_kv import FP32, Case, ec, i32, starts_of  # noqa: F401 (ec is a fixture)
from test_gpu_kv_rows import check, normal, row_bounds, stored

pytestmark = pytest.mark.gpu
INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("window,sinks", [(20, INT_MAX), (20, INT_MAX - 14), (20, 350), (INT_MAX, 0), (INT_MAX, INT_MAX), (349, INT_MAX)])
@pytest.mark.parametrize("qh", [4, 80])
def test_sinks_and_windows_past_every_token(ec, window, sinks, qh):
    """Sinks and windows of any size, also where rows lie before the first token."""
    lens, new = [350, 3, 40], [6, 5, 1]
    c = Case(ec, lens, 1, 128, 16)
    k, v = normal(30, sum(lens), 1, 128), normal(31, sum(lens), 1, 128)
    c.fill(k, v)
    check(ec, c, k, v, new, normal(32, sum(new), qh, 128), FP32, window=window, sinks=sinks)


def test_one_buffer_for_the_longest_chunk(ec):
    """A buffer sized once for the largest call serves every smaller one."""
    lens = [3000, 2500]
    c = Case(ec, lens, 2, 128, 64)
    c.fill(normal(33, sum(lens), 2, 128), normal(34, sum(lens), 2, 128))
    most = ec.kv_attend_work_bytes(c.cache, 2, 1000, 8, 500, 3000)
    work = torch.empty(most, dtype=torch.uint8, device="cuda")
    for new in ([500, 500], [400, 3], [100, 64], [20, 7], [12, 1], [9, 0], [1, 1]):
        for dtype in (torch.bfloat16, FP32):
            q = normal(35, sum(new), 8, 128).to(dtype)
            outs = [torch.empty_like(q) for _ in range(2)]
            ec.kv_attend(c.cache, 0, c.seqs, q, outs[0], starts=starts_of(new), max_new=max(new), max_len=3000, work=work)
            ec.kv_attend(c.cache, 0, c.seqs, q, outs[1], starts=starts_of(new), max_new=max(new), max_len=3000)
            assert ec.status() == 0 and torch.equal(outs[0], outs[1]), new


def test_buffers_sized_with_the_defaults(ec):
    """Sizes asked for without a length are accepted by a call without one."""
    lens = [9000, 3, 700, 5000]
    c = Case(ec, lens, 8, 128, 64)
    k, v = normal(36, sum(lens), 8, 128), normal(37, sum(lens), 8, 128)
    c.fill(k, v)
    work = torch.empty(ec.kv_attend_work_bytes(c.cache, 4, 4, 32), dtype=torch.uint8, device="cuda")
    q = normal(38, 4, 32, 128)
    a, b = torch.empty_like(q), torch.empty_like(q)
    ec.kv_attend(c.cache, 0, c.seqs, q, a, work=work)
    ec.kv_attend(c.cache, 0, c.seqs, q, b)
    assert ec.status() == 0 and torch.equal(a, b)


def streams_with_memory():
    return {s["stream"] for s in torch.cuda.memory_snapshot()}


@pytest.mark.parametrize("raw", [False, True])
def test_calls_on_a_stream_of_their_own_allocate_there(ec, raw):
    """Without a work buffer: neither the current stream's earlier work nor its later
    allocations share bytes with the call."""
    lens = [3000, 700]
    c = Case(ec, lens, 2, 128, 64, spare=9)
    c.fill(normal(39, sum(lens), 2, 128), normal(40, sum(lens), 2, 128))
    q = normal(41, 2, 8, 128)
    want = torch.empty_like(q)
    ec.kv_attend(c.cache, 0, c.seqs, q, want)
    refs = i32([sum(p in row for row in c.rows) for p in range(c.n_pages)])
    to = [ec.kv_seqs(torch.empty_like(c.table), torch.empty_like(c.dlens)) for _ in range(2)]
    refs_out = [torch.empty_like(refs) for _ in range(2)]
    ec.kv_fork(c.cache, c.seqs, refs, to[0], refs_out[0])
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    assert s.cuda_stream not in streams_with_memory()
    s.wait_stream(torch.cuda.current_stream())
    stream = s.cuda_stream if raw else s
    ec.kv_attend(c.cache, 0, c.seqs, q, out, stream=stream)
    ec.kv_fork(c.cache, c.seqs, refs, to[1], refs_out[1], stream=stream)
    s.synchronize()
    assert s.cuda_stream in streams_with_memory()
    assert torch.equal(out, want) and torch.equal(to[0].table, to[1].table) and torch.equal(refs_out[0], refs_out[1])
    ec.kv_attend(c.cache, 0, c.seqs, q, out, stream=0)  # the default stream by its handle
    torch.cuda.synchronize()
    assert torch.equal(out, want) and ec.status() == 0


@pytest.mark.parametrize("op", ["fork", "compact"])
def test_page_operations_flag_lengths_past_the_table(ec, op):
    """More tokens than a row of the table holds are an inconsistency, as in the other calls."""
    c = Case(ec, [40, 16], 1, 64, 16, spare=5)
    c.table.copy_(i32([[0, 1, 2, 3], [4, 5, 6, 7]]))  # every place of a row names a page
    refs = i32([1] * 8 + [0] * (c.n_pages - 8))
    out = torch.empty_like(refs)
    to = ec.kv_seqs(torch.empty_like(c.table), torch.empty_like(c.dlens))
    call = ec.kv_fork if op == "fork" else ec.kv_compact
    cap = c.table.shape[1] * 16
    for n, code in ((16, 0), (cap, 0), (cap + 1, -5), (1 << 30, -5), (2 ** 31 - 1, -5), (-3, 0)):
        c.dlens[1] = n
        call(c.cache, c.seqs, refs, to, out)
        assert ec.status() == code, n


def test_sequences_at_the_end_of_31_bits(ec):
    """2^31 - 16 tokens (most of them in one page that the table names again and again): new
    tokens, what a window sees of them, and the pages that a dropped sequence gives up."""
    n, pages, new = 2 ** 31 - 16, 1 << 23, 40
    cache = ec.kv_cache(1, 4, 1, 64, 256)
    cache.pool.fill_(255)
    table = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    table[0, -1], table[0, -2] = 2, 1
    seqs, starts = ec.kv_seqs(table, i32([n])), i32([0, new])
    k, v = normal(42, new, 1, 64), normal(43, new, 1, 64)
    ec.kv_append(cache, 0, seqs, k, v, starts=starts, max_new=100)
    held = torch.empty((2, new, 1, 64), device="cuda")
    ec.kv_read(cache, 0, seqs, held[0], held[1], starts=starts, max_new=100)
    assert ec.status() == 0
    assert torch.equal(held[0].double(), stored(k)) and torch.equal(held[1].double(), stored(v))
    for qh in (2, 80):
        q = normal(44, 3, qh, 64)
        out = torch.empty_like(q)
        ec.kv_attend(cache, 0, seqs, q, out, starts=i32([0, 3]), max_new=3, window=30)
        r = R.attend(q.double(), stored(k), stored(v), new - 3, None, 30)
        e, _ = row_bounds(r, q.double(), stored(k), stored(v), new - 3, None, 30, 0, FP32)
        assert ec.status() == 0 and bool(((out.double() - r.out).abs() <= e).all())
    refs, out = i32([pages - 2, 1, 1, 5]), torch.empty(4, dtype=torch.int32, device="cuda")
    none = ec.kv_seqs(torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"))
    for tokens in (n, 2 ** 31 - 1):
        seqs.lens.fill_(tokens)
        ec.kv_fork(cache, seqs, refs, none, out, parents=torch.empty(0, dtype=torch.int32, device="cuda"))
        assert ec.status() == 0 and out.tolist() == [0, 0, 0, 5], tokens
