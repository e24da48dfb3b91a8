"""Paths of the cache that only large or simultaneous calls take."""
import math
import random

import pytest
import torch

import kv_ref as R
from test_gpu_kv import BF16, FP32, Case, ec, i32, starts_of  # noqa: F401 (ec is a fixture)
from test_gpu_kv_rows import check, normal, row_bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("loud", [0, 20])
def test_a_tile_in_more_parts_than_a_warp_has_lanes(ec, loud):
    """One long sequence over one key/value head: every share of the GPU holds a part of its tile."""
    n = 200003
    c = Case(ec, [n], 1, 64, 64)
    k, v = normal(50, n, 1, 64) * 0.5, normal(51, n, 1, 64)
    k[n // 3] *= 6
    if loud:
        v[n // 2] *= 2.0 ** loud
    c.fill(k, v)
    held = c.read()
    q = normal(52, 1, 5, 64) * 2
    out, lse = torch.empty_like(q), torch.empty((1, 5), device="cuda")
    ec.kv_attend(c.cache, 0, c.seqs, q, out, lse=lse)
    again = torch.empty_like(q)
    ec.kv_attend(c.cache, 0, c.seqs, q, again)
    assert ec.status() == 0 and torch.equal(out, again)
    qd, kd, vd = q.double(), held[0].double(), held[1].double()
    r = R.attend(qd, kd, vd, n - 1)
    eo, el = row_bounds(r, qd, kd, vd, n - 1, None, 0, 0, FP32)
    assert bool(((out.double() - r.out).abs() <= eo).all()) and bool(((lse.double() - r.lse).abs() <= el).all())


def test_compaction_of_a_large_pool(ec):
    """More pages than one pass of the planning threads."""
    r = random.Random(4)
    lens = [r.randint(1, 9000) for _ in range(12)]
    c = Case(ec, lens, 1, 64, 16, 4, spare=9000)
    c.pool.random_(0, 256)
    refs = [0] * c.n_pages
    for row in c.rows:
        for p in row:
            if p >= 0:
                refs[p] += 1
    for p in r.sample(range(c.n_pages), 2000):  # held by tables that are not in this call
        refs[p] += 1
    to = ec.kv_seqs(torch.empty_like(c.table), torch.empty_like(c.dlens))
    out, page_map = torch.empty(c.n_pages, dtype=torch.int32, device="cuda"), torch.empty(c.n_pages, dtype=torch.int32, device="cuda")
    before = c.pool.clone()
    ec.kv_compact(c.cache, c.seqs, i32(refs), to, out, page_map=page_map)
    assert ec.status() == 0 and c.n_pages > 10000
    rows, new_refs, m, moves = R.compact(c.rows, refs)
    assert to.table.cpu().tolist() == rows and out.cpu().tolist() == new_refs and page_map.cpu().tolist() == m
    src, dst = zip(*moves)
    before[list(dst)] = before[list(src)]
    assert torch.equal(c.pool, before)


@pytest.mark.parametrize("new", [[1, 1], [200, 60]])
def test_calls_at_once_on_two_streams(ec, new):
    """Two calls on one cache, each with a work buffer of its own."""
    lens = [7000, 300]
    c = Case(ec, lens, 2, 128, 64)
    c.fill(normal(53, sum(lens), 2, 128), normal(54, sum(lens), 2, 128))
    qs = [normal(55 + i, sum(new), 8, 128).to(BF16) for i in range(2)]
    want, outs = [], [[torch.empty_like(q) for _ in range(30)] for q in qs]
    for q in qs:
        want.append(torch.empty_like(q))
        ec.kv_attend(c.cache, 0, c.seqs, q, want[-1], starts=starts_of(new), max_new=max(new))
    n = ec.kv_attend_work_bytes(c.cache, 2, sum(new), 8, max(new))
    works = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams, starts = [torch.cuda.Stream() for _ in range(2)], starts_of(new)
    torch.cuda.synchronize()
    for i in range(30):
        for s, q, o, w in zip(streams, qs, outs, works):
            ec.kv_attend(c.cache, 0, c.seqs, q, o[i], starts=starts, max_new=max(new), work=w, stream=s)
    torch.cuda.synchronize()
    assert ec.status() == 0
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)


@pytest.mark.parametrize("qh", [4, 80])
def test_loud_values_beside_nan(ec, qh):
    """What FP16 does not span, with keys and values of NaN that some rows see."""
    n = 300
    c = Case(ec, [n, 41], 1, 128, 32)
    k, v = normal(57, n + 41, 1, 128) * 0.5, normal(58, n + 41, 1, 128)
    v[::17] *= 2.0 ** 40
    v[n - 4, 0, 32:64] = math.nan
    v[20] = math.nan
    k[n - 2] = math.inf
    v[n + 30:n + 35] = 0
    c.fill(k, v)
    q = normal(59, 9, qh, 128)
    out, _ = check(ec, c, k, v, [6, 3], q, window=100, sinks=4)
    assert not torch.isnan(out[:2]).any() and torch.isnan(out[2:4, :, 32:64]).all() and not torch.isnan(out[2:4, :, :32]).any()
    assert torch.isnan(out[4:6]).all() and not torch.isnan(out[6:]).any()
