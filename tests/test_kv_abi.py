"""The 4-bit cache's C ABI on the CPU: sizes, argument checks, and the 64-bit forms that
the GPU tests compare with against their definitions."""
import ctypes

import numpy as np
import pytest
import torch

import kv_ref as R


@pytest.fixture(scope="module")
def ec():
    from lossless_entropy_coded_gb300 import build
    build.build()
    import lossless_entropy_coded_gb300 as ec
    return ec


@pytest.fixture(scope="module")
def e(ec):
    from lossless_entropy_coded_gb300 import _ec
    return _ec


def test_pool_bytes(ec, e):
    # 32 layers x 8 heads x 128 channels: 4.25 bits for every key and value
    assert ec.kv_pool_bytes(32, 10, 8, 128, 64) == 10 * 32 * 8 * 64 * 2 * 128 * 17 // 32
    for args, code in (((0, 1, 1, 64, 16), e.EC_ERR_SHAPE), ((1, 0, 1, 64, 16), e.EC_ERR_SHAPE),
                       ((1, 1, -1, 64, 16), e.EC_ERR_SHAPE), ((1, 1, 1, 96, 16), e.EC_ERR_UNSUPPORTED),
                       ((1, 1, 1, 64, 48), e.EC_ERR_UNSUPPORTED), ((1, 1, 1, 64, 512), e.EC_ERR_UNSUPPORTED),
                       ((1025, 1, 1, 64, 16), e.EC_ERR_UNSUPPORTED), ((1, (1 << 30) + 1, 1, 64, 16), e.EC_ERR_UNSUPPORTED),
                       ((1024, 1 << 30, 1024, 256, 256), e.EC_ERR_OVERFLOW)):
        with pytest.raises(ec.EcError) as x:
            ec.kv_pool_bytes(*args)
        assert x.value.code == code, args
    assert ec.lib.ec_kv_pool_bytes(None, None) == e.EC_ERR_INVALID_ARG


def test_create(ec, e):
    p = e.KvParams(2, 4, 128, 64, 100)
    h = ctypes.c_void_p()
    lib = ec.lib
    assert lib.ec_kv_create(ctypes.byref(p), None, 0, -1, None) == e.EC_ERR_INVALID_ARG
    assert lib.ec_kv_create(None, None, 0, -1, ctypes.byref(h)) == e.EC_ERR_INVALID_ARG
    need = ec.kv_pool_bytes(2, 100, 4, 128, 64)
    for pool, n in ((0, need), (4096 + 8, need), (4096, need - 1)):  # none, misaligned, too small
        assert lib.ec_kv_create(ctypes.byref(p), pool, n, 0, ctypes.byref(h)) == e.EC_ERR_INVALID_ARG
        assert not h.value
    lib.ec_kv_free(None)
    c = ec.kv_cache(2, 100, 4, 128, 64, device=-1)
    c.free()
    c.free()


class Seqs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p), ("n_seqs", ctypes.c_int32)]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class Attn(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("scale", ctypes.c_float)]


class Tokens(ctypes.Structure):
    _fields_ = [("seqs", Seqs), ("starts", ctypes.c_void_p), ("n_rows", ctypes.c_int64), ("layer", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("k", Rows), ("v", Rows)]


class Attention(ctypes.Structure):
    _fields_ = [("seqs", Seqs), ("starts", ctypes.c_void_p), ("n_rows", ctypes.c_int64), ("layer", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("max_len", ctypes.c_int64), ("attn", Attn), ("q", Rows), ("out", Rows),
                ("lse", ctypes.c_void_p), ("work", ctypes.c_void_p), ("work_bytes", ctypes.c_size_t)]


class Pages(ctypes.Structure):
    _fields_ = [("frm", Seqs), ("to", Seqs), ("refs", ctypes.c_void_p), ("refs_out", ctypes.c_void_p), ("parents", ctypes.c_void_p),
                ("grow", ctypes.c_void_p), ("map", ctypes.c_void_p), ("work", ctypes.c_void_p), ("work_bytes", ctypes.c_size_t)]


def test_packed_arguments_have_the_structures_sizes(e):
    for a, b in ((e._SEQS, Seqs), (e._ROWS, Rows), (e._TOKENS, Tokens), (e._ATTENTION, Attention), (e._PAGES, Pages)):
        assert a.size == ctypes.sizeof(b)


class Host:
    """A cache without a device and arguments that are right otherwise (host addresses that
    no call gets as far as using)."""

    def __init__(self, ec, e, heads=4, dim=128):
        self.ec, self.e, self.lib = ec, e, ec.lib
        self.cache = ec.kv_cache(2, 100, heads, dim, 64, device=-1)
        self.buf = np.zeros(1 << 16, np.int32)
        self.at = self.buf.ctypes.data & ~15
        self.seqs = (self.at, 10, self.at, 3)
        self.rows = (self.at, heads * dim, dim, 0)
        self.attn = (4 * heads, 0, 0, 0.0)

    def append(self, fn="ec_kv_append", cache=0, args=0, seqs=None, n_rows=3, layer=0, max_new=1, k=None, v=None):
        t = Tokens(Seqs(*(seqs or self.seqs)), 0, n_rows, layer, max_new, Rows(*(k or self.rows)), Rows(*(v or self.rows)))
        return getattr(self.lib, fn)(self.cache.handle if cache == 0 else cache, ctypes.addressof(t) if args == 0 else args, None)

    def attend(self, cache=0, args=0, seqs=None, n_rows=3, layer=0, max_new=1, max_len=0, attn=None, q=None, out=None, lse=0, work=0, n=0):
        t = Attention(Seqs(*(seqs or self.seqs)), 0, n_rows, layer, max_new, max_len, Attn(*(attn or self.attn)),
                      Rows(*(q or self.rows)), Rows(*(out or self.rows)), lse, work, n)
        return self.lib.ec_kv_attend(self.cache.handle if cache == 0 else cache, ctypes.addressof(t) if args == 0 else args, None)


@pytest.fixture()
def host(ec, e):
    return Host(ec, e)


@pytest.mark.parametrize("fn", ["ec_kv_append", "ec_kv_read"])
def test_append_and_read_refuse(host, e, fn):
    at = host.at
    assert host.append(fn) == e.EC_ERR_INVALID_ARG  # no pool: every check before that passed
    assert host.append(fn, cache=None) == e.EC_ERR_INVALID_ARG and host.append(fn, args=None) == e.EC_ERR_INVALID_ARG
    for layer in (-1, 2):
        assert host.append(fn, layer=layer) == e.EC_ERR_INVALID_ARG
    for s, code in (((0, 10, at, 3), e.EC_ERR_INVALID_ARG), ((at, 10, 0, 3), e.EC_ERR_INVALID_ARG), ((at, -1, at, 3), e.EC_ERR_SHAPE),
                    ((at, 10, at, -1), e.EC_ERR_SHAPE), ((at, 10, at, 1025), e.EC_ERR_UNSUPPORTED)):
        assert host.append(fn, seqs=s, n_rows=2000) == code, s
    assert host.append(fn, n_rows=-1) == e.EC_ERR_SHAPE and host.append(fn, max_new=-1) == e.EC_ERR_SHAPE
    assert host.append(fn, n_rows=2) == e.EC_ERR_SHAPE  # fewer rows than sequences, one each
    assert host.append(fn, max_new=(1 << 24) + 1) == e.EC_ERR_UNSUPPORTED
    for r, code in (((at, 512, 128, 1), e.EC_ERR_INVALID_ARG), ((at, 512, 128, 9), e.EC_ERR_INVALID_ARG),
                    ((at + 1, 512, 128, 0), e.EC_ERR_INVALID_ARG), ((at + 2, 512, 128, 4), e.EC_ERR_INVALID_ARG),
                    ((at, -512, 128, 0), e.EC_ERR_SHAPE), ((at, 512, -128, 0), e.EC_ERR_SHAPE),
                    ((at, 1 << 60, 128, 0), e.EC_ERR_OVERFLOW), ((at, 512, 1 << 60, 0), e.EC_ERR_OVERFLOW)):
        assert host.append(fn, k=r) == code, r
        assert host.append(fn, v=r) == code, r
    none = (0, 512, 128, 0)
    assert host.append(fn, k=none) == e.EC_ERR_INVALID_ARG and host.append(fn, k=none, v=none) == e.EC_ERR_INVALID_ARG


def test_attend_refuses(host, e):
    a, at = ctypes.addressof, host.at
    assert host.attend() == e.EC_ERR_INVALID_ARG
    assert host.attend(cache=None) == e.EC_ERR_INVALID_ARG and host.attend(args=None) == e.EC_ERR_INVALID_ARG
    assert host.attend(layer=2) == e.EC_ERR_INVALID_ARG
    for t, code in (((15, 0, 0, 0), e.EC_ERR_SHAPE), ((0, 0, 0, 0), e.EC_ERR_SHAPE), ((16, -1, 0, 0), e.EC_ERR_INVALID_ARG),
                    ((16, 5, -1, 0), e.EC_ERR_INVALID_ARG), ((16, 0, 3, 0), e.EC_ERR_INVALID_ARG), ((16, 0, 0, -1.0), e.EC_ERR_INVALID_ARG),
                    ((16, 0, 0, float("nan")), e.EC_ERR_INVALID_ARG), ((16, 0, 0, float("inf")), e.EC_ERR_INVALID_ARG)):
        assert host.attend(attn=t) == code, t
    assert host.attend(max_len=-1) == e.EC_ERR_SHAPE
    for r, code in (((0, 512, 128, 0), e.EC_ERR_INVALID_ARG), ((at, 512, 128, 2), e.EC_ERR_INVALID_ARG), ((at, -1, 128, 0), e.EC_ERR_SHAPE)):
        assert host.attend(q=r) == code and host.attend(out=r) == code
    assert host.attend(lse=at + 2) == e.EC_ERR_INVALID_ARG
    assert host.attend(seqs=(at, 10, at, 1025), n_rows=2000) == e.EC_ERR_UNSUPPORTED and host.attend(n_rows=2) == e.EC_ERR_SHAPE
    n, own = ctypes.c_size_t(), Attn(*host.attn)
    lib = host.lib
    assert lib.ec_kv_attend_work_bytes(host.cache.handle, 3, 3, 1, 640, a(own), None) == e.EC_ERR_INVALID_ARG
    assert lib.ec_kv_attend_work_bytes(None, 3, 3, 1, 640, a(own), a(n)) == e.EC_ERR_INVALID_ARG
    assert lib.ec_kv_attend_work_bytes(host.cache.handle, -3, 3, 1, 640, a(own), a(n)) == e.EC_ERR_SHAPE
    assert lib.ec_kv_attend_work_bytes(host.cache.handle, 3, 3, 1, 640, a(own), a(n)) == 0


def test_pages_refuse(host, e, ec):
    a, at, lib = ctypes.addressof, host.at, host.lib
    need = ec.kv_pages_work_bytes(host.cache, 3, 5)
    assert need > 0
    far = at + 40000
    frm, to = (at, 10, at + 4096, 3), (far, 10, far + 4096, 3)

    def call(name, c, f, r, t, o, m, w, n):
        x = Pages(Seqs(*f), Seqs(*t), r, o, 0, 0, m, w, n)
        return getattr(lib, name)(c, a(x), None)

    def fork(c=host.cache.handle, f=frm, r=at + 8192, t=to, o=far + 8192, w=at + 16384, n=1 << 20):
        return call("ec_kv_fork", c, f, r, t, o, 0, w, n)

    def compact(c=host.cache.handle, f=frm, r=at + 8192, t=to, o=far + 8192, m=0, w=at + 16384, n=1 << 20):
        return call("ec_kv_compact", c, f, r, t, o, m, w, n)

    assert lib.ec_kv_fork(host.cache.handle, None, None) == e.EC_ERR_INVALID_ARG
    assert lib.ec_kv_compact(host.cache.handle, None, None) == e.EC_ERR_INVALID_ARG
    for fn in (fork, compact):
        assert fn() == e.EC_ERR_INVALID_ARG  # no pool
        assert fn(c=None) == e.EC_ERR_INVALID_ARG
        assert fn(r=0) == e.EC_ERR_INVALID_ARG and fn(o=0) == e.EC_ERR_INVALID_ARG and fn(w=0) == e.EC_ERR_INVALID_ARG
        assert fn(w=at + 8) == e.EC_ERR_INVALID_ARG and fn(n=63) == e.EC_ERR_INVALID_ARG
        assert fn(o=at + 8192 + 16) == e.EC_ERR_INVALID_ARG  # overlaps refs
        assert fn(t=(at + 8, 10, far, 3)) == e.EC_ERR_INVALID_ARG
        assert fn(t=(far, 10, far + 4096, 2)) == e.EC_ERR_SHAPE
    assert compact(t=(far, 9, far + 4096, 3)) == e.EC_ERR_SHAPE
    assert compact(m=at + 8192) == e.EC_ERR_INVALID_ARG
    with pytest.raises(ec.EcError):
        ec.kv_pages_work_bytes(host.cache, 1025, 1)


def test_binding_refuses_host_tensors_and_types(ec, e):
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for t, n in ((table, lens), (table.long(), lens), (table.T, lens), (table[0], lens), (table, lens[:1])):
        with pytest.raises(ec.EcError):
            ec.kv_seqs(t, n)
    cache = ec.kv_cache(1, 4, 2, 64, 16, device=-1)

    class Some:
        n, packed, pages, device = 2, bytes(32), 3, -1
    x = torch.zeros((2, 2, 64))
    for k in (x, x.double(), x[..., :32], x[:, :1], x.transpose(1, 2)):
        with pytest.raises(ec.EcError):
            ec.kv_append(cache, 0, Some, k, k)
        with pytest.raises(ec.EcError):
            ec.kv_attend(cache, 0, Some, k, k, work=x)
    with pytest.raises(ec.EcError):
        ec.kv_cache(1, 4, 2, 64, 16, pool=torch.zeros(1 << 20, dtype=torch.uint8), device=0)


# ------------------------------------------------------------------ the 64-bit forms themselves
def test_quantiser_against_a_search():
    """Brute force over all scales and levels: the scale is the smallest that needs no
    clipping, each element the nearest level."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 32)) * 2.0 ** rng.integers(-20, 20, (200, 1))
    x[0], x[1] = 0, 6.0
    x[2, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    x[2, 8:] = 0
    codes, byte = R.quantise(x)
    v = R.values(codes, byte)
    for i in range(200):
        top = np.abs(x[i]).max()
        if top == 0:
            assert byte[i, 0] == 0 and not codes[i].any()
            continue
        fits = [e for e in range(1, 255) if top <= 6 * 2.0 ** (e - 127)]
        assert byte[i, 0] == fits[0]
        grid = np.concatenate([-R.LEVELS, R.LEVELS]) * 2.0 ** (fits[0] - 127)
        assert np.array_equal(np.abs(v[i] - x[i]), np.abs(grid[:, None] - x[i]).min(0))
    assert v[2, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]  # ties


def test_units_take_every_place_once():
    for dim in (64, 128, 192, 256):
        rng = np.random.default_rng(dim)
        kc, vc = (rng.integers(0, 16, (16, dim)).astype(np.uint8) for _ in range(2))
        ks, vs = (rng.integers(0, 256, (16, dim // 32)).astype(np.uint8) for _ in range(2))
        u = R.unit_bytes(kc, ks, vc, vs)
        nib = lambda x: np.bincount(np.concatenate([x & 15, x >> 4]), minlength=16)
        assert np.array_equal(nib(u[:8 * dim]), np.bincount(kc.ravel(), minlength=16))
        assert np.array_equal(nib(u[8 * dim:16 * dim]), np.bincount(vc.ravel(), minlength=16))
        assert np.array_equal(np.sort(u[16 * dim:16 * dim + dim // 2]), np.sort(ks.ravel()))
        assert np.array_equal(np.sort(u[16 * dim + dim // 2:]), np.sort(vs.ravel()))


def test_attention_form_on_a_case_by_hand():
    q = torch.tensor([[[1.0] + [0.0] * 31]], dtype=torch.float64).repeat(2, 1, 1)
    k = torch.zeros((3, 1, 32), dtype=torch.float64)
    k[1, 0, 0] = np.log(3.0)
    v = torch.arange(3, dtype=torch.float64)[:, None, None].repeat(1, 1, 32)
    r = R.attend(q, k, v, 1, scale=1.0)
    assert torch.allclose(r.out[0], torch.tensor(3 / 4, dtype=torch.float64))      # weights 1, 3
    assert torch.allclose(r.out[1], torch.tensor(1.0, dtype=torch.float64))        # weights 1, 3, 1
    assert torch.allclose(r.lse, torch.log(torch.tensor([[4.0], [5.0]], dtype=torch.float64)))
    w = R.attend(q, k, v, 1, scale=1.0, window=1)
    assert w.out[0, 0, 0] == 1 and w.out[1, 0, 0] == 2
    w = R.attend(q, k, v, 1, scale=1.0, window=1, sinks=1)
    assert w.out[1, 0, 0] == 1 and R.attend(q, k, v, -1).out[0].abs().max() == 0


def test_page_rules_on_a_case_by_hand():
    # pages of 16: sequence 0 has 20 tokens in pages 3, 1; sequence 1 has 5 in page 0
    rows, lens, refs, copies = R.fork(16, 6, [[3, 1], [0, -1]], [20, 5], [1, 1, 0, 1, 0, 0], [0, 0, -1], [0, 13, 4], 3)
    assert rows == [[3, 1, -1], [3, 0, 2], [-1, -1, -1]] and lens == [20, 33, 0]
    assert refs == [1, 1, 1, 2, 0, 0] and copies == [(1, 0, 1)]
    rows, lens, refs, _ = R.fork(16, 4, [[3, 1], [0, 2]], [20, 32], [1, 1, 1, 1], [0, 1], [20, 1], 3)
    assert lens == [-1, -1] and refs == [0, 0, 0, 0]  # nothing is free
    out, refs, m, moves = R.compact([[3, 1], [5, -1]], [0, 1, 0, 2, 0, 1])
    assert out == [[0, 1], [2, -1]] and refs == [2, 1, 1, 0, 0, 0] and m == [-1, 1, -1, 0, -1, 2] and moves == [(3, 0), (5, 2)]
