"""What ec_kv_attend_work_bytes answers on the CPU: sizes at the ends of their ranges."""
import os
import subprocess
import sys

import pytest
import torch

INT_MAX = 2 ** 31 - 1
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ec():
    from lossless_entropy_coded_gb300 import build
    build.build()
    import lossless_entropy_coded_gb300 as ec
    return ec


@pytest.fixture(scope="module")
def cache(ec):
    return ec.kv_cache(1, 100, 8, 128, 64, device=-1)


@pytest.mark.parametrize("max_new", [1, 5, 500])
@pytest.mark.parametrize("max_len", [100, 8192, 400000])
def test_sinks_and_windows_past_every_token(ec, cache, max_new, max_len):
    """As many sinks or as wide a window as a number holds: the same as all tokens."""
    def work(window, sinks):
        return ec.kv_attend_work_bytes(cache, 4, 4 * max_new, 32, max_new, max_len, window, sinks)
    whole = work(0, 0)
    for sinks in (max_len, max_len + 1, INT_MAX - 16, INT_MAX - 14, INT_MAX):
        assert work(64, sinks) == work(64, max_len) == whole, sinks
        assert work(max_len - 1, sinks) == whole
        assert work(INT_MAX, sinks) == whole
    for window in (max_len, INT_MAX - 16, INT_MAX):
        assert work(window, 0) == work(window, 4) == whole, window


def test_rows_past_31_bits_are_refused(ec):
    """Row numbers of a key/value head, rounded up to a tile, have to fit 31 bits."""
    cache = ec.kv_cache(1, 100, 1, 128, 64, device=-1)
    for heads, max_new in ((256, 1 << 24), (128, 1 << 24), (65536, 32768), (65536, 1 << 24)):
        with pytest.raises(ec.EcError) as x:
            ec.kv_attend_work_bytes(cache, 1, 1, heads, max_new, 1000)
        assert x.value.code == -4, (heads, max_new)
    for heads, max_new in ((64, 1 << 24), (256, 1 << 22), (65536, 16384)):
        ec.kv_attend_work_bytes(cache, 1, 1, heads, max_new, 1000)


def test_work_of_no_sequences(ec):
    """A call without sequences or new tokens, whatever its bounds, needs no buffer (the question
    is asked in a process of its own: a division by the number of row tiles would end it)."""
    code = ("import lossless_entropy_coded_gb300 as ec\n"
            "c = ec.kv_cache(1, 100, 8, 128, 64, device=-1)\n"
            "print([ec.kv_attend_work_bytes(c, n, 0, 32, m, 100000) for n, m in ((0, 1), (0, 500), (0, 5000), (3, 0))])")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    assert eval(r.stdout) == [0, 0, 0, 0]


SIZES = [(n, m, t) for n in (1, 2, 7, 64) for m in (1, 2, 5, 9, 16, 64, 100, 400, 5003) for t in (1, 100, 700, 3000, 20000, 500000)]


@pytest.mark.parametrize("heads,kvh,dim", [(32, 8, 128), (8, 8, 64), (48, 1, 128), (12, 4, 192), (16, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (600, 4)])
def test_a_buffer_for_larger_sizes_serves_smaller_ones(ec, heads, kvh, dim, window, sinks):
    """The work size grows with every bound, so one buffer for the largest serves all."""
    cache = ec.kv_cache(1, 100, kvh, dim, 64, device=-1)
    work = {s: ec.kv_attend_work_bytes(cache, s[0], s[0] * s[1], heads, s[1], s[2], window, sinks) for s in SIZES}
    for a in SIZES:
        for b in SIZES:
            if all(x <= y for x, y in zip(a, b)):
                assert work[a] <= work[b], (a, b)
    for n, m, t in SIZES:  # fewer rows of the same bounds
        assert ec.kv_attend_work_bytes(cache, n, 1, heads, m, t, window, sinks) <= work[n, m, t]


@pytest.mark.parametrize("max_new", [1, 5, 100])
@pytest.mark.parametrize("window", [0, 600])
def test_a_buffer_for_any_length(ec, cache, max_new, window):
    """max_len 0 is any length, as in the call itself, and serves all."""
    any_len = ec.kv_attend_work_bytes(cache, 4, 4 * max_new, 32, max_new, window=window)
    for t in (1, 100, 8192, 500000, INT_MAX - 15):
        assert ec.kv_attend_work_bytes(cache, 4, 4 * max_new, 32, max_new, t, window=window) <= any_len
    assert any_len > 0


def test_a_table_that_holds_more_than_a_sequence(ec):
    """The binding's own buffer is sized for the tokens that the call takes from such a table."""
    cache = ec.kv_cache(1, 100, 8, 128, 256, device=-1)

    class Some:
        n, packed, pages, device = 2, bytes(32), 1 << 24, -1
    x = torch.zeros((2, 8, 128))
    with pytest.raises(ec.EcError) as e:
        ec.kv_attend(cache, 0, Some, x, x)
    assert "work_bytes" not in str(e.value) and e.value.code == -1  # the library's answer: no pool


def test_a_work_tensor_has_to_hold_its_bytes(ec, cache):
    """An expanded or strided tensor has fewer bytes, or other ones, than its shape says."""
    class Some:
        n, packed, pages, device = 2, bytes(32), 3, -1
    x, refs = torch.zeros((2, 8, 128)), torch.zeros(100, dtype=torch.int32)
    for work in (torch.zeros(1, dtype=torch.uint8).expand(1 << 25), torch.zeros(1 << 10)[::2]):
        for call in (lambda: ec.kv_attend(cache, 0, Some, x, x.clone(), work=work), lambda: ec.kv_fork(cache, Some, refs, Some, refs.clone(), work=work),
                     lambda: ec.kv_compact(cache, Some, refs, Some, refs.clone(), work=work)):
            with pytest.raises(ec.EcError, match="contiguous"):
                call()
