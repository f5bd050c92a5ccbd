"""tc_rotary refuses an output that overlaps its input without being it, whatever their strides, and no other. Without a GPU: no
call has frequencies, so what passes that check is refused for them."""
import ctypes
import random

import pytest

from topology_construction_amd import binding

BASE = 1 << 20  # an address that is never read
SIZES = {0: 4, 1: 2, 2: 2}


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def _answer(lib, at_x, x, at_out, out, rows, heads, dim, dtype=0):
    """at_x, at_out: bytes; x, out: strides of rows and of heads."""
    sections = (ctypes.c_int32 * 1)(1)
    status = lib.tc_rotary(BASE + at_x, x[0], x[1], rows, heads, dim, dtype, BASE, 1, 1, sections, None, 0, 0, BASE + at_out, out[0],
                           out[1], None)
    assert status == 1
    return {b"d_out overlaps d_x without being d_x": "overlap", b"the rows or heads of d_out overlap": "itself",
            b"d_freqs is NULL": "fine"}[lib.tc_last_error()]


def _bytes(at, strides, rows, heads, dim, size):
    return {at + size * (r * strides[0] + h * strides[1] + c) + b for r in range(rows) for h in range(heads) for c in range(dim)
            for b in range(size)}


@pytest.mark.parametrize("dtype", [0, 1])
def test_against_the_bytes_themselves(lib, dtype):
    rng = random.Random(dtype)
    seen = {"overlap": 0, "itself": 0, "fine": 0}
    size = SIZES[dtype]
    for _ in range(4000):
        rows, heads, dim = rng.randint(1, 5), rng.randint(1, 4), rng.randint(2, 4)
        head = rng.choice((dim, dim, 2 * dim, rng.randint(dim, 3 * dim)))
        row = rng.choice((heads * head, 2 * heads * head, rng.randint(1, 4 * heads * head)))
        out = (row, head) if rng.random() < 0.7 else (head, rows * head)
        x = out if rng.random() < 0.6 else rng.choice(((0, head), (row, 0), (2 * row, head), (rng.randint(0, 40), rng.randint(0, 12))))
        at_x = 4 * 100
        at_out = at_x + (size * rng.randint(-60, 60) if rng.random() < 0.9 else rng.randint(-60, 60))
        same = at_x == at_out and (rows < 2 or x[0] == out[0]) and (heads < 2 or x[1] == out[1])
        answer = _answer(lib, at_x, x, at_out, out, rows, heads, dim, dtype)
        seen[answer] += 1
        if answer != "itself":
            shared = _bytes(at_x, x, rows, heads, dim, size) & _bytes(at_out, out, rows, heads, dim, size)
            assert answer == ("overlap" if shared and not same else "fine"), (at_x, x, at_out, out, rows, heads, dim)
    assert min(seen.values()) > 100


def test_parts_of_packed_rows(lib):
    """Queries, keys and values in one row of 3 x 16 heads of 64; a million rows."""
    rows, heads, dim = 1_000_000, 16, 64
    packed = (3 * heads * dim, dim)
    each = 4 * heads * dim
    assert _answer(lib, 0, packed, each, packed, rows, heads, dim) == "fine"
    assert _answer(lib, 2 * each, packed, 0, packed, rows, heads, dim) == "fine"
    assert _answer(lib, 0, packed, each - 4 * dim, packed, rows, heads, dim) == "overlap"
    assert _answer(lib, 0, packed, each - 4, packed, rows, heads, dim) == "overlap"
    assert _answer(lib, each, packed, 0, packed, rows, heads + 1, dim) == "overlap"
    assert _answer(lib, 0, packed, 2 * each + 4, packed, rows, heads, dim) == "overlap"  # the next row's first
    # every other head, every other row, heads before rows
    assert _answer(lib, 0, (64 * 32, 128), 4 * 64, (64 * 32, 128), rows, 16, 64) == "fine"
    assert _answer(lib, 0, (64 * 32, 128), 4 * 63, (64 * 32, 128), rows, 16, 64) == "overlap"
    assert _answer(lib, 0, (2 * 1024, 64), 4 * 1024, (2 * 1024, 64), rows, 16, 64) == "fine"
    assert _answer(lib, 0, (64, rows * 64), 4 * 16 * rows * 64, (64, rows * 64), rows, 16, 64) == "fine"
    assert _answer(lib, 0, (64, rows * 64), 4 * 15 * rows * 64, (64, rows * 64), rows, 16, 64) == "overlap"
    # one row for all, of the same buffer
    assert _answer(lib, 0, (0, 64), 4 * 1024, (3 * 1024, 64), rows, 16, 64) == "fine"
    assert _answer(lib, 4 * 1024, (0, 64), 0, (3 * 1024, 64), rows, 16, 64) == "fine"
    assert _answer(lib, 4 * 1000, (0, 64), 0, (3 * 1024, 64), rows, 16, 64) == "overlap"


def test_other_strides(lib):
    """Rows of one step among rows of two steps: told apart while they are few, refused where they are not."""
    assert _answer(lib, 0, (2048, 64), 4 * 64, (1024, 64), 1000, 1, 64) == "fine"
    assert _answer(lib, 0, (2048, 64), 4 * 63, (1024, 64), 1000, 1, 64) == "overlap"
    assert _answer(lib, 0, (2048, 64), 4 * 64, (1024, 64), 10_000_000, 1, 64) == "overlap"
    assert _answer(lib, 0, (2 ** 62, 2 ** 62), 8, (64, 2 ** 50), 1000, 2, 2) == "fine"
