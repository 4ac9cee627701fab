"""The rotary table's fractions of a turn and the refusals of overlapping
arguments (CPU: pointers here are made up, and a refused call reads nothing)."""
import ctypes
import math

import pytest

import varlen_gqa_split_b200 as vg

OK, INVALID = 0, -1


@pytest.fixture(scope="module")
def L():
    from varlen_gqa_split_b200 import build
    build.build()
    return vg.lib()


def _create(L, D=8, n=4, axes=2, freq=None):
    h = ctypes.c_void_p()
    f, a = (ctypes.c_double * n)(*(freq or [1.0] * n)), (ctypes.c_int32 * n)(*[0] * n)
    return L.attn_rope_create(ctypes.byref(h), D, n, axes, f, a, 0, 1.0), h


def _apply(L, h, x=0x10000, T=4, pos=0x900000, out=0x20000):
    return L.attn_rope_apply(h, 0, x, 16, T, 2, pos, 4, 0, out, 16, None)


def _one_over_two_pi(bits):
    """2^bits / 2 pi, rounded down, by Machin's formula in integers."""
    one = 1 << (bits + 64)

    def arctan_of_inverse(x):
        total, term, n, sign = 0, one // x, 1, 1
        while term:
            total += sign * (term // n)
            term //= x * x
            n, sign = n + 2, -sign
        return total

    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    return (1 << (2 * bits + 63)) // pi


def test_rope_table_turns_are_exact_for_frequencies_of_any_size(L):
    """The table's fractions of a turn against integer arithmetic, in units of
    2^-64: small frequencies and ones of many turns a position."""
    freqs = [1e4 ** (-i / 20) for i in range(20)]
    freqs += [0.5, 1.0, math.pi, 2 * math.pi, 6.0, 7.0, 100.0, 1e4, 12345.678, 1e15, 2.0 ** 100, 1e300, 5e-324, 0.0]
    freqs += [-f for f in freqs]
    rc, h = _create(L, D=256, n=len(freqs), axes=1, freq=freqs)
    assert rc == OK
    turns = (ctypes.c_uint64 * len(freqs)).from_address(h.value)       # the table is what the object begins with
    bits = 2300
    inv = _one_over_two_pi(bits)
    for f, got in zip(freqs, turns):
        num, den = abs(f).as_integer_ratio()
        exact = ((num * inv) << 64) // den >> bits                      # floor(|f| / 2 pi * 2^64)
        exact = (-exact if f < 0 else exact) % (1 << 64)
        off = (got - exact) % (1 << 64)
        assert min(off, (1 << 64) - off) <= 2 + 1, f                    # 2 units, and the floor's one
    L.attn_rope_destroy(h)


def test_rope_positions_lie_apart_from_the_result(L):
    rc, h = _create(L)                                       # D = 8, two axes, T = 4, H = 2: out is 128 bytes, pos 32
    assert rc == OK
    for pos in (0x20000, 0x20000 + 124, 0x20000 - 28, 0x20000 - 32 + 4):
        assert _apply(L, h, pos=pos) == INVALID
    assert _apply(L, h, pos=0x20000, x=0x20000, T=0) == OK   # nothing is read or written
    L.attn_rope_destroy(h)
