"""Angles as fractions of a turn (csrc/turn.cuh), built as plain C++ and compared with exact arithmetic."""
import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# 2^300 / 2 pi, from pi by Machin's formula in whole numbers
BITS = 300


def _turns():
    one = 1 << (BITS + 64)

    def atan(n):
        term, total, k = one // n, one // n, 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total

    pi = 4 * (4 * atan(5) - atan(239))
    return (1 << (2 * BITS + 64)) // (2 * pi)


TURNS = _turns()


def exact(f, scale=64):
    """f / 2 pi turns times 2^scale, modulo 2^scale, with 32 more bits."""
    num, den = f.as_integer_ratio()
    return (num * TURNS * 2 ** (scale + 32) // (den << BITS)) % 2 ** (scale + 32)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("turn")
    src, so = d / "turn.cc", d / "turn.so"
    src.write_text('#include "turn.cuh"\nextern "C" uint64_t turn_fraction(double f) { return pkv::turn_fraction(f); }\n'
                   'extern "C" void turns_of(const uint32_t *u, float *out, int64_t n)\n'
                   '{ for (int64_t i = 0; i < n; ++i) pkv::turn_of(u[i], out[2 * i], out[2 * i + 1]); }\n')
    subprocess.run([cxx, "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-x", "c++", "-I",
                    os.path.join(ROOT, "gqa_decode_attention_paged_gb300", "csrc"), str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.turn_fraction.restype, lib.turn_fraction.argtypes = ctypes.c_uint64, [ctypes.c_double]
    lib.turns_of.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64]
    return lib


def test_turn_fraction_is_the_nearest_64_bits_of_every_frequency(lib):
    rng = random.Random(3)
    freqs = [0.0, 1.0, -1.0, 2.0 ** 20, -2.0 ** 20, 2.0 ** 20 - 2.0 ** -33, 1e-300, 5e-324, 2.0 ** -62, 2.0 ** -63, 6.28318530717958]
    freqs += [base ** (-i / 64) for base in (1e4, 5e5, 1e6) for i in range(64)]
    freqs += [rng.choice([-1, 1]) * rng.uniform(0.5, 1) * 2.0 ** rng.randint(-80, 20) for _ in range(4000)]
    for f in freqs:
        off = (lib.turn_fraction(f) * 2 ** 32 - exact(f)) % 2 ** 96
        assert min(off, 2 ** 96 - off) <= 2 ** 31 + 2 ** 22, f  # half of the 64th bit, and 2^-74 of a turn


def test_the_angle_is_good_to_2_to_the_minus_32_of_a_turn_at_every_position(lib):
    """The kernel's own steps: the 64-bit product, and its top 32 bits rounded."""
    rng = random.Random(4)
    for _ in range(4000):
        f = rng.choice([-1, 1]) * rng.uniform(0.5, 1) * 2.0 ** rng.randint(-30, 20)
        pos = rng.choice([-1, 1]) * (2 ** 31 - 1 - rng.randint(0, 10 ** rng.randint(0, 9)))
        got = (((lib.turn_fraction(f) * pos % 2 ** 64) + 2 ** 31) % 2 ** 64) >> 32
        num, den = f.as_integer_ratio()
        want = (num * pos * TURNS * 2 ** 64 // (den << BITS)) % 2 ** 64
        off = (got * 2 ** 32 - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 2 ** 32, (f, pos)  # 2^-32 of a turn


def test_sine_and_cosine_are_within_0_73_of_a_last_place(lib):
    """A million angles of all sizes around every eighth of a turn, against double (good to 2^-29 of such a place)."""
    rng = np.random.default_rng(5)
    away = (2.0 ** rng.uniform(0, 29, 2 ** 20)).astype(np.int64) * rng.choice([-1, 1], 2 ** 20)
    u = (rng.integers(0, 8, 2 ** 20) * 2 ** 29 + away) % 2 ** 32
    u = np.concatenate([u, np.arange(8) * 2 ** 29, np.arange(8) * 2 ** 29 + 1, (np.arange(8) * 2 ** 29 - 1) % 2 ** 32])
    u32, got = u.astype(np.uint32), np.empty((len(u), 2), np.float32)
    lib.turns_of(u32.ctypes.data, got.ctypes.data, len(u))
    quarter, rest = (u + 2 ** 29) >> 30 & 3, (u + 2 ** 29) % 2 ** 30 - 2 ** 29
    a = rest * (np.pi * 2.0 ** -31)
    s, c = np.sin(a), np.cos(a)
    want = np.stack((np.choose(quarter, (s, c, -s, -c)), np.choose(quarter, (c, -s, -c, s))), -1)
    place = np.ldexp(1.0, np.frexp(np.where(want == 0, 1, want))[1] - 24)
    off = np.abs(got - want) / place
    assert off.max() <= 0.73 and off.mean() < 0.26
    assert (got[want == 0] == 0).all()
