"""Host parts of the library that no entry point shows by itself, compiled alone (g++) and called."""
import ctypes
import os
import subprocess
import threading

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_kv_page_gb300", "csrc")


def compiled(tmp_path, name, code):
    src, lib = tmp_path / f"{name}.cpp", tmp_path / f"{name}.so"
    src.write_text(code)
    subprocess.run([os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC,
                    str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


# ------------------------------------------------------------ raise_once.h

@pytest.fixture
def limits(tmp_path):
    lib = compiled(tmp_path, "limits", '''
        #include "raise_once.h"
        extern "C" void* make() { return new locks::RaiseOnce; }
        extern "C" void drop(void* r) { delete static_cast<locks::RaiseOnce*>(r); }
        extern "C" int raise_to(void* r, int device, int value, int (*set)(int)) {
            return static_cast<locks::RaiseOnce*>(r)->raise(device, value, [&] { return set(value); });
        }''')
    lib.make.restype = ctypes.c_void_p
    lib.drop.argtypes = [ctypes.c_void_p]
    SET = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_int)
    lib.raise_to.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, SET]
    r = lib.make()
    yield lambda device, value, f: lib.raise_to(r, device, value, SET(f))
    lib.drop(r)


def test_a_limit_is_set_once_and_only_goes_up(limits):
    calls = []

    def ok(v):
        calls.append(v)
        return 0

    for device, value in ((0, 0), (0, 0), (0, 100), (0, 50), (0, 100), (1, 50), (0, 101), (63, 7)):
        assert limits(device, value, ok) == 0
    assert calls == [0, 100, 50, 101, 7]
    assert limits(2, 10, lambda v: 3) == 3        # a failed call is made again
    assert limits(2, 10, ok) == 0 and calls[-1] == 10
    assert limits(2, 10, lambda v: 3) == 0


def test_of_two_threads_the_smaller_size_does_not_stay(limits):
    """The smaller one is held up between its check and its call until the larger one's is through,
    or a while passes (it may have to wait)."""
    now, started, larger = [0], threading.Event(), threading.Event()

    def slow(v):
        started.set()
        larger.wait(0.5)
        now[0] = v
        return 0

    def fast(v):
        now[0] = v
        larger.set()
        return 0

    a = threading.Thread(target=limits, args=(0, 100, slow))
    a.start()
    assert started.wait(5)
    b = threading.Thread(target=limits, args=(0, 5000, fast))
    b.start()
    a.join(10), b.join(10)
    limits(0, 5000, fast)
    assert now[0] == 5000


# ------------------------------------------------------------ rope_turns.h

def inverse_two_pi(bits):
    """1 / (2 pi) * 2^bits, from pi = 16 atan(1/5) - 4 atan(1/239) in integers."""
    one = 1 << (bits + 32)

    def atan(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return (one << bits) // (2 * (16 * atan(5) - 4 * atan(239)))


def test_turns_per_position_to_the_last_bit(tmp_path):
    lib = compiled(tmp_path, "turns", '''
        #include "rope_turns.h"
        extern "C" uint64_t turns(double x) { return locks::turn_fraction(x); }''')
    lib.turns.argtypes, lib.turns.restype = [ctypes.c_double], ctypes.c_uint64
    bits = 320
    scale = inverse_two_pi(bits)
    sizes = [0.75, 1.0, 0.1, 1e-3, 1e-6, 2.6e-6, 1e-12, 6.283185307179586, 6.3, 3.0, 100.0, 4095.9, 4096.0]
    sizes += [500000.0 ** (-i / 64) for i in range(64)]
    for x in [0.0, -0.0] + sizes + [-v for v in sizes]:
        num, den = x.as_integer_ratio()
        # units of 2^-64 turns, with 64 bits behind the point
        exact = (num * scale << 64 >> (bits - 64)) // den
        off = ((lib.turns(x) << 64) - exact) % (1 << 128)
        off = min(off, (1 << 128) - off) / 2.0 ** 64
        assert off <= 0.5 + 2.0 ** -20, (x, off)
