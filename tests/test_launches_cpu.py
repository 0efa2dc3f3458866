"""The library's host code against a stand-in for the CUDA runtime
(fake_cudart.cpp): launches that fail, calls of two threads at once."""

import ctypes
import os
import random
import shutil
import subprocess
import threading
import time

import pytest

from test_rope_evict_cpu import ARG, A, B, C, D_
from turboquant_bit_kv_gb300 import build_lib, tq as real

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def linked(tmp_path_factory):
    """The library linked with the stand-in."""
    build_lib.build()
    out = str(tmp_path_factory.mktemp("fake") / "libtq_fake.so")
    objs = [os.path.join(build_lib.BUILD, s + ".o") for s in build_lib.SOURCES]
    cuda = os.path.dirname(os.path.dirname(shutil.which(build_lib.NVCC) or build_lib.NVCC))
    r = subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I" + os.path.join(cuda, "include"), "-o", out,
                        os.path.join(HERE, "fake_cudart.cpp")] + objs + ["-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.fixture
def lib(linked, tmp_path):
    """A copy of it (with state of its own), its functions typed as the binding's."""
    path = str(tmp_path / "libtq_fake.so")
    shutil.copy(linked, path)
    fake, typed = ctypes.CDLL(path), real.lib()
    for name in ("tq_insert_kv", "tq_attn_decode_weights", "tq_attn_weights_workspace_bytes", "tq_evict_select",
                 "tq_evict_compact", "tq_rope_apply", "tq_attn_decode", "tq_attn_decode_paged", "tq_attn_decode_d"):
        getattr(fake, name).argtypes = getattr(typed, name).argtypes
        getattr(fake, name).restype = getattr(typed, name).restype
    fake.fake_reset()
    return fake


def insert(lib, heads, n):
    kcb, vcb, rope = real.tq_codebook_load(128, 4), real.tq_codebook_load(128, 2), real.tq_rope_load()
    return lib.tq_insert_kv(A, 128 * heads, 128, B, 128 * heads, 128, real.TQ_BF16, n, heads, C, n, rope, kcb, vcb,
                            real.tq_signs(), C, D_, n * heads, A, n, None)


def test_stand_in_takes_calls(lib):
    assert insert(lib, 8, 16) == 0 and insert(lib, 8, 5000) == 0 and insert(lib, 1, 50000) == 0
    assert lib.fake_launches() == 3


def test_first_large_inserts_of_two_threads(lib):
    """Two threads make the first large calls at once, one of which needs more shared memory: later calls of either
    kind still launch."""
    lib.fake_slow_limit(60 * 1024)      # (one head: four tables of sines)
    got = {}
    a = threading.Thread(target=lambda: got.update(one=insert(lib, 1, 50000)))
    a.start()
    while not lib.fake_in_slow_limit():
        time.sleep(0.001)
    b = threading.Thread(target=lambda: got.update(eight=insert(lib, 8, 5000)))
    b.start()
    b.join()
    a.join()
    assert got == {"one": 0, "eight": 0}
    assert insert(lib, 1, 50000) == 0 and insert(lib, 8, 5000) == 0


def calls(lib):
    """Name -> a valid call of the library (its pointers are never read)."""
    k4, v2 = real.tq_codebook_load(128, 4), real.tq_codebook_load(128, 2)
    k4d = real.tq_codebook_load(96, 4)
    s, big = real.tq_signs(), 1 << 40
    return {
        "weights": lambda: lib.tq_attn_decode_weights(A, real.TQ_BF16, B, k4, C, v2, None, 0, 0, None, 2, 8, 2, 512, 500,
                                                      0.1, s, D_, 500, 1.0, A, real.TQ_F32, B, big, None),
        "weights, pages": lambda: lib.tq_attn_decode_weights(A, real.TQ_BF16, B, v2, C, v2, D_, 16, 40, None, 2, 8, 2, 0, 500,
                                                             0.1, s, D_, 500, 1.0, A, real.TQ_F32, B, big, None),
        "decode": lambda: lib.tq_attn_decode(A, real.TQ_BF16, B, k4, C, v2, None, 2, 8, 2, 512, 500, 0.1, s, None, None, None,
                                             A, B, big, None),
        "decode, pages": lambda: lib.tq_attn_decode_paged(A, real.TQ_BF16, B, k4, C, v2, D_, 16, 32, None, 2, 8, 2, 500, 0.1,
                                                          s, A, B, big, None),
        "decode, 96": lambda: lib.tq_attn_decode_d(A, real.TQ_BF16, B, k4d, C, k4d, None, 2, 8, 2, 512, 500, 96, 0.1, D_, A,
                                                   B, big, None),
        "select": lambda: lib.tq_evict_select(A, 500, B, 2, 2, 500, 100, 4, 10, C, D_, None),
        "compact": lambda: lib.tq_evict_compact(A, 66, B, 34, C, 500, D_, 100, A, None, 0, 0, 0, 2, 2, 512, 500, None),
        "insert": lambda: insert(lib, 8, 5000),
        "insert, few": lambda: insert(lib, 8, 16),
        "rope": lambda: lib.tq_rope_apply(A, real.TQ_BF16, 4, 2, 256, 128, B, 4, real.tq_rope_load(), C, 256, 128, None),
    }


NAMES = ["weights", "weights, pages", "decode", "decode, pages", "decode, 96", "select", "compact", "insert",
         "insert, few", "rope"]


@pytest.mark.parametrize("name", NAMES)
def test_a_failed_launch_does_not_fail_the_next_call(lib, name):
    """Each launch of a call in turn fails: the call says so, and the next one, whose launches succeed, does not."""
    call = calls(lib)[name]
    assert sorted(calls(lib)) == sorted(NAMES)
    assert call() == 0
    n = lib.fake_launches()
    assert n >= 1
    for i in range(1, n + 1):
        lib.fake_fail_at(i)
        assert call() == real.TQ_ERR_CUDA, i
        assert lib.fake_launches() == i     # (and nothing is launched after it)
        lib.fake_fail_at(0)
        assert calls(lib)["rope"]() == 0, i
        assert call() == 0, i


def test_rope_refuses_rows_that_overlap(lib):
    """Layouts of the output in which two (token, head) rows share an element are refused, the others are not: against
    all pairs of rows."""
    rng = random.Random(1)
    rope = real.tq_rope_load()
    seen = [0, 0]
    layouts = [(2, 128, 2, 128), (5, 128, 1, 64), (1, 8, 7, 128), (4, 256, 2, 128), (4, 128, 3, 512), (3, 128, 3, 376),
               (2, 256, 2, 384), (2, 256, 3, 384), (4, 136, 4, 136), (1000, 128, 1000, 128000), (1000, 128, 1000, 127992),
               (3000, 128, 2, 3000 * 128 - 8), (2, 1 << 40, 2, 1 << 40)]
    layouts += [(rng.randint(1, 9), 8 * rng.randint(12, 80), rng.randint(1, 9), 8 * rng.randint(12, 80)) for _ in range(2000)]
    for n, s, m, t in layouts:
        if n * m <= 10000:
            at = sorted(i * s + j * t for i in range(n) for j in range(m))
            overlap = any(b - a < 128 for a, b in zip(at, at[1:]))
        else:
            overlap = not (s >= (m - 1) * t + 128 or t >= (n - 1) * s + 128)
        got = lib.tq_rope_apply(A, real.TQ_BF16, n, m, 0, 0, B, 0, rope, C, s, t, None)
        assert got == (ARG if overlap else 0), (n, s, m, t, overlap)
        seen[overlap] += 1
    assert min(seen) > 200


def test_launches_of_an_insert(lib):
    """One launch, of very many tokens a few: a CTA has places for the rows that it takes again among 15200 rows."""
    for heads, n, want in ((8, 16, 1), (8, 131072, 1), (8, 460000, 1), (8, 1000000, 3), (1, 2000000, 1), (1, 10000000, 5),
                           (40, 200000, 3), (100000, 100, 2)):
        lib.fake_reset()
        assert insert(lib, heads, n) == 0
        assert lib.fake_launches() == want, (heads, n, lib.fake_launches())
