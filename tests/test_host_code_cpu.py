"""Host-callable code of the library's headers, compiled into small programs
of their own (with fakes of the runtime's calls where a test needs them)."""

import os
import subprocess

import pytest

from turboquant_bit_kv_gb300 import build_lib


def program(tmp_path, source, *flags):
    """Compile a CUDA C++ source that runs on the host alone; its path."""
    src, out = tmp_path / "prog.cu", tmp_path / "prog"
    src.write_text(source)
    r = subprocess.run([build_lib.NVCC] + build_lib.ARCH + ["-std=c++17", "-I" + os.path.join(build_lib.ROOT, "include"),
                        "-I" + build_lib.CSRC, *flags, "-o", str(out), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(out)


def run(prog, *args):
    r = subprocess.run([prog, *map(str, args)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
    return r.stdout


def test_pieces_of_a_chunk(tmp_path):
    """The pieces that pages cut a chunk of 32 tokens into: every token once, no piece across a page's end, in order,
    for pages of 8 tokens to nearly 2^31 (products of a lane and the page size pass 32 bits from 71.6 million on)."""
    prog = program(tmp_path, r"""
#include <cstdio>
#include <cstdlib>
#include "tq_attn_mma.h"
int main(int argc, char **argv) {
    for (int i = 1; i + 1 < argc; i += 2) {
        for (int p = 0; p < tq::kMmaPieces; ++p) {
            int t, len;
            tq::chunk_piece(atoi(argv[i]), atoi(argv[i + 1]), p, t, len);
            std::printf("%d %d ", t, len);
        }
        std::printf("\n");
    }
}
""")
    pages = [8, 16, 24, 32, 40, 48, 72, 104, 1000, 71582792, 134217736, 536870920, 1073741832, 2147483640]
    calls = []
    for page in pages:
        last = (2**31 - 33) // 32 * 32
        starts = [0, 32, 64, 96, 320, page // 32 * 32, page * 3 // 32 * 32, (page * 28 // 32) * 32, last]
        calls += [(t0, page) for t0 in starts if t0 <= last]
    out = run(prog, *[x for c in calls for x in c]).splitlines()
    assert len(out) == len(calls)
    for (t0, page), line in zip(calls, out):
        v = list(map(int, line.split()))
        pieces = [(t, n) for t, n in zip(v[::2], v[1::2]) if n > 0]
        want, t = [], t0
        while t < t0 + 32:
            n = min(page - t % page, t0 + 32 - t)
            want.append((t, n))
            t += n
        assert pieces == want, (t0, page)
        assert all(n >= 0 for n in v[1::2])


def test_weights_ctas_cover_every_context(tmp_path):
    """CTAs of equal shares cover the context once, none without a token, for contexts up to the longest."""
    prog = program(tmp_path, r"""
#include <cstdio>
#include <cstdlib>
#include "tq_attn_mma.h"
int main(int argc, char **argv) {
    std::printf("%d\n", tq::kMmaMaxTokens);
    for (int i = 1; i + 2 < argc; i += 3) {
        int64_t per;
        const int parts = tq::weights_parts(atoi(argv[i]), atoll(argv[i + 1]), atoi(argv[i + 2]), per);
        std::printf("%d %lld\n", parts, (long long)per);
    }
}
""")
    longest = 2**31 - 8192
    calls = [(sms, segs, T) for sms in (1, 152) for segs in (1, 3, 32, 256, 5000, 10**6)
             for T in (1, 31, 33, 1024, 1025, 32769, 10**6 + 1, 2**30, 2**30 + 5, 2**31 - 450000, longest)]
    out = run(prog, *[x for c in calls for x in c]).splitlines()
    assert int(out[0]) == longest
    for (sms, segs, T), line in zip(calls, out[1:]):
        parts, per = map(int, line.split())
        assert parts >= 1 and per % 32 == 0 and parts * per >= T > (parts - 1) * per, (sms, segs, T)
        assert parts <= max(1, -(-sms * 32 // segs)) and (per >= 512 or parts == 1)   # (1025 tokens: 2 x 544)
