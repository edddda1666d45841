"""The walk over packed sequences that the convolution's and the scan's kernels share (Run in
csrc/gdn_layer.h), compiled for the CPU: every token of a tile in one run of the sequence
that holds it, for well-formed offsets, padded and ill-formed ones, and token
counts near 2^31."""
import ctypes
import os
import random
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HARNESS = r"""
#include <algorithm>
#include <cstdint>
using std::max; using std::min;
#define __device__
#define __forceinline__ inline
#define __builtin_amdgcn_readfirstlane(v) (v)
%s
// One tile's runs as (n, start, ta, tb, end); returns their number, or -1 beyond `most`.
extern "C" int walk(const int64_t* cu, int T, int N, int tile, int ntiles, int len, int most, int* out, int* rest) {
  Run<true> r;
  int k = 0;
  for (r.init(cu, T, N, tile, ntiles, len); !r.done(); r.next()) {
    if (k == most) return -1;
    const int v[5] = {r.n, r.start, r.ta, r.tb, r.end};
    std::copy(v, v + 5, out + 5 * k++);
  }
  rest[0] = r.rest;
  rest[1] = r.t1;
  return k;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    text = open(os.path.join(ROOT, "gated_deltanet_chunkwise_amd", "csrc", "gdn_layer.h")).read()
    part = re.search(r"// Packed sequences\..*(?=}  // namespace gdn)", text, re.S).group(0)
    d = tmp_path_factory.mktemp("walk")
    src, out = d / "walk.cc", d / "walk.so"
    src.write_text(HARNESS % part)
    # (sums that pass 2^31 wrap, as on the device)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-o", str(out), str(src)], check=True)
    return ctypes.CDLL(str(out))


def walk(lib, cu, T, N, tile, ntiles, length):
    most = 64
    out, rest = (ctypes.c_int * (5 * most))(), (ctypes.c_int * 2)()
    arr = None if cu is None else (ctypes.c_int64 * len(cu))(*cu)
    k = lib.walk(arr, T, N, tile, ntiles, length, most, out, rest)
    assert 0 <= k
    return [tuple(out[5 * i:5 * i + 5]) for i in range(k)], rest[0], rest[1]


def tiles(lib, cu, T, N, length):
    n = max(-(-T // length), 1)
    return [walk(lib, cu, T, N, t, n, length) for t in range(n)] if T else []


def test_well_formed_offsets(lib):
    rng = random.Random(1)
    for _ in range(400):
        N, T = rng.choice([1, 2, 3, 9, 40]), rng.choice([1, 5, 33, 64, 150])
        cu = sorted(rng.randint(0, T) for _ in range(N + 1))
        cu[0] = 0
        if rng.random() < 0.5:
            cu[-1] = T
        if rng.random() < 0.3:  # padded to a fixed count
            cu += [cu[-1]] * 500
        length, runs = rng.choice([8, 13, 16, 32, 77]), []
        for i, (r, rest, t1) in enumerate(tiles(lib, cu, T, len(cu) - 1, length)):
            assert t1 == min((i + 1) * length, T) and rest == max(min(cu[-1], t1), i * length)
            runs += r
        want = []
        for n in range(len(cu) - 1):
            for t in range(cu[n], cu[n + 1]):
                if want and want[-1][0] == n and t % length:
                    want[-1][3] = t + 1
                else:
                    want.append([n, cu[n], t, t + 1, cu[n + 1]])
        assert runs == [tuple(w) for w in want], (cu, T, length)


def test_ill_formed_offsets(lib):
    """Whatever the offsets: runs lie in their tile one after the other, within a sequence's
    bounds, and only a tile's first run continues one that began before it."""
    rng = random.Random(2)
    for _ in range(2000):
        N, T = rng.choice([1, 2, 3, 9]), rng.choice([1, 5, 33, 150])
        cu = [rng.choice([rng.randint(-5, T + 5), rng.randint(0, T), -2 ** 62, 2 ** 62]) for _ in range(N + 1)]
        length = rng.choice([8, 13, 32])
        for i, (runs, rest, t1) in enumerate(tiles(lib, cu, T, N, length)):
            at = i * length
            for k, (n, start, ta, tb, end) in enumerate(runs):
                assert 0 <= n < N and at <= ta < tb <= t1 and 0 <= start <= ta and tb <= end <= T
                assert k == 0 or start == ta
                at = tb
            assert i * length <= rest <= t1 <= T


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("length", [16, 262144, 1 << 20])
def test_token_counts_near_the_limit(lib, packed, length):
    """Long tiles (few channels leave a tile hundreds of thousands of tokens) at the last
    token counts that are allowed: the sums of token and tile length pass 2^31."""
    T = (1 << 31) - 5000
    n = -(-T // length)
    cu = [0, T - 3, T] if packed else None
    runs, rest, t1 = walk(lib, cu, T, 2 if packed else 1, n - 1, n, length)
    assert t1 == T and rest == T and runs[-1][3] == T and runs[0][2] == (n - 1) * length
    runs, _, t1 = walk(lib, cu, T, 2 if packed else 1, 0, n, length)
    assert t1 == length and [r[2:4] for r in runs] == [(0, length)]


def test_rows_of_a_batch(lib):
    T, B, length = 50, 3, 16
    n = -(-T // length)
    got = [walk(lib, None, T, B, t, n, length)[0] for t in range(B * n)]
    assert got == [[(b, b * T, b * T + k * length, min(b * T + (k + 1) * length, (b + 1) * T), (b + 1) * T)]
                   for b in range(B) for k in range(n)]
