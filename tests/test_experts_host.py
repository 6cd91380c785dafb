"""Functions of the expert products run on the host, from their own source text in
csrc/: the search for a block's tile with a block's threads as fibers, one wave as
far ahead of the others as the barriers let it, the sigmoid over the whole range of
its argument, and the rules that bound a launch."""

from __future__ import annotations

import ctypes
import math
import os
import random
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_get_dispatch_05_amd",
                    "csrc")


def source(start: str, end: str, name: str = "gemm.h") -> str:
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert text.count(start) == 1 and text.count(end) >= 1, (start, end)
    return text[text.index(start):text.index(end, text.index(start))]


def compiled(tmp_path_factory, name: str, code: str) -> ctypes.CDLL:
    d = tmp_path_factory.mktemp(name)
    src, lib = d / (name + ".cpp"), d / (name + ".so")
    src.write_text(code)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-ffp-contract=off", "-shared", "-fPIC", "-o", str(lib), str(src)])
    return ctypes.CDLL(str(lib))


# A wave's lanes run one after the other up to a place where the hardware has them
# together (a lane exchange, a value told to be uniform, a barrier); a wave runs up to
# a barrier before the next wave gets a turn, in ascending or descending order.
FIBERS = r"""
#include <stdint.h>
#include <stdlib.h>
#include <ucontext.h>
#include <vector>
#define __device__
#define __forceinline__ inline
#define __shared__ static
#define __builtin_amdgcn_update_dpp emulated_dpp
constexpr int kThreads = 512, kWave = 64, kLanes = 64;
struct Dim { unsigned x; };
static thread_local Dim threadIdx;
enum State { kRun, kLaneWait, kBlockWait, kDone };
struct Fiber { ucontext_t c; std::vector<char> stack; State state; };
static std::vector<Fiber> fibers;
static ucontext_t scheduler;
static unsigned at;
static int lane_value[kThreads];
static void (*body)(unsigned);
static void wait_as(State s)
{
    const unsigned me = at;
    fibers[me].state = s;
    swapcontext(&fibers[me].c, &scheduler);
    at = me;
    threadIdx.x = me;
}
static void __syncthreads() { wait_as(kBlockWait); }
static int exchange(int v, int from, bool valid)
{
    const unsigned me = at;
    lane_value[me] = v;
    wait_as(kLaneWait);
    const int got = valid ? lane_value[from] : 0;
    wait_as(kLaneWait);
    return got;
}
// the wave scan's controls: shift right by 1, 2, 4, 8 inside 16 lanes, a row's last lane
// to the next row, lane 31 to the rows after it
static int emulated_dpp(int, int v, int ctrl, int rows, int, bool)
{
    const int wave = at / kLanes * kLanes, lane = at % kLanes;
    int from = -1;
    if (ctrl > 0x110 && ctrl < 0x120)
        from = lane % 16 >= (ctrl & 15) ? lane - (ctrl & 15) : -1;
    else if (ctrl == 0x142)
        from = lane >= 16 ? lane / 16 * 16 - 1 : -1;
    else if (ctrl == 0x143)
        from = lane >= 32 ? 31 : -1;
    else
        abort();
    const bool valid = from >= 0 && (rows >> (lane / 16) & 1);
    return exchange(v, wave + (from < 0 ? 0 : from), valid);
}
static int uniform(int v) { return exchange(v, at / kLanes * kLanes, true); }
static void entry() { body(at); fibers[at].state = kDone; swapcontext(&fibers[at].c, &scheduler); }
static void run_block(void (*f)(unsigned), bool descending)
{
    body = f;
    if (fibers.empty())
        fibers.resize(kThreads);
    for (auto &b : fibers) {
        b.stack.resize(1 << 16);
        getcontext(&b.c);
        b.c.uc_stack.ss_sp = b.stack.data();
        b.c.uc_stack.ss_size = b.stack.size();
        b.c.uc_link = &scheduler;
        makecontext(&b.c, entry, 0);
        b.state = kRun;
    }
    for (bool alive = true; alive;) {
        for (int i = 0; i < kThreads / kLanes; ++i) {
            const int w = (descending ? kThreads / kLanes - 1 - i : i) * kLanes;
            for (bool moved = true; moved;) {
                moved = false;
                for (int l = w; l < w + kLanes; ++l)
                    if (fibers[l].state == kRun) {
                        at = l;
                        threadIdx.x = l;
                        swapcontext(&scheduler, &fibers[l].c);
                        moved = true;
                    }
                int waits = 0, alive_lanes = 0;
                for (int l = w; l < w + kLanes; ++l) {
                    waits += fibers[l].state == kLaneWait;
                    alive_lanes += fibers[l].state != kDone;
                }
                if (waits > 0 && waits == alive_lanes)
                    for (int l = w; l < w + kLanes; ++l)
                        if (fibers[l].state == kLaneWait) {
                            fibers[l].state = kRun;
                            moved = true;
                        }
            }
        }
        alive = false;  // all at the barrier, or done: past it, as far as there is one
        for (auto &b : fibers) {
            if (b.state == kLaneWait)
                abort();  // lanes of a wave went different ways
            if (b.state == kBlockWait) {
                b.state = kRun;
                alive = true;
            }
        }
    }
}
"""

TILES = r"""
static Groups G;
static unsigned first_block, step, columns;
static int tile_height;
static Tile seen[2][kThreads];
template <int BM> static void two_tiles(unsigned tid)
{
    // as a block that works through tiles: the next one is looked up without a barrier since
    seen[0][tid] = find_tile<BM, kThreads>(G, first_block, columns);
    if (seen[0][tid].group < 0)
        return;
    seen[1][tid] = find_tile<BM, kThreads>(G, first_block + step, columns);
}
extern "C" void look_up(const int32_t *offsets, const int32_t *counts, int slots, int num, int bm, unsigned block,
                        unsigned grid, unsigned nt, int descending, int32_t *out)
{
    G = Groups{offsets, counts, slots, num, 1, num, 1, 0x7fffffff};
    first_block = block;
    step = grid;
    columns = nt;
    for (auto &s : seen)
        for (auto &t : s)
            t = Tile{-2, 0, 0, 0};
    run_block(bm == 256 ? two_tiles<256> : two_tiles<64>, descending != 0);
    for (int c = 0; c < 2; ++c)
        for (int i = 0; i < kThreads; ++i) {
            const Tile &t = seen[c][i];
            const int32_t v[4] = {t.group, t.m0, t.rows, t.n};
            for (int k = 0; k < 4; ++k)
                out[(c * kThreads + i) * 4 + k] = v[k];
        }
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    body = source("struct Groups {", "__device__ __forceinline__ f32x4 mfma_bf16")
    return compiled(tmp_path_factory, "tiles", FIBERS + body + TILES)


THREADS = 512


def look_up(lib, rows, cells, bm, block, grid, nt, descending):
    """Every thread's results of the two look-ups of a block."""
    offsets = [0]
    for r in rows:
        offsets.append(offsets[-1] + r)
    arr = (ctypes.c_int32 * (len(rows) + 1))(*(list(rows) + [0] if cells else offsets))
    out = (ctypes.c_int32 * (2 * THREADS * 4))()
    lib.look_up(None if cells else arr, arr if cells else None, 1 << 20, len(rows), bm, block, grid, nt, descending, out)
    got = [tuple(out[i * 4:i * 4 + 4]) for i in range(2 * THREADS)]
    return got[:THREADS], got[THREADS:]


# rows of the groups; past 512 groups a thread looks after several
MANY = [0] * 640
for _i in (0, 3, 511, 512, 513, 639):
    MANY[_i] = 40 + _i % 7
TILE_CASES = [([300, 0, 70, 256, 129], False, 256, 3), ([5, 64, 65, 0, 33, 200], True, 64, 2), (MANY, False, 64, 1),
              (MANY, True, 256, 2), ([0, 0, 0], True, 64, 4), ([1], False, 256, 1)]


@pytest.mark.parametrize("descending", [0, 1], ids=["first wave ahead", "last wave ahead"])
@pytest.mark.parametrize("rows,cells,bm,nt", TILE_CASES)
def test_every_tile_is_found_once_by_all_waves(tiles, rows, cells, bm, nt, descending):
    count = sum(-(-r // bm) for r in rows) * nt
    blocks = (count // 8 + 2) * 8
    grid = min(blocks, 16)
    first, second = {}, {}
    for b in range(blocks):
        one, two = look_up(tiles, rows, cells, bm, b, grid, nt, descending)
        assert len(set(one)) == 1, f"block {b}: waves that differ in their first tile: {sorted(set(one))}"
        first[b] = one[0]
        if one[0][0] >= 0:
            assert len(set(two)) == 1, f"block {b}: waves that differ in their second tile: {sorted(set(two))}"
            second[b + grid] = two[0]
    want = {(g, m, r, n) for g, r in enumerate(rows) for m in range(0, r, bm) for n in range(nt)}
    real = [t for t in first.values() if t[0] >= 0]
    assert len(real) == len(want) and set(real) == want
    for b, t in second.items():
        assert t == first.get(b, t), b
        assert t[0] < 0 or t in want


# The hardware's 2^x and reciprocal, rounded from 64 bits; their results below the
# normal numbers are zero there.
SIGMOID = r"""
#include <cmath>
#define __device__
#define __forceinline__ inline
#define __builtin_amdgcn_exp2f emulated_exp2
#define __builtin_amdgcn_rcpf emulated_rcp
#define __builtin_amdgcn_fmed3f emulated_med3
static float flushed(double v) { const float f = float(v); return std::fabs(f) < 1.17549435e-38f ? 0.0f : f; }
static float emulated_exp2(float v) { return flushed(std::exp2(double(v))); }
static float emulated_med3(float v, float lo, float hi) { return std::isnan(v) || v < lo ? lo : v > hi ? hi : v; }
static float emulated_rcp(float v) { return flushed(1.0 / double(v)); }
using std::fmaf;
"""


@pytest.fixture(scope="module")
def sigmoid(tmp_path_factory):
    body = source("// 1 / (1 + e^-v)", "__device__ __forceinline__ uint2 pack4")
    lib = compiled(tmp_path_factory, "sigmoid", SIGMOID + body + 'extern "C" float sigmoid(float v) { return sigmoidf(v); }')
    lib.sigmoid.restype, lib.sigmoid.argtypes = ctypes.c_float, [ctypes.c_float]
    return lib.sigmoid


def test_sigmoid_over_its_range(sigmoid):
    v = np.concatenate([np.linspace(-87, 87, 4001), np.logspace(-20, 1.9, 300), -np.logspace(-20, 1.9, 300)])
    for x in v.astype(np.float32):
        want = 1 / (1 + math.exp(-float(x)))
        # the exponential, the sum, the Newton step and the last product: at most a unit each
        assert abs(sigmoid(x) - want) <= 4 * 2.0 ** -23 * want, x


def test_sigmoid_at_its_ends(sigmoid):
    """1 for large arguments and +inf, 0 below the normal results and at -inf."""
    for x in (87.5, 88.8, 1e4, 2.3e38, 2.4e38, 3.4e38, math.inf):
        assert sigmoid(x) == 1.0, x
    for x in (-88.0, -89.0, -104.0, -1e4, -2.4e38, -3.4e38, -math.inf):
        # what is left out there is below the smallest normal number and a half
        assert 0.0 <= sigmoid(x) <= 1.7e-38, x
        assert x >= -104 or sigmoid(x) == 0.0, x
    assert 0.0 <= sigmoid(math.nan) <= 1.0  # its uses multiply by the argument too


RULES = """
#include <stdint.h>
static int units;
static int compute_units() { return units; }
"""
RULES_OUT = """
extern "C" int height(int64_t rows, int64_t groups, int64_t columns, int cus)
{
    units = cus;
    return tile_rows(rows, groups, columns);
}
extern "C" int64_t needed(int64_t rows, int64_t groups, int64_t columns, int cus)
{
    return row_tiles(rows, groups, height(rows, groups, columns, cus)) * columns;
}
extern "C" int64_t at_most(int64_t rows, int64_t groups, int64_t columns)
{
    return tiles_at_most(rows, groups, columns);
}
"""


def test_no_launch_needs_more_tiles_than_the_check_allows(tmp_path_factory):
    """What the entry points check before the first launch bounds every launch, whatever
    height it takes, also one that is left only the groups of more than 64 rows."""
    body = source("inline int tile_rows", "// Shared with the entry points", "ep_internal.h")
    lib = compiled(tmp_path_factory, "rules", RULES + body + RULES_OUT)
    i64 = ctypes.c_int64
    lib.height.argtypes = lib.needed.argtypes = [i64, i64, i64, ctypes.c_int]
    lib.at_most.argtypes = [i64, i64, i64]
    lib.needed.restype = lib.at_most.restype = i64
    rng = random.Random(5)
    seen = set()
    for _ in range(20000):
        rows = int(2 ** rng.uniform(0, 28))
        groups = int(2 ** rng.uniform(0, 13))
        columns = int(2 ** rng.uniform(0, 13))
        cus = rng.choice([32, 256])
        most = lib.at_most(rows, groups, columns)
        assert lib.needed(rows, groups, columns, cus) <= most
        left = min(rows // 65, groups)
        assert lib.needed(rows, left, columns, cus) <= most
        seen.add((lib.height(rows, groups, columns, cus), rows // groups > 64))
    assert seen == {(64, False), (64, True), (256, True)}
