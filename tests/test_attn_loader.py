"""The warps that load attention tiles, compiled for the CPU with recorded barriers.

A tile that has been asked for must have landed before the CTA leaves, also when a wait gave up: the loader's code is taken
from the kernel's source as it stands, its barriers and loads are replaced by records, and at every way out of it the
phases of all loads must have been waited for.
"""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dynamic_draft_tree_gb300", "csrc")

BEFORE = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <algorithm>
#include <map>
#include "dt_internal.cuh"
using std::max;
using std::min;
#undef __syncwarp
#define __syncwarp() ((void)0)
#define __syncthreads() ((void)0)
#define __umulhi(a, b) ((unsigned)(((uint64_t)(a) * (b)) >> 32))
#define __shfl_up_sync(m, v, d) (v)
#define __uint_as_float(x) (0.0f * (float)(x))
#define __half2float(x) (0.0f)
#define __ushort_as_half(x) (x)
#define threadIdx (dt::kNoIndex)
#define blockIdx (dt::kNoIndex)
#define gridDim (dt::kOneIndex)
namespace dt {
static const uint3 kNoIndex = {0, 0, 0}, kOneIndex = {1, 1, 1};
static int g_status;
static void set_status(int32_t*, int32_t bits) { g_status |= bits; }
static const float kLog2e = 1.442695f;
namespace tc {
// phases asked for on each barrier, and the latest one that was waited for
static std::map<uint64_t*, int> asked, landed;
static uint64_t *seg_lo, *seg_hi, *empty_lo, *empty_hi;
static int seg_left, empty_left, boxes;  // waits that succeed before one gives up
static bool bar_wait_warp(uint64_t* b, uint32_t, volatile int* stop) {
  int* left = b >= seg_lo && b < seg_hi ? &seg_left : b >= empty_lo && b < empty_hi ? &empty_left : nullptr;
  if (left && --*left < 0) {
    *stop = 1;
    return false;
  }
  return true;
}
static void bar_arrive(uint64_t*) {}
static void bar_expect(uint64_t* b, uint32_t) { ++asked[b]; }
static void bar_drain(uint64_t* b, uint32_t parity) {
  if (asked[b] > 0 && ((asked[b] - 1) & 1) == (int)parity) landed[b] = asked[b];
}
static void tma_load_4d(uint32_t, const CUtensorMap*, int, int, int, int, uint64_t*) { ++boxes; }
static void tma_load_3d(uint32_t, const CUtensorMap*, int, int, int, uint64_t*) { ++boxes; }
}  // namespace tc
}  // namespace dt
"""

AFTER = r"""
template <int DP, bool IS_K>
int leave(int tiles, int segments, int seg_left, int empty_left) {
  static Shared sh;
  memset(&sh, 0, sizeof(sh));
  AttnParams p{};
  int32_t table[4096] = {0};
  p.a.page = 128;
  p.page_shift = 7;
  p.tree_box = 8;
  p.a.n_blocks = 1;
  p.a.block_table = table;
  p.a.max_blocks = 4096;
  for (int i = 0; i < segments; ++i) {
    sh.seg[i].t1 = tiles;
    sh.seg[i].tree = tiles;  // cached tokens alone
    sh.seg[i].len = tiles * kTile;
  }
  uint64_t* empty = IS_K ? sh.kempty : sh.vempty;
  tc::asked.clear();
  tc::landed.clear();
  tc::boxes = 0;
  tc::seg_lo = sh.segfull;
  tc::seg_hi = sh.segfull + kSegs;
  tc::empty_lo = empty;
  tc::empty_hi = empty + kMostStages;
  tc::seg_left = seg_left;
  tc::empty_left = empty_left;
  load_tiles<DP, IS_K>(p, sh, nullptr, nullptr, 0, 0);
  int lost = 0;
  for (auto& x : tc::asked) lost += tc::landed[x.first] != x.second;
  printf("DP %d K %d tiles %d segments %d seg_left %d empty_left %d: %d boxes, %d not waited for\n", DP, IS_K, tiles, segments,
         seg_left, empty_left, tc::boxes, lost);
  return lost + (tc::boxes == 0);
}
template <int DP, bool IS_K>
int all() {
  int bad = 0;
  for (int tiles = 1; tiles <= 20; ++tiles) {
    bad += leave<DP, IS_K>(tiles, 1, 1, 1000);          // the wait for the next segment gives up
    bad += leave<DP, IS_K>(tiles, 1, 1000, 1000);       // the line's end
    bad += leave<DP, IS_K>(tiles, 3, 2, 1000);          // after two segments
    bad += leave<DP, IS_K>(tiles, 2, 1000, tiles);      // a stage is not given back
  }
  return bad;
}
}  // namespace
}  // namespace dt
int main() {
  const int bad = dt::all<64, true>() + dt::all<64, false>() + dt::all<128, true>() + dt::all<128, false>();
  return bad != 0;
}
"""


@pytest.fixture(scope="module")
def leave(tmp_path_factory):
    text = open(os.path.join(CSRC, "k_attn.cu")).read()
    end = "__device__ __forceinline__ int uniform("
    assert text.count(end) == 1
    body = "\n".join(x for x in text[:text.index(end)].split("\n") if not x.startswith("#include"))
    tmp = tmp_path_factory.mktemp("loader")
    src = tmp / "loader.cpp"
    src.write_text("#include <string.h>\n" + BEFORE + body + AFTER)
    exe = tmp / "loader"
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I",
                    "/usr/local/cuda/include", str(src), "-o", str(exe)], check=True)
    return exe


def test_loads_have_landed_at_every_way_out(leave):
    r = subprocess.run([str(leave)], capture_output=True, text=True)
    assert r.returncode == 0, [x for x in r.stdout.splitlines() if not x.endswith(" 0 not waited for")]


def test_barriers_are_made_once():
    """A barrier that is in use is not initialised again: its memory holds one for the CTA's whole life."""
    text = open(os.path.join(CSRC, "k_attn.cu")).read()
    made = re.findall(r"bar_init\(&sh\.(\w+(?:\[[^\]]*\])*)", text)
    assert len(made) == len(set(made)) and made.count("drained") == 1, made
