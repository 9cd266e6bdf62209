"""The kernels' bounded waits, whole warps at a time, compiled for the CPU from the kernels' source.

A flag in shared memory says that a role gave up; another warp may set it between the reads of two lanes, and lanes look at the
clock one after the other. What follows a wait is for whole warps, so that all lanes of it leave together, with one answer: no lane may be
gone while others meet in a vote. Here 32 lanes run one after the other, each up to its next vote, and the flag is set at every
place between two of them.
"""
import os
import re
import subprocess

import pytest

from test_attn_loader import CSRC

LANES = r"""
#include <stdint.h>
#include <stdio.h>
#include <ucontext.h>
#include <vector>
#define __device__
#define __forceinline__ inline
static const int kLanes = 32;
struct Shared { int stop; } sh;
static ucontext_t main_ctx, ctx[kLanes];
static std::vector<char> stacks(kLanes * 65536);
static int lane, voted[kLanes], gone[kLanes], answer[kLanes], result, tries_left;
static int64_t now[kLanes];
static int slow;  // the lane whose clock runs ahead, or -1
static int vote(int x) {
  voted[lane] = x;
  swapcontext(&ctx[lane], &main_ctx);
  return result;
}
static int all_, any_;
static int __all_sync(unsigned, bool x) { return vote(x ? 1 : 0) & 1; }
static int __any_sync(unsigned, bool x) { return vote(x ? 1 : 0) >> 1; }
static int64_t ticks() { return now[lane] += lane == slow ? 5000000000ll : 300000000ll; }
#define clock() ticks()
#define clock64() ticks()
namespace tc {
static bool bar_try(uint64_t*, uint32_t) { return tries_left > 0 && --tries_left == 0; }
"""

RUN = r"""
static bool call(int which) {
  switch (which) {
    case 0: return wait(nullptr, 0, sh);
    case 1: return wait_soon(nullptr, 0, sh);
    default: return tc::bar_wait_warp(nullptr, 0, &sh.stop);
  }
}
static int which_;
static void lane_main() {
  answer[lane] = call(which_);
  gone[lane] = 1;
  swapcontext(&ctx[lane], &main_ctx);
}
// The flag is set behind lane `at` of turn `turn`. True if the lanes part ways.
static bool parts(int which, int turn, int at, int slow_lane) {
  which_ = which;
  slow = slow_lane;
  sh.stop = 0;
  tries_left = 0;
  for (int i = 0; i < kLanes; ++i) {
    getcontext(&ctx[i]);
    ctx[i].uc_stack.ss_sp = stacks.data() + i * 65536;
    ctx[i].uc_stack.ss_size = 65536;
    ctx[i].uc_link = &main_ctx;
    makecontext(&ctx[i], lane_main, 0);
    gone[i] = 0;
    now[i] = 0;
  }
  for (int t = 0; t < 100; ++t) {
    int left = 0;
    for (int i = 0; i < kLanes; ++i) {
      lane = i;
      swapcontext(&main_ctx, &ctx[i]);
      left += gone[i];
      if (t == turn && i == at) sh.stop = 1;
    }
    if (left == kLanes) {
      for (int i = 1; i < kLanes; ++i)
        if (answer[i] != answer[0]) return true;
      return false;
    }
    if (left) return true;
    int all = 1, any = 0;
    for (int i = 0; i < kLanes; ++i) all &= voted[i], any |= voted[i];
    result = all | any << 1;
  }
  return true;  // no end
}
int main() {
  int bad = 0;
  for (int which = 0; which < 3; ++which) {
    int n = 0;
    for (int turn = 0; turn < 6; ++turn)
      for (int at = 0; at < kLanes; ++at) n += parts(which, turn, at, -1);
    for (int s = -1; s < kLanes; ++s) n += parts(which, -1, 0, s);
    printf("wait %d: lanes part ways in %d of the orders\n", which, n);
    bad += n;
  }
  return bad != 0;
}
"""


def _function(text, head):
    at = text.index(head)
    return text[at:text.index("\n}\n", at) + 3]


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    prompt, tc = (open(os.path.join(CSRC, name)).read() for name in ("k_prompt.cu", "tc.cuh"))
    parts = [LANES, "constexpr long long kWaitClocks = 4000000000ll;\n",
             _function(tc, "__device__ __forceinline__ bool bar_wait("), _function(tc, "__device__ __forceinline__ bool bar_wait_warp("),
             "}  // namespace tc\nconstexpr uint32_t kWaitTicks = 2000000000u;\n",
             _function(prompt, "__device__ __forceinline__ bool wait("), _function(prompt, "__device__ __forceinline__ bool wait_soon("),
             RUN]
    tmp = tmp_path_factory.mktemp("waits")
    (tmp / "waits.cpp").write_text("".join(parts))
    subprocess.run(["g++", "-std=c++17", "-O0", "-w", str(tmp / "waits.cpp"), "-o", str(tmp / "waits")], check=True)
    return tmp / "waits"


def test_a_warp_leaves_its_waits_together(program):
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_flags_that_steer_a_warp_are_read_by_a_vote():
    """What the prompts' kernel reads while another warp may write it decides what whole warps do: one answer for all lanes."""
    text = open(os.path.join(CSRC, "k_prompt.cu")).read()
    reads = [x.strip() for x in text.split("\n") if "*(volatile int*)&sh." in x]
    reads = [x for x in reads if not re.search(r"\*\(volatile int\*\)&sh\.\w+ = ", x)]
    assert len(reads) == 2, reads  # the flag of a wait that gave up, and that of values that are no numbers
    for x in reads:
        assert re.search(r"__(any|all)_sync\(0xFFFFFFFFu, !?\*\(volatile int\*\)&sh\.\w+\)", x), x
