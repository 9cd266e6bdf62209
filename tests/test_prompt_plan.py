"""The prompt attention's line of work and its loading warp, compiled for the CPU from the kernel's source.

The line: whatever the lengths, every tile of every item belongs to exactly one CTA, and what the CTAs say about items
that are cut (first CTA, number of parts) is what the join needs. The loader: at every way out, all loads that were asked
for have been waited for.
"""
import os
import subprocess

import pytest

from test_attn_loader import BEFORE, CSRC, ROOT

MORE = r"""
#define __all_sync(m, v) (v)
static uint32_t ticks() {
  static uint32_t now = 0;
  return now += 2100000000u;
}
#define clock ticks
namespace dt {
static uint64_t shfl_u64(uint64_t v, int) { return v; }
namespace tc {
static bool bar_try(uint64_t* b, uint32_t parity) {
  int never = 0;
  return bar_wait_warp(b, parity, &never);  // which counts the waits that succeed
}
}  // namespace tc
}  // namespace dt
"""

AFTER = r"""
static PromptParams params_for(int G, int H_kv, int B, int page, int max_blocks, const int32_t* off, const int32_t* len) {
  PromptParams p{};
  p.a.B = B;
  p.a.H_kv = H_kv;
  p.a.H_q = H_kv * G;
  p.a.rows = off[B];
  p.a.row_off = off;
  p.a.seq_len = len;
  p.a.page = page;
  p.a.max_blocks = max_blocks;
  shape_params(p);
  return p;
}
static uint32_t seed_ = 12345;
static int rnd(int n) {
  seed_ = seed_ * 1664525u + 1013904223u;
  return (int)((seed_ >> 8) % (uint32_t)n);
}
static int check(int G, int H_kv, int B, int most_n, int most_len, int ctas, bool whole = false) {
  std::vector<int32_t> off(B + 1, 0), len(B, 0);
  for (int b = 0; b < B; ++b) {
    const int kind = rnd(4);
    off[b + 1] = off[b] + (kind == 0 ? 0 : kind == 1 ? 1 : rnd(most_n + 1));
    len[b] = rnd(3) ? rnd(most_len + 1) : 0;
  }
  PromptParams p = params_for(G, H_kv, B, 16, most_len / 16 + 1, off.data(), len.data());
  p.whole = whole;
  int bad = 0;
  int64_t total = 0;
  std::vector<int64_t> before(B + 1, 0);
  for (int b = 0; b < B; ++b) {
    const Request r = request_of(p, b);
    bad += r.bad || r.n != off[b + 1] - off[b] || r.len != len[b];
    const Extent e = extent_of(p, r);
    int64_t tiles = 0, units = 0;
    for (int i = 0; i * p.w < r.n; ++i) {
      bad += units_before(p, e.ct, i) != units;
      const int end = std::min(r.n, (i + 1) * p.w), t = e.ct + (end + 127) / 128;
      units += kItemUnits + t;
    }
    bad += e.head != units;
    before[b + 1] = before[b] + H_kv * e.head;
  }
  total = before[B];
  const int64_t per = std::max<int64_t>(1, (total + ctas - 1) / ctas);
  std::map<std::tuple<int, int, int>, std::vector<std::array<int, 3>>> got;  // item -> (t0, t1, CTA), in order
  std::map<std::tuple<int, int, int>, Segment> first;
  std::map<std::tuple<int, int, int>, int> parts;
  for (int c = 0; c < ctas; ++c) {
    Plan pl{};
    pl.x0 = std::min(total, per * c);
    pl.x1 = std::min(total, pl.x0 + per);
    pl.per = (int)per;
    for (int b = 0; b < B; ++b)
      if (before[b] <= pl.x0 && pl.x0 < before[b + 1]) {
        pl.b = b;
        pl.t_b = before[b];
      }
    Walk w{};
    w.start(p, pl);
    int cuts = 0, firsts = 0;
    for (int k = 0;; ++k) {
      Segment s{};
      w.next(p, pl, s);
      if (s.t1 == s.t0) break;
      const auto key = std::make_tuple(s.b, s.h, s.i0);
      if (s.t0 == 0) first[key] = s;
      got[key].push_back({s.t0, s.t1, c});
      cuts += s.t0 == 0 && s.t1 < s.tt;
      firsts += s.t0 > 0;
      bad += whole && (s.t0 != 0 || s.t1 != s.tt);
      bad += s.t0 > 0 && k > 0;  // only a CTA's first segment goes on with another CTA's item
      if (s.t0 == 0 && s.t1 < s.tt) parts[key] = parts_of(pl, s);
      bad += s.rows != (s.iend - s.i0) * G || s.rows > kItemRows || s.iend > off[s.b + 1] - off[s.b];
      bad += s.tiles0 > s.tt || (s.tiles1 != 0 && s.tiles1 != s.tt);
    }
    bad += cuts > 1 || firsts > 1;  // two places for parts
  }
  int64_t items = 0;
  for (int b = 0; b < B; ++b)
    for (int h = 0; h < H_kv; ++h)
      for (int i0 = 0; i0 < off[b + 1] - off[b]; i0 += p.w, ++items) {
        const auto& v = got[std::make_tuple(b, h, i0)];
        const int end = std::min(off[b + 1] - off[b], i0 + p.w), tt = (len[b] + 127) / 128 + (end + 127) / 128;
        int t = 0;
        for (size_t k = 0; k < v.size(); ++k) {
          bad += v[k][0] != t || (k > 0 && v[k][2] != v[k - 1][2] + 1);
          t = v[k][1];
        }
        bad += t != tt;
        if (!v.empty()) {
          const Segment& s = first[std::make_tuple(b, h, i0)];
          bad += s.tt != tt || (v.size() > 1 && parts[std::make_tuple(b, h, i0)] != (int)v.size());
        }
      }
  bad += items != (int64_t)got.size();
  if (bad) printf("G %d H_kv %d B %d n %d len %d ctas %d: %d wrong\n", G, H_kv, B, most_n, most_len, ctas, bad);
  return bad;
}
enum { kKeys, kValues, kQueries };  // whose place is not given back
template <int DP>
int leave(int tiles, int segments, int seg_left, int which, int left, int cached) {
  static Shared sh;
  memset(&sh, 0, sizeof(sh));
  int32_t table[4096] = {0}, off[2] = {0, 1 << 20};
  PromptParams p = params_for(4, 1, 1, 128, 4096, off, nullptr);
  p.page_shift = 7;
  p.a.page = 128;
  p.a.n_blocks = 1;
  p.a.block_table = table;
  for (int i = 0; i < segments; ++i) {
    sh.seg[i].t1 = sh.seg[i].tiles0 = sh.seg[i].tiles1 = tiles;
    sh.seg[i].ct = std::min(cached, tiles);
    sh.seg[i].len = sh.seg[i].ct * kTile;
  }
  tc::asked.clear();
  tc::landed.clear();
  tc::boxes = 0;
  tc::seg_lo = sh.segfull;
  tc::seg_hi = sh.segfull + kSegs;
  tc::empty_lo = which == kKeys ? sh.kempty : which == kValues ? sh.vempty : sh.qempty;
  tc::empty_hi = tc::empty_lo + (which == kQueries ? 2 : kMostStages);
  tc::seg_left = seg_left;
  tc::empty_left = left;
  load_tiles<DP>(p, sh, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, 0, 0);
  int lost = 0;
  for (auto& x : tc::asked) lost += tc::landed[x.first] != x.second;
  if (lost || (tc::boxes == 0 && left > 0))
    printf("DP %d tiles %d segments %d seg_left %d which %d left %d: %d boxes, %d not waited for\n", DP, tiles, segments, seg_left,
           which, left, tc::boxes, lost);
  return lost + (tc::boxes == 0 && left > 0);
}
template <int DP>
int all() {
  int bad = 0;
  for (int tiles = 1; tiles <= 20; ++tiles)
    for (int cached : {0, 1, 100})
      for (int which : {kKeys, kValues, kQueries}) {
        bad += leave<DP>(tiles, 1, 1, which, 1000, cached);     // the wait for the next segment gives up
        bad += leave<DP>(tiles, 1, 1000, which, 1000, cached);  // the line's end
        bad += leave<DP>(tiles, 3, 2, which, 1000, cached);     // after two segments
        for (int left = 0; left < 2 * tiles; ++left) bad += leave<DP>(tiles, 2, 1000, which, left, cached);
      }
  return bad;
}
}  // namespace
}  // namespace dt
int main() {
  int bad = 0;
  const int groups[] = {1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 31, 32, 64, 65, 128};
  for (int G : groups) {
    for (int k = 0; k < 30; ++k)
      bad += dt::check(G, 1 + dt::rnd(5), 1 + dt::rnd(12), 1 + dt::rnd(700), dt::rnd(900), k % 3 ? 152 : 1 + dt::rnd(20), k % 5 == 0);
    bad += dt::check(G, 2, 400, 3, 300, 152) + dt::check(G, 3, 40, 9, 0, 152, true) + dt::check(G, 1, 1, 300, 0, 152, true);
    bad += dt::check(G, 1, 2, 20000, 20000, 152);
  }
  bad += dt::all<64>() + dt::all<128>();
  return bad != 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    text = open(os.path.join(CSRC, "k_prompt.cu")).read()
    end = "__device__ __forceinline__ int uniform("
    shape = text[text.index("void shape_params(PromptParams& p)"):]
    shape = shape[:shape.index("\n}\n") + 3]  # the host's part of the plan
    assert text.count(end) == 1
    body = "\n".join(x for x in text[:text.index(end)].split("\n") if not x.startswith("#include"))
    tmp = tmp_path_factory.mktemp("prompt")
    src = tmp / "plan.cpp"
    src.write_text("#include <string.h>\n#include <array>\n#include <tuple>\n#include <vector>\n" + BEFORE + MORE + body + shape + AFTER)
    exe = tmp / "plan"
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I",
                    "/usr/local/cuda/include", str(src), "-o", str(exe)], check=True)
    return exe


def test_every_tile_has_one_owner_and_loads_land(program):
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
