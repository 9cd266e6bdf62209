// Causal attention over whole prompts, packed one behind the other, each behind the tokens that its request has in pages.
//
// For query row f = (position i, head of the group) of request b and key head h, with c = scale * log2 e:
//   out_f = sum_j 2^(c s_fj - m_f) v_j / sum_j 2^(c s_fj - m_f),  s_fj = q_f k_j,
// j over the request's cached tokens and its new positions up to i. G = H_q / H_kv rows of one position read the same keys,
// so a block of 128 rows is 128 / G positions of all G heads: it has the narrowest diagonal, and short prompts fill it.
//
// Work. An item is up to 256 rows (two groups of 128) of one key head over tiles of 128 tokens: the cached tokens', then
// those of the new positions up to the item's last one. Tiles above the diagonal do not exist. All tiles in item order
// (request, key head, block of positions) form one line that the CTAs, one an SM, cut into equal runs, whatever the lengths;
// a CTA's run of one item is a segment. An item in one CTA is written by it; of others every CTA leaves sum, maximum and
// unnormalised result in fp32, joined in the order of the line by join_kernel. Every CTA derives the cuts from the lengths
// on the device, so a captured call follows them.
//
// A CTA: warps 0-3 and 4-7 are two softmax groups (thread = row), warp 8 loads tiles (TMA), warps 9 and
// 11 issue a group's matrix instructions each, warp 10 walks along the line and clears value rows. Every wait is bounded
// (DT_DEV_TIMEOUT). S = Q K^T of a group's next tile is issued right behind O += P V of its last one, over the ends of
// segments too: Q has a buffer a group that is loaded again when the group's last S of a segment is done. S (fp32), P (16-bit,
// over S) and O live in tensor memory, which they fill (2 x 128 + 2 x 128 columns at D = 128).
//
// Bound by the chain S, softmax, P V of the two groups in turn: a tile of both takes 2815 clocks at D = 128, of which the tensor
// cores need 2048 (pages of 64 to 256 tokens as whole boxes, pages of 16 tokens 3280), and by power where all SMs are at it: one
// prompt of 16384 tokens, 8 x 4 heads of 128, bf16: 1310 to 1340 us, 1.65 PFLOP/s, in a few runs and 1480 us, 1.49 PFLOP/s, when
// it goes on. An item's ends cost 1.2 to 1.5 tiles more: its masked tile, and the softmax of the next item, which begins when the
// rows have left.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dt_internal.cuh"
#include "tc.cuh"
#include "tma_map.cuh"

namespace dt {
namespace {

constexpr int kTile = 128;      // tokens of a tile, rows of a group
constexpr int kItemRows = 256;  // rows of an item, at most (whole positions: 2 * (128 / G) * G)
constexpr int kPromptThreads = 384;
constexpr float kLazy = 8.0f;   // the reference maximum moves when a row passes it by 2^kLazy
constexpr float kShift = 6.0f;  // weights are held as 2^kShift times themselves: up to 2^14, inside fp16, and
                                // small ones stay normal in fp16 for longer; it cancels in the quotient
constexpr float kFar = 256.0f;  // scores of rows whose maximum is beyond this (log2 units) become distances first (softmax_group)
// Units of the line: a tile, for one group of rows (whose chain of softmax and products takes as long) as for two; an item has
// kItemUnits more in front for its ends. Tile t of an item at unit u is at u + kItemUnits + t, and belongs to the CTA that this
// falls to. 16 prompts of up to 2000 tokens, whose CTAs have 8 to 33 items each, take 189 us with one unit for an item, 195 with two
// and 207 with three (one and a half: no difference).
constexpr int kItemUnits = 1;

// An item that is cut: left by its first CTA for the join.
struct Cut {
  int32_t parts, rows;  // parts 0: none begins in this CTA
  int32_t h, pad;
  int64_t row;          // row of its first position
};

struct PromptParams {
  dt_prompt_args a;
  int32_t G, page_shift;
  int32_t pos, rows2;   // whole positions of a group's 128 rows (128 / G), rows of an item (2 pos G)
  int32_t w;            // positions of an item, 2 pos
  uint32_t g_magic;     // ceil(2^32 / G), for position_of
  float c, lazy, far;   // scale * log2 e, kLazy / c, kFar / c
  int32_t period, step; // w / 128 = step / period in lowest terms, period a power of two
  int32_t period_shift;
  int32_t warp_box;     // 32 rows of a group are a box of the output: whole positions, or a part of one
  int32_t whole;        // no item is cut: a CTA takes those that begin in its run
  uint16_t part[128];   // part[r] = sum of ceil(k step / period), k = 1 .. r < period
  int32_t part_all;     // the same up to r = period
  Cut* cuts;            // [CTAs]
  float2* ml;           // [2 CTAs][kItemRows] (m, l)
  float* o;             // [2 CTAs][kItemRows][D]
  int32_t* status;
  int32_t test_stop;    // test only: every wait that is not over at once gives up
};

// x / G for a row x < 256 of an item: exact, as x (g_magic G - 2^32) < 2^32.
__device__ __forceinline__ int position_of(const PromptParams& p, int x) {
  return p.G == 1 ? x : (int)__umulhi((uint32_t)x, p.g_magic);
}

struct Request {
  int len, n;    // cached tokens, positions
  int64_t base;  // row of position 0
  bool bad;
};

__device__ __forceinline__ Request request_of(const PromptParams& p, int b) {
  const dt_prompt_args& a = p.a;
  Request r;
  const int64_t r0 = a.row_off[b], r1 = a.row_off[b + 1];
  const int len = a.seq_len ? a.seq_len[b] : 0;
  const int64_t most = a.seq_len ? min((int64_t)a.max_blocks << p.page_shift, (int64_t)0x7FFFFF00) : 0;
  r.base = r0;
  r.len = (int)min((int64_t)max(len, 0), most);
  r.bad = len < 0 || len > most || r0 < 0 || r1 < r0 || r1 > a.rows;
  r.n = r0 < 0 || r1 < r0 || r1 > a.rows ? 0 : (int)(r1 - r0);
  return r;
}

// sum of ceil(k w / 128), k = 1 .. m: tiles of new positions in the first m items of a prompt. Whole periods first.
__device__ __forceinline__ int64_t new_tiles(const PromptParams& p, int m) {
  const int64_t q = m >> p.period_shift;
  const int r = m & (p.period - 1);
  return (int64_t)p.step * p.period * (q * (q - 1) / 2) + q * p.part_all + r * q * p.step + p.part[r];
}

// Items of a request and key head.
struct Extent {
  int items, ct;  // items; tiles of cached tokens
  int64_t head;   // units of a key head
};
__device__ __forceinline__ int64_t units_before(const PromptParams& p, int ct, int i) {  // of items 0 .. i - 1, not the last
  return (int64_t)i * (kItemUnits + ct) + new_tiles(p, i);
}
__device__ __forceinline__ Extent extent_of(const PromptParams& p, const Request& r) {
  Extent e;
  e.items = (r.n + p.w - 1) / p.w;
  e.ct = (r.len + kTile - 1) / kTile;
  e.head = r.n > 0 ? units_before(p, e.ct, e.items - 1) + kItemUnits + e.ct + (r.n + kTile - 1) / kTile : 0;
  return e;
}

// A CTA's run.
struct Plan {
  int64_t x0, x1;  // units of the line
  int64_t t_b;     // unit offset of request b
  int32_t per;     // units of a CTA
  int32_t b;       // first request
};

struct Segment {
  int t0, t1;           // tiles; none: the line is at its end
  int tiles0, tiles1;   // tiles of the item for each group
  int tt;               // tiles of the item
  int b, h;
  int ct, len;          // tiles of cached tokens, cached tokens
  int i0, iend;         // the item's positions
  int rows;             // rows of the item
  int64_t next_u;       // unit where tile t1 begins
  int64_t base;         // row of position 0
};

// One lane walks along the CTA's run.
struct Walk {
  int64_t x;
  int z;                // units from the current item's first to x
  int b, h, i;          // the current item
  Request r;
  Extent e;

  __device__ void start(const PromptParams& p, const Plan& pl) {
    x = pl.x0;
    if (x >= pl.x1) return;
    b = pl.b;
    r = request_of(p, b);
    e = extent_of(p, r);
    const int64_t y = x - pl.t_b;
    h = (int)(y / e.head);
    const int64_t at = y - h * e.head;
    int lo = 0, hi = e.items - 1;  // the last item that starts at or before `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (units_before(p, e.ct, mid) <= at) lo = mid;
      else hi = mid - 1;
    }
    i = lo;
    z = (int)(at - units_before(p, e.ct, i));
  }
  // The next segment that has tiles (a run may end or begin inside an item's first units).
  __device__ __forceinline__ void next(const PromptParams& p, const Plan& pl, Segment& s) {
    do {
      s.t0 = s.t1 = 0;
      if (x >= pl.x1) return;
      s.b = b;
      s.h = h;
      s.ct = e.ct;
      s.len = r.len;
      s.base = r.base;
      s.i0 = i * p.w;
      s.iend = min(r.n, s.i0 + p.w);
      s.rows = (s.iend - s.i0) * p.G;
      s.tiles0 = e.ct + (min(s.iend, s.i0 + p.pos) + kTile - 1) / kTile;
      s.tt = e.ct + (s.iend + kTile - 1) / kTile;
      s.tiles1 = s.iend - s.i0 > p.pos ? s.tt : 0;
      const int units = kItemUnits + s.tt, end = p.whole ? units : (int)min((int64_t)units, z + pl.x1 - x);
      s.t0 = max(0, z - kItemUnits);
      s.t1 = p.whole && z > 0 ? s.t0 : max(0, end - kItemUnits);  // (one that begins in the run before)
      s.next_u = x - z + kItemUnits + s.t1;
      x += end - z;
      z = end;
      if (end == units) {
        z = 0;
        if (++i == e.items) {
          i = 0;
          if (++h == p.a.H_kv) {
            h = 0;
            while (x < pl.x1) {  // the next request with positions (units left: there is one)
              if (++b >= p.a.B) {
                x = pl.x1;
                break;
              }
              r = request_of(p, b);
              if (r.n > 0) {
                e = extent_of(p, r);
                break;
              }
            }
          }
        }
      }
    } while (s.t1 == s.t0);
  }
};

// CTAs with tiles of an item that is cut behind this, its first segment.
__device__ __forceinline__ int parts_of(const Plan& pl, const Segment& s) {
  const int over = (int)(s.next_u - pl.x1) + s.tt - 1 - s.t1;  // from the first unit behind the run to the last tile
  return 2 + over / pl.per;
}

// Columns of tile t that are in use: cached tokens, or new positions up to the item's last one.
__device__ __forceinline__ int tile_valid(int t, int ct, int len, int iend) {
  return min(kTile, t < ct ? len - t * kTile : iend - (t - ct) * kTile);
}
// Whether value rows of tile t are cleared before it is used: rows past its end, and positions that the item's first rows
// do not attend to.
__device__ __forceinline__ bool tile_fixed(int t, int ct, int valid, int i0) {
  return valid < kTile || (t >= ct && (t - ct) * kTile + valid > i0 + 1);
}

template <int DP>
struct Smem {
  static constexpr int kHalf = kTile * 128;         // bytes of 64 elements of 128 rows
  static constexpr int kBlock = (DP / 64) * kHalf;  // a tile of Q, K or V
  static constexpr int kK = DP == 128 ? 2 : 4, kV = DP == 128 ? 2 : 6;  // tiles of K and of V in flight
  static constexpr int kOut = 8 * 32 * 128;         // where results turn from a row a thread to rows side by side
  static constexpr int kTiles = (2 + kK + kV) * kBlock + kOut;
};
constexpr int kMostStages = 6;
constexpr int kSegs = 4;  // segments that warp 10 is ahead of the slowest reader, at most

struct Shared {
  uint64_t kfull[kMostStages], kempty[kMostStages], vfull[kMostStages], vempty[kMostStages], vfix[kMostStages];
  uint64_t sfull[2], phalf[2][2], odone[2], qfull[2], qempty[2], turn[2], drained[2];
  uint64_t segfull[kSegs], segempty[kSegs];
  Segment seg[kSegs];
  Plan plan;
  int64_t sums[kPromptThreads / 32];
  uint32_t tmem;
  int stop, odd_values, cut;
};

template <int DP>
constexpr int kSmemBytes = Smem<DP>::kTiles + (int)sizeof(Shared);
static_assert(kSmemBytes<128> <= 232448 && kSmemBytes<64> <= 232448, "227 KB a CTA");

// The whole warp waits and leaves with one answer: as tc::bar_wait_warp, in fewer instructions. What the CTA's roles run must
// stay in the SM's instruction cache: with softmax code for 128 columns at once and three copies of the products' code one
// fetch in seven missed it, and the cache behind it, which several SMs share, was busy for 75 % of the time.
constexpr uint32_t kWaitTicks = 2000000000u;  // about a second
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Shared& sh) {
  const uint32_t t0 = (uint32_t)clock();
#pragma unroll 1
  do {
    if (__all_sync(0xFFFFFFFFu, tc::bar_try(bar, parity))) return true;
    if ((uint32_t)clock() - t0 > kWaitTicks) *(volatile int*)&sh.stop = 1;
    // another warp may set it between two lanes' reads: they leave by a vote
  } while (__all_sync(0xFFFFFFFFu, !*(volatile int*)&sh.stop));
  return false;
}

// The same with the first look in front, for the waits that the pipeline hangs on.
__device__ __forceinline__ bool wait_soon(uint64_t* bar, uint32_t parity, Shared& sh) {
  return __all_sync(0xFFFFFFFFu, tc::bar_try(bar, parity)) || wait(bar, parity, sh);
}

// The other warps read the segments that warp 10 puts down, in order. `lead`: the lane that gives the place back.
struct Segments {
  uint32_t n = 0;
  __device__ __forceinline__ bool next(Shared& sh, Segment& s, bool lead) {
    const int at = (int)(n % kSegs);
    const uint32_t parity = n / kSegs & 1;
    ++n;
    if (!wait(&sh.segfull[at], parity, sh)) return false;
    s = sh.seg[at];
    __syncwarp();
    if (lead) tc::bar_arrive(&sh.segempty[at]);
    return s.t1 > s.t0;
  }
  // The same in two halves, for a reader that has no registers for all of it: where the segment is, and that it is done with.
  __device__ __forceinline__ bool begin(Shared& sh) {
    if (!wait(&sh.segfull[n % kSegs], n / kSegs & 1, sh)) return false;
    return sh.seg[n % kSegs].t1 > sh.seg[n % kSegs].t0;
  }
  __device__ __forceinline__ const Segment& here(Shared& sh) const { return sh.seg[n % kSegs]; }
  __device__ __forceinline__ void end(Shared& sh) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::bar_arrive(&sh.segempty[n % kSegs]);
    ++n;
  }
};
constexpr int kSegReaders = 11;  // eight softmax warps, the loading warp, two issuing warps

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t d;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <bool BF16>
__device__ __forceinline__ float unpack16(uint16_t x) {
  return BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}

// Every CTA: the line's length and where its own run starts.
__device__ __forceinline__ void make_plan(const PromptParams& p, Shared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (p.a.B + kPromptThreads - 1) / kPromptThreads, b0 = tid * chunk, b1 = min(p.a.B, b0 + chunk);
  int64_t units = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(p, b);
    units += p.a.H_kv * extent_of(p, r).head;
    if (blockIdx.x == 0 && r.bad) set_status(p.status, DT_DEV_BAD_PAGE);
  }
  int64_t su = units;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = (int64_t)shfl_u64((uint64_t)su, max(lane - d, 0));
    if (lane >= d) su += o;
  }
  if (lane == 31) sh.sums[warp] = su;
  if (tid == 0) sh.cut = 0;
  __syncthreads();
  int64_t total = 0, t_b = su - units;
#pragma unroll
  for (int w = 0; w < kPromptThreads / 32; ++w) {
    const int64_t o = sh.sums[w];
    if (w < warp) t_b += o;
    total += o;
  }
  // at least one: no CTA between an item's first and last one is without a tile
  const int64_t per = max((int64_t)1, (total + (int64_t)gridDim.x - 1) / (int64_t)gridDim.x);
  const int64_t x0 = min(total, per * (int64_t)blockIdx.x), x1 = min(total, x0 + per);
  if (tid == 0) {
    sh.plan.x0 = x0;
    sh.plan.x1 = x1;
    sh.plan.per = (int32_t)per;
  }
  if (x0 >= x1) return;
  for (int b = b0; b < b1; ++b) {
    int64_t u = units;
    if (chunk > 1) u = p.a.H_kv * extent_of(p, request_of(p, b)).head;
    if (t_b <= x0 && x0 < t_b + u) {
      sh.plan.b = b;
      sh.plan.t_b = t_b;
    }
    t_b += u;
  }
}

// Ring position of the n-th tile: stage and the parity of its use.
template <int N>
__device__ __forceinline__ void ring(uint32_t n, int& stage, uint32_t& parity) {
  stage = (int)(n % N);
  parity = (n / N) & 1;
}

// One warp loads the tiles of the CTA's line in order, K and then V of each; a segment's rows of Q stand behind its first K
// tile, whose place is free earlier.
template <int DP>
__device__ void load_tiles(const PromptParams& p, Shared& sh, const CUtensorMap* k_pages, const CUtensorMap* v_pages,
                           const CUtensorMap* k_map, const CUtensorMap* v_map, const CUtensorMap* q_map, uint32_t q_smem,
                           uint32_t k_smem, uint32_t v_smem, int lane) {
  using S = Smem<DP>;
  constexpr int kHalves = DP / 64;
  const int shift = p.page_shift, page = p.a.page;
  const int box = min(page, kTile);  // tokens of a page box
  const int box_shift = min(shift, 7);
  Segments segs;
  Segment s;
  uint32_t n = 0, nv = 0;     // K and V tiles so far
  uint32_t nq0 = 0, nq1 = 0;  // loads of each group's Q so far
  bool ok = true;
  const int half = lane & (kHalves - 1), part = lane / kHalves;  // this lane's box of a tile
  while (ok && segs.next(sh, s, lane == 0)) {
    const int32_t* table = p.a.block_table + (int64_t)s.b * p.a.max_blocks;
    // block id of this lane's box in tile t (-1: none)
    auto block_at = [&](int t) {
      const int tok = t * kTile + (part << box_shift);
      if (t >= s.ct || (part << box_shift) >= kTile || tok >= s.len) return -1;
      int id = table[tok >> shift];
      if (id < 0 || id >= p.a.n_blocks) {
        set_status(p.status, DT_DEV_BAD_PAGE);
        id = p.a.n_blocks;  // outside the tensor: zeros
      }
      return id;
    };
    int id = block_at(s.t0);
    for (int t = s.t0; ok && t < s.t1; ++t) {
      const int next_id = t + 1 < s.t1 ? block_at(t + 1) : -1;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        int stage;
        uint32_t parity;
        if (kv) ring<S::kV>(nv, stage, parity);
        else ring<S::kK>(n, stage, parity);
        ok = wait(&(kv ? sh.vempty : sh.kempty)[stage], parity ^ 1, sh);
        if (!ok) break;
        uint64_t* full = &(kv ? sh.vfull : sh.kfull)[stage];
        const uint32_t at = (kv ? v_smem : k_smem) + stage * S::kBlock;
        if (t < s.ct) {
          const int boxes = (min(kTile, s.len - t * kTile) + box - 1) >> box_shift;
          if (lane == 0) tc::bar_expect(full, kHalves * 128 * boxes * box);
          __syncwarp();
          if (part < boxes) {
            const int tok = t * kTile + (part << box_shift);
            tc::tma_load_4d(at + half * S::kHalf + (part << box_shift) * 128, kv ? v_pages : k_pages, half * 64, s.h,
                            tok & (page - 1), id, full);
          }
        } else {  // new positions; rows behind the request's last one are masked
          if (lane == 0) tc::bar_expect(full, S::kBlock);
          __syncwarp();
          if (lane < kHalves)
            tc::tma_load_3d(at + lane * S::kHalf, kv ? v_map : k_map, lane * 64, s.h, (int)s.base + (t - s.ct) * kTile, full);
        }
        if (kv) ++nv;
        else ++n;
        if (kv || t > s.t0) continue;
        // Whole positions of G heads, once the group's last S of the segment before is done. Rows past the item's belong
        // to other positions or lie past the buffer (zeros); nobody reads theirs.
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          if (t >= (g ? s.tiles1 : s.tiles0)) continue;
          ok = wait(&sh.qempty[g], ((g ? nq1 : nq0) & 1) ^ 1, sh);
          if (!ok) break;
          if (g) ++nq1;
          else ++nq0;
          if (lane == 0) tc::bar_expect(&sh.qfull[g], kHalves * p.pos * p.G * 128);
          __syncwarp();
          if (lane < kHalves)
            tc::tma_load_3d(q_smem + g * S::kBlock + lane * S::kHalf, q_map, lane * 64, s.h * p.G, (int)s.base + s.i0 + g * p.pos,
                            &sh.qfull[g]);
        }
        if (!ok) break;
      }
      id = next_id;
    }
  }
  // No load may land once the CTA is gone, and any wait, here or of a reader, may be the one that gave up: the last tiles
  // are waited for whatever ended the loop (in a call that runs through, the products wait for them too).
  for (uint32_t k = n > S::kK ? n - S::kK : 0; k < n; ++k) {
    int stage;
    uint32_t parity;
    ring<S::kK>(k, stage, parity);
    tc::bar_drain(&sh.kfull[stage], parity);
  }
  for (uint32_t k = nv > S::kV ? nv - S::kV : 0; k < nv; ++k) {
    int stage;
    uint32_t parity;
    ring<S::kV>(k, stage, parity);
    tc::bar_drain(&sh.vfull[stage], parity);
  }
  if (nq0) tc::bar_drain(&sh.qfull[0], (nq0 - 1) & 1);
  if (nq1) tc::bar_drain(&sh.qfull[1], (nq1 - 1) & 1);
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// One warp issues the matrix instructions of a group along the CTA's line, all lanes on one path and one thread elected for
// the instructions themselves, so that descriptors stay in uniform registers. A step is a tile n of the line: O += P V of the
// tile before (if the group had it), then S of this one (if it has it). The two groups' warps take turns, so that one group's
// softmax runs beside the other's products, and each does its waiting while the other one issues.
template <int DP, bool BF16>
__device__ void issue_mma(const PromptParams& p, Shared& sh, uint32_t q_smem, uint32_t k_smem, uint32_t v_smem, int g, int lane) {
  using S = Smem<DP>;
  constexpr uint32_t kDescS = tc::instr_desc(BF16, kTile, kTile, false), kDescHalf = tc::instr_desc(BF16, kTile, kTile / 2, false);
  constexpr uint32_t kDescO = tc::instr_desc(BF16, kTile, DP, true);
  const int steps = (p.a.D + 15) / 16;  // the padding elements of a row are zero
  const uint32_t tm = uniform(sh.tmem);
  // shared memory lies below 2^18 bytes, so offsets add up inside a descriptor's address field
  const uint64_t q_desc = tc::smem_desc(uniform(q_smem + g * S::kBlock), 16, 1024), k_desc = tc::smem_desc(uniform(k_smem), 16, 1024),
                 v_desc = tc::smem_desc(uniform(v_smem), S::kHalf, 1024);
  const uint32_t s_at = tm + g * kTile, o_at = tm + 2 * kTile + g * DP;
  const bool elected = tc::elect();
  Segments segs;
  Segment s;
  uint32_t n = 0;      // tiles so far
  uint32_t np = 0;     // products with V so far (phase of phalf)
  uint32_t nq = 0;     // segments of the group so far (phase of qfull)
  uint32_t turns = 0;  // this warp's turns so far
  uint32_t fix = 0;    // parity of every stage's vfix
  int owe = 0;         // of the tile before: bit 0 a product with V, bit 1 it begins the accumulator, bit 2 it ends a segment
  int steps_v = 0;     // 16 tokens each, of the tile before
  bool fixed = false;
  int v_stage = 0;
  int t = 0, t1 = 0, ct = 0, len = 0, iend = 0, i0 = 0, tiles = 0;
  auto take_turn = [&] {
    const uint32_t k = turns++;
    return wait_soon(&sh.turn[g], (k & 1) ^ (g ? 0 : 1), sh);
  };
  auto pass_turn = [&] {
    if (elected) tc::bar_arrive(&sh.turn[g ^ 1]);
  };
#pragma unroll 1
  while (true) {
    int stage;
    uint32_t parity;
    ring<S::kK>(n, stage, parity);
    const bool fresh = t == t1;  // the next tile is another segment's
    // What a step waits for has been waited for before its weights are there: with K and the turn behind the weights one prompt of
    // 16384 tokens took 1494 us when it took 1335.
    if (n > 0) {
      uint32_t v_parity;
      ring<S::kV>(n - 1, v_stage, v_parity);
      if (!wait_soon(&sh.vfull[v_stage], v_parity, sh)) return;
      if (fixed) {
        if (!wait(&sh.vfix[v_stage], fix >> v_stage & 1, sh)) return;
        fix ^= 1u << v_stage;
      }
    }
    bool more = true;
    if (fresh) {
      more = segs.next(sh, s, lane == 0);
      t = uniform(s.t0);
      t1 = uniform(s.t1);
      ct = uniform(s.ct);
      len = uniform(s.len);
      iend = uniform(s.iend);
      i0 = uniform(s.i0);
      tiles = min(t1, uniform(g ? s.tiles1 : s.tiles0));
    }
    // waited for and let go by a group without this tile too, so that it does not run ahead of the ring
    if (!fresh && !wait_soon(&sh.kfull[stage], parity, sh)) return;
    if (!take_turn()) return;
    if (owe) {  // O += P V of the tile before, which is then let go
      const uint64_t va = v_desc + (uint32_t)(v_stage * (S::kBlock >> 4));
      // the first half's products run while the group works on the second half's weights
      if (!wait_soon(&sh.phalf[g][0], np & 1, sh)) return;
      tc::fence_after();
      if (elected) {
        tc::mma_ts(o_at, s_at, va, kDescO, !(owe & 2));
#pragma unroll
        for (int x = 1; x < kTile / 32; ++x)
          if (x < steps_v) tc::mma_ts(o_at, s_at + x * 8, va + x * 128, kDescO, true);
      }
      if (!wait_soon(&sh.phalf[g][1], np++ & 1, sh)) return;
      tc::fence_after();
      if (elected) {
#pragma unroll
        for (int x = kTile / 32; x < kTile / 16; ++x)
          if (x < steps_v) tc::mma_ts(o_at, s_at + x * 8, va + x * 128, kDescO, true);
        if (owe & 4) tc::mma_commit(&sh.odone[g]);  // else S's commit says so too
        tc::mma_commit(&sh.vempty[v_stage]);
      }
    } else if (n > 0 && elected) {
      tc::bar_arrive(&sh.vempty[v_stage]);
    }
    // The turn is kept for another segment's Q and K too, which are mostly there. (Given to the other group in between, S came
    // behind that group's products: 16 prompts of up to 2000 tokens 190 us instead of 186.)
    if (fresh) {
      if (!more) {
        pass_turn();
        return;
      }
      if (t < tiles && !wait(&sh.qfull[g], nq++ & 1, sh)) return;
      if (!wait_soon(&sh.kfull[stage], parity, sh)) return;
    }
    owe = 0;
    const int valid = tile_valid(t, ct, len, iend);
    steps_v = (valid + 15) / 16;
    fixed = tile_fixed(t, ct, valid, i0);
    if (t < tiles) {
      tc::fence_after();
      const uint64_t ka = k_desc + (uint32_t)(stage * (S::kBlock >> 4));
      owe = 1 | (fresh ? 2 : 0) | (t + 1 == tiles ? 4 : 0);
      const uint32_t desc = valid > kTile / 2 ? kDescS : kDescHalf;
      if (elected) {
        tc::mma_ss(s_at, q_desc, ka, desc, false);
#pragma unroll
        for (int x = 1; x < DP / 16; ++x) {
          const uint32_t off = ((x >> 2) * S::kHalf + (x & 3) * 32) >> 4;
          if (x < steps) tc::mma_ss(s_at, q_desc + off, ka + off, desc, true);
        }
        tc::mma_commit(&sh.sfull[g]);
        if (owe & 4) tc::mma_commit(&sh.qempty[g]);
        tc::mma_commit(&sh.kempty[stage]);
      }
    } else if (elected) {
      tc::bar_arrive(&sh.kempty[stage]);
    }
    pass_turn();
    ++t;
    ++n;
  }
}

// The larger absolute values of two pairs; NaN stays.
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One warp puts down the segments for the other roles, and clears values. Value rows past the end of a tile become zero
// (a weight of zero times what lies there need not be zero), and so do NaN and infinities at positions that only some rows
// of the item attend to: the rows that do add them in add_odd_values.
template <int DP, bool BF16>
__device__ void fix_values(const PromptParams& p, Shared& sh, uint8_t* v_smem, int lane) {
  using S = Smem<DP>;
  constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
  Walk w;
  w.start(p, sh.plan);
  Segment s;
  uint32_t n = 0, put = 0;
  // The segment after the one whose tiles are looked at is put down first: the others work ahead. That waits only
  // for readers of segments long past, never for tiles of this one.
  auto put_next = [&]() {
    const int at = (int)(put % kSegs);
    const uint32_t parity = put / kSegs & 1;
    ++put;
    if (!wait(&sh.segempty[at], parity ^ 1, sh)) return false;
    if (lane == 0) {
      w.next(p, sh.plan, sh.seg[at]);
      const Segment& q = sh.seg[at];
      if (q.t0 == 0 && q.t1 > 0 && q.t1 < q.tt) {  // it begins here and goes on in the next CTAs
        p.cuts[blockIdx.x] = Cut{parts_of(sh.plan, q), q.rows, q.h, 0, q.base + q.i0};
        sh.cut = 1;
      }
      if (q.t1 == q.t0 && !sh.cut) p.cuts[blockIdx.x] = Cut{0, 0, 0, 0, 0};
      tc::bar_arrive(&sh.segfull[at]);
    }
    __syncwarp();
    return true;
  };
  for (int seg = -1;; ++seg) {
    if (seg >= 0) {
      s = sh.seg[seg % kSegs];  // not written again before this warp puts down kSegs more
      if (s.t1 == s.t0) return;
    }
    if (!put_next()) return;
    if (seg < 0) continue;
    for (int t = s.t0; t < s.t1; ++t, ++n) {
      const int valid = tile_valid(t, s.ct, s.len, s.iend);
      int stage;
      uint32_t parity;
      ring<S::kV>(n, stage, parity);
      // every tile is waited for and let go here too, so that the ring never runs ahead of this warp
      if (!wait(&sh.vfull[stage], parity, sh)) return;
      if (!tile_fixed(t, s.ct, valid, s.i0)) {
        if (lane == 0) tc::bar_arrive(&sh.vempty[stage]);
        continue;
      }
      uint8_t* at = v_smem + stage * S::kBlock;
      const int upto = (valid + 15) / 16 * 16;
      const int some = t < s.ct ? valid : max(0, s.i0 + 1 - (t - s.ct) * kTile);  // the first that not all rows attend to
      // whether there is a NaN or an infinity, and only then where (an instruction a word: the products wait for this)
      uint32_t most = 0;
      for (int hf = 0; hf < DP / 64; ++hf) {
        uint8_t* rows = at + hf * S::kHalf;
        for (int c = valid * 8 + lane; c < upto * 8; c += 32) *(uint4*)(rows + c * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll 8
        for (int c = some * 8 + lane; c < valid * 8; c += 32) {
          const uint4 q = *(const uint4*)(rows + c * 16);
          most = max_abs<BF16>(most, q.x);
          most = max_abs<BF16>(most, q.y);
          most = max_abs<BF16>(most, q.z);
          most = max_abs<BF16>(most, q.w);
        }
      }
      const bool odd = __any_sync(0xFFFFFFFFu, (most & kExp) == kExp || (most >> 16 & kExp) == kExp);
      if (odd) {
        for (int hf = 0; hf < DP / 64; ++hf) {
          uint32_t* words = (uint32_t*)(at + hf * S::kHalf);
          for (int c = some * 32 + lane; c < valid * 32; c += 32) {
            uint32_t e = words[c];
            if ((e & kExp) == kExp) e &= 0xFFFF0000u;
            if ((e >> 16 & kExp) == kExp) e &= 0xFFFFu;
            words[c] = e;
          }
        }
      }
      if (odd) *(volatile int*)&sh.odd_values = 1;
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::bar_arrive(&sh.vfix[stage]);
        tc::bar_arrive(&sh.vempty[stage]);
      }
    }
  }
}

// What a softmax thread keeps of its row.
struct Row {
  float m, l;  // reference maximum (a score, without c), sum of weights
};

// Scores of the columns from `n` to `upto` become -inf in tensor memory, whatever they were: few tiles of an item need it.
__device__ __noinline__ void mask_scores(uint32_t s_at, int n, int upto) {
#pragma unroll 1
  for (int c = 0; c < upto; c += 32) {
    if (__all_sync(0xFFFFFFFFu, n >= c + 32)) continue;
    uint32_t raw[32];
    tc::tmem_ld32(s_at + c, raw);
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (c + x >= n) raw[x] = 0xFF800000u;
    tc::tmem_st32(s_at + c, raw);
  }
  tc::wait_st();
}

// Scores become distances from `ref`, of rows that are far; others' stay as they are (ref 0).
__device__ __noinline__ void far_scores(uint32_t s_at, float ref, int upto) {
#pragma unroll 1
  for (int c = 0; c < upto; c += 32) {
    uint32_t raw[32];
    tc::tmem_ld32(s_at + c, raw);
#pragma unroll
    for (int x = 0; x < 32; ++x) raw[x] = __float_as_uint(__uint_as_float(raw[x]) - ref);
    tc::tmem_st32(s_at + c, raw);
  }
  tc::wait_st();
}

// Values that are no numbers, which were cleared: a row that attends to one (positions j0 .. j1 - 1) shows it, whatever its
// weight, which is positive. Added to the row where it lies: in the result, or in the part that is to be joined.
template <bool BF16>
__device__ __noinline__ void add_odd_values(const PromptParams& p, int h, int64_t base, int j0, int j1, uint16_t* out, float* part) {
  for (int j = j0; j < j1; ++j) {
    const uint16_t* v = (const uint16_t*)p.a.v_new + (base + j) * p.a.vn_row + h * p.a.vn_head;
    for (int d = 0; d < p.a.D; ++d) {
      const float x = unpack16<BF16>(v[d]);
      if (isfinite(x)) continue;
      if (out) out[d] = (uint16_t)pack16<BF16>(unpack16<BF16>(out[d]) + x, 0.0f);
      else part[d] += x;
    }
  }
}

// The warp's place in shared memory is free: its last store has read what it took.
__device__ __forceinline__ void place_free() {
  if ((threadIdx.x & 31) == 0) tc::tma_stores_read();
  __syncwarp();
}

// A group's rows of a segment leave tensor memory, 128 bytes of a row a turn, through 4 KB of shared memory of each warp's own
// (2500 clocks; 4000 with one store for a group's rows, 6500 with a row a thread). An item in one piece: the quotient, rounded. A warp whose 32 rows are in use stores them by TMA (where they are whole positions,
// or whole parts of one); other rows are stored by the threads, eight of them a row.
template <bool BF16>
__device__ __forceinline__ void write_rows(const PromptParams& p, const Segment& s, int group, int wl, bool odd, float l, int end,
                                           uint32_t o_at, uint8_t* place, const CUtensorMap* out_map) {
  const int lane = threadIdx.x & 31, eighth = lane & 7, half = p.rows2 >> 1, r0 = group * half + (wl & 96);
  const bool full = end == 32 && p.warp_box && !odd;
  const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;  // NaN stays
  const int i0 = position_of(p, r0), h0 = r0 - i0 * p.G;  // the warp's first row
#pragma unroll 1
  for (int d0 = 0; d0 < p.a.D; d0 += 64) {
    uint32_t raw[64];
    tc::tmem_ld64(o_at + d0, raw);
#pragma unroll
    for (int k = 0; k < 64; ++k) raw[k] = __float_as_uint(__uint_as_float(raw[k]) * inv);
    place_free();
#pragma unroll
    for (int k = 0; k < 64; k += 8) {
      uint32_t w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) w[x] = pack16<BF16>(__uint_as_float(raw[k + 2 * x]), __uint_as_float(raw[k + 2 * x + 1]));
      *(uint4*)(place + lane * 128 + (((k / 8) ^ eighth) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (full) {
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::tma_store_3d(out_map, tc::smem_addr(place), d0, s.h * p.G + h0, (int)s.base + s.i0 + i0);
    } else {
      __syncwarp();
      uint16_t* out = (uint16_t*)p.a.out + (s.base + s.i0) * p.a.o_row + (int64_t)s.h * p.G * p.a.o_head + eighth * 8 + d0;
#pragma unroll 1
      for (int x = lane >> 3; x < end; x += 4) {
        const int f = r0 + x, i = position_of(p, f);
        if (d0 + eighth * 8 < p.a.D)
          *(uint4*)(out + i * p.a.o_row + (f - i * p.G) * p.a.o_head) = *(const uint4*)(place + x * 128 + ((eighth ^ (x & 7)) << 4));
      }
      __syncwarp();
    }
  }
}

// A part of one: as it is, in fp32, to be joined.
template <bool BF16>
__device__ __noinline__ void leave_rows(const PromptParams& p, const Segment& s, int r, int end, uint32_t o_at, uint8_t* stage) {
  const int lane = threadIdx.x & 31, eighth = lane & 7, r0 = r - lane;
  float* part = p.o + ((int64_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * kItemRows + r0 + (lane >> 3)) * p.a.D + eighth * 4;
  uint8_t *mine = stage + lane * 128, *theirs = stage + (lane >> 3) * 128;
#pragma unroll 1
  for (int d0 = 0; d0 < p.a.D; d0 += 32) {
    uint32_t raw[32];
    tc::tmem_ld32(o_at + d0, raw);
#pragma unroll
    for (int k = 0; k < 32; k += 4) *(uint4*)(mine + (((k / 4) ^ eighth) << 4)) = make_uint4(raw[k], raw[k + 1], raw[k + 2], raw[k + 3]);
    __syncwarp();
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = *(const uint4*)(theirs + u * 512 + ((eighth ^ ((u * 4 + (lane >> 3)) & 7)) << 4));
    if (d0 + eighth * 4 < p.a.D) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (u * 4 + (lane >> 3) < end) *(uint4*)(part + u * 4 * p.a.D + d0) = v[u];
    }
    __syncwarp();
  }
}

// A group of 128 threads turns every S of its tiles into weights.
template <int DP, bool BF16>
__device__ void softmax_group(const PromptParams& p, Shared& sh, const CUtensorMap* out_map, uint8_t* out_smem, int group) {
  const int wl = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)(threadIdx.x & 96) << 16, tm = sh.tmem;
  const uint32_t s_at = tm + lanes + group * kTile, o_at = tm + lanes + 2 * kTile + group * DP;
  const int half = p.rows2 >> 1, r = group * half + wl;  // this thread's row of an item
  uint8_t* place = out_smem + (threadIdx.x >> 5) * 4096;  // this warp's
  Segments segs;
  uint32_t ns = 0, no = 0;  // phases of sfull and odone of this group
  while (segs.begin(sh)) {
    const int t0 = segs.here(sh).t0, ct = segs.here(sh).ct, len = segs.here(sh).len, iend = segs.here(sh).iend;
    const bool live = wl < half && r < segs.here(sh).rows;
    const int i = live ? segs.here(sh).i0 + position_of(p, r) : -1;  // this thread's position
    const int tiles = min(segs.here(sh).t1, group ? segs.here(sh).tiles1 : segs.here(sh).tiles0);
    Row row{-INFINITY, 0.0f};
    const bool work = __any_sync(0xFFFFFFFFu, live);
    for (int t = t0; t < tiles; ++t) {
      const int valid = tile_valid(t, ct, len, iend);
      // columns that this row attends to: all, or up to its own position
      const int see = !live ? kTile : t < ct ? valid : min(valid, i + 1 - (t - ct) * kTile);
      if (!wait_soon(&sh.sfull[group], ns++ & 1, sh)) return;
      // the tile before this one has been added up too: S of this one was issued behind it
      tc::fence_after();
      if (work) {
        const int upto = valid > 64 ? kTile : 64;  // columns past the tile's end are in no product
        if (__any_sync(0xFFFFFFFFu, see < upto)) mask_scores(s_at, see, upto);
        uint32_t raw[64];
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < upto; c += 64) {
          tc::tmem_ld64(s_at + c, raw);
#pragma unroll
          for (int x = 0; x < 64; x += 8) {
#pragma unroll
            for (int y = 0; y < 4; ++y) tops[y] = fmaxf(fmaxf(tops[y], __uint_as_float(raw[x + 2 * y])), __uint_as_float(raw[x + 2 * y + 1]));
          }
        }
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        const bool is_far = live && fabsf(top) > p.far && fabsf(top) < INFINITY;
        const bool up = t > t0 && top > __fadd_rd(row.m, p.lazy);
        if (t == t0) row.m = top;
        float ref = row.m;
        if (__any_sync(0xFFFFFFFFu, up || is_far)) {
          if (__any_sync(0xFFFFFFFFu, up)) {
            // the accumulator of the tiles so far moves to the new reference
            const float fac = up ? (row.m == -INFINITY ? 0.0f : exp2f((row.m - top) * p.c)) : 1.0f;
            if (up) {
              row.m = ref = top;
              row.l *= fac;
            }
#pragma unroll 1
            for (int d0 = 0; d0 < DP; d0 += 16) {
              uint32_t acc[16];
              tc::tmem_ld16(o_at + d0, acc);
#pragma unroll
              for (int x = 0; x < 16; ++x) acc[x] = __float_as_uint(__uint_as_float(acc[x]) * fac);
              tc::tmem_st16(o_at + d0, acc);
            }
            tc::wait_st();
          }
          // A weight is 2^(c s + off), one multiply-add. off is rounded by up to 2^-24 of itself, a factor that all weights of a row
          // have in common; it cancels, but against other tiles' and parts' (2^-16 up to kFar) and but for what 16 bits hold:
          // with c m of 2^27 it may overflow fp16, later any type, or leave a sum of zero. Far scores are taken as distances
          // from the reference first. (A tile whose scores are near has weights of zero beside a reference beyond 2 kFar.)
          // With all scores as distances, another addition a pair, 16 prompts of up to 2000 tokens take 191 us instead of 189.
          if (__any_sync(0xFFFFFFFFu, is_far)) {
            far_scores(s_at, is_far ? row.m : 0.0f, upto);
            if (is_far) ref = 0.0f;
          }
        }
        const float off = fmaf(ref == -INFINITY ? 0.0f : -ref, p.c, kShift);
        const float2 c2 = make_float2(p.c, p.c), off2 = make_float2(off, off);
        float2 l2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        // P's 64 columns lie over S's first half: the second half of S is read before P reaches it
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          if (hf * 64 < upto) {
            tc::tmem_ld64(s_at + hf * 64, raw);
            uint32_t pk[32];
#pragma unroll
            for (int x = 0; x < 64; x += 2) {
              float2 e = __ffma2_rn(make_float2(__uint_as_float(raw[x]), __uint_as_float(raw[x + 1])), c2, off2);
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              l2[x >> 1 & 1] = __fadd2_rn(l2[x >> 1 & 1], e);
              pk[x >> 1] = pack16<BF16>(e.x, e.y);
            }
            tc::tmem_st32(s_at + hf * 32, pk);
            tc::wait_st();
          }
          tc::fence_before();
          tc::bar_arrive(&sh.phalf[group][hf]);
        }
        row.l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
      } else {
        tc::fence_before();
        tc::bar_arrive(&sh.phalf[group][0]);
        tc::bar_arrive(&sh.phalf[group][1]);
      }
    }
    const bool some = tiles > t0;
    if (some) {
      if (!wait(&sh.odone[group], no++ & 1, sh)) break;
      tc::fence_after();
    }
    // O is read before this group's next weights are handed over, and with them the next segment's first product
    const Segment s = segs.here(sh);
    segs.end(sh);
    const bool odd = __any_sync(0xFFFFFFFFu, *(volatile int*)&sh.odd_values) && s.t1 > s.ct;  // another warp may set it just now
    const int end = max(0, min(32, min(half, s.rows - group * half) - (wl & 96)));  // the warp's rows in use
    if (s.t1 - s.t0 == s.tt) {
      if (some && end > 0) write_rows<BF16>(p, s, group, wl, odd, row.l, end, o_at, place, out_map);
    } else {
      if (live) p.ml[(int64_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * kItemRows + r] = make_float2(row.m, row.l);
      // without a tile of this segment the group has no result: m = -inf, l = 0 say so
      if (some && end > 0) {
        place_free();
        leave_rows<BF16>(p, s, r, end, o_at, place);
      }
    }
    if (odd && some) {
      __syncwarp();  // the warp's rows have been written, by other lanes
      const int pos = position_of(p, r);
      if (live)
        add_odd_values<BF16>(p, s.h, s.base, max(s.i0 + 1, (max(s.t0, s.ct) - s.ct) * kTile), min(i + 1, (s.t1 - s.ct) * kTile),
                             s.t1 - s.t0 < s.tt ? nullptr
                                                : (uint16_t*)p.a.out + (s.base + i) * p.a.o_row + ((int64_t)s.h * p.G + r - pos * p.G) * p.a.o_head,
                             p.o + ((int64_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * kItemRows + r) * p.a.D);
      __syncwarp();
    }
  }
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap q_map,
                  const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const __grid_constant__ CUtensorMap kn_map, const __grid_constant__ CUtensorMap vn_map,
                  const __grid_constant__ CUtensorMap out_map) {
  using S = Smem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *q_smem = smem, *k_smem = smem + 2 * S::kBlock, *v_smem = k_smem + S::kK * S::kBlock;
  Shared& sh = *(Shared*)(smem + S::kTiles);
  if (tc::smem_addr(smem) & 1023) {  // the swizzle goes by address; dynamic shared memory alone starts on 1024
    if (threadIdx.x == 0) {
      set_status(p.status, DT_DEV_INTERNAL);
      p.cuts[blockIdx.x] = Cut{0, 0, 0, 0, 0};
    }
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 9) tc::tmem_alloc<512>(&sh.tmem);
  if (tid == 0) {
    for (int i = 0; i < kMostStages; ++i) {
      tc::bar_init(&sh.kfull[i], 1);
      tc::bar_init(&sh.kempty[i], 2);
      tc::bar_init(&sh.vfull[i], 1);
      tc::bar_init(&sh.vempty[i], 3);  // the end of both groups' products and the fixing warp
      tc::bar_init(&sh.vfix[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      tc::bar_init(&sh.sfull[g], 1);
      tc::bar_init(&sh.phalf[g][0], kTile);
      tc::bar_init(&sh.phalf[g][1], kTile);
      tc::bar_init(&sh.odone[g], 1);
      tc::bar_init(&sh.qfull[g], 1);
      tc::bar_init(&sh.qempty[g], 1);
      tc::bar_init(&sh.turn[g], 1);
      tc::bar_init(&sh.drained[g], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      tc::bar_init(&sh.segfull[i], 1);
      tc::bar_init(&sh.segempty[i], kSegReaders);
    }
    tc::bar_init_fence();
    sh.stop = p.test_stop;
    sh.odd_values = 0;
    tc::tma_prefetch_map(&q_map);
    tc::tma_prefetch_map(&k_map);
    tc::tma_prefetch_map(&v_map);
    tc::tma_prefetch_map(&kn_map);
    tc::tma_prefetch_map(&vn_map);
    tc::tma_prefetch_map(&out_map);
  }
  pdl_begin();
  make_plan(p, sh);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp < 8) {
    softmax_group<DP, BF16>(p, sh, &out_map, v_smem + S::kV * S::kBlock, warp >> 2);
    if (lane == 0) tc::tma_stores_done();  // whichever way it left
  } else if (warp == 8) {
    load_tiles<DP>(p, sh, &k_map, &v_map, &kn_map, &vn_map, &q_map, tc::smem_addr(q_smem), tc::smem_addr(k_smem),
                   tc::smem_addr(v_smem), lane);
  } else if (warp == 10) {
    fix_values<DP, BF16>(p, sh, v_smem, lane);
  } else {
    issue_mma<DP, BF16>(p, sh, tc::smem_addr(q_smem), tc::smem_addr(k_smem), tc::smem_addr(v_smem), warp == 11, lane);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (sh.stop) {  // products in flight end before their memory goes, waited for by the threads that issued them
    if ((warp == 9 || warp == 11) && tc::elect()) {
      tc::mma_commit(&sh.drained[warp == 11]);
      tc::bar_drain(&sh.drained[warp == 11], 0);
    }
    __syncthreads();
    if (tid == 0) {
      set_status(p.status, DT_DEV_TIMEOUT);
      p.cuts[blockIdx.x] = Cut{0, 0, 0, 0, 0};  // what it has left of a cut item is not joined
    }
  }
  if (warp == 9) tc::tmem_free<512>(sh.tmem);
}

// ------------------------------------------------------------------------------- join -----------
constexpr int kJoinWarps = 4;
constexpr int kJoinRows = 4 * kJoinWarps;  // rows of a CTA: eight lanes a row, each up to 16 elements of it
// CTA (c, y): rows [y kJoinRows, ...) of the item that is cut and begins in CTA c of the kernel before.
template <bool BF16>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ PromptParams p) {
  pdl_begin();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31, e = lane & 7;
  const Cut cut = p.cuts[c0];
  const int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5) * 4 + (lane >> 3);
  if (r >= cut.rows) return;
  auto slot = [&](int k) { return ((int64_t)2 * (c0 + k) + (k == 0 ? 1 : 0)) * kItemRows + r; };
  float m = -INFINITY;
  for (int k = 0; k < cut.parts; ++k) m = fmaxf(m, p.ml[slot(k)].x);
  const float ref = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  float4 o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = make_float4(0, 0, 0, 0);
#pragma unroll 2
  for (int k = 0; k < cut.parts; ++k) {
    const float2 x = p.ml[slot(k)];
    if (x.x == -INFINITY && x.y == 0.0f) continue;  // no tile of the row's group: its result was not written
    const float w = exp2f((x.x - ref) * p.c);
    l += x.y * w;
    const float* src = p.o + slot(k) * p.a.D + e * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j * 32 + e * 4 < p.a.D) {
        const float4 v = *(const float4*)(src + j * 32);
        o[j].x = fmaf(v.x, w, o[j].x);
        o[j].y = fmaf(v.y, w, o[j].y);
        o[j].z = fmaf(v.z, w, o[j].z);
        o[j].w = fmaf(v.w, w, o[j].w);
      }
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
  const int i = position_of(p, r);
  uint16_t* out = (uint16_t*)p.a.out + (cut.row + i) * p.a.o_row + ((int64_t)cut.h * p.G + r - i * p.G) * p.a.o_head + e * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j * 32 + e * 4 < p.a.D)
      *(uint2*)(out + j * 32) = make_uint2(pack16<BF16>(o[j].x * inv, o[j].y * inv), pack16<BF16>(o[j].z * inv, o[j].w * inv));
}

// ------------------------------------------------------------------------------- host -----------
// What follows from the heads and the page.
void shape_params(PromptParams& p) {
  p.G = p.a.H_q / p.a.H_kv;
  p.pos = kTile / p.G;
  p.rows2 = 2 * p.pos * p.G;
  p.w = 2 * p.pos;
  p.warp_box = 32 % p.G == 0 || p.G % 32 == 0;
  p.g_magic = (uint32_t)((0x100000000ull + p.G - 1) / p.G);
  while ((1 << p.page_shift) < p.a.page) ++p.page_shift;
  p.period = kTile;
  p.step = p.w;
  while (p.period > 1 && p.step % 2 == 0) {
    p.period /= 2;
    p.step /= 2;
  }
  while ((1 << p.period_shift) < p.period) ++p.period_shift;
  for (int r = 1, sum = 0; r <= p.period; ++r) {
    sum += (r * p.step + p.period - 1) / p.period;
    if (r < p.period) p.part[r] = (uint16_t)sum;
    p.part_all = sum;
  }
}

struct Layout {
  int64_t ml, o, total;
};
Layout layout_of(const dt_handle* h, int D) {
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  Layout L;
  L.ml = up((int64_t)sizeof(Cut) * h->num_sms);
  L.o = up(L.ml + 8ll * 2 * h->num_sms * kItemRows);
  L.total = up(L.o + 4ll * 2 * h->num_sms * kItemRows * D);
  return L;
}

// Items of few tiles are not cut: a launch to join them costs more than an uneven share. One prompt, four heads a key head, heads
// of 128, cut and whole, us: eight key heads 93 tokens 12.1 and 8.8, 512 17.1 and 13.8, 1024 23.9 and 19.8, 1500 30.5 and 32.7,
// 2000 40.5 and 49.8; one key head 93 11.8 and 8.5, 512 16.3 and 13.3, 1024 18.7 and 19.0, 1500 21.2 and 24.6; 16 prompts of 93
// 15.4 and 12.3, with one key head 12.7 and 9.3. The host decides, which knows the buffers and not the lengths: by what the tables
// and rows could hold. So a short prompt of a cache that may grow past these tiles is cut, and joined (93 tokens, room for 8192:
// 12.1 us), and so are several whose rows together are more.
constexpr int kWholeTiles = 8;
template <int DP, bool BF16>
cudaError_t launch_t(dt_handle* h, const PromptParams& p, const CUtensorMap* m, cudaStream_t s) {
  launch_k(prompt_kernel<DP, BF16>, dim3(h->num_sms), dim3(kPromptThreads), kSmemBytes<DP>, s, p, m[0], m[1], m[2], m[3], m[4], m[5]);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.whole) return e;
  launch_k(join_kernel<BF16>, dim3(h->num_sms, (p.rows2 + kJoinRows - 1) / kJoinRows), dim3(32 * kJoinWarps), 0, s, p);
  return cudaGetLastError();
}

template <int DP, bool BF16>
cudaError_t init_t() {
  return cudaFuncSetAttribute(prompt_kernel<DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<DP>);
}

}  // namespace

cudaError_t init_prompt_attributes() {
  cudaError_t e = init_t<64, true>();
  if (e == cudaSuccess) e = init_t<64, false>();
  if (e == cudaSuccess) e = init_t<128, true>();
  if (e == cudaSuccess) e = init_t<128, false>();
  return e;
}

bool prompt_line_fits(const dt_handle* h, const dt_prompt_args* a) {
  const int w = 2 * (kTile / (a->H_q / a->H_kv));
  const double tiles = (double)(a->seq_len ? (double)a->max_blocks * a->page / kTile : 0.0) + (double)a->rows / kTile + 2;
  return (double)a->H_kv * ((double)a->rows / w + a->B) * (kItemUnits + tiles) < 2.0e9 * h->num_sms;
}

int64_t prompt_workspace_bytes(const dt_handle* h, int D) { return layout_of(h, D).total; }

cudaError_t launch_prompt(dt_handle* h, const dt_prompt_args* a, cudaStream_t s) {
  PromptParams p{};
  p.a = *a;
  const bool cached = a->seq_len != nullptr;
  if (!cached) p.a.page = kTile;
  shape_params(p);
  p.c = a->scale * kLog2e;
  p.lazy = kLazy / p.c;
  p.far = kFar / p.c;
  // tiles of an item, at most
  const int64_t most = (cached ? ((int64_t)a->max_blocks * a->page + kTile - 1) / kTile : 0) + (a->rows + kTile - 1) / kTile;
  p.whole = most <= kWholeTiles;
  const Layout L = layout_of(h, a->D);
  char* ws = (char*)a->workspace;
  p.cuts = (Cut*)ws;
  p.ml = (float2*)(ws + L.ml);
  p.o = (float*)(ws + L.o);
  p.status = h->ws.status;
  p.test_stop = h->cfg.flags & DT_FLAG_TEST_TIMEOUT ? 1 : 0;
  CUtensorMap m[6];
  const int64_t nd[3] = {a->D, a->H_kv, a->rows};
  const int64_t kn[3] = {1, a->kn_head, a->kn_row}, vn[3] = {1, a->vn_head, a->vn_row};
  const int nb[3] = {64, 1, kTile};
  const int64_t qd[3] = {a->D, a->H_q, a->rows}, qs[3] = {1, a->q_head, a->q_row};
  const int qb[3] = {64, p.G, p.pos}, ob[3] = {64, std::min(p.G, 32), std::max(32 / p.G, 1)};
  const int64_t os[3] = {1, a->o_head, a->o_row};
  bool ok = encode(&m[0], a->dtype, a->q, 3, qd, qs, qb) && encode(&m[5], a->dtype, a->out, 3, qd, os, ob) && encode(&m[3], a->dtype, a->k_new, 3, nd, kn, nb) &&
            encode(&m[4], a->dtype, a->v_new, 3, nd, vn, nb);
  if (cached) {
    const int64_t pd[4] = {a->D, a->H_kv, a->page, a->n_blocks};
    const int64_t ks[4] = {1, a->k_head, a->k_tok, a->k_block}, vs[4] = {1, a->v_head, a->v_tok, a->v_block};
    const int pb[4] = {64, 1, std::min<int>(a->page, kTile), 1};
    ok = ok && encode(&m[1], a->dtype, a->k_pages, 4, pd, ks, pb) && encode(&m[2], a->dtype, a->v_pages, 4, pd, vs, pb);
  } else {  // never read
    m[1] = m[3];
    m[2] = m[4];
  }
  if (!ok) return cudaErrorInvalidValue;
  if (a->D <= 64) return a->dtype == DT_BF16 ? launch_t<64, true>(h, p, m, s) : launch_t<64, false>(h, p, m, s);
  return a->dtype == DT_BF16 ? launch_t<128, true>(h, p, m, s) : launch_t<128, false>(h, p, m, s);
}

}  // namespace dt
