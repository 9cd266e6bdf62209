// Attention of the verify tree over a paged cache.
//
// For query row f = (position, head of the group) of request b and key head h, with c = scale * log2 e:
//   out_f = sum_j 2^(c s_fj - m_f) v_j / sum_j 2^(c s_fj - m_f),  s_fj = q_f k_j,
// j over the cached tokens and the tree positions that f's mask row allows. The n_pos * G rows of a request and
// key head attend to the same cached tokens, so they are the 128-row operand of the matrix instructions and
// every key and value is read once for up to 256 of them; a prefix that all requests share is read once for
// 256 rows of any requests.
//
// Work. An item is up to 256 rows of one key head over a list of 128-token tiles: the shared prefix's, or one
// request's own cached tokens and then its tree positions. All tiles in item order form one line that the CTAs
// (one a SM) cut into equal runs, whatever the lengths; a CTA's run of one item is a segment. A segment that is a
// whole item of an unshared call writes the result; others leave sum, maximum and unnormalised result in
// fp32, joined in a fixed order by the CTA that comes last to the item (few rows, no shared prefix) or by
// attn_merge_kernel. Every CTA derives the cuts from the lengths on the device, so a captured call follows them.
//
// A CTA: warps 0-3 and 4-7 are two softmax groups (thread = row), warp 8 loads K tiles, warp 11 V tiles (TMA, one
// box a page and 64 elements), warp 9 loads Q rows and issues the matrix instructions, warp 10 walks along the line
// and clears value rows past the end. Every wait is bounded (DT_DEV_TIMEOUT).
// The line of work is a sequence of units u = 0, 1, ... for groups u & 1: with more than 128 rows a tile gives two
// units, one for each half of the rows; with fewer, tiles alternate between the groups, whose results are
// joined at the end. S = Q K^T of unit u + 2 is issued right behind O += P V of unit u, so the tensor cores
// work for one group while the other takes its softmax; P goes over in halves. S (fp32), P (16-bit, over S) and O
// live in tensor memory, which they fill (2 x 128 + 2 x 128 columns at D = 128).
//
// What bounds it, at D = 128 on one GB300: few rows, the cache's bytes (64 requests, 5100 cached tokens on average:
// 6.3 TB/s, 0.93 of the measured copy peak); a shared prefix, the chain of one group's softmax (about 1400 clocks a tile
// of 128 x 128, 450 of them for 64 columns' powers, where the unit for them would need 260) and its two products (1030),
// of which the tensor cores are busy 2060 of 2750 clocks; small calls,
// latency (11 us: 1.3 for the plan, 1 for the first segment, 2.5 for the first tiles, 1.1 softmax, 3 for the join).
// One issuing thread behind `if (lane == 0)` instead of the uniform path cost 70 clocks an instruction (attend to 64
// requests behind a prefix: 436 against 294 us); fully unrolled softmax code for masked and unmasked tiles missed the
// instruction cache and made a segment's ends 4 to 12 us long instead of 2 to 3.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dt_internal.cuh"
#include "tc.cuh"

namespace dt {
namespace {

constexpr int kTile = 128;      // tokens of a tile, rows of a group
constexpr int kItemRows = 256;  // rows of an item, at most (whole positions: 2 * (128 / G) * G)
constexpr int kAttnThreads = 384;
constexpr float kLazy = 8.0f;   // the reference maximum moves when a row passes it by 2^kLazy
constexpr float kShift = 6.0f;  // weights are held as 2^kShift times themselves: up to 2^14, inside fp16, and
                                // small ones stay normal in fp16 for longer; it cancels in the quotient

struct AttnHead {  // start of the workspace, written by CTA 0 for the merge
  int32_t per;     // units of a CTA
  int32_t w_shared;
  int32_t sh_head, mp_s, rows_s;
};

struct AttnParams {
  dt_attn_args a;
  int32_t G, page_shift, tree_box;
  int32_t join;       // split items are joined by the CTA that comes last (items of at most kJoinRows rows, unshared)
  unsigned* tickets;  // [CTAs] arrivals at the split item whose first CTA this is; zero between calls
  int32_t test_stop;  // test only: every wait that is not over at once gives up
  int32_t pos, rows2; // whole positions of a group's 128 rows (128 / G), rows of an item (2 pos G)
  uint32_t g_magic;   // ceil(2^32 / G), for position_of
  float c;            // scale * log2 e
  int32_t ns;         // tiles of the shared prefix as items of its own; 0: requests read it with their own tokens
  int32_t skip;       // tokens that a request's own items leave to it
  int64_t own_rows;   // rows of an own item's partials
  int32_t by_cut;     // their slots go by the CTA of the first cut instead of by item: layout_of
  AttnHead* head;
  int32_t* t_pre;     // [B] unit offset of a request among the own units
  int32_t* k_pre;     // [B] item offset
  float2* ml_own;     // [slot][own_rows] (m, l)
  float* o_own;       // [slot][own_rows][D]
  float2* ml_sh;      // [slot][kItemRows]
  float* o_sh;
  int32_t* status;
};

// x / G for a row x < 256 of an item: exact, as x (g_magic G - 2^32) < 2^32.
__device__ __forceinline__ int position_of(const AttnParams& p, int x) {
  return p.G == 1 ? x : (int)__umulhi((uint32_t)x, p.g_magic);
}

struct Request {
  int len, n;      // cached tokens, positions
  int64_t base;    // row of position 0
  bool bad;
};

// Rows that belong to requests.
__device__ __forceinline__ int64_t rows_used(const dt_attn_args& a) {
  const int64_t padded = (int64_t)a.B * a.P;
  return a.row_off ? min(max((int64_t)a.row_off[a.B], (int64_t)0), min(padded, a.rows)) : padded;
}

__device__ __forceinline__ Request request_of(const dt_attn_args& a, int page_shift, int b) {
  Request r;
  const int len = a.seq_len[b], n = a.n_pos[b];
  r.base = a.row_off ? (int64_t)a.row_off[b] : (int64_t)b * a.P;
  const int64_t most = min((int64_t)a.max_blocks << page_shift, (int64_t)0x7FFFFF00);
  r.len = (int)min((int64_t)max(len, a.shared_len), most);
  r.n = min(max(n, 0), a.P);
  // one without positions (an idle place in the batch) needs no prefix
  r.bad = (n != 0 && len < a.shared_len) || len > most || n < 0 || n > a.P;
  // the rows behind a packed batch's end are no request's (and no shared item's)
  if (r.base < 0 || r.base + r.n > rows_used(a)) {
    r.bad = true;
    r.n = 0;
  }
  return r;
}

// The line in units of about 0.5 us: a tile takes three for two halves of rows and two for one (1.55 and 1.05 us measured),
// and an item kItemUnits more in front, for what it costs beside its tiles: an empty pipeline at its begin and end, and
// its rows' way out (about 6 us). Tile t of an item at unit u starts at u + kItemUnits + t * units of a tile, and belongs
// to the CTA that unit falls to.
constexpr int kItemUnits = 12;
__device__ __forceinline__ int tile_units(const AttnParams& p, int rows) { return rows > p.rows2 >> 1 ? 3 : 2; }

// Items of a request for all key heads, tiles of one item.
// The tree's positions begin a tile of their own or, where the last cached tokens and all positions fit into one, stand
// in that tile behind the tokens' pages: position 0 is column `col` of tile `tree`.
struct Extent {
  int mp, tt;            // row blocks a head; tiles
  int tree, col;
  int full, last;        // units of an item of all its rows, of a head's last item
  __device__ __forceinline__ int head() const { return (mp - 1) * full + last; }
  __device__ __forceinline__ int all(int heads) const { return tt > 0 ? heads * head() : 0; }
};
__device__ __forceinline__ Extent extent_of(const AttnParams& p, const Request& r) {
  Extent e;
  e.mp = (r.n + 2 * p.pos - 1) / (2 * p.pos);
  const int cached = r.len - p.skip, rest = cached & (kTile - 1), box = min(p.a.page, kTile);
  e.tree = (cached + kTile - 1) / kTile;
  e.col = (rest + box - 1) & -box;  // pages are loaded whole
  const bool with = rest > 0 && e.col + ((r.n + p.tree_box - 1) & -p.tree_box) <= kTile;
  if (with) --e.tree;
  else e.col = 0;
  e.tt = r.n > 0 ? e.tree + (e.col + r.n + kTile - 1) / kTile : 0;
  e.full = kItemUnits + 3 * e.tt;
  e.last = kItemUnits + tile_units(p, r.n * p.G - (e.mp - 1) * p.rows2) * e.tt;
  return e;
}

// Items of its own for a shared prefix cost a launch to join them and an item's ends; they pay from about ten units an SM
// that the requests' own items would have more. 8 key heads of 128, groups of 4, as items of their own against with the
// requests' tokens: 8 requests behind 512 tokens (2.7 units an SM) 17.0 and 15.2 us, 20 behind 1024 (7.2) 21.6 and 18.5,
// 8 behind 2048 (10.9) 19.1 and 20.2, 32 behind 1024 (26) 25 and 32, 64 behind 2048 (105) 40 and 75.
constexpr int kShareUnits = 10;

// A CTA's share and where it starts.
struct Plan {
  int32_t x0, x1, per;  // units [x0, x1) of the line, units of a CTA
  int32_t w_shared;
  int32_t t_b;          // own unit offset of request b
  int32_t b, k_b;       // first own request, its item offset
  int32_t ts, mp_s, rows_s, sh_head;  // shared: tiles, row blocks, rows, units of a key head
};

struct Segment {
  int shared, whole;    // whole: an item without other parts, written straight to the result
  int b, h, mp;
  int t0, t1;           // tiles; none: the line is at its end
  int len, tok0;        // cached tokens, the first tile's first one
  int tree, col;        // tile and column of position 0
  int n;                // positions (0 for the shared prefix)
  int rows;             // rows of the item
  int i0;               // position of its first rows
  int c0, parts;        // first CTA of the item and how many have tiles of it
  int64_t base;         // row of the first position
  int64_t slot;
};

// One lane walks along the CTA's run.
struct Walk {
  int x, t_b;
  int b, k_b;
  int loaded;           // request whose extent is held
  Request r;
  Extent e;

  __device__ void start(const Plan& pl) {
    x = pl.x0;
    t_b = pl.t_b;
    b = pl.b;
    k_b = pl.k_b;
    loaded = -1;
  }
  // The next segment that has tiles (a run may end or begin inside an item's first units).
  __device__ __forceinline__ void next(const AttnParams& p, const Plan& pl, Segment& s) {
    do {
      s.t0 = s.t1 = 0;
      if (x >= pl.x1) return;
      int item, tt, at;  // item of its kind, its tiles, our place in its units
      if (x < pl.w_shared) {
        tt = pl.ts;
        const int full = kItemUnits + 3 * tt;
        s.h = x / pl.sh_head;
        const int y = x - s.h * pl.sh_head;
        s.mp = min(y / full, pl.mp_s - 1);
        at = y - s.mp * full;
        item = s.h * pl.mp_s + s.mp;
        s.shared = 1;
        s.b = 0;
        s.tree = tt;
        s.col = 0;
        s.len = p.a.shared_len;
        s.tok0 = 0;
        s.n = 0;
        s.base = 0;
        s.rows = min(p.rows2, pl.rows_s - s.mp * p.rows2);
      } else {
        const int z = x - pl.w_shared;
        while (true) {
          if (b >= p.a.B) return;
          if (loaded != b) {
            r = request_of(p.a, p.page_shift, b);
            e = extent_of(p, r);
            loaded = b;
          }
          const int w = e.all(p.a.H_kv);
          if (z < t_b + w) break;
          t_b += w;
          k_b += p.a.H_kv * e.mp;
          ++b;
        }
        tt = e.tt;
        s.h = (z - t_b) / e.head();
        const int y = z - t_b - s.h * e.head();
        s.mp = min(y / e.full, e.mp - 1);
        at = y - s.mp * e.full;
        item = k_b + s.h * e.mp + s.mp;
        s.shared = 0;
        s.b = b;
        s.tree = e.tree;
        s.col = e.col;
        s.len = r.len;
        s.tok0 = p.skip;
        s.n = r.n;
        s.base = r.base;
        s.rows = min(p.rows2, r.n * p.G - s.mp * p.rows2);
      }
      const int tw = tile_units(p, s.rows);
      const int end = min(tt * tw + kItemUnits, at + pl.x1 - x), u0 = x - at + kItemUnits;
      s.c0 = u0 / pl.per;
      s.parts = (u0 + (tt - 1) * tw) / pl.per - s.c0 + 1;
      x += end - at;
      s.t0 = (max(0, at - kItemUnits) + tw - 1) / tw;
      s.t1 = (max(0, end - kItemUnits) + tw - 1) / tw;
      s.slot = (int64_t)(p.by_cut ? s.c0 : item) + blockIdx.x;
      s.whole = s.t0 == 0 && s.t1 == tt && p.ns == 0;
      s.i0 = s.mp * 2 * p.pos;
    } while (s.t1 == s.t0);
  }
};

// Columns of tile t that are in use, and whether it holds tree positions.
__device__ __forceinline__ int tile_valid(const Segment& s, int t, bool& tree) {
  tree = t >= s.tree;  // (a shared prefix: never)
  return min(kTile, tree ? s.col + s.n - (t - s.tree) * kTile : s.len - s.tok0 - t * kTile);
}
// Its columns of cached tokens.
__device__ __forceinline__ int tile_cached(const Segment& s, int t) {
  return max(0, min(kTile, s.len - s.tok0 - t * kTile));
}

template <int DP>
struct Smem {
  static constexpr int kHalf = kTile * 128;              // bytes of 64 elements of 128 rows
  static constexpr int kBlock = (DP / 64) * kHalf;       // a tile of Q, K or V
  // tiles of K and of V in flight: a V tile is held longer, from its load until the weights have come
  static constexpr int kK = DP == 128 ? 2 : 5, kV = DP == 128 ? 3 : 6;
  static constexpr int kTiles = (2 + kK + kV) * kBlock;
};
constexpr int kMostStages = 6;

constexpr int kSegs = 4;  // segments that warp 10 is ahead of the slowest reader, at most

struct Shared {
  uint64_t kfull[kMostStages], kempty[kMostStages], vfull[kMostStages], vempty[kMostStages], vfix[kMostStages];
  uint64_t sfull[2], phalf[2][2], odone[2], qfull, qfree, mlready, parts_in, ticket_in, drained;
  uint64_t segfull[kSegs], segempty[kSegs];
  Segment seg[kSegs];
  float2 ml[2][kTile];
  Plan plan;
  int32_t sums[2][12];
  uint32_t tmem;
  int stop, odd_values, last;
};

template <int DP>
constexpr int kSmemBytes = Smem<DP>::kTiles + (int)sizeof(Shared);
static_assert(kSmemBytes<128> <= 232448 && kSmemBytes<64> <= 232448, "227 KB a CTA");

// The other warps read the segments that warp 10 puts down, in order. `lead`: the lane that gives the place back.
struct Segments {
  uint32_t n = 0;
  __device__ __forceinline__ bool next(Shared& sh, Segment& s, bool lead) {
    const int at = (int)(n % kSegs);
    const uint32_t parity = n / kSegs & 1;
    ++n;
    if (!tc::bar_wait_warp(&sh.segfull[at], parity, &sh.stop)) return false;
    s = sh.seg[at];
    __syncwarp();
    if (lead) tc::bar_arrive(&sh.segempty[at]);
    return s.t1 > s.t0;
  }
};
constexpr int kSegReaders = 11;  // eight softmax warps, two loading warps, the issuing warp

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

// Units of a key head's items over the shared prefix.
__device__ __forceinline__ int shared_head(const AttnParams& p, int rows_s, int mp_s, int ts) {
  return (mp_s - 1) * (kItemUnits + 3 * ts) + kItemUnits + tile_units(p, rows_s - (mp_s - 1) * p.rows2) * ts;
}

// Every CTA: the line's length and where its own run starts.
__device__ __forceinline__ void make_plan(const AttnParams& p, Shared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (p.a.B + kAttnThreads - 1) / kAttnThreads, b0 = tid * chunk, b1 = min(p.a.B, b0 + chunk);
  int units = 0, items = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(p.a, p.page_shift, b);
    const Extent e = extent_of(p, r);
    units += e.all(p.a.H_kv);
    items += p.a.H_kv * e.mp;
    if (blockIdx.x == 0 && r.bad) set_status(p.status, DT_DEV_BAD_PAGE);
  }
  if (p.a.row_off && blockIdx.x == 0 && tid == 0) {
    const int64_t last = p.a.row_off[p.a.B];
    if (last < 0 || last > min((int64_t)p.a.B * p.a.P, p.a.rows)) set_status(p.status, DT_DEV_BAD_PAGE);
  }
  int su = units, si = items;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, su, d), c = __shfl_up_sync(0xFFFFFFFFu, si, d);
    if (lane >= d) {
      su += a;
      si += c;
    }
  }
  if (lane == 31) {
    sh.sums[0][warp] = su;
    sh.sums[1][warp] = si;
  }
  __syncthreads();
  int total = 0, t_b = su - units, k_b = si - items;
#pragma unroll
  for (int w = 0; w < kAttnThreads / 32; ++w) {
    const int a = sh.sums[0][w], c = sh.sums[1][w];
    if (w < warp) {
      t_b += a;
      k_b += c;
    }
    total += a;
  }
  const int rows_s = p.ns ? (int)rows_used(p.a) * p.G : 0;
  const int mp_s = (rows_s + p.rows2 - 1) / p.rows2;
  const int sh_head = mp_s > 0 ? shared_head(p, rows_s, mp_s, p.ns) : 0;
  const int w_shared = p.a.H_kv * sh_head;
  total += w_shared;
  // at least a tile's units: no CTA between an item's first and last one is without a tile
  const int per = max(3, (total + (int)gridDim.x - 1) / (int)gridDim.x);
  const int x0 = min(total, per * (int)blockIdx.x), x1 = min(total, x0 + per);
  if (tid == 0) {
    Plan& pl = sh.plan;
    pl.x0 = x0;
    pl.x1 = x1;
    pl.per = per;
    pl.w_shared = w_shared;
    pl.ts = p.ns;
    pl.mp_s = mp_s;
    pl.rows_s = rows_s;
    pl.sh_head = sh_head;
    if (x0 <= w_shared) {  // the own requests from the first
      pl.b = 0;
      pl.t_b = 0;
      pl.k_b = 0;
    }
    if (blockIdx.x == 0) *p.head = AttnHead{per, w_shared, sh_head, mp_s, rows_s};
  }
  const int y0 = x0 - w_shared;
  for (int b = b0; b < b1; ++b) {
    int w = units, k = items;
    if (chunk > 1) {
      const Extent e = extent_of(p, request_of(p.a, p.page_shift, b));
      w = e.all(p.a.H_kv);
      k = p.a.H_kv * e.mp;
    }
    if (y0 > 0 && t_b <= y0 && y0 < t_b + w) {
      sh.plan.b = b;
      sh.plan.t_b = t_b;
      sh.plan.k_b = k_b;
    }
    if (blockIdx.x == 0) {
      p.t_pre[b] = t_b;
      p.k_pre[b] = k_b;
    }
    t_b += w;
    k_b += k;
  }
}

// Ring position of the n-th tile: stage and the parity of its use.
template <int N>
__device__ __forceinline__ void ring(uint32_t n, int& stage, uint32_t& parity) {
  stage = (int)(n % N);
  parity = (n / N) & 1;
}

// One warp loads the K (or V) tiles of the CTA's line in order.
template <int DP, bool IS_K>
__device__ void load_tiles(const AttnParams& p, Shared& sh, const CUtensorMap* pages, const CUtensorMap* tree_map,
                           uint32_t smem, int lane) {
  using S = Smem<DP>;
  uint64_t* full = IS_K ? sh.kfull : sh.vfull;
  uint64_t* empty = IS_K ? sh.kempty : sh.vempty;
  constexpr int kHalves = DP / 64, kStages = IS_K ? S::kK : S::kV;
  const int shift = p.page_shift, page = p.a.page;
  const int box = min(page, kTile);  // tokens of a page box
  const int box_shift = min(shift, 7);
  Segments segs;
  Segment s;
  uint32_t n = 0;
  bool ok = true;
  const int half = lane & (kHalves - 1), part = lane / kHalves;  // this lane's box of a tile
  while (ok && segs.next(sh, s, lane == 0)) {
    const int32_t* table = p.a.block_table + (int64_t)s.b * p.a.max_blocks;
    const int tok0 = s.tok0;
    // block id of this lane's box in tile t (-1: none)
    auto block_at = [&](int t) {
      const int tok = tok0 + t * kTile + (part << box_shift);
      if ((part << box_shift) >= kTile || tok >= s.len) return -1;
      int id = (tok < p.a.shared_len ? p.a.block_table : table)[tok >> shift];
      if (id < 0 || id >= p.a.n_blocks) {
        set_status(p.status, DT_DEV_BAD_PAGE);
        id = p.a.n_blocks;  // outside the tensor: zeros
      }
      return id;
    };
    int id = block_at(s.t0);
    for (int t = s.t0; t < s.t1; ++t, ++n) {
      int stage;
      uint32_t parity;
      ring<kStages>(n, stage, parity);
      const int next_id = t + 1 < s.t1 ? block_at(t + 1) : -1;
      ok = tc::bar_wait_warp(&empty[stage], parity ^ 1, &sh.stop);
      if (!ok) break;
      const uint32_t at = smem + stage * S::kBlock;
      bool tree;
      const int valid = tile_valid(s, t, tree);
      // page boxes of the cached tokens, then boxes of tree_box positions
      const int boxes = (tile_cached(s, t) + box - 1) >> box_shift, col = t == s.tree ? s.col : 0;
      const int tree_boxes = tree ? (valid - col + p.tree_box - 1) / p.tree_box : 0;
      if (lane == 0) tc::bar_expect(&full[stage], kHalves * 128 * (boxes * box + tree_boxes * p.tree_box));
      __syncwarp();
      if (part < boxes) {
        const int tok = tok0 + t * kTile + (part << box_shift);
        tc::tma_load_4d(at + half * S::kHalf + (part << box_shift) * 128, pages, half * 64, s.h, tok & (page - 1), id,
                        &full[stage]);
      }
      for (int k = lane; k < tree_boxes * kHalves; k += 32) {
        const int hf = k & (kHalves - 1), i = k / kHalves * p.tree_box;
        tc::tma_load_3d(at + hf * S::kHalf + (col + i) * 128, tree_map, hf * 64, s.h,
                        (int)s.base + (t - s.tree) * kTile - s.col + col + i, &full[stage]);
      }
      id = next_id;
    }
  }
  // No load may land once the CTA is gone, and any wait, here or of a reader, may be the one that gave up: the last tiles
  // are waited for whatever ended the loop (in a call that runs through, the products wait for them too).
  for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k) {
    int stage;
    uint32_t parity;
    ring<kStages>(k, stage, parity);
    tc::bar_drain(&full[stage], parity);
  }
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// One warp issues the matrix instructions of the CTA's line, all lanes on one path and one thread elected for the
// instructions themselves, so that descriptors stay in uniform registers.
template <int DP, bool BF16>
__device__ void issue_mma(const AttnParams& p, Shared& sh, const CUtensorMap* q_map, uint32_t q_smem, uint32_t k_smem, uint32_t v_smem, int lane) {
  using S = Smem<DP>;
  constexpr uint32_t kDescS = tc::instr_desc(BF16, kTile, kTile, false);
  constexpr uint32_t kDescO = tc::instr_desc(BF16, kTile, DP, true);
  const int steps = (p.a.D + 15) / 16;  // the padding elements of a row are zero
  const uint32_t tm = uniform(sh.tmem);
  // shared memory lies below 2^18 bytes, so offsets add up inside a descriptor's address field
  const uint64_t q_desc = tc::smem_desc(uniform(q_smem), 16, 1024), k_desc = tc::smem_desc(uniform(k_smem), 16, 1024),
                 v_desc = tc::smem_desc(uniform(v_smem), S::kHalf, 1024);
  const bool elected = tc::elect();
  Segments segs;
  Segment s;
  uint32_t kn = 0, vn = 0;    // K and V tiles so far
  uint32_t np0 = 0, np1 = 0;  // units of each group so far (phase of phalf)
  uint32_t nq = 0;            // segments so far
  uint32_t fix = 0;           // parity of every stage's vfix
  while (segs.next(sh, s, lane == 0)) {
    const bool dual = uniform(s.rows) > p.rows2 >> 1;
    const int t0 = uniform(s.t0), first = uniform(s.tree), n = uniform(s.col + s.n), cached = uniform(s.len - s.tok0);
    const int units = uniform(s.t1 - s.t0) << (dual ? 1 : 0);
    // The rows of Q, once both groups are through with the last segment's (and its accumulators): whole positions of
    // G heads. Rows past the item's belong to other positions or lie past the buffer (zeros); nobody reads theirs.
    if (!tc::bar_wait_warp(&sh.qfree, (nq & 1) ^ 1, &sh.stop)) return;
    if (elected) {
      constexpr int kHalves = DP / 64;
      const int groups = dual ? 2 : 1, bytes = p.pos * p.G * 128;
      tc::bar_expect(&sh.qfull, groups * kHalves * bytes);
      for (int x = 0; x < groups * kHalves; ++x)
        tc::tma_load_3d(q_smem + x * S::kHalf, q_map, (x % kHalves) * 64, s.h * p.G, (int)s.base + s.i0 + x / kHalves * p.pos,
                        &sh.qfull);
    }
    if (!tc::bar_wait_warp(&sh.qfull, nq & 1, &sh.stop)) {
      tc::bar_drain(&sh.qfull, nq & 1);  // no load may land once the CTA is gone
      return;
    }
    ++nq;
    int t = t0;
    // O += P V of unit v - 2, then S of unit v
    for (int v = 0; v < units + 2; ++v) {
      const int g = v & 1;
      if (v >= 2) {
        int stage;
        uint32_t parity;
        ring<S::kV>(vn, stage, parity);
        const bool tree = t >= first;  // as tile_valid
        const int valid = min(kTile, tree ? n - (t - first) * kTile : cached - t * kTile);
        if (!dual || g == 0) {
          if (!tc::bar_wait_warp(&sh.vfull[stage], parity, &sh.stop)) return;
          if (tree || valid < kTile) {
            if (!tc::bar_wait_warp(&sh.vfix[stage], fix >> stage & 1, &sh.stop)) return;
            fix ^= 1u << stage;
          }
        }
        const uint64_t va = v_desc + (uint32_t)(stage * (S::kBlock >> 4));
        const uint32_t o = tm + 2 * kTile + g * DP, pr = tm + g * kTile;
        const uint32_t np = g ? np1++ : np0++;
        const bool last = !dual || g == 1;
        // the first half's products run while the group works on the second half's weights
        if (!tc::bar_wait_warp(&sh.phalf[g][0], np & 1, &sh.stop)) return;
        tc::fence_after();
        if (elected) {
          tc::mma_ts(o, pr, va, kDescO, v >= 4);  // the group's first unit starts its accumulator
#pragma unroll
          for (int x = 1; x < kTile / 32; ++x)
            if (x * 16 < valid) tc::mma_ts(o, pr + x * 8, va + x * 128, kDescO, true);
        }
        if (!tc::bar_wait_warp(&sh.phalf[g][1], np & 1, &sh.stop)) return;
        tc::fence_after();
        if (elected) {
#pragma unroll
          for (int x = kTile / 32; x < kTile / 16; ++x)
            if (x * 16 < valid) tc::mma_ts(o, pr + x * 8, va + x * 128, kDescO, true);
          if (v >= units) tc::mma_commit(&sh.odone[g]);  // else S's commit says so too
          if (last) tc::mma_commit(&sh.vempty[stage]);
        }
        if (last) {
          ++vn;
          ++t;
        }
      }
      if (v < units) {
        int stage;
        uint32_t parity;
        ring<S::kK>(kn, stage, parity);
        if (!dual || g == 0) {
          if (!tc::bar_wait_warp(&sh.kfull[stage], parity, &sh.stop)) return;
        }
        tc::fence_after();
        const uint64_t qa = q_desc + (uint32_t)((dual ? g : 0) * (S::kBlock >> 4)), ka = k_desc + (uint32_t)(stage * (S::kBlock >> 4));
        const uint32_t d = tm + g * kTile;
        const bool last = !dual || g == 1;
        if (elected) {
          tc::mma_ss(d, qa, ka, kDescS, false);
#pragma unroll
          for (int x = 1; x < DP / 16; ++x) {
            const uint32_t off = ((x >> 2) * S::kHalf + (x & 3) * 32) >> 4;
            if (x < steps) tc::mma_ss(d, qa + off, ka + off, kDescS, true);
          }
          tc::mma_commit(&sh.sfull[g]);
          if (last) tc::mma_commit(&sh.kempty[stage]);
        }
        if (last) ++kn;
      }
    }
  }
}

// One warp puts down the segments for the other roles, and clears values. Value rows past the end of a tile become zero
// (a weight of zero times what lies there need not be zero), and so do NaN and infinities at tree positions, which only
// some rows attend to: the rows that do add them in finish_rows.
template <int DP, bool BF16>
__device__ void fix_values(const AttnParams& p, Shared& sh, uint8_t* v_smem, int lane) {
  using S = Smem<DP>;
  constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
  Walk w;
  w.start(sh.plan);
  Segment s;
  uint32_t n = 0, put = 0;
  // The segment after the one whose tiles are looked at is put down first: the others work ahead. That waits only
  // for readers of segments long past, never for tiles of this one.
  auto put_next = [&]() {
    const int at = (int)(put % kSegs);
    const uint32_t parity = put / kSegs & 1;
    ++put;
    if (!tc::bar_wait_warp(&sh.segempty[at], parity ^ 1, &sh.stop)) return false;
    if (lane == 0) {
      w.next(p, sh.plan, sh.seg[at]);
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
      bool tree;
      const int valid = tile_valid(s, t, tree);
      int stage;
      uint32_t parity;
      ring<S::kV>(n, stage, parity);
      // every tile is waited for and let go here too, so that the ring never runs ahead of this warp
      if (!tc::bar_wait_warp(&sh.vfull[stage], parity, &sh.stop)) return;
      if (!tree && valid == kTile) {
        if (lane == 0) tc::bar_arrive(&sh.vempty[stage]);
        continue;
      }
      uint8_t* at = v_smem + stage * S::kBlock;
      const int upto = (valid + 15) / 16 * 16, cached = tree ? tile_cached(s, t) : valid;
      const int col = tree && t == s.tree ? s.col : tree ? 0 : upto;  // clear: between tokens and positions, and behind
      for (int hf = 0; hf < DP / 64; ++hf) {
        for (int c = cached * 8 + lane; c < col * 8; c += 32) *(uint4*)(at + hf * S::kHalf + c * 16) = make_uint4(0, 0, 0, 0);
        if (tree) {
          for (int c = valid * 8 + lane; c < upto * 8; c += 32) *(uint4*)(at + hf * S::kHalf + c * 16) = make_uint4(0, 0, 0, 0);
          bool odd = false;
          for (int c = col * 8 + lane; c < valid * 8; c += 32) {
            uint4 q = *(uint4*)(at + hf * S::kHalf + c * 16);
            uint32_t* e = &q.x;
            bool mine = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if ((e[k] & kExp) == kExp) {
                e[k] &= 0xFFFF0000u;
                mine = true;
              }
              if ((e[k] >> 16 & kExp) == kExp) {
                e[k] &= 0xFFFFu;
                mine = true;
              }
            }
            if (mine) *(uint4*)(at + hf * S::kHalf + c * 16) = q;
            odd |= mine;
          }
          if (odd) *(volatile int*)&sh.odd_values = 1;
        }
      }
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
  float m, l;  // reference maximum (log2 units), sum of weights
};

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

// The 128 columns of tile t, which holds tree positions, that position i (-1: none) attends to, as bits; all lanes of the
// warp.
__device__ __forceinline__ void tree_bits(const AttnParams& p, const Segment& s, int t, int i, uint32_t* bits) {
  const int lane = threadIdx.x & 31, j0 = (t - s.tree) * kTile - s.col;  // position of column 0
  const int cached = t == s.tree && s.col > 0 ? tile_cached(s, t) : 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) bits[w] = low_bits(cached - 32 * w);
  if (!p.a.mask) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int c = j0 + 32 * w;  // positions max(c, 0) .. i
      if (i >= 0) bits[w] |= low_bits(i + 1 - c) & ~low_bits(-c);
    }
    return;
  }
  // rows of a warp are neighbours: positions first..last, one coalesced read and ballot for 32 columns of each
  const int first = __shfl_sync(0xFFFFFFFFu, i, 0);
  const int last = __reduce_max_sync(0xFFFFFFFFu, i);
  if (last < 0) return;
  const uint8_t* m = p.a.mask + (int64_t)s.b * p.a.P * p.a.P;
  for (int x = first; x <= last; ++x) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int j = j0 + 32 * w + lane;
      const uint32_t word = __ballot_sync(0xFFFFFFFFu, j >= 0 && j < s.n && m[(int64_t)x * p.a.P + j] != 0);
      if (x == i) bits[w] |= word;
    }
  }
}

// Scores of columns that are not attended to become -inf in tensor memory, whatever they were (few tiles of an item
// need it: a short loop of its own keeps the common path short).
__device__ __noinline__ void mask_scores(uint32_t s_at, uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
#pragma unroll 1
  for (int c = 0; c < kTile; c += 16) {
    uint32_t raw[16];
    tc::tmem_ld16(s_at + c, raw);
    const uint32_t w = (c < 64 ? c < 32 ? b0 : b1 : c < 96 ? b2 : b3) >> (c & 16);
#pragma unroll
    for (int x = 0; x < 16; ++x)
      if (!(w >> x & 1)) raw[x] = 0xFF800000u;
    tc::tmem_st16(s_at + c, raw);
  }
  tc::wait_st();
}

// Values that are no numbers at tree positions this row attends to: weight times value, from global memory.
template <bool BF16>
__device__ __noinline__ void add_odd_row(const AttnParams& p, int b, int h, int64_t base, int j0, int j1, int i, int g,
                                         float m, float scale, int d0, float* o) {
  const uint16_t* q = (const uint16_t*)p.a.q + (base + i) * p.a.q_row + ((int64_t)h * p.G + g) * p.a.q_head;
  for (int j = j0; j < j1; ++j) {
    if (p.a.mask ? p.a.mask[((int64_t)b * p.a.P + i) * p.a.P + j] == 0 : j > i) continue;
    const uint16_t* v = (const uint16_t*)p.a.v_new + (base + j) * p.a.vn_row + h * p.a.vn_head;
    const uint16_t* k = (const uint16_t*)p.a.k_new + (base + j) * p.a.kn_row + h * p.a.kn_head;
    bool odd = false;
    for (int d = d0; d < min(d0 + 32, p.a.D); ++d) odd |= !isfinite(unpack16<BF16>(v[d]));
    if (!odd) continue;
    float dot = 0.0f;
    for (int d = 0; d < p.a.D; ++d) dot += unpack16<BF16>(q[d]) * unpack16<BF16>(k[d]);
    const float wgt = exp2f(dot * p.c - m + kShift);
    for (int d = 0; d < min(32, p.a.D - d0); ++d) {
      const float x = unpack16<BF16>(v[d0 + d]);
      if (!isfinite(x)) o[d] += wgt * x * scale;
    }
  }
}

template <int DP, bool BF16>
__device__ __forceinline__ void add_odd_values(const AttnParams& p, const Segment& s, int r, float m, float scale, int d0,
                                               float (&o)[32]) {
  float x[32];  // its own array: one whose address is taken does not stay in registers
#pragma unroll
  for (int k = 0; k < 32; ++k) x[k] = o[k];
  add_odd_row<BF16>(p, s.b, s.h, s.base, max(0, (max(s.t0, s.tree) - s.tree) * kTile - s.col),
                    min(s.n, (s.t1 - s.tree) * kTile - s.col), s.i0 + r / p.G,
                    r % p.G, m, scale, d0, x);
#pragma unroll
  for (int k = 0; k < 32; ++k) o[k] = x[k];
}

// The segment's rows of a softmax group leave tensor memory. `both`: the two groups hold parts of the same rows, and this
// one takes the even (group 0) or odd blocks of 32 elements.
template <int DP, bool BF16>
__device__ void finish_rows(const AttnParams& p, Shared& sh, const Segment& s, int group, Row row, bool both, uint32_t tm,
                            uint8_t* q_smem) {
  const int wl = threadIdx.x & 127, lane = wl & 31, half = p.rows2 >> 1;
  const int r = (s.rows > half ? group * half : 0) + wl;  // row of the item
  const bool live = r < s.rows && wl < half;
  if (!__any_sync(0xFFFFFFFFu, live)) return;
  float f0 = 1.0f, f1 = 0.0f, m = row.m, l = row.l;
  if (both) {
    const float2 o = sh.ml[group ^ 1][wl];
    m = fmaxf(row.m, o.x);
    f0 = row.m == -INFINITY ? 0.0f : exp2f(row.m - m);
    f1 = o.x == -INFINITY ? 0.0f : exp2f(o.x - m);
    l = row.l * f0 + o.y * f1;
  }
  const bool odd = *(volatile int*)&sh.odd_values && s.t1 > s.tree;
  // 16-byte stores along rows, through the warp's own 32 rows of the Q buffer (its products are done), 32 elements of a
  // row a turn: four lanes a row of the result, eight of a partial.
  const int row0 = r - lane, end = min(s.rows - row0, min(32, half - (wl - lane)));  // the warp's first row, its live rows
  uint8_t* stage = q_smem + group * Smem<DP>::kBlock + (wl >> 5) * 32 * 128;
  const uint32_t o_at = tm + ((uint32_t)(threadIdx.x & 96) << 16) + 2 * kTile;
  float* part = nullptr;
  uint16_t* out[4];
  const float inv = !s.whole ? 1.0f : l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;  // nothing attended to: zeros; NaN stays
  if (s.whole) {
    f0 *= inv;
    f1 *= inv;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int ri = row0 + u * 8 + (lane >> 2), i = position_of(p, ri);
      out[u] = (uint16_t*)p.a.out + (s.base + s.i0 + i) * p.a.o_row + ((int64_t)s.h * p.G + ri - i * p.G) * p.a.o_head + (lane & 3) * 8;
    }
  } else {
    const int64_t at = s.shared ? s.slot * kItemRows : s.slot * p.own_rows;
    if (live && !(both && group == 1)) (s.shared ? p.ml_sh : p.ml_own)[at + r] = make_float2(m, l);
    part = (s.shared ? p.o_sh : p.o_own) + (at + row0 + (lane >> 3)) * p.a.D + (lane & 7) * 4;
  }
#pragma unroll 1
  for (int d0 = both ? 32 * group : 0; d0 < p.a.D; d0 += both ? 64 : 32) {
    uint32_t raw[32];
    float o[32];
    tc::tmem_ld32(o_at + group * DP + d0, raw);
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(raw[k]) * f0;
    if (both) {
      tc::tmem_ld32(o_at + (group ^ 1) * DP + d0, raw);
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = fmaf(__uint_as_float(raw[k]), f1, o[k]);
    }
    if (odd && live) add_odd_values<DP, BF16>(p, s, r, m == -INFINITY ? 0.0f : m, inv, d0, o);
    if (s.whole) {
#pragma unroll
      for (int k = 0; k < 32; k += 8)
        *(uint4*)(stage + lane * 128 + (((k / 8) ^ (lane & 7)) << 4)) =
            make_uint4(pack16<BF16>(o[k], o[k + 1]), pack16<BF16>(o[k + 2], o[k + 3]), pack16<BF16>(o[k + 4], o[k + 5]),
                       pack16<BF16>(o[k + 6], o[k + 7]));
    } else {
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        *(float4*)(stage + lane * 128 + (((k / 4) ^ (lane & 7)) << 4)) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
    }
    __syncwarp();
    if (s.whole) {
      const int c = lane & 3;
      if (d0 + c * 8 < p.a.D) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int rr = u * 8 + (lane >> 2);
          if (rr < end) *(uint4*)(out[u] + d0) = *(const uint4*)(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
        }
      }
    } else {
      const int c = lane & 7;
      if (d0 + c * 4 < p.a.D) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int rr = u * 4 + (lane >> 3);
          if (rr < end) *(uint4*)(part + u * 4 * p.a.D + d0) = *(const uint4*)(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
        }
      }
    }
    __syncwarp();
  }
}

// Items of few rows: the CTA that comes last to a split item joins its parts, so that no second launch is needed. Both
// groups; returns false after a give-up. Eight lanes hold a row, a warp four of them; with fewer rows than that the
// warps share the parts out and add up through shared memory (the Q rows' memory).
// Joined here or by a second launch, eight key heads of 128, us: one request of 2000 cached tokens, 4 rows 12.9 and 15.6, 16
// rows 14.3 and 19.2, 32 rows 16.4 and 19.1; eight requests of 2000, 32 rows 20.4 and 23.6; 64 of 300, 32 rows 31.0 and 35.5;
// 64 of 2000, 4 rows 90.8 and 92.7, 32 rows 95.3 and 97.2. With 68 rows of one request, when this took any number of
// rows, 22.5 and 18.3 (one CTA's rows against all CTAs'); not measured for many items of more than 32 rows. Behind a shared
// prefix a row's parts belong to two items, which one item's arrivals do not count.
constexpr int kJoinRows = 32;
template <int DP, bool BF16>
__device__ bool join_parts(const AttnParams& p, Shared& sh, const Segment& s, uint8_t* q_smem, uint32_t& n_in, uint32_t& n_ticket) {
  __threadfence();  // this thread's part of the rows
  tc::bar_arrive(&sh.parts_in);
  if (threadIdx.x < 32) {
    if (!tc::bar_wait_warp(&sh.parts_in, n_in & 1, &sh.stop)) return false;
    if (threadIdx.x == 0) {
      __threadfence();
      sh.last = atomicInc(&p.tickets[s.c0], s.parts - 1) == s.parts - 1;
      __threadfence();
      tc::bar_arrive(&sh.ticket_in);
    }
    __syncwarp();
  }
  ++n_in;
  if (!tc::bar_wait_warp(&sh.ticket_in, n_ticket++ & 1, &sh.stop)) return false;
  if (!*(volatile int*)&sh.last) return true;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 7;
  int blocks = 1;  // of four rows: 1, 2, 4 or 8
  while (blocks * 4 < s.rows) blocks *= 2;
  const int r = (warp & (blocks - 1)) * 4 + (lane >> 3), k0 = warp / blocks, step = 8 / blocks;
  const bool live = r < s.rows;
  const int64_t at = (s.slot - (int)blockIdx.x + s.c0) * p.own_rows + r;  // part 0's row
  float m = -INFINITY, l = 0.0f;
  float4 o[DP / 32];
#pragma unroll
  for (int j = 0; j < DP / 32; ++j) o[j] = make_float4(0, 0, 0, 0);
  if (live) {
#pragma unroll 4
    for (int k = k0; k < s.parts; k += step) m = fmaxf(m, __ldcg((const float*)(p.ml_own + at + k * p.own_rows)));
    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll 2
    for (int k = k0; k < s.parts; k += step) {
      const float2 x = __ldcg(p.ml_own + at + k * p.own_rows);
      const float w = exp2f(x.x - ref);  // a part that attends to nothing: 0
      l += x.x == -INFINITY && x.y == 0.0f ? 0.0f : x.y * w;
      const float* src = p.o_own + (at + k * p.own_rows) * p.a.D + c * 4;
#pragma unroll
      for (int j = 0; j < DP / 32; ++j) {
        if (j * 32 + c * 4 < p.a.D) {
          const float4 v = __ldcg((const float4*)(src + j * 32));
          o[j].x = fmaf(v.x, w, o[j].x);
          o[j].y = fmaf(v.y, w, o[j].y);
          o[j].z = fmaf(v.z, w, o[j].z);
          o[j].w = fmaf(v.w, w, o[j].w);
        }
      }
    }
  }
  // warps of the same rows: through shared memory to the first of them
  constexpr int kRowFloats = DP + 2;
  float* mine = (float*)q_smem + (warp * 4 + (lane >> 3)) * kRowFloats;
  if (step > 1) {
    if (k0 > 0) {
#pragma unroll
      for (int j = 0; j < DP / 32; ++j) {
        float* d = mine + j * 32 + c * 4;
        d[0] = o[j].x;
        d[1] = o[j].y;
        d[2] = o[j].z;
        d[3] = o[j].w;
      }
      if (c == 0) {
        mine[DP] = m;
        mine[DP + 1] = l;
      }
    }
    tc::bar_arrive(&sh.parts_in);
    if (!tc::bar_wait_warp(&sh.parts_in, n_in++ & 1, &sh.stop)) return false;
    if (k0 > 0) return true;
    for (int y = 1; y < step; ++y) {
      const float* other = mine + y * blocks * 4 * kRowFloats;
      const float mo = other[DP], lo = other[DP + 1], top = fmaxf(m, mo), ref = top == -INFINITY ? 0.0f : top;
      const float a = exp2f(m - ref), w = exp2f(mo - ref);
      l = l * a + lo * w;
      m = top;
#pragma unroll
      for (int j = 0; j < DP / 32; ++j) {
        const float* d = other + j * 32 + c * 4;
        o[j].x = fmaf(d[0], w, o[j].x * a);
        o[j].y = fmaf(d[1], w, o[j].y * a);
        o[j].z = fmaf(d[2], w, o[j].z * a);
        o[j].w = fmaf(d[3], w, o[j].w * a);
      }
    }
  }
  if (live) {
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    const int i = position_of(p, r);
    uint16_t* out = (uint16_t*)p.a.out + (s.base + s.i0 + i) * p.a.o_row + ((int64_t)s.h * p.G + r - i * p.G) * p.a.o_head + c * 4;
#pragma unroll
    for (int j = 0; j < DP / 32; ++j)
      if (j * 32 + c * 4 < p.a.D)
        *(uint2*)(out + j * 32) = make_uint2(pack16<BF16>(o[j].x * inv, o[j].y * inv), pack16<BF16>(o[j].z * inv, o[j].w * inv));
  }
  return true;
}

// A group of 128 threads turns every S of its units into weights.
template <int DP, bool BF16>
__device__ void softmax_group(const AttnParams& p, Shared& sh, uint8_t* q_smem, int group) {
  using S = Smem<DP>;
  const int wl = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)(threadIdx.x & 96) << 16, tm = sh.tmem;
  const uint32_t s_at = tm + lanes + group * kTile, o_at = tm + lanes + 2 * kTile + group * DP;
  Segments segs;
  Segment s;
  uint32_t ns = 0, no = 0, nml = 0;  // phases of sfull and odone of this group; of mlready
  uint32_t n_in = 0, n_ticket = 0;   // of parts_in and ticket_in
  for (uint32_t seg = 0; segs.next(sh, s, (threadIdx.x & 31) == 0); ++seg) {
    const bool dual = s.rows > p.rows2 >> 1;
    const int tiles = s.t1 - s.t0;
    const int mine = dual ? tiles : (tiles + 1 - group) / 2;
    const int r = (dual ? group * (p.rows2 >> 1) : 0) + wl;  // this thread's row of the item
    const bool live = r < s.rows && wl < p.rows2 >> 1;
    Row row{-INFINITY, 0.0f};
    const bool work = __any_sync(0xFFFFFFFFu, live);
    for (int k = 0; k < mine; ++k) {
      const int t = s.t0 + (dual ? k : 2 * k + group);
      bool tree;
      const int valid = tile_valid(s, t, tree);
      uint32_t bits[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
      const bool masked = tree || valid < kTile;
      if (tree && work) tree_bits(p, s, t, live ? s.i0 + position_of(p, r) : -1, bits);
      if (masked) {
#pragma unroll
        for (int x = 0; x < 4; ++x) bits[x] &= low_bits(valid - 32 * x);
      }
      if (!tc::bar_wait_warp(&sh.sfull[group], ns++ & 1, &sh.stop)) return;
      // the unit before this one has been added up too: S of this one was issued behind it
      tc::fence_after();
      if (work) {
        if (masked) mask_scores(s_at, bits[0], bits[1], bits[2], bits[3]);
        uint32_t raw[64];
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          tc::tmem_ld64(s_at + hf * 64, raw);
#pragma unroll
          for (int x = 0; x < 64; x += 8) {
#pragma unroll
            for (int y = 0; y < 4; ++y) tops[y] = fmaxf(fmaxf(tops[y], __uint_as_float(raw[x + 2 * y])), __uint_as_float(raw[x + 2 * y + 1]));
          }
        }
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * p.c;
        if (k == 0) {
          row.m = top;
        } else {
          const bool up = top > row.m + kLazy;
          if (__any_sync(0xFFFFFFFFu, up)) {
            // the accumulator of the rows so far moves to the new reference
            const float fac = up ? (row.m == -INFINITY ? 0.0f : exp2f(row.m - top)) : 1.0f;
            if (up) {
              row.m = top;
              row.l *= fac;
            }
#pragma unroll 1
            for (int d0 = 0; d0 < DP; d0 += 32) {
              tc::tmem_ld32(o_at + d0, raw);
#pragma unroll
              for (int x = 0; x < 32; ++x) raw[x] = __float_as_uint(__uint_as_float(raw[x]) * fac);
              tc::tmem_st32(o_at + d0, raw);
            }
            tc::wait_st();
          }
        }
        const float off = kShift - (row.m == -INFINITY ? 0.0f : row.m);
        const float2 c2 = make_float2(p.c, p.c), off2 = make_float2(off, off);
        float2 l2 = make_float2(0.0f, 0.0f);
        // P's 64 columns lie over S's first half: the second half of S is read before P reaches it
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          tc::tmem_ld64(s_at + hf * 64, raw);
          uint32_t pk[32];
#pragma unroll
          for (int x = 0; x < 64; x += 2) {
            float2 e = __ffma2_rn(make_float2(__uint_as_float(raw[x]), __uint_as_float(raw[x + 1])), c2, off2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            l2 = __fadd2_rn(l2, e);
            pk[x >> 1] = pack16<BF16>(e.x, e.y);
          }
          tc::tmem_st32(s_at + hf * 32, pk);
          tc::wait_st();
          tc::fence_before();
          tc::bar_arrive(&sh.phalf[group][hf]);
        }
        row.l += l2.x + l2.y;
      } else {
        tc::fence_before();
        tc::bar_arrive(&sh.phalf[group][0]);
        tc::bar_arrive(&sh.phalf[group][1]);
      }
    }
    // A group without a unit in this segment still comes along: its arrival on qfree below must not fall into the last
    // segment's phase, which is over once this segment's Q has been loaded.
    if (mine == 0 && !tc::bar_wait_warp(&sh.qfull, seg & 1, &sh.stop)) return;
    // the group's last product, with no S behind it
    if (mine > 0) {
      if (!tc::bar_wait_warp(&sh.odone[group], no++ & 1, &sh.stop)) return;
      tc::fence_after();
    }
    if (!dual && tiles > 1) {
      // both groups hold sums over the same rows: each takes half of the elements of the joined ones
      sh.ml[group][wl] = make_float2(row.m, row.l);
      tc::fence_before();
      tc::bar_arrive(&sh.mlready);
      if (!tc::bar_wait_warp(&sh.mlready, nml++ & 1, &sh.stop)) return;
      tc::fence_after();
    }
    if (dual || tiles > 1 || group == 0) finish_rows<DP, BF16>(p, sh, s, group, row, !dual && tiles > 1, tm, q_smem);
    if (p.join && !s.whole && !join_parts<DP, BF16>(p, sh, s, q_smem, n_in, n_ticket)) return;
    tc::fence_async_smem();  // the Q rows' memory, written and read above, goes to the next load
    tc::fence_before();
    tc::bar_arrive(&sh.qfree);
  }
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ CUtensorMap kn_map, const __grid_constant__ CUtensorMap vn_map) {
  using S = Smem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *q_smem = smem, *k_smem = smem + 2 * S::kBlock, *v_smem = k_smem + S::kK * S::kBlock;
  Shared& sh = *(Shared*)(smem + S::kTiles);
  if (tc::smem_addr(smem) & 1023) {  // the swizzle goes by address; dynamic shared memory alone starts on 1024
    if (threadIdx.x == 0) set_status(p.status, DT_DEV_INTERNAL);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 9) tc::tmem_alloc<512>(&sh.tmem);
  if (tid == 0) {
    for (int i = 0; i < kMostStages; ++i) {
      tc::bar_init(&sh.kfull[i], 1);
      tc::bar_init(&sh.kempty[i], 1);
      tc::bar_init(&sh.vfull[i], 1);
      tc::bar_init(&sh.vempty[i], 2);  // the products' end and the fixing warp
      tc::bar_init(&sh.vfix[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      tc::bar_init(&sh.sfull[g], 1);
      tc::bar_init(&sh.phalf[g][0], kTile);
      tc::bar_init(&sh.phalf[g][1], kTile);
      tc::bar_init(&sh.odone[g], 1);
    }
    tc::bar_init(&sh.qfull, 1);
    tc::bar_init(&sh.qfree, 2 * kTile);
    tc::bar_init(&sh.mlready, 2 * kTile);
    tc::bar_init(&sh.parts_in, 2 * kTile);
    tc::bar_init(&sh.ticket_in, 1);
    tc::bar_init(&sh.drained, 1);
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
  }
  pdl_begin();
  make_plan(p, sh);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp < 8) {
    softmax_group<DP, BF16>(p, sh, q_smem, warp >> 2);
  } else if (warp == 8) {
    load_tiles<DP, true>(p, sh, &k_map, &kn_map, tc::smem_addr(k_smem), lane);
  } else if (warp == 9) {
    issue_mma<DP, BF16>(p, sh, &q_map, tc::smem_addr(q_smem), tc::smem_addr(k_smem), tc::smem_addr(v_smem), lane);
  } else if (warp == 10) {
    fix_values<DP, BF16>(p, sh, v_smem, lane);
  } else {
    load_tiles<DP, false>(p, sh, &v_map, &vn_map, tc::smem_addr(v_smem), lane);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 9) {
    if (sh.stop) {  // products in flight end before their memory goes
      if (tc::elect()) {  // the thread that issued them
        set_status(p.status, DT_DEV_TIMEOUT);
        tc::mma_commit(&sh.drained);
        tc::bar_drain(&sh.drained, 0);
      }
      __syncwarp();
    }
    tc::tmem_free<512>(sh.tmem);
  }
}

// ------------------------------------------------------------------------------- merge ----------
constexpr int kMergeWarps = 4;
// A warp joins the partial results of HEADS heads of one position: the shared prefix's parts, then the request's own, in
// the order of the line. 32 / HEADS lanes take the (m, l) of a head's parts at once; then every lane adds up four
// elements of each part.
template <bool BF16, int HEADS>
__global__ void __launch_bounds__(32 * kMergeWarps) attn_merge_kernel(const __grid_constant__ AttnParams p) {
  pdl_begin();
  constexpr int kLanes = 32 / HEADS;
  const int i = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31;
  const int x0 = (blockIdx.z * kMergeWarps + (threadIdx.x >> 5)) * HEADS;  // the warp's first head
  const AttnHead hd = *p.head;
  const int t_b = p.t_pre[b], k_b = p.k_pre[b];
  const Request rq = request_of(p.a, p.page_shift, b);
  if (i >= rq.n || x0 >= p.a.H_q) return;
  const Extent e = extent_of(p, rq);
  // this lane's head: where its parts are
  const int x = x0 + lane / kLanes, k_lane = lane % kLanes;
  const int h = x / p.G, f = i * p.G + x - h * p.G, blk = f / p.rows2, item = h * e.mp + blk;
  const int u0 = hd.w_shared + t_b + h * e.head() + blk * e.full + kItemUnits;  // the item's first tile
  const int tw = tile_units(p, rq.n * p.G - blk * p.rows2);
  const int c0 = u0 / hd.per, own = (u0 + (e.tt - 1) * tw) / hd.per - c0 + 1;
  const int64_t own_at = ((p.by_cut ? (int64_t)c0 : (int64_t)k_b + item) + c0) * p.own_rows + f - blk * p.rows2;
  int parts_s = 0;
  int64_t sh_at = 0;
  if (p.ns) {
    const int64_t fl = (rq.base + i) * p.G + x - h * p.G;
    const int ms = (int)(fl / p.rows2), is = h * hd.mp_s + ms;
    const int su = h * hd.sh_head + ms * (kItemUnits + 3 * p.ns) + kItemUnits, s0 = su / hd.per;
    parts_s = (su + (p.ns - 1) * tile_units(p, hd.rows_s - ms * p.rows2)) / hd.per - s0 + 1;
    sh_at = ((int64_t)is + s0) * kItemRows + fl - (int64_t)ms * p.rows2;
  }
  // an unshared item in one part was written by its segment
  const int parts = x >= p.a.H_q || (!p.ns && own == 1) ? 0 : parts_s + own;
  const int most = __reduce_max_sync(0xFFFFFFFFu, parts);
  const int d = lane * 4;
  float m = -INFINITY, l = 0.0f;  // of this lane's head
  float4 o[HEADS];
#pragma unroll
  for (int q = 0; q < HEADS; ++q) o[q] = make_float4(0, 0, 0, 0);
  for (int k0 = 0; k0 < most; k0 += kLanes) {
    const int k = k0 + k_lane;
    const bool is_shared = k < parts_s;
    const int64_t at = is_shared ? sh_at + (int64_t)k * kItemRows : own_at + (k - parts_s) * p.own_rows;
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (k < parts) ml = is_shared ? p.ml_sh[at] : p.ml_own[at];
    const float* src = (is_shared ? p.o_sh : p.o_own) + at * p.a.D;
    float top = fmaxf(m, ml.x);
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
    // a part that attends to nothing has weight 0 (and l = 0); one with NaN keeps it
    const float wgt = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
    float lw = ml.x == -INFINITY && ml.y == 0.0f ? 0.0f : ml.y * wgt;
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) lw += __shfl_xor_sync(0xFFFFFFFFu, lw, s);
    const float old = m == -INFINITY ? 0.0f : exp2f(m - top);
    l = l * old + lw;
    m = top;
    const int here = min(kLanes, parts - k0);  // parts of this lane's head in this turn
    const int turns = min(kLanes, most - k0);
    if (k0 > 0) {
#pragma unroll
      for (int q = 0; q < HEADS; ++q) {
        const float c = __shfl_sync(0xFFFFFFFFu, old, q * kLanes);
        o[q] = make_float4(o[q].x * c, o[q].y * c, o[q].z * c, o[q].w * c);
      }
    }
#pragma unroll 2
    for (int y = 0; y < turns; ++y) {
#pragma unroll
      for (int q = 0; q < HEADS; ++q) {
        const float w = __shfl_sync(0xFFFFFFFFu, wgt, q * kLanes + y);
        const float* from = (const float*)shfl_u64((uint64_t)src, q * kLanes + y);
        const int cnt = __shfl_sync(0xFFFFFFFFu, here, q * kLanes);
        if (y < cnt && d < p.a.D) {
          const float4 v = __ldcs((const float4*)(from + d));
          o[q].x = fmaf(v.x, w, o[q].x);
          o[q].y = fmaf(v.y, w, o[q].y);
          o[q].z = fmaf(v.z, w, o[q].z);
          o[q].w = fmaf(v.w, w, o[q].w);
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < HEADS; ++q) {
    const float lq = __shfl_sync(0xFFFFFFFFu, l, q * kLanes);
    if (__shfl_sync(0xFFFFFFFFu, parts, q * kLanes) > 0 && d < p.a.D) {
      const float inv = lq > 0.0f ? 1.0f / lq : lq == 0.0f ? 0.0f : lq;
      uint16_t* out = (uint16_t*)p.a.out + (rq.base + i) * p.a.o_row + (int64_t)(x0 + q) * p.a.o_head + d;
      *(uint2*)out = make_uint2(pack16<BF16>(o[q].x * inv, o[q].y * inv), pack16<BF16>(o[q].z * inv, o[q].w * inv));
    }
  }
}

// ------------------------------------------------------------------------------- host -----------
struct Layout {
  int64_t items, own_slots, own_rows, sh_slots;
  int64_t t_pre, k_pre, ml_own, o_own, ml_sh, o_sh, total;
};

Layout layout_of(const dt_handle* h, int B, int P, int H_q, int H_kv, int D, bool shared) {
  Layout L{};
  const int64_t G = H_q / H_kv, rows = (int64_t)P * G;
  // A segment's slot is item + CTA: the pair grows along the line, so slots are distinct. Without a shared prefix only
  // items that are cut have parts, and with more items than CTAs a slot is first CTA of the item + CTA: an item in CTAs
  // a .. a + m, m > 0, takes 2 a .. 2 a + m, and the next cut one begins in CTA a + m or later, from 2 a + 2 m on.
  const int64_t rows2 = 2 * (kTile / G) * G;
  L.items = (int64_t)B * H_kv * ((rows + rows2 - 1) / rows2);
  L.own_slots = h->num_sms + (shared ? L.items : std::min<int64_t>(L.items, h->num_sms));
  L.own_rows = std::min<int64_t>(kItemRows, rows);
  L.sh_slots = shared ? (int64_t)H_kv * ((B * rows + rows2 - 1) / rows2) + h->num_sms : 0;
  int64_t at = 256;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  L.t_pre = take(4ll * B);
  L.k_pre = take(4ll * B);
  L.ml_own = take(8 * L.own_slots * L.own_rows);
  L.o_own = take(4 * L.own_slots * L.own_rows * D);
  L.ml_sh = take(8 * L.sh_slots * kItemRows);
  L.o_sh = take(4 * L.sh_slots * kItemRows * D);
  L.total = at;
  return L;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder (a host function that touches no device state).
EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (EncodeFn)f;
  }();
  return fn;
}

// 64 elements of `box` rows a copy, 128-byte rows swizzled; strides in elements, the innermost one is 1.
bool encode(CUtensorMap* m, int dtype, const void* at, int rank, const int64_t* dims, const int64_t* strides,
            const int* box) {
  cuuint64_t d[4], st[3];
  cuuint32_t bx[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    bx[i] = (cuuint32_t)box[i];
    if (i) st[i - 1] = (cuuint64_t)strides[i] * 2;
  }
  const EncodeFn fn = encoder();
  return fn && fn(m, dtype == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                  const_cast<void*>(at), d, st, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, bool BF16>
cudaError_t launch_t(dt_handle* h, const AttnParams& p, const CUtensorMap* m, cudaStream_t s) {
  launch_k(attn_kernel<DP, BF16>, dim3(h->num_sms), dim3(kAttnThreads), kSmemBytes<DP>, s, p, m[0], m[1], m[2], m[3], m[4]);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.join) return e;
  // Few rows: a warp a head, all of its parts at once; many: four heads a warp.
  const int heads = (int64_t)p.a.P * p.a.B * p.a.H_q > 16ll * h->num_sms ? 4 : 1;
  const dim3 grid(p.a.P, p.a.B, (p.a.H_q + kMergeWarps * heads - 1) / (kMergeWarps * heads));
  if (heads == 4)
    launch_k(attn_merge_kernel<BF16, 4>, grid, dim3(32 * kMergeWarps), 0, s, p);
  else
    launch_k(attn_merge_kernel<BF16, 1>, grid, dim3(32 * kMergeWarps), 0, s, p);
  return cudaGetLastError();
}

template <int DP, bool BF16>
cudaError_t init_t() {
  return cudaFuncSetAttribute(attn_kernel<DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<DP>);
}

}  // namespace

cudaError_t init_attn_attributes() {
  cudaError_t e = init_t<64, true>();
  if (e == cudaSuccess) e = init_t<64, false>();
  if (e == cudaSuccess) e = init_t<128, true>();
  if (e == cudaSuccess) e = init_t<128, false>();
  return e;
}

bool attn_line_fits(const dt_attn_args* a) {
  const int pos2 = 2 * (kTile / (a->H_q / a->H_kv));  // positions of an item
  const double own_tiles = ((double)a->max_blocks * a->page + a->P) / kTile + 2, sh_tiles = (double)a->shared_len / kTile + 1;
  const double own = (double)a->B * a->H_kv * ((a->P + pos2 - 1) / pos2) * (kItemUnits + 3 * own_tiles);
  const double sh = a->shared_len > 0 ? a->H_kv * ((double)a->B * a->P / pos2 + 1) * (kItemUnits + 3 * sh_tiles) : 0.0;
  return own + sh < 2.0e9;
}

int64_t attn_workspace_bytes(const dt_handle* h, int B, int P, int H_q, int H_kv, int D, int shared) {
  return layout_of(h, B, P, H_q, H_kv, D, shared != 0).total;
}

cudaError_t launch_attention(dt_handle* h, const dt_attn_args* a, cudaStream_t s) {
  AttnParams p{};
  p.a = *a;
  p.G = a->H_q / a->H_kv;
  p.pos = kTile / p.G;
  p.rows2 = 2 * p.pos * p.G;
  p.g_magic = (uint32_t)((0x100000000ull + p.G - 1) / p.G);
  while ((1 << p.page_shift) < a->page) ++p.page_shift;
  p.tree_box = 8;  // positions of a tree box: a power of two that covers P, up to a tile
  while (p.tree_box < a->P && p.tree_box < kTile) p.tree_box *= 2;
  p.c = a->scale * kLog2e;
  p.ns = (a->shared_len + kTile - 1) / kTile;
  // units that the requests' own items would have more if they read the prefix with their own tokens
  const int64_t blocks = (a->P + 2 * p.pos - 1) / (2 * p.pos), blocks_s = ((int64_t)a->B * a->P + 2 * p.pos - 1) / (2 * p.pos);
  const int64_t more = (int64_t)a->H_kv * p.ns * (a->B * blocks * (a->P * p.G > p.rows2 / 2 ? 3 : 2) - blocks_s * 3);
  if (more < kShareUnits * h->num_sms) p.ns = 0;
  p.skip = p.ns ? a->shared_len : 0;
  const Layout L = layout_of(h, a->B, a->P, a->H_q, a->H_kv, a->D, a->shared_len > 0);
  char* ws = (char*)a->workspace;
  p.own_rows = L.own_rows;
  p.by_cut = a->shared_len == 0 && L.items > h->num_sms;
  p.head = (AttnHead*)ws;
  p.t_pre = (int32_t*)(ws + L.t_pre);
  p.k_pre = (int32_t*)(ws + L.k_pre);
  p.ml_own = (float2*)(ws + L.ml_own);
  p.o_own = (float*)(ws + L.o_own);
  p.ml_sh = (float2*)(ws + L.ml_sh);
  p.o_sh = (float*)(ws + L.o_sh);
  p.status = h->ws.status;
  p.join = p.ns == 0 && (int64_t)a->P * p.G <= kJoinRows;
  p.tickets = h->ws.attn_tickets;
  p.test_stop = h->cfg.flags & DT_FLAG_TEST_TIMEOUT ? 1 : 0;
  CUtensorMap m[5];
  const int64_t pd[4] = {a->D, a->H_kv, a->page, a->n_blocks};
  const int64_t ks[4] = {1, a->k_head, a->k_tok, a->k_block}, vs[4] = {1, a->v_head, a->v_tok, a->v_block};
  const int pb[4] = {64, 1, std::min<int>(a->page, kTile), 1};
  const int64_t td[3] = {a->D, a->H_kv, a->rows};
  const int64_t kn[3] = {1, a->kn_head, a->kn_row}, vn[3] = {1, a->vn_head, a->vn_row};
  const int tb[3] = {64, 1, p.tree_box};
  const int64_t qd[3] = {a->D, a->H_q, a->rows}, qs[3] = {1, a->q_head, a->q_row};
  const int qb[3] = {64, p.G, p.pos};
  if (!encode(&m[0], a->dtype, a->q, 3, qd, qs, qb) || !encode(&m[1], a->dtype, a->k_pages, 4, pd, ks, pb) ||
      !encode(&m[2], a->dtype, a->v_pages, 4, pd, vs, pb) || !encode(&m[3], a->dtype, a->k_new, 3, td, kn, tb) ||
      !encode(&m[4], a->dtype, a->v_new, 3, td, vn, tb))
    return cudaErrorInvalidValue;
  if (a->D <= 64) return a->dtype == DT_BF16 ? launch_t<64, true>(h, p, m, s) : launch_t<64, false>(h, p, m, s);
  return a->dtype == DT_BF16 ? launch_t<128, true>(h, p, m, s) : launch_t<128, false>(h, p, m, s);
}

}  // namespace dt
