// Log probabilities of given tokens under rows of logits, with the row's entropy, the token's rank and the best alternatives.
//
// With m = max x, S = sum exp(x - m):  log p(t) = x_t - m - log S,  H = log S + (1 / S) sum exp(x - m) (m - x),
// rank = tokens with a larger logit, or an equal one and a lower id.
//
// Every row is read once. A warp takes a piece of a row, 1024 tokens at a time (32 a lane), and shares nothing with other warps:
// sums a lane, relative to a reference that moves when a lane passes it by 2^8, the count in front of the token, and the largest
// logit of every step. Pieces' sums are put together in a fixed order, a warp an entry. The K alternatives are read again: the
// K-th largest of a row's steps' maxima is no larger than the K-th largest token, so that only the steps that reach it are
// looked at (K of 126 for 128256 tokens, but for ties), a CTA an entry.
//
// Bound by the instructions of the sums (two exponentials a pair of tokens among about twenty): 2048 rows of 128256 bf16, 525 MB,
// take 92 us (5.7 TB/s, 0.84 of the measured copy), with the ranks 104, with one alternative 104 and with twenty 119; 512 rows
// of fp32, 263 MB, 44 us (6.0 TB/s). A few rows take the latency of two or three launches (one row: 6.3 us).
// With lists of the K largest that every warp kept as it went, one alternative made the 2048 rows three times as long (301 us),
// and CTAs of 256 threads that met four times in 8192 tokens were no faster (302 us with ranks).
#include <cuda_bf16.h>
#include <string.h>

#include <algorithm>

#include "dt_internal.cuh"

namespace dt {
namespace {

constexpr int kLpWarps = 4;
constexpr int kLpThreads = 32 * kLpWarps;
constexpr int kLpPer = 32;            // tokens of a lane at a time
constexpr int kLpStep = 32 * kLpPer;  // tokens of a warp at a time
constexpr int kLpMost = 8;            // steps of a piece, at most
constexpr float kLpLazy = 8.0f;       // the reference moves when a lane passes it by 2^kLpLazy
// CTAs of an SM: warps enough that a step's loads run beside others' sums. With the next step's tokens loaded in front of this
// one's sums, and so twice the registers, 2287 rows of 128256 bf16 took 151 us instead of 131 (8 CTAs), 734 of 128255 fp32
// 95 instead of 87 (4).
constexpr int kLpCtas = 8;

struct LpArgs {
  dt_logprob_args a;
  const void* logits;
  int64_t ld;
  int32_t V, per;     // entries of a request (path, padded)
  uint32_t S, steps;  // pieces of a row, steps of a piece
  int64_t entries;
  uint32_t all;       // pieces of all entries
  bool direct;        // the pieces' warps look their entry up
  int2* what;         // [entries] (row, token); row -1: none, token -1: none
  float4* sums;       // [entries][S] (m, s, t, count): t = sum 2^d d, d = log2 e (x - m)
  float* tops;        // [entries][S * steps] largest logit of a step
  int32_t* status;
};

// What entry e is, after checks of its request's counts and its positions.
__device__ __forceinline__ int2 entry_of(const LpArgs& p, int64_t e) {
  const dt_logprob_args& a = p.a;
  const int2 none = make_int2(-1, -1);
  int b, j;
  const bool packed = !a.path && a.row_off;
  if (packed) {  // the request whose rows hold e
    int lo = 0, hi = a.B;  // row_off[lo] <= e < row_off[hi], if it is anybody's
    if (e < a.row_off[0] || e >= a.row_off[a.B]) return none;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.row_off[mid] <= e) lo = mid;
      else hi = mid;
    }
    b = lo;
    j = (int)(e - a.row_off[b]);
  } else {
    b = (int)(e / p.per);
    j = (int)(e - (int64_t)b * p.per);
  }
  const int64_t n = (int64_t)a.n_new[b] + a.n_extra;
  const int64_t first = a.row_off ? (int64_t)a.row_off[b] : (int64_t)b * a.P;
  const int64_t rows = a.row_off ? (int64_t)a.row_off[b + 1] - first : a.P;  // the request's: a path leads to no other's
  const int64_t room = packed ? rows : min((int64_t)p.per, min(rows, (int64_t)a.P));
  if (n < 0 || n > room) {
    if (j == 0) set_status(p.status, DT_DEV_BAD_TREE);
    return none;
  }
  if (j >= n) return none;
  const int64_t k = (int64_t)j + a.shift;
  int pos = j, next = -1;
  if (a.path) {
    pos = a.path[(int64_t)b * a.D_path + j];
    if (k < n) next = a.path[(int64_t)b * a.D_path + k];
    if (pos < 0 || pos >= a.P || pos >= rows) {
      set_status(p.status, DT_DEV_BAD_TREE);
      return none;
    }
  }
  const int64_t row = first + pos;
  if (row < 0 || row >= a.rows) {
    set_status(p.status, DT_DEV_BAD_TREE);
    return none;
  }
  int token = -1;
  if (k >= n) {
    if (a.last) token = a.last[b];
  } else if (a.tokens) {
    const int64_t at = !a.path ? first + k : next >= 0 && next < a.P && next < rows ? (int64_t)b * a.P + next : -1;
    if (at >= 0 && at < a.n_tokens) token = a.tokens[at];
    else set_status(p.status, DT_DEV_BAD_TREE);
  }
  if (token < -1 || token >= p.V) {
    set_status(p.status, DT_DEV_BAD_TOKEN);
    token = -1;
  }
  return make_int2((int)row, token);
}

// Packed requests whose entries are no rows of the buffer, so that no entry's look-up meets them (b = first, first + stride, ...).
__device__ __forceinline__ void check_requests(const LpArgs& p, int first, int stride) {
  if (p.a.path || !p.a.row_off) return;
  for (int b = first; b < p.a.B; b += stride) {
    const int64_t n = (int64_t)p.a.n_new[b] + p.a.n_extra, r0 = p.a.row_off[b], r1 = p.a.row_off[b + 1];
    if (n < 0 || n > r1 - r0 || (n > 0 && (r0 < 0 || r0 + n > p.a.rows))) set_status(p.status, DT_DEV_BAD_TREE);
  }
}

// The entries' rows and tokens first where a warp takes many pieces: a search in front of every piece is five loads one after
// the other before its row's.
__global__ void __launch_bounds__(kLpThreads) logprob_entries_kernel(const __grid_constant__ LpArgs p) {
  pdl_begin();
  const int64_t e = (int64_t)blockIdx.x * kLpThreads + threadIdx.x;
  check_requests(p, (int)min(e, (int64_t)p.a.B), (int)min((int64_t)gridDim.x * kLpThreads, (int64_t)p.a.B));
  if (e < p.entries) p.what[e] = entry_of(p, e);
}

template <typename T>
__device__ __forceinline__ float logit_at(const void* logits, int64_t at) {
  if (sizeof(T) == 4) return ((const float*)logits)[at];
  return __uint_as_float((uint32_t)((const uint16_t*)logits)[at] << 16);
}

// A lane's tokens of a step: kVecs 16-byte vectors, 32 apart.
template <typename T>
struct Held {
  static constexpr int E = 16 / (int)sizeof(T), kVecs = kLpPer / E;
  uint32_t w[kLpPer * sizeof(T) / 4];
  __device__ __forceinline__ float get(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(w[i]);
    return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  }
  // v0: token of the step's first place (negative in front of a row that does not start on 16 bytes). Vectors that lie in
  // the row are read whole, others token by token; places without a token get -inf.
  __device__ __forceinline__ void load(const T* row, int v0, int V) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int v = token(v0, u * E);
      uint4 q;
      if (v >= 0 && v <= V - E) {
        q = __ldcs((const uint4*)(row + v));
      } else {
        uint32_t* x = &q.x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (sizeof(T) == 4) {
            x[k] = v + k >= 0 && v + k < V ? ((const uint32_t*)row)[v + k] : 0xFF800000u;
          } else {
            const uint32_t lo = v + 2 * k >= 0 && v + 2 * k < V ? ((const uint16_t*)row)[v + 2 * k] : 0xFF80u;
            const uint32_t hi = v + 2 * k + 1 >= 0 && v + 2 * k + 1 < V ? ((const uint16_t*)row)[v + 2 * k + 1] : 0xFF80u;
            x[k] = lo | hi << 16;
          }
        }
      }
      w[4 * u] = q.x;
      w[4 * u + 1] = q.y;
      w[4 * u + 2] = q.z;
      w[4 * u + 3] = q.w;
    }
  }
  __device__ __forceinline__ static int token(int v0, int i) {  // of place i
    return v0 + (i / E * 32 + (int)(threadIdx.x & 31)) * E + i % E;
  }
  __device__ __forceinline__ float top() const {  // the largest; NaN is left out
    if constexpr (sizeof(T) == 4) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kLpPer; i += 2) m = fmaxf(fmaxf(m, get(i)), get(i + 1));
      return m;
    } else {
      uint32_t m = w[0];
#pragma unroll
      for (int i = 1; i < kLpPer / 2; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
      return fmaxf(fmaxf(-INFINITY, bf16_lo(m)), bf16_hi(m));
    }
  }
  // Two tokens' logits, no smaller than `least` (NaN stays).
  __device__ __forceinline__ float2 pair(int i, uint32_t least) const {
    if constexpr (sizeof(T) == 4) {
      float2 r;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.x) : "f"(get(i)), "f"(__uint_as_float(least)));
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.y) : "f"(get(i + 1)), "f"(__uint_as_float(least)));
      return r;
    } else {
      uint32_t q;
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(q) : "r"(w[i >> 1]), "r"(least));
      return make_float2(bf16_lo(q), bf16_hi(q));
    }
  }
  // Logits below this are taken as this: their weight is zero, and log2 e times their distance from the reference is a number,
  // as zero times it is to be zero. (Where the reference is the type's lowest value, others are -inf and taken as they are:
  // every weight times its distance is zero or no number there, see lowest().)
  __device__ __forceinline__ static uint32_t least(float ref) {
    const uint32_t x = ref > 1.5e38f ? 0x7EB48E52u : ref > -1e29f ? 0xF149F2CAu : ref > -1.2e38f ? 0xFF2D0864u : lowest(ref) ? 0xFF800000u : kLowest;
    return sizeof(T) == 4 ? x : x >> 16 | (x & 0xFFFF0000u);
  }
  static constexpr uint32_t kLowest = sizeof(T) == 4 ? 0xFF7FFFFFu : 0xFF7F0000u;
  __device__ __forceinline__ static bool lowest(float ref) { return __float_as_uint(ref) == kLowest; }
  // How many stand in front of a token with logit xt: larger ones, and equal ones with a lower id.
  __device__ __forceinline__ int before(float xt, int token_, int v0) const {
    const uint32_t x2 = (__float_as_uint(xt) >> 16) * 0x10001u;
    uint32_t sum = 0;  // bf16: a pair of bf16, up to 16 each, exact
    int cnt = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int v = token(v0, u * E);
      if (v + E <= token_) {
        count<true>(u, xt, x2, cnt, sum);
      } else {
        count<false>(u, xt, x2, cnt, sum);
        if (v <= token_) {  // the token's own vector
#pragma unroll
          for (int k = 0; k < E; ++k) cnt += get(u * E + k) == xt && v + k < token_ && v + k >= 0;
        }
      }
    }
    if (sizeof(T) == 2) cnt += (int)bf16_lo(sum) + (int)bf16_hi(sum);
    // places in front of the row hold -inf
    const int v = token(v0, 0);
    if (v < 0 && xt == -INFINITY && v + E <= token_) cnt -= min(E, -v);
    return cnt;
  }
  template <bool EQ>
  __device__ __forceinline__ void count(int u, float xt, uint32_t x2, int& cnt, uint32_t& sum) const {
#pragma unroll
    for (int k = 0; k < E; k += 4 / (int)sizeof(T)) {
      if constexpr (sizeof(T) == 4) {
        const float y = get(u * E + k);
        cnt += EQ ? y >= xt : y > xt;
      } else {
        __nv_bfloat162 x, y, n;
        memcpy(&x, &w[(u * E + k) / 2], 4);
        memcpy(&y, &x2, 4);
        memcpy(&n, &sum, 4);
        n = __hadd2(n, EQ ? __hge2(x, y) : __hgt2(x, y));
        memcpy(&sum, &n, 4);
      }
    }
  }
};

template <typename T, bool RANK, bool TOP>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) logprob_pieces_kernel(const __grid_constant__ LpArgs p) {
  using H = Held<T>;
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
  for (uint32_t at = blockIdx.x * kLpWarps + warp; at < p.all; at += gridDim.x * kLpWarps) {
    const uint32_t e = at / p.S;
    const int2 en = p.direct ? entry_of(p, e) : p.what[e];
    if (p.direct && at == e * p.S && lane == 0) p.what[e] = en;
    if (en.x < 0) continue;
    const T* row = (const T*)p.logits + (int64_t)en.x * p.ld;
    int v0 = (int)(at - e * p.S) * (int)p.steps * kLpStep - (int)((uintptr_t)row % 16 / sizeof(T));
    const int end = min(p.V, v0 + (int)p.steps * kLpStep);  // the piece's end
    H x;
    x.load(row, v0, p.V);
    const float xt = RANK && en.y >= 0 ? logit_at<T>(row, en.y) : INFINITY;
    float ref = -INFINITY, minus = 0.0f;  // the reference, and what is added to logits
    uint32_t least = H::least(0.0f);
    float2 s2 = make_float2(0.0f, 0.0f), t2 = make_float2(0.0f, 0.0f);
    int cnt = 0;
    float* tops = p.tops + (int64_t)at * p.steps;
#pragma unroll 1
    while (true) {
      const int v1 = v0 + kLpStep;
      const float mt = x.top();
      if (TOP) {
        const float top = ord2f(__reduce_max_sync(0xFFFFFFFFu, f2ord(mt)));
        if (lane == 0) *tops = top;
        ++tops;
      }
      if (__any_sync(0xFFFFFFFFu, mt > ref && (mt - ref) * kLog2e > kLpLazy)) {
        const float top = ord2f(__reduce_max_sync(0xFFFFFFFFu, f2ord(mt)));
        if (ref != -INFINITY) {  // the sums so far move to the new reference
          const float d = fmaxf(ref - top, -1e30f) * kLog2e, f = ex2(d);
          if (H::lowest(ref)) t2 = make_float2(0.0f, 0.0f);
          t2 = make_float2((t2.x + s2.x * d) * f, (t2.y + s2.y * d) * f);
          s2 = make_float2(s2.x * f, s2.y * f);
        }
        ref = top;
        minus = -top;
        least = H::least(top);
      }
      // the reference is subtracted before log2 e is multiplied: in one step, with log2 e times the reference rounded, weights
      // would be off by 2^-24 of the reference, at -1e30, as masks leave in whole pieces, by any factor
      const float2 c2 = make_float2(kLog2e, kLog2e), m2 = make_float2(minus, minus);
      float2 s1 = make_float2(0.0f, 0.0f), t1 = s1;  // (16 terms a sum, then 8: fewer roundings than 128 in a row)
#pragma unroll
      for (int i = 0; i < kLpPer; i += 2) {
        const float2 d = __fmul2_rn(__fadd2_rn(x.pair(i, least), m2), c2);
        const float2 w = make_float2(ex2(d.x), ex2(d.y));
        s1 = __fadd2_rn(s1, w);
        t1 = __ffma2_rn(w, d, t1);
      }
      s2 = __fadd2_rn(s2, s1);
      t2 = __fadd2_rn(t2, t1);
      if (RANK) cnt += x.before(xt, en.y, v0);
      if (v1 >= end) break;
      x.load(row, v1, p.V);
      v0 = v1;
    }
    float s = s2.x + s2.y, t = H::lowest(ref) ? 0.0f : t2.x + t2.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
    }
    if (RANK) cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
    if (lane == 0) p.sums[at] = make_float4(ref, s, t, __int_as_float(cnt));
  }
}

// What a row's pieces add up to.
struct Total {
  float M;
  double logS;
  bool bad;
};
// One warp: lanes take entry e's pieces; writes its log probability, entropy and rank.
template <typename T>
__device__ __forceinline__ Total finish_entry(const LpArgs& p, int64_t e, int2 en) {
  const int lane = threadIdx.x & 31;
  const dt_logprob_args& a = p.a;
  const float4* part = p.sums + e * p.S;
  const float xt = en.y >= 0 ? logit_at<T>(p.logits, (int64_t)en.x * p.ld + en.y) : 0.0f;
  float M = -INFINITY;
  for (int k = lane; k < (int)p.S; k += 32) M = fmaxf(M, part[k].x);
  M = ord2f(__reduce_max_sync(0xFFFFFFFFu, f2ord(M)));
  // sums over pieces in 64 bits: the row's largest token alone is 1 of S, and what the others add may be small beside it
  double S = 0.0, T2 = 0.0;
  int cnt = 0;
  for (int k = lane; k < (int)p.S; k += 32) {
    const float4 q = part[k];
    const float d = q.x == -INFINITY ? 0.0f : fmaxf(q.x - M, -1e30f) * kLog2e, f = exp2f(d);
    S += (double)(q.y * f);
    T2 += (double)((q.z + q.y * d) * f);
    cnt += __float_as_int(q.w);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    S += __longlong_as_double((long long)shfl_xor_u64((uint64_t)__double_as_longlong(S), d));
    T2 += __longlong_as_double((long long)shfl_xor_u64((uint64_t)__double_as_longlong(T2), d));
  }
  cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
  const bool bad = !(S > 0.0) || !(M > -INFINITY) || M == INFINITY || S > 1e300;
  if (bad && lane == 0) set_status(p.status, DT_DEV_BAD_LOGITS);
  // log S: the exponent, and the fp32 logarithm of the mantissa in [1, 2)
  const uint64_t bits = (uint64_t)__double_as_longlong(S);
  const double mant = __longlong_as_double((long long)((bits & 0x000FFFFFFFFFFFFFull) | 0x3FF0000000000000ull));
  const double logS = bad ? __longlong_as_double(0x7FF8000000000000ll)
                          : (double)((int)(bits >> 52 & 0x7FF) - 1023) * 0.6931471805599453 + (double)logf((float)mant);
  if (lane == 0) {
    const bool none = bad || en.y < 0;
    const float nan = __int_as_float(0x7FC00000);
    if (a.logp) a.logp[e] = none ? nan : (float)((double)xt - (double)M - logS);
    if (a.rank) a.rank[e] = none ? -1 : cnt;
    if (a.entropy) a.entropy[e] = bad ? nan : (float)(logS - 0.6931471805599453 * T2 / S);
  }
  return Total{M, logS, bad};
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprob_finish_kernel(const __grid_constant__ LpArgs p) {
  pdl_begin();
  const int64_t e = (int64_t)blockIdx.x * kLpWarps + (threadIdx.x >> 5);
  if (e >= p.entries) return;
  const int2 en = p.what[e];
  if (en.x >= 0) finish_entry<T>(p, e, en);
}

constexpr int kTopWarps = 8;
constexpr int kTopThreads = 32 * kTopWarps;
constexpr int kTopSteps = 1024;  // maxima that are ranked at once; with more steps, K times the largest below the last one
constexpr int kTopCand = 512;    // candidates that are ranked by counting; with more, the same
struct TopShared {
  alignas(16) float tops[kTopSteps];
  uint64_t cand[kTopCand], best[kTopWarps];
  int n, n_steps;
  int list[kTopSteps];
  uint32_t tau;  // as f2ord
  Total total;
};

// The largest over the CTA.
__device__ __forceinline__ uint64_t cta_max(uint64_t x, uint64_t* best) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = max(x, shfl_xor_u64(x, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = x;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTopWarps; ++w) x = max(x, best[w]);
  return x;
}

// A CTA an entry: its sums, and its K alternatives. LANES: rows of at most K steps, where maxima of parts of steps take the place
// of the steps' (16 rows of 16000 bf16, K = 20: 11.9 us, and 69 with all tokens as candidates; 512 rows: 16.5 and 285).
template <typename T, bool LANES>
__global__ void __launch_bounds__(kTopThreads) logprob_top_kernel(const __grid_constant__ LpArgs p) {
  __shared__ TopShared sh;
  pdl_begin();
  const int64_t e = blockIdx.x;
  const int2 en = p.what[e];
  if (en.x < 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = p.a.K;
  const T* row = (const T*)p.logits + (int64_t)en.x * p.ld;
  const int first = -(int)((uintptr_t)row % 16 / sizeof(T));  // token of the row's first place
  const int steps = (p.V - first + kLpStep - 1) / kLpStep;
  const float* tops = p.tops + e * p.S * p.steps;
  using H = Held<T>;
  const bool few = steps <= kTopSteps;
  int group = 32;  // lanes whose tokens have a maximum: so many that there are 2 K of these, or one
  while (LANES && group > 1 && steps * 32 / group < 2 * K) group >>= 1;
  const int maxima = steps * (32 / group);
  static_assert(kMaxK * 32 <= kTopSteps, "the lanes' maxima of up to K steps");
  if (tid == 0) sh.n = sh.n_steps = 0;
  float tau = -INFINITY;
  if (LANES) {
    for (int s = warp; s < steps; s += kTopWarps) {
      H x;
      x.load(row, first + s * kLpStep, p.V);
      float m = x.top();
      for (int d = 1; d < group; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      if (!(lane & (group - 1))) sh.tops[(s * 32 + lane) / group] = m;
    }
    if (tid < (-maxima & 3)) sh.tops[maxima + tid] = -INFINITY;
  } else if (few) {
    for (int k = tid; k < (steps + 3) / 4 * 4; k += kTopThreads) sh.tops[k] = k < steps ? tops[k] : -INFINITY;
  }
  if (tid == 0) sh.tau = 0xFFFFFFFFu;
  __syncthreads();
  if (warp == kTopWarps - 1) {
    const Total total = finish_entry<T>(p, e, en);
    if (lane == 0) sh.total = total;
  } else if (few) {
    // the K-th largest is the smallest that fewer than K are larger than
    for (int s = tid; s < maxima; s += kTopThreads - 32) {
      const float x = sh.tops[s];
      int larger = 0;
#pragma unroll 4
      for (int k = 0; k < maxima; k += 4) {
        const float4 o = *(const float4*)(sh.tops + k);
        larger += (o.x > x) + (o.y > x) + (o.z > x) + (o.w > x);
      }
      if (larger < K) atomicMin(&sh.tau, f2ord(x));
    }
  }
  __syncthreads();
  if (sh.total.bad) {
    for (int k = tid; k < K; k += kTopThreads) {
      p.a.top_ids[e * K + k] = -1;
      p.a.top_logp[e * K + k] = -INFINITY;
    }
    return;
  }
  if (few) {
    tau = ord2f(sh.tau);
  } else {
    uint64_t last = ~0ull;
    for (int k = 0; k < K; ++k) {
      uint64_t best = 0;
      for (int s = tid; s < steps; s += kTopThreads) {
        const uint64_t key = make_key(tops[s], (uint32_t)s);
        if (key < last && key > best) best = key;
      }
      last = cta_max(best, sh.best);
    }
    tau = key_value(last);
  }
  // tokens that reach it, of the steps that do
  auto add = [&](int s) {
    H x;
    const int v0 = first + s * kLpStep;
    x.load(row, v0, p.V);
#pragma unroll
    for (int i = 0; i < kLpPer; ++i) {
      const float y = x.get(i);
      if (y >= tau && y > -INFINITY) {
        const int c = atomicAdd(&sh.n, 1);
        if (c < kTopCand) sh.cand[c] = make_key(y, (uint32_t)H::token(v0, i));
      }
    }
  };
  if (few) {
    for (int s = tid; s < steps; s += kTopThreads)
      if (LANES || sh.tops[s] >= tau) sh.list[atomicAdd(&sh.n_steps, 1)] = s;
    __syncthreads();
    for (int k = warp; k < sh.n_steps; k += kTopWarps) add(sh.list[k]);
  } else {
    for (int s = warp; s < steps; s += kTopWarps)
      if (tops[s] >= tau) add(s);
  }
  __syncthreads();
  auto put = [&](int k, uint64_t key) {
    p.a.top_ids[e * K + k] = key ? (int32_t)key_id(key) : -1;
    p.a.top_logp[e * K + k] = key ? (float)((double)key_value(key) - (double)sh.total.M - sh.total.logS) : -INFINITY;
  };
  const int n = sh.n;
  if (n <= kTopCand) {
    // the order in which candidates came does not matter: their ranks among each other are unique
    for (int c = tid; c < n; c += kTopThreads) {
      const uint64_t key = sh.cand[c];
      int before = 0;
      for (int k = 0; k < n; ++k) before += sh.cand[k] > key;
      if (before < K) put(before, key);
    }
    for (int k = n + tid; k < K; k += kTopThreads) put(k, 0);
  } else {
    // many equal logits: the largest key below the last one, K times. A grammar by a finite mask that leaves tokens in fewer than K
    // steps comes here: 512 rows of 128256 bf16 with three tokens left take 680 us for five alternatives and 2.3 ms for
    // twenty, with 400 left 40 and 45, and 74 where the mask is -inf.
    uint64_t last = ~0ull;
    for (int k = 0; k < K; ++k) {
      uint64_t best = 0;
      for (int v = tid; v < p.V; v += kTopThreads) {
        const float y = logit_at<T>(row, v);
        const uint64_t key = y >= tau && y > -INFINITY ? make_key(y, (uint32_t)v) : 0;
        if (key < last && key > best) best = key;
      }
      last = cta_max(best, sh.best);
      if (tid == 0) put(k, last);
    }
  }
}

int64_t steps_of(const dt_handle* h) { return ((int64_t)h->cfg.V + (h->cfg.dtype == DT_BF16 ? 7 : 3) + kLpStep - 1) / kLpStep; }
int64_t warps_of(const dt_handle* h) { return (int64_t)h->num_sms * kLpWarps * kLpCtas; }
// Steps of a piece and pieces of a row: as many pieces as warps are resident, of one to kLpMost steps. (4 steps at most: 139 us
// instead of 131 for 2287 rows of 128256 bf16, 82 instead of 87 for 734 of 128255 fp32, whose last turn is fuller with them.)
void split_of(const dt_handle* h, int64_t entries, int& steps, int64_t& S) {
  const int64_t most = steps_of(h);
  steps = (int)std::max<int64_t>(1, std::min<int64_t>(kLpMost, most * entries / warps_of(h)));
  S = (most + steps - 1) / steps;
}

template <typename T>
cudaError_t launch_t(const LpArgs& p, int num_sms, bool lanes, cudaStream_t s) {
  const dim3 block(kLpThreads);
  cudaError_t e = cudaSuccess;
  if (!p.direct) {
    launch_k(logprob_entries_kernel, dim3((unsigned)((p.entries + kLpThreads - 1) / kLpThreads)), block, 0, s, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(std::min<uint32_t>((p.all + kLpWarps - 1) / kLpWarps, (uint32_t)num_sms * kLpCtas));  // as many as are resident
  if (p.a.rank)
    p.a.K ? launch_k(logprob_pieces_kernel<T, true, true>, grid, block, 0, s, p) : launch_k(logprob_pieces_kernel<T, true, false>, grid, block, 0, s, p);
  else
    p.a.K ? launch_k(logprob_pieces_kernel<T, false, true>, grid, block, 0, s, p) : launch_k(logprob_pieces_kernel<T, false, false>, grid, block, 0, s, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.a.K)
    lanes ? launch_k(logprob_top_kernel<T, true>, dim3((unsigned)p.entries), dim3(kTopThreads), 0, s, p)
          : launch_k(logprob_top_kernel<T, false>, dim3((unsigned)p.entries), dim3(kTopThreads), 0, s, p);
  else
    launch_k(logprob_finish_kernel<T>, dim3((unsigned)((p.entries + kLpWarps - 1) / kLpWarps)), block, 0, s, p);
  return cudaGetLastError();
}

// A workspace serves calls of fewer entries too, which may have more pieces: fewer than two for each of the resident warps and
// one an entry where a piece has fewer than kLpMost steps.
struct LpLayout {
  int64_t sums, tops, total;
};
LpLayout layout_of(const dt_handle* h, int64_t entries, int K) {
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  const int64_t most = steps_of(h);
  const int64_t n = std::max(entries * ((most + kLpMost - 1) / kLpMost), std::min(entries * most, 2 * warps_of(h) + entries));
  LpLayout L;
  L.sums = up(8 * entries);
  L.tops = up(L.sums + 16 * n);
  L.total = L.tops + (K ? 4 * entries * (most + kLpMost - 1) : 0);
  return L;
}

}  // namespace

int64_t logprob_pieces(const dt_handle* h, int64_t entries) {
  int steps;
  int64_t S;
  split_of(h, entries, steps, S);
  return entries * S;
}

int64_t logprob_workspace_bytes(const dt_handle* h, int64_t entries, int K) { return layout_of(h, entries, K).total; }

cudaError_t launch_logprobs(dt_handle* h, const void* logits, int64_t ld, const dt_logprob_args* a, cudaStream_t s) {
  LpArgs p{};
  p.a = *a;
  p.logits = logits;
  p.ld = ld;
  p.V = h->cfg.V;
  p.per = a->path ? a->D_path : a->P;
  p.entries = a->n_out;
  int steps;
  int64_t S;
  split_of(h, p.entries, steps, S);
  p.steps = (uint32_t)steps;
  p.S = (uint32_t)S;
  p.all = (uint32_t)(p.entries * S);
  // one piece a warp, and no search among packed requests: the look-up instead of a launch
  p.direct = steps == 1 && (a->path || !a->row_off);
  const LpLayout L = layout_of(h, p.entries, a->K);
  p.what = (int2*)a->workspace;
  p.sums = (float4*)((char*)a->workspace + L.sums);
  p.tops = (float*)((char*)a->workspace + L.tops);
  p.status = h->ws.status;
  const bool lanes = steps_of(h) <= a->K;
  return h->cfg.dtype == DT_BF16 ? launch_t<uint16_t>(p, h->num_sms, lanes, s) : launch_t<float>(p, h->num_sms, lanes, s);
}

}  // namespace dt
