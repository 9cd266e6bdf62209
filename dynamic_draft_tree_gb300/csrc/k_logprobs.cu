// Log probabilities of given tokens under rows of logits, with the row's entropy, the token's rank and the best alternatives.
//
// With m = max x, S = sum exp(x - m):  log p(t) = x_t - m - log S,  H = log S + (1 / S) sum exp(x - m) (m - x),
// rank = tokens with a larger logit, or an equal one and a lower id.
//
// Every row is read once, in pieces of 8192 tokens that a CTA holds in registers: a maximum a warp, then sums relative to it
// (sums of 32 terms a thread, then trees), and the count in front of the token. The K largest of a piece need no order over
// it: the K-th largest of the maxima of 64 groups of four threads is no larger than the K-th largest token, so that a handful of tokens
// reach it (about 24 for K = 20), which are ranked by counting. Pieces' results (24 to 280 bytes for 16 or 32 KB read) are put together by a
// warp an entry in a second launch, in a fixed order.
// Bound by DRAM in large calls.
#include <algorithm>

#include "dt_internal.cuh"

namespace dt {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpPer = 32;                        // tokens of a thread
constexpr int kLpPiece = kLpThreads * kLpPer;     // tokens of a CTA
constexpr int kLpGroups = kLpThreads / 4;
constexpr int kLpCand = 512;                      // candidates that are ranked by counting; more are taken one by one
static_assert(kLpGroups >= kMaxK, "as many groups as alternatives");

struct LpArgs {
  dt_logprob_args a;
  const void* logits;
  int64_t ld;
  int32_t V, S, per;  // pieces of a row; entries of a request (path, padded)
  int64_t entries;
  float4* sums;       // [entries][S] (m, s, t, count): t = sum e d, d = log2 e
  uint64_t* keys;     // [entries][S][K], descending
  int32_t* status;
};

struct Entry {
  bool used;
  int64_t row;
  int32_t token;  // -1: none
};

// What entry e is. Its request's counts are checked, and its positions; `report`: by whom.
__device__ Entry entry_of(const LpArgs& p, int64_t e, bool report) {
  const dt_logprob_args& a = p.a;
  Entry r{false, 0, -1};
  int b, j;
  const bool packed = !a.path && a.row_off;
  if (packed) {  // the request whose rows hold e: 32 looks at once
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.B;  // row_off[lo] <= e < row_off[hi], if it is anybody's
    if (e < a.row_off[0] || e >= a.row_off[a.B]) return r;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = min(hi, lo + (lane + 1) * step);
      const uint32_t le = __ballot_sync(0xFFFFFFFFu, at < hi && a.row_off[at] <= e);
      const int k = __popc(le);
      hi = min(hi, lo + (k + 1) * step);
      lo += k * step;
    }
    b = lo;
    j = (int)(e - a.row_off[b]);
  } else {
    b = (int)(e / p.per);
    j = (int)(e - (int64_t)b * p.per);
  }
  const int64_t n = (int64_t)a.n_new[b] + a.n_extra;
  const int64_t first = a.row_off ? (int64_t)a.row_off[b] : (int64_t)b * a.P;
  const int64_t room = packed ? (int64_t)a.row_off[b + 1] - first : p.per;
  if (n < 0 || n > room) {
    if (report && j == 0) set_status(p.status, DT_DEV_BAD_TREE);
    return r;
  }
  if (j >= n) return r;
  int64_t pos = j;
  if (a.path) {
    pos = a.path[(int64_t)b * a.D_path + j];
    if (pos < 0 || pos >= a.P) {
      if (report) set_status(p.status, DT_DEV_BAD_TREE);
      return r;
    }
  }
  r.row = first + pos;
  if (r.row < 0 || r.row >= a.rows) {
    if (report) set_status(p.status, DT_DEV_BAD_TREE);
    return r;
  }
  r.used = true;
  if (a.tokens) {
    const int64_t k = (int64_t)j + a.shift;
    int64_t at = -1;
    if (k < n) {
      if (!a.path) at = first + k;
      else {
        const int next = a.path[(int64_t)b * a.D_path + k];
        if (next >= 0 && next < a.P) at = (int64_t)b * a.P + next;
        else if (report) set_status(p.status, DT_DEV_BAD_TREE);
      }
      if (at >= 0 && at < a.n_tokens) r.token = a.tokens[at];
      else if (at >= 0 && report) set_status(p.status, DT_DEV_BAD_TREE);
    } else if (a.last) {
      r.token = a.last[b];
    }
    if (r.token < -1 || r.token >= p.V) {
      if (report) set_status(p.status, DT_DEV_BAD_TOKEN);
      r.token = -1;
    }
  }
  return r;
}

template <typename T>
__device__ __forceinline__ float logit_at(const void* logits, int64_t at) {
  if (sizeof(T) == 4) return ((const float*)logits)[at];
  return __uint_as_float((uint32_t)((const uint16_t*)logits)[at] << 16);
}

// A thread's tokens: kVecs 16-byte vectors, kLpThreads apart.
template <typename T>
struct Held {
  static constexpr int E = 16 / (int)sizeof(T), kVecs = kLpPer / E;
  uint32_t w[kLpPer * sizeof(T) / 4];
  __device__ __forceinline__ float get(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(w[i]);
    return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  }
  // v0: token of the piece's first place (negative in front of a row that does not start on 16 bytes). Vectors that lie in
  // the row are read whole, others token by token; places without a token get -inf.
  __device__ __forceinline__ void load(const T* row, int64_t v0, int V) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int64_t v = v0 + ((int64_t)u * kLpThreads + threadIdx.x) * E;
      uint4 q;
      if (v >= 0 && v + E <= V) {
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
  __device__ __forceinline__ static int64_t token(int64_t v0, int i) {  // of place i
    return v0 + ((int64_t)(i / E) * kLpThreads + threadIdx.x) * E + i % E;
  }
};

struct LpShared {
  float m[kLpThreads / 32], s[kLpThreads / 32], t[kLpThreads / 32];
  int cnt[kLpThreads / 32];
  float group[kLpGroups];
  float tau;
  int n_cand;
  uint64_t cand[kLpCand];
  uint64_t best[kLpThreads / 32];
};

template <typename T, bool RANK, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) logprob_pieces_kernel(const __grid_constant__ LpArgs p) {
  __shared__ LpShared sh;
  using H = Held<T>;
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t e = blockIdx.x / p.S;
  const int piece = (int)(blockIdx.x - e * p.S);
  const Entry en = entry_of(p, e, piece == 0 && tid == 0);
  if (!en.used) return;
  const T* row = (const T*)p.logits + en.row * p.ld;
  const int64_t v0 = (int64_t)piece * kLpPiece - (int64_t)((uintptr_t)row % 16 / sizeof(T));
  H x;
  x.load(row, v0, p.V);
  const float xt = RANK && en.token >= 0 ? logit_at<T>(row, en.token) : INFINITY;
  // maxima: this thread's, its group's, its warp's
  float mt = -INFINITY;
#pragma unroll
  for (int i = 0; i < kLpPer; i += 2) mt = fmaxf(fmaxf(mt, x.get(i)), x.get(i + 1));
  const float mw = ord2f(__reduce_max_sync(0xFFFFFFFFu, f2ord(mt)));
  if (TOP) {
    float mg = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, 1));
    mg = fmaxf(mg, __shfl_xor_sync(0xFFFFFFFFu, mg, 2));
    if ((tid & 3) == 0) sh.group[tid >> 2] = mg;
    if (tid == 0) sh.n_cand = 0;
  }
  // sums relative to the warp's maximum; a weight of zero adds nothing to t, whatever its distance
  const float off = mw == -INFINITY ? 0.0f : -mw * kLog2e;
  const float2 c2 = make_float2(kLog2e, kLog2e), off2 = make_float2(off, off);
  float2 s2 = make_float2(0.0f, 0.0f), t2 = make_float2(0.0f, 0.0f);
  int cnt = 0;
#pragma unroll
  for (int i = 0; i < kLpPer; i += 2) {
    const float2 d = __ffma2_rn(make_float2(x.get(i), x.get(i + 1)), c2, off2);
    const float2 w = make_float2(ex2(d.x), ex2(d.y));
    s2 = __fadd2_rn(s2, w);
    t2 = __ffma2_rn(w, make_float2(fmaxf(d.x, -200.0f), fmaxf(d.y, -200.0f)), t2);
  }
  if (RANK) {
#pragma unroll
    for (int u = 0; u < H::kVecs; ++u) {
      const int64_t v = H::token(v0, u * H::E);
#pragma unroll
      for (int k = 0; k < H::E; ++k) {
        const float y = x.get(u * H::E + k);
        cnt += y > xt || (y == xt && v + k < en.token && v + k >= 0);
      }
    }
  }
  float s = s2.x + s2.y, t = t2.x + t2.y;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
  }
  if (RANK) cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
  if (lane == 0) {
    sh.m[warp] = mw;
    sh.s[warp] = s;
    sh.t[warp] = t;
    sh.cnt[warp] = cnt;
  }
  __syncthreads();
  if (tid == kLpThreads - 32) {  // one thread of a warp without candidates to rank
    float M = -INFINITY, ss = 0.0f, tt = 0.0f;
    int c = 0;
#pragma unroll
    for (int k = 0; k < kLpThreads / 32; ++k) M = fmaxf(M, sh.m[k]);
#pragma unroll
    for (int k = 0; k < kLpThreads / 32; ++k) {
      const float d = sh.m[k] == -INFINITY ? 0.0f : (sh.m[k] - M) * kLog2e, f = ex2(d);
      ss += sh.s[k] * f;
      tt += (sh.t[k] + sh.s[k] * fmaxf(d, -1000.0f)) * f;
      c += sh.cnt[k];
    }
    p.sums[e * p.S + piece] = make_float4(M, ss, tt, __int_as_float(c));
  }
  if constexpr (TOP) {
    const int K = p.a.K;
    // the K-th largest of the groups' maxima
    if (tid < kLpGroups) {
      const float g = sh.group[tid];
      int before = 0;
#pragma unroll 8
      for (int k = 0; k < kLpGroups; ++k) {
        const float o = sh.group[k];
        before += o > g || (o == g && k < tid);
      }
      if (before == K - 1) sh.tau = g;
    }
    __syncthreads();
    const float tau = sh.tau;
    if (mt >= tau && mt > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kLpPer; ++i) {
        const float y = x.get(i);
        if (y >= tau && y > -INFINITY) {
          const int at = atomicAdd(&sh.n_cand, 1);
          if (at < kLpCand) sh.cand[at] = make_key(y, (uint32_t)H::token(v0, i));
        }
      }
    }
    __syncthreads();
    uint64_t* out = p.keys + (e * p.S + piece) * K;
    const int n = sh.n_cand;
    if (n <= kLpCand) {
      // the order in which candidates came does not matter: their ranks among each other are unique
      for (int c = tid; c < n; c += kLpThreads) {
        const uint64_t key = sh.cand[c];
        int before = 0;
        for (int k = 0; k < n; ++k) before += sh.cand[k] > key;
        if (before < K) out[before] = key;
      }
      for (int k = n + tid; k < K; k += kLpThreads) out[k] = 0;
    } else {  // many equal logits: the largest key below the last one, K times
      uint64_t last = ~0ull;
      for (int k = 0; k < K; ++k) {
        uint64_t best = 0;
        for (int i = 0; i < kLpPer; ++i) {
          float y = 0.0f;
#pragma unroll
          for (int q = 0; q < kLpPer; ++q)
            if (q == i) y = x.get(q);
          const uint64_t key = y > -INFINITY ? make_key(y, (uint32_t)H::token(v0, i)) : 0;
          if (key < last && key > best) best = key;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) best = max(best, shfl_xor_u64(best, d));
        if (lane == 0) sh.best[warp] = best;
        __syncthreads();
        for (int q = 0; q < kLpThreads / 32; ++q) best = max(best, sh.best[q]);
        __syncthreads();
        if (tid == 0) out[k] = best;
        last = best;
      }
    }
  }
}

constexpr int kFinishWarps = 4;
// A warp an entry: lanes take its pieces.
template <typename T>
__global__ void __launch_bounds__(32 * kFinishWarps) logprob_finish_kernel(const __grid_constant__ LpArgs p) {
  __shared__ uint64_t top_s[kFinishWarps][kMaxK];
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t e = (int64_t)blockIdx.x * kFinishWarps + warp;
  if (e >= p.entries) return;
  const Entry en = entry_of(p, e, false);
  if (!en.used) return;
  const dt_logprob_args& a = p.a;
  const float4* part = p.sums + e * p.S;
  const float xt = en.token >= 0 ? logit_at<T>(p.logits, en.row * p.ld + en.token) : 0.0f;
  float M = -INFINITY;
  for (int k = lane; k < p.S; k += 32) M = fmaxf(M, part[k].x);
  M = ord2f(__reduce_max_sync(0xFFFFFFFFu, f2ord(M)));
  // sums over pieces in 64 bits: the row's largest token alone is 1 of S, and what the others add may be small beside it
  double S = 0.0, T2 = 0.0;
  int cnt = 0;
  for (int k = lane; k < p.S; k += 32) {
    const float4 q = part[k];
    const float d = q.x == -INFINITY ? 0.0f : (q.x - M) * kLog2e, f = exp2f(d);
    S += (double)(q.y * f);
    T2 += (double)((q.z + q.y * fmaxf(d, -1000.0f)) * f);
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
    const bool none = bad || en.token < 0;
    const float nan = __int_as_float(0x7FC00000);
    if (a.logp) a.logp[e] = none ? nan : (float)((double)xt - (double)M - logS);
    if (a.rank) a.rank[e] = none ? -1 : cnt;
    if (a.entropy) a.entropy[e] = bad ? nan : (float)(logS - 0.6931471805599453 * T2 / S);
  }
  if (a.K == 0) return;
  // 31 pieces' lists and the one of the pieces before them at a time: every lane shows its list's largest key
  uint64_t* top = top_s[warp];
  top[lane] = 0;
  __syncwarp();
  for (int k0 = 0; k0 < p.S; k0 += 31) {
    const bool carry = lane == 31;
    const bool mine = carry ? k0 > 0 : k0 + lane < p.S;
    const uint64_t* list = carry ? top : p.keys + (e * p.S + min(k0 + lane, p.S - 1)) * a.K;
    int at = 0;
    uint64_t key = mine ? list[0] : 0, kept = 0;
    for (int k = 0; k < a.K; ++k) {
      const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key >> 32));
      const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
      const uint64_t best = (uint64_t)hi << 32 | lo;
      if (lane == k) kept = best;
      if (best == 0) break;
      if (key == best) key = ++at < a.K ? list[at] : 0;
    }
    __syncwarp();
    top[lane] = kept;
    __syncwarp();
  }
  if (lane < a.K) {
    const uint64_t key = bad ? 0 : top[lane];
    a.top_ids[e * a.K + lane] = key ? (int32_t)key_id(key) : -1;
    a.top_logp[e * a.K + lane] = key ? (float)((double)key_value(key) - (double)M - logS) : -INFINITY;
  }
}

int pieces_of(int V, int dtype) { return (int)(((int64_t)V + (dtype == DT_BF16 ? 7 : 3) + kLpPiece - 1) / kLpPiece); }

template <typename T>
cudaError_t launch_t(const LpArgs& p, cudaStream_t s) {
  const dim3 grid((unsigned)(p.entries * p.S)), block(kLpThreads);
  if (p.a.rank)
    p.a.K ? launch_k(logprob_pieces_kernel<T, true, true>, grid, block, 0, s, p) : launch_k(logprob_pieces_kernel<T, true, false>, grid, block, 0, s, p);
  else
    p.a.K ? launch_k(logprob_pieces_kernel<T, false, true>, grid, block, 0, s, p) : launch_k(logprob_pieces_kernel<T, false, false>, grid, block, 0, s, p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  launch_k(logprob_finish_kernel<T>, dim3((unsigned)((p.entries + kFinishWarps - 1) / kFinishWarps)), dim3(32 * kFinishWarps), 0, s, p);
  return cudaGetLastError();
}

}  // namespace

int64_t logprob_ctas(const dt_handle* h, int64_t entries) { return entries * pieces_of(h->cfg.V, h->cfg.dtype); }

int64_t logprob_workspace_bytes(const dt_handle* h, int64_t entries, int K) {
  const int64_t n = entries * pieces_of(h->cfg.V, h->cfg.dtype);
  return (16 * n + 255) / 256 * 256 + 8 * n * K;
}

cudaError_t launch_logprobs(dt_handle* h, const void* logits, int64_t ld, const dt_logprob_args* a, cudaStream_t s) {
  LpArgs p{};
  p.a = *a;
  p.logits = logits;
  p.ld = ld;
  p.V = h->cfg.V;
  p.S = pieces_of(h->cfg.V, h->cfg.dtype);
  p.per = a->path ? a->D_path : a->P;
  p.entries = a->n_out;
  p.sums = (float4*)a->workspace;
  p.keys = (uint64_t*)((char*)a->workspace + (16 * p.entries * p.S + 255) / 256 * 256);
  p.status = h->ws.status;
  return h->cfg.dtype == DT_BF16 ? launch_t<uint16_t>(p, s) : launch_t<float>(p, s);
}

}  // namespace dt
