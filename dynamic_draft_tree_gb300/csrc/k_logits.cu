// Target rows prepared for the verify pass: penalties for repeated tokens, biases, grammar masks.
//
// Every row is read and written once. A CTA owns a chunk of the vocabulary for one request and goes
// through a group of that request's rows, so the request's counts and biases of the chunk are read once
// a group into registers. What differs from row to row is the tree path: the path tokens that fall into the chunk (a few
// of D <= 17 over V / 1024 chunks) have a bit a row in shared memory, made before the row loop, so that the loop has one
// multiply-add and two selects an element and only threads with a bit set look further. Rows wait in a ring of
// asynchronous copies that every thread fills and waits for by itself. Bound by DRAM in large calls: 330 rows of 128256
// bf16 with a grammar mask 38 us (4.7 TB/s of what has to move; a plain device copy of the rows takes 55), 766 MB of fp32
// rows of an odd vocabulary 131 us (5.8 TB/s), of a vocabulary of whole 16 bytes 6.1 TB/s. Loads into registers instead of the ring: 48 us (more registers, fewer CTAs); 16 tokens
// a thread instead of 8: 52 us; 8 CTAs an SM instead of 6 (spills): 58 us.
#include <algorithm>

#include "dt_internal.cuh"

namespace dt {
namespace {

constexpr int kLogThreads = 128;
// CTAs an SM holds; a launch of fewer gives each of them fewer rows. 16 rows always against this rule: one request of 17
// positions and 32000 tokens 9.8 and 4.3 us, four of 85 15.8 and 10.6 us, eight of 61 and 128256 34.2 us both.
constexpr int kLogFill = 6;
constexpr int kPer = 8;                          // tokens of a thread
constexpr int kLogChunk = kLogThreads * kPer;    // tokens of a CTA
template <typename T>
constexpr int kWords = kPer * (int)sizeof(T) / 4;  // 32-bit words of a row that a thread holds
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);        // tokens of 16 bytes
template <typename T>
constexpr int kChunks = kPer / kVec<T>;
constexpr int kLogRows = 16;                     // rows of a CTA, at most (bits of a word)

// How a row's tokens are divided among the threads.
// kAligned: every row starts on a 16-byte boundary; a thread's tokens are 16 bytes in every 16 kLogThreads (a warp's
//   accesses are whole lines; fp32 tokens of a thread as one run of 32 bytes, half lines an access: 16 x up to 65 rows of
//   128256 149 us, so 110 us).
// kShifted: the first row starts on a 16-byte boundary, and every `step`-th one equally far from one, in the logits and in
//   the output. A CTA takes such rows, and its chunk begins that far in front of the vocabulary's, so that accesses are those
//   of aligned rows (the end of the row before is read with a row's first tokens, never used or written).
// kSingle: one token in every kLogThreads (single elements; bf16 ones are too small for an asynchronous copy and are loaded
//   one row ahead of their use): rows of other alignments, and few rows, whose tables weigh more the fewer rows a CTA has of
//   its kind: kShiftRows. Single and shifted, 16 requests: fp32, every fourth row alike, 128255
//   tokens: 16 positions 40 and 47 us, 32 66.5 and 68, 48 105 and 96, 65 146 and 131; bf16, every second row alike, 128252
//   tokens: 8 positions 21 and 24 us, 24 44 and 40, 65 98 and 80; every eighth, 128255 tokens, 65 positions: 108 and 111 us.
enum { kSingle, kAligned, kShifted };
constexpr int kShiftRows = 10;

struct LogitsArgs {
  dt_logits_params p;
  const void* logits;
  int64_t ld;
  void* out;
  int64_t ld_out;
  int32_t V;
  int32_t rows;   // rows of a CTA
  int32_t step;   // kShifted: from one of its rows to the next, else 1
  bool counts16;  // every counts row starts on a 16-byte boundary
  int32_t* status;
};

template <typename T>
__device__ __forceinline__ float element(const uint32_t* w, int u) {
  if (sizeof(T) == 4) return __uint_as_float(w[u]);
  return u & 1 ? bf16_hi(w[u >> 1]) : bf16_lo(w[u >> 1]);
}
template <typename T>
__device__ __forceinline__ void pack_words(const float* y, uint32_t* w) {
#pragma unroll
  for (int k = 0; k < kWords<T>; ++k) {
    if constexpr (sizeof(T) == 4)
      w[k] = __float_as_uint(y[k]);
    else
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(y[2 * k + 1]), "f"(y[2 * k]));
  }
}

struct Penalty {
  float rep, inv, freq, pres;
};
// y = x * factor + add: a token that has not been seen has factor 1 and add = bias; a seen one 1 / repetition or, where
// x is not positive, repetition, and add = bias - frequency c - presence.
__device__ __forceinline__ float factor_of(const Penalty& p, bool seen, float x) {
  const float f = x > 0.0f ? p.inv : p.rep;
  return seen ? f : 1.0f;
}
__device__ __forceinline__ float add_of(const Penalty& p, int c, float bias) {
  return bias - (c > 0 ? fmaf(p.freq, (float)c, p.pres) : 0.0f);
}

// 128 bytes a thread on their way.
template <typename T>
constexpr int kRingRows = sizeof(T) == 2 ? 8 : 4;
template <typename T, int MODE>
constexpr int kSaid = (MODE == kShifted ? 2 : 1) * kChunks<T>;  // allow words that a thread has of a row
template <typename T, int MODE>
constexpr int kRingBytes = kRingRows<T> * (kWords<T> + kSaid<T, MODE>) * kLogThreads * 4;

__device__ __forceinline__ void copy16(uint32_t* dst, const void* src, int bytes) {  // the rest of the 16 becomes zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups are there
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kLogThreads, 6) logits_kernel(LogitsArgs a) {
  // A row's elements wait in shared memory, kDepth rows ahead, every thread's in places of its own (asynchronous copies
  // that only the thread itself waits for), and the allow words that hold (VEC) or lend its warp their bits.
  constexpr bool VEC = MODE != kSingle, SHIFT = MODE == kShifted;
  constexpr int W = kWords<T>, kDepth = kRingRows<T>, E = kVec<T>, C = kChunks<T>, A = kSaid<T, MODE>;
  extern __shared__ __align__(16) uint32_t dyn[];
  const int P = a.p.P;
  uint32_t* ring = dyn;                                          // [kDepth][W][kLogThreads]
  uint32_t* said = ring + kDepth * W * kLogThreads;              // [kDepth][A][kLogThreads]
  int32_t* path_tok = (int32_t*)(said + kDepth * A * kLogThreads);  // [P] chunk offset of a position's token, its position
  int32_t* path_pos = path_tok + P;                              // [P]
  uint32_t* on_rows = (uint32_t*)(path_pos + P);                 // [P] bit r: on row r's path
  __shared__ int n_path, twice;
  __shared__ uint32_t hit[kLogRows][kLogChunk / 32];  // bit = the token is on the row's path
  __shared__ float bias_s[kLogChunk];
  __shared__ uint32_t biased[kLogChunk / 32];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  const int step = SHIFT ? a.step : 1;
  const int row0 = SHIFT ? (int)(blockIdx.z % step + blockIdx.z / step * a.rows * step) : (int)blockIdx.z * a.rows;
  // everything that depends on the request alone is asked for at once
  const bool with_bias = a.p.bias_ids != nullptr && a.p.n_bias > 0;
  const int32_t* ids = a.p.bias_ids + (int64_t)b * a.p.n_bias;
  const float* vals = a.p.bias_vals + (int64_t)b * a.p.n_bias;
  const int n = min(max(a.p.n_pos[b], 0), P);
  const int64_t base = a.p.row_off ? (int64_t)a.p.row_off[b] : (int64_t)b * P;
  constexpr int kTok = kMaxP / kLogThreads;
  int path[kTok];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    const int j = tid + k * kLogThreads;
    path[k] = a.p.tokens && j < P ? a.p.tokens[(int64_t)b * P + j] : -1;
  }
  const int id0 = with_bias && tid < a.p.n_bias ? ids[tid] : -1;
  const float val0 = with_bias && tid < a.p.n_bias ? vals[tid] : 0.0f;
  Penalty pen;
  pen.rep = a.p.repetition ? a.p.repetition[b] : 1.0f;
  pen.freq = a.p.frequency ? a.p.frequency[b] : 0.0f;
  pen.pres = a.p.presence ? a.p.presence[b] : 0.0f;
  if (row0 >= n) return;
  const int rows = min(a.rows, (n - row0 + step - 1) / step);
  if (base < 0 || base + n > a.p.rows) {
    if (tid == 0) set_status(a.status, DT_DEV_BAD_PAGE);
    return;
  }
  int v0 = blockIdx.x * kLogChunk;  // token of the chunk's first place
  if (SHIFT) v0 -= (int)((uint64_t)(base + row0) * a.ld % E);
  auto place = [&](int u) { return VEC ? u / E * E * kLogThreads + tid * E + u % E : tid + u * kLogThreads; };  // in the chunk
  constexpr bool kHalves = !VEC && W < kPer;  // strided bf16
  const T* src = (const T*)a.logits + (base + row0) * a.ld + v0 + (VEC ? tid * E : tid);  // the next row to fetch
  T* dst = (T*)a.out + (base + row0) * a.ld_out + v0 + (VEC ? tid * E : tid);
  constexpr int kWordStep = E * kLogThreads / 32;  // VEC: words from one 16 bytes' bits to the next
  const int word_at = VEC ? tid * E >> 5 : lane * (kLogThreads / 32) + warp;
  const int word_shift = tid * E & 31;  // VEC: this thread's first bit
  const bool word_in = a.p.allow && (VEC ? v0 + tid * E < a.V : lane < kPer && v0 + word_at * 32 < a.V);
  const int allow_shift = SHIFT ? (v0 + tid * E) & 31 : word_shift;  // where its bits begin in the allow word
  const uint32_t* allow_at = a.p.allow + (base + row0) * a.p.allow_ld + (SHIFT ? (v0 + tid * E) >> 5 : (v0 >> 5) + word_at);
  const int left = (a.V - v0 - tid * E) * (int)sizeof(T);  // VEC: bytes of the row from this thread's first token
  constexpr int kStep = 16 * kLogThreads;                  // VEC: bytes from one 16 to the next
  uint32_t* mine = ring + tid * (VEC ? 4 : 1);
  auto fetch = [&](int r) {
    if (r < rows) {
      uint32_t* to = mine + (r % kDepth) * W * kLogThreads;
      if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < W / 4; ++c)
          if (left > kStep * c) copy16(to + c * kLogThreads * 4, (const char*)src + kStep * c, min(16, left - kStep * c));
      } else if constexpr (!kHalves) {
#pragma unroll
        for (int u = 0; u < kPer; ++u)
          if (v0 + place(u) < a.V) copy4(to + u * kLogThreads, src + u * kLogThreads);
      }
      uint32_t* word = said + (r % kDepth) * A * kLogThreads + tid;
      if constexpr (SHIFT) {  // the bits of 16 bytes may lie in two words
        if (a.p.allow) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int v = v0 + c * E * kLogThreads + tid * E;
            if (v >= 0 && v < a.V) copy4(word + 2 * c * kLogThreads, allow_at + c * kWordStep);
            if (allow_shift > 32 - E && (v | 31) + 1 < a.V) copy4(word + (2 * c + 1) * kLogThreads, allow_at + c * kWordStep + 1);
          }
        }
      } else {
        if (word_in) copy4(word, allow_at);
        if constexpr (VEC && C > 1)
          if (a.p.allow && left > kStep) copy4(word + kLogThreads, allow_at + kWordStep);
      }
      if constexpr (!kHalves) src += step * a.ld;
      allow_at += step * a.p.allow_ld;
    }
    copies_close();
  };
  uint16_t half[kPer];  // strided bf16: the next row's
  auto load_halves = [&]() {
    if constexpr (kHalves) {
#pragma unroll
      for (int u = 0; u < kPer; ++u)
        if (v0 + place(u) < a.V) half[u] = src[u * kLogThreads];
      src += a.ld;  // (step 1)
    }
  };
  // the first rows and the counts are on their way while the tables are made
#pragma unroll 1
  for (int k = 0; k < kDepth; ++k) fetch(k);
  load_halves();
  const int32_t* counts = a.p.counts ? a.p.counts + (int64_t)b * a.V + v0 : nullptr;
  int cnt[kPer];
#pragma unroll
  for (int u = 0; u < kPer; u += 4) {
    if (counts && VEC && !SHIFT && a.counts16 && v0 + place(u) < a.V) {  // (V is a multiple of 4)
      const int4 q = *(const int4*)(counts + place(u));
      cnt[u] = q.x, cnt[u + 1] = q.y, cnt[u + 2] = q.z, cnt[u + 3] = q.w;
    } else {
#pragma unroll
      for (int k = u; k < u + 4; ++k) cnt[k] = counts && v0 + place(k) < a.V && (!SHIFT || v0 + place(k) >= 0) ? counts[place(k)] : 0;
    }
  }
  if (tid == 0) n_path = twice = 0;
  for (int i = tid; i < kLogRows * (kLogChunk / 32); i += kLogThreads) (&hit[0][0])[i] = 0;
  if (with_bias) {
    for (int i = tid; i < kLogChunk; i += kLogThreads) bias_s[i] = 0.0f;
    if (tid < kLogChunk / 32) biased[tid] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    const int j = tid + k * kLogThreads, at = path[k];
    if (j < n && at != -1) {
      if (at < 0 || at >= a.V) {
        if (blockIdx.x == 0) set_status(a.status, DT_DEV_BAD_TOKEN);
      } else if (at >= v0 && at - v0 < kLogChunk) {
        const int q = atomicAdd(&n_path, 1);
        path_tok[q] = at - v0;
        path_pos[q] = j;
        on_rows[q] = 0;
      }
    }
  }
  if (with_bias) {
    for (int k = tid; k < a.p.n_bias; k += kLogThreads) {
      const int id = k == tid ? id0 : ids[k];
      const float val = k == tid ? val0 : vals[k];
      if (id < -1 || id >= a.V) {
        if (blockIdx.x == 0) set_status(a.status, DT_DEV_BAD_TOKEN);
      } else if (id >= max(v0, 0) && id - v0 < kLogChunk) {
        const int off = id - v0;
        if (atomicOr(&biased[off >> 5], 1u << (off & 31)) >> (off & 31) & 1)
          twice = 1;
        else
          bias_s[off] = val;
      }
    }
  }
  __syncthreads();
  if (with_bias && twice) {
    // ids that come twice add up in list order: once more, by one warp that goes through the list
    for (int i = tid; i < kLogChunk; i += kLogThreads) bias_s[i] = 0.0f;
    __syncthreads();
    if (warp == 0) {
      for (int k0 = 0; k0 < a.p.n_bias; k0 += 32) {
        const int k = k0 + lane, id = k < a.p.n_bias ? ids[k] : -1;
        const bool inside = id >= max(v0, 0) && id - v0 < kLogChunk && id < a.V;
        const float val = inside ? vals[k] : 0.0f;
        for (uint32_t m = __ballot_sync(0xFFFFFFFFu, inside); m; m &= m - 1) {
          if (lane == __ffs(m) - 1) bias_s[id - v0] += val;
          __syncwarp();
        }
      }
    }
    __syncthreads();
  }
  const int np = n_path;
  auto on_path_of = [&](int r, int k) {  // is path entry k on row r's path
    const int i = row0 + r * step, j = path_pos[k];
    return a.p.mask ? a.p.mask[((int64_t)b * P + i) * P + j] != 0 : j <= i;
  };
  // bits of the rows' path tokens: the first mask byte of a thread travels while the additions are made up
  auto mark = [&](int r, int k) {
    atomicOr(&hit[r][path_tok[k] >> 5], 1u << (path_tok[k] & 31));
    atomicOr(&on_rows[k], 1u << r);
  };
  const int r1 = np > 0 ? tid / np : 0, k1 = tid - r1 * np;
  const bool on1 = tid < np * rows && on_path_of(r1, k1);
  pen.inv = 1.0f / pen.rep;
  float add[kPer];
  uint32_t seen = 0, made = 0;  // bits: in the history at all; generated before
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    add[u] = with_bias ? bias_s[place(u)] : 0.0f;
    if (cnt[u]) add[u] = add_of(pen, cnt[u] & (DT_SEEN_PROMPT - 1), add[u]);
    seen |= (cnt[u] != 0 ? 1u : 0u) << u;
    made |= (cnt[u] & (DT_SEEN_PROMPT - 1) ? 1u : 0u) << u;
  }
  if (on1) mark(r1, k1);
  for (int x = tid + kLogThreads; x < np * rows; x += kLogThreads) {
    const int r = x / np, k = x - r * np;
    if (on_path_of(r, k)) mark(r, k);
  }
  __syncthreads();
  for (int r = 0; r < rows; ++r) {
    copies_wait<kDepth - 1>();
    uint32_t in[W];
    const uint32_t* from = mine + (r % kDepth) * W * kLogThreads;
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < W / 4; ++c) {
        const uint4 q = *(const uint4*)(from + c * kLogThreads * 4);
        in[4 * c] = q.x;
        in[4 * c + 1] = q.y;
        in[4 * c + 2] = q.z;
        in[4 * c + 3] = q.w;
      }
    } else if constexpr (!kHalves) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) in[u] = from[u * kLogThreads];
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) in[k] = (uint32_t)half[2 * k] | (uint32_t)half[2 * k + 1] << 16;
      if (r + 1 < rows) load_halves();
    }
    // bit u: the thread's token u may be said
    uint32_t allow = 0xFFFFFFFFu;
    if (a.p.allow) {
      const uint32_t* words = said + (r % kDepth) * A * kLogThreads + tid;
      const uint32_t word = words[0];
      if constexpr (SHIFT) {
        allow = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
          allow |= (__funnelshift_r(words[2 * c * kLogThreads], words[(2 * c + 1) * kLogThreads], allow_shift) & ((1u << E) - 1)) << c * E;
      } else if constexpr (VEC) {
        allow = word >> word_shift;
        if constexpr (C > 1) allow = (allow & ((1u << E) - 1)) | words[kLogThreads] >> word_shift << E;
      } else {  // the warp's tokens of u are the 32 of one word
        allow = 0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) allow |= (__shfl_sync(0xFFFFFFFFu, word, u) >> lane & 1u) << u;
      }
    }
    float y[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const float x = element<T>(in, u);
      y[u] = fmaf(x, factor_of(pen, seen & 1u << u, x), add[u]);
    }
    if (np > 0) {  // tokens on the row's path count beside the history
      uint32_t on_path = 0;
      if (VEC) {
#pragma unroll
        for (int c = 0; c < C; ++c) on_path |= (hit[r][word_at + c * kWordStep] >> word_shift & ((1u << E) - 1)) << c * E;
      } else {
#pragma unroll
        for (int u = 0; u < kPer; ++u) on_path |= (hit[r][u * (kLogThreads / 32) + warp] >> lane & 1u) << u;
      }
      for (; on_path; on_path &= on_path - 1) {
        const int u = __ffs(on_path) - 1, off = place(u);
        int c = 0;  // occurrences on the path
        for (int q = 0; q < np; ++q) c += path_tok[q] == off && on_rows[q] >> r & 1;
        const float more = fmaf(pen.freq, (float)c, made & 1u << u ? 0.0f : pen.pres);
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          if (q == u) {
            const float x = element<T>(in, q);
            y[q] = fmaf(x, factor_of(pen, true, x), add[q] - more);
          }
        }
      }
    }
    if (a.p.allow) {
#pragma unroll
      for (int u = 0; u < kPer; ++u)
        if (!(allow & 1u << u)) y[u] = -INFINITY;
    }
    uint32_t res[W];
    pack_words<T>(y, res);
    if (VEC && left >= kStep * (C - 1) + 16 && (!SHIFT || v0 + tid * E >= 0)) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        *(uint4*)((char*)dst + kStep * c) = make_uint4(res[4 * c], res[4 * c + 1], res[4 * c + 2], res[4 * c + 3]);
    } else {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        if (v0 + place(u) < a.V && (!SHIFT || v0 + place(u) >= 0)) {
          T* to = dst + (VEC ? u / E * E * kLogThreads + u % E : u * kLogThreads);
          if constexpr (sizeof(T) == 4)
            *(uint32_t*)to = res[u];
          else
            *(uint16_t*)to = (uint16_t)(res[u >> 1] >> (16 * (u & 1)));
        }
      }
    }
    dst += step * a.ld_out;
    fetch(r + kDepth);
  }
  copies_wait<0>();
}

struct CountArgs {
  int32_t* counts;
  const int32_t* tokens;
  int64_t n_tokens;
  int32_t P;
  const int32_t* row_off;
  const int32_t* path;
  int32_t D_path;
  const int32_t* n_new;
  int32_t n_extra, prompt, V;
  int32_t* status;
};

// CTA (c, b): every gridDim.x-th group of kLogThreads tokens of request b. Integer atomics: order does not matter.
__global__ void __launch_bounds__(kLogThreads) count_kernel(CountArgs a) {
  pdl_begin();
  const int b = blockIdx.y;
  const int64_t n = (int64_t)a.n_new[b] + a.n_extra;
  const int64_t base = a.row_off ? (int64_t)a.row_off[b] : (int64_t)b * a.P;
  const int64_t rows = a.row_off ? (int64_t)a.row_off[b + 1] - base : a.P;  // the request's
  if (n < 0 || n > (a.path ? (int64_t)a.D_path : rows)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(a.status, DT_DEV_BAD_TREE);
    return;
  }
  for (int64_t j = (int64_t)blockIdx.x * kLogThreads + threadIdx.x; j < n; j += (int64_t)gridDim.x * kLogThreads) {
    const int pos = a.path ? a.path[(int64_t)b * a.D_path + j] : (int)j;
    if (pos < 0 || pos >= rows || (a.path && pos >= a.P) || base < 0 || base + pos >= a.n_tokens) {
      set_status(a.status, DT_DEV_BAD_TREE);
      continue;
    }
    const int t = a.tokens[base + pos];
    if (t < 0 || t >= a.V) {
      set_status(a.status, DT_DEV_BAD_TOKEN);
      continue;
    }
    int32_t* c = a.counts + (int64_t)b * a.V + t;
    if (a.prompt)
      atomicOr(c, DT_SEEN_PROMPT);
    else
      atomicAdd(c, 1);
  }
}

template <typename T, int MODE>
cudaError_t launch_logits_m(dt_handle* h, int B, LogitsArgs a, cudaStream_t s) {
  const int chunks = (a.V + (MODE == kShifted ? kVec<T> - 1 : 0) + kLogChunk - 1) / kLogChunk;
  // a CTA's tables pay over many rows, but few CTAs leave SMs idle
  const int classes = std::min(a.step, a.p.P), most = (a.p.P + a.step - 1) / a.step;
  auto groups = [&]() { return (most + a.rows - 1) / a.rows; };
  a.rows = kLogRows;
  while (a.rows > 1 && (int64_t)chunks * B * classes * groups() < h->num_sms * kLogFill) a.rows /= 2;
  const size_t smem = kRingBytes<T, MODE> + (size_t)a.p.P * 12;
  launch_k(logits_kernel<T, MODE>, dim3(chunks, B, (groups() - 1) * a.step + classes), dim3(kLogThreads), smem, s, a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_logits_t(dt_handle* h, int B, LogitsArgs a, cudaStream_t s) {
  constexpr int E = kVec<T>;
  const uintptr_t in = (uintptr_t)a.logits, out = (uintptr_t)a.out;
  a.step = 1;
  if (a.ld % E == 0 && a.ld_out % E == 0 && (in | out) % 16 == 0) return launch_logits_m<T, kAligned>(h, B, a, s);
  int step = 1;
  while (step * a.ld % E != 0) step *= 2;
  if ((in | out) % 16 != 0 || (a.ld - a.ld_out) % E != 0 || a.p.P < kShiftRows * step) return launch_logits_m<T, kSingle>(h, B, a, s);
  a.step = step;
  return launch_logits_m<T, kShifted>(h, B, a, s);
}

}  // namespace

cudaError_t launch_logits(dt_handle* h, int B, const void* logits, int64_t ld, void* out, int64_t ld_out,
                          const dt_logits_params* p, cudaStream_t s) {
  LogitsArgs a{*p, logits, ld, out, ld_out, h->cfg.V, 0, 1, h->cfg.V % 4 == 0 && (uintptr_t)p->counts % 16 == 0, h->ws.status};
  return h->cfg.dtype == DT_BF16 ? launch_logits_t<uint16_t>(h, B, a, s) : launch_logits_t<float>(h, B, a, s);
}

cudaError_t launch_count_tokens(dt_handle* h, int B, int32_t* counts, const int32_t* tokens, int64_t n_tokens, int P,
                                const int32_t* row_off, const int32_t* path, int D_path, const int32_t* n_new,
                                int n_extra, int prompt, cudaStream_t s) {
  CountArgs a{counts, tokens, n_tokens, P, row_off, path, D_path, n_new, n_extra, prompt, h->cfg.V, h->ws.status};
  const int64_t most = path ? D_path : P;
  const int chunks = (int)min((int64_t)64, max((int64_t)1, (most + kLogThreads - 1) / kLogThreads));
  launch_k(count_kernel, dim3(chunks, B), dim3(kLogThreads), 0, s, a);
  return cudaGetLastError();
}

}  // namespace dt
