// Target rows prepared for the verify pass: penalties for repeated tokens, biases, grammar masks.
//
// Every row is read and written once. A CTA owns a chunk of the vocabulary for one request and goes
// through a group of that request's rows, so the request's counts and biases of the chunk are read once
// a group into registers. What differs from row to row is the tree path: the path tokens that fall into
// the chunk (a few of D <= 17 over V / 2048 chunks) are listed a row in shared memory before the row loop, with a
// bit a token, so that the loop has one multiply-add and two selects an element and only threads with a bit set look
// at the list. Bound by DRAM: 64 bytes a thread are in flight, the next row's load behind every row's store.
#include <cuda_bf16.h>

#include "dt_internal.cuh"

namespace dt {
namespace {

constexpr int kLogThreads = 256;
constexpr int kLogPer = 8;                       // tokens of a thread
constexpr int kLogChunk = kLogThreads * kLogPer;  // tokens of a CTA
constexpr int kLogRows = 16;                     // rows of a CTA

struct LogitsArgs {
  dt_logits_params p;
  const void* logits;
  int64_t ld;
  void* out;
  int64_t ld_out;
  int32_t V;
  int32_t* status;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float y, float& o) { o = y; }
__device__ __forceinline__ void from_f(float y, __nv_bfloat16& o) { o = __float2bfloat16_rn(y); }

// What the row loop needs of a token: y = x * (x > 0 ? pos : neg) - sub. A token that has not been seen has
// pos = neg = 1 and sub = -bias; a seen one 1 / repetition, repetition and frequency c + presence - bias.
struct Token {
  float pos, neg, sub;
};
struct Penalty {
  float rep, inv, freq, pres;
};
__device__ __forceinline__ Token token_of(const Penalty& p, int c, bool prompt, float bias) {
  const bool seen = c > 0 || prompt;
  Token t;
  t.pos = seen ? p.inv : 1.0f;
  t.neg = seen ? p.rep : 1.0f;
  t.sub = (c > 0 ? fmaf(p.freq, (float)c, p.pres) : 0.0f) - bias;
  return t;
}

// VEC: every row starts on a 16-byte boundary; a thread's tokens are then kLogPer neighbours (one or two
// 16-byte accesses), else one token in every kLogThreads (coalesced single elements).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kLogThreads, 3) logits_kernel(LogitsArgs a) {
  extern __shared__ char dyn[];
  const int P = a.p.P;
  int32_t* path_tok = (int32_t*)dyn;               // [P] chunk offset of a position's token, its position
  int32_t* path_pos = path_tok + P;                // [P]
  uint16_t* row_list = (uint16_t*)(path_pos + P);  // [kLogRows][P] chunk offsets of the row's path tokens
  __shared__ int n_path, n_row[kLogRows];
  __shared__ uint32_t hit[kLogRows][kLogChunk / 32];  // bit = the token is on the row's path
  __shared__ float bias_s[kLogChunk];
  pdl_begin();
  const int tid = threadIdx.x, b = blockIdx.y;
  const int v0 = blockIdx.x * kLogChunk;
  const int row0 = blockIdx.z * kLogRows;
  const int n = min(max(a.p.n_pos[b], 0), P);
  if (row0 >= n) return;
  const int rows = min(kLogRows, n - row0);
  int64_t base = a.p.row_off ? (int64_t)a.p.row_off[b] : (int64_t)b * P;
  if (base < 0 || base + n > a.p.rows) {
    if (tid == 0) set_status(a.status, DT_DEV_BAD_PAGE);
    return;
  }
  auto place = [&](int u) { return VEC ? tid * kLogPer + u : tid + u * kLogThreads; };  // in the chunk
  // the first rows are on their way while the tables are made
  constexpr int kTurn = VEC && sizeof(T) == 4 ? 2 : 4;  // rows in flight: 64 bytes a thread
  const bool full = VEC && v0 + (tid + 1) * kLogPer <= a.V;
  T in[kTurn][kLogPer];
  auto load = [&](int r, T* x) {
    const T* src = (const T*)a.logits + (base + row0 + r) * a.ld;
    if (full) {
      constexpr int kVec = (int)sizeof(T) * kLogPer / 16;
      uint4 q[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) q[k] = __ldcs((const uint4*)(src + v0 + tid * kLogPer) + k);
      memcpy(x, q, sizeof(q));
    } else {
#pragma unroll
      for (int u = 0; u < kLogPer; ++u)
        if (v0 + place(u) < a.V) x[u] = src[v0 + place(u)];
    }
  };
#pragma unroll
  for (int k = 0; k < kTurn; ++k)
    if (k < rows) load(k, in[k]);
  if (tid == 0) n_path = 0;
  if (tid < kLogRows) n_row[tid] = 0;
  for (int i = tid; i < kLogRows * (kLogChunk / 32); i += kLogThreads) (&hit[0][0])[i] = 0;
  const bool with_bias = a.p.bias_ids != nullptr && a.p.n_bias > 0;
  if (with_bias)
    for (int i = tid; i < kLogChunk; i += kLogThreads) bias_s[i] = 0.0f;
  __syncthreads();
  if (a.p.tokens) {
    for (int j = tid; j < n; j += kLogThreads) {
      const int t = a.p.tokens[(int64_t)b * P + j];
      if (t < -1 || t >= a.V) {
        if (blockIdx.x == 0) set_status(a.status, DT_DEV_BAD_TOKEN);
      } else if (t >= v0 && t - v0 < kLogChunk) {
        const int k = atomicAdd(&n_path, 1);
        path_tok[k] = t - v0;
        path_pos[k] = j;
      }
    }
  }
  if (with_bias && tid < 32) {
    // warp 0 goes through the list in order; equal ids add up in list order
    for (int k0 = 0; k0 < a.p.n_bias; k0 += 32) {
      const int k = k0 + tid;
      int id = k < a.p.n_bias ? a.p.bias_ids[(int64_t)b * a.p.n_bias + k] : -1;
      if (id < -1 || id >= a.V) {
        if (blockIdx.x == 0) set_status(a.status, DT_DEV_BAD_TOKEN);
        id = -1;
      }
      const bool inside = id >= v0 && id - v0 < kLogChunk;
      const float val = inside ? a.p.bias_vals[(int64_t)b * a.p.n_bias + k] : 0.0f;
      for (uint32_t m = __ballot_sync(0xFFFFFFFFu, inside); m; m &= m - 1) {
        if (tid == __ffs(m) - 1) bias_s[id - v0] += val;
        __syncwarp();
      }
    }
  }
  __syncthreads();
  const int np = n_path;
  for (int x = tid; x < np * rows; x += kLogThreads) {
    const int r = x / np, k = x - r * np, i = row0 + r, j = path_pos[k];
    const bool on = a.p.mask ? a.p.mask[((int64_t)b * P + i) * P + j] != 0 : j <= i;
    if (on) {
      const int off = path_tok[k];
      row_list[r * P + atomicAdd(&n_row[r], 1)] = (uint16_t)off;
      atomicOr(&hit[r][off >> 5], 1u << (off & 31));
    }
  }
  Penalty pen;
  pen.rep = a.p.repetition ? a.p.repetition[b] : 1.0f;
  pen.inv = 1.0f / pen.rep;
  pen.freq = a.p.frequency ? a.p.frequency[b] : 0.0f;
  pen.pres = a.p.presence ? a.p.presence[b] : 0.0f;
  Token tok[kLogPer];
  const int32_t* counts = a.p.counts ? a.p.counts + (int64_t)b * a.V + v0 : nullptr;
#pragma unroll
  for (int u = 0; u < kLogPer; ++u) {
    const int c = counts && v0 + place(u) < a.V ? counts[place(u)] : 0;
    tok[u] = token_of(pen, c & (DT_SEEN_PROMPT - 1), c & DT_SEEN_PROMPT, with_bias ? bias_s[place(u)] : 0.0f);
  }
  __syncthreads();
  const int lane = tid & 31, warp = tid >> 5;
  for (int r0 = 0; r0 < rows; r0 += kTurn) {
#pragma unroll
    for (int k = 0; k < kTurn; ++k) {
      const int r = r0 + k;
      if (r >= rows) break;
      const int64_t row = base + row0 + r;
      // bit u: the thread's token u may be said
      uint32_t allow = 0xFFu;
      if (a.p.allow) {
        const uint32_t* w = a.p.allow + row * a.p.allow_ld + (v0 >> 5);
        if (VEC) {
          allow = v0 + tid * kLogPer < a.V ? w[tid >> 2] >> (8 * (tid & 3)) : 0u;
        } else {
          // the warp's tokens of u are the 32 of one word
          const uint32_t word = lane < kLogPer && v0 + lane * kLogThreads + warp * 32 < a.V ? w[lane * (kLogThreads / 32) + warp] : 0u;
          allow = 0;
#pragma unroll
          for (int u = 0; u < kLogPer; ++u) allow |= (__shfl_sync(0xFFFFFFFFu, word, u) >> lane & 1u) << u;
        }
      }
      // tokens on the row's path, past the history
      uint32_t on_path = 0;
      if (np > 0) {
        if (VEC) {
          on_path = hit[r][tid >> 2] >> (8 * (tid & 3)) & 0xFFu;
        } else {
#pragma unroll
          for (int u = 0; u < kLogPer; ++u) on_path |= (hit[r][u * (kLogThreads / 32) + warp] >> lane & 1u) << u;
        }
      }
      T res[kLogPer];
#pragma unroll
      for (int u = 0; u < kLogPer; ++u) {
        const float x = to_f(in[k][u]);
        float y = fmaf(x, x > 0.0f ? tok[u].pos : tok[u].neg, -tok[u].sub);
        if (!(allow >> u & 1)) y = -INFINITY;
        from_f(y, res[u]);
      }
      if (on_path) {
        const int nr = n_row[r];
        for (uint32_t m = on_path; m; m &= m - 1) {
          const int u = __ffs(m) - 1, off = place(u);
          int c = counts ? counts[off] : 0;
          const bool prompt = c & DT_SEEN_PROMPT;
          c &= DT_SEEN_PROMPT - 1;
          for (int q = 0; q < nr; ++q) c += row_list[r * P + q] == off;
          const Token t = token_of(pen, c, prompt, with_bias ? bias_s[off] : 0.0f);
          T o;
          float x = 0.0f;
#pragma unroll
          for (int q = 0; q < kLogPer; ++q)
            if (q == u) x = to_f(in[k][q]);
          from_f(allow >> u & 1 ? fmaf(x, x > 0.0f ? t.pos : t.neg, -t.sub) : -INFINITY, o);
#pragma unroll
          for (int q = 0; q < kLogPer; ++q)
            if (q == u) res[q] = o;
        }
      }
      T* dst = (T*)a.out + row * a.ld_out + v0;
      if (full) {
        constexpr int kVec = (int)sizeof(T) * kLogPer / 16;
        uint4 q[kVec];
        memcpy(q, res, sizeof(q));
#pragma unroll
        for (int c = 0; c < kVec; ++c) ((uint4*)(dst + tid * kLogPer))[c] = q[c];
      } else {
#pragma unroll
        for (int u = 0; u < kLogPer; ++u)
          if (v0 + place(u) < a.V) dst[place(u)] = res[u];
      }
      if (r + kTurn < rows) load(r + kTurn, in[k]);
    }
  }
}

struct CountArgs {
  int32_t* counts;
  const int32_t* tokens;
  int32_t P;
  const int32_t* row_off;
  const int32_t* path;
  int32_t D_path;
  const int32_t* n_new;
  int32_t n_extra, prompt, V;
  int32_t* status;
};

// CTA (c, b): every gridDim.x-th group of 256 tokens of request b. Integer atomics: order does not matter.
__global__ void __launch_bounds__(kLogThreads) count_kernel(CountArgs a) {
  pdl_begin();
  const int b = blockIdx.y;
  const int64_t n = (int64_t)a.n_new[b] + a.n_extra;
  const int64_t room = a.path ? a.D_path : a.row_off ? (int64_t)a.row_off[b + 1] - a.row_off[b] : a.P;
  if (n < 0 || n > room) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(a.status, DT_DEV_BAD_TREE);
    return;
  }
  const int64_t base = a.row_off ? (int64_t)a.row_off[b] : (int64_t)b * a.P;
  for (int64_t j = (int64_t)blockIdx.x * kLogThreads + threadIdx.x; j < n; j += (int64_t)gridDim.x * kLogThreads) {
    const int pos = a.path ? a.path[(int64_t)b * a.D_path + j] : (int)j;
    if (pos < 0 || (a.path && pos >= a.P)) {
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

size_t logits_smem(int P) { return (size_t)P * 8 + (size_t)kLogRows * P * 2; }

template <typename T>
cudaError_t launch_logits_t(dt_handle* h, int B, const LogitsArgs& a, cudaStream_t s) {
  const int per16 = 16 / (int)sizeof(T);
  const bool vec = a.ld % per16 == 0 && a.ld_out % per16 == 0 && ((uintptr_t)a.logits | (uintptr_t)a.out) % 16 == 0;
  const dim3 grid((a.V + kLogChunk - 1) / kLogChunk, B, (a.p.P + kLogRows - 1) / kLogRows);
  if (vec)
    launch_k(logits_kernel<T, true>, grid, dim3(kLogThreads), logits_smem(a.p.P), s, a);
  else
    launch_k(logits_kernel<T, false>, grid, dim3(kLogThreads), logits_smem(a.p.P), s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logits(dt_handle* h, int B, const void* logits, int64_t ld, void* out, int64_t ld_out,
                          const dt_logits_params* p, cudaStream_t s) {
  LogitsArgs a{*p, logits, ld, out, ld_out, h->cfg.V, h->ws.status};
  return h->cfg.dtype == DT_BF16 ? launch_logits_t<__nv_bfloat16>(h, B, a, s) : launch_logits_t<float>(h, B, a, s);
}

cudaError_t launch_count_tokens(dt_handle* h, int B, int32_t* counts, const int32_t* tokens, int P,
                                const int32_t* row_off, const int32_t* path, int D_path, const int32_t* n_new,
                                int n_extra, int prompt, cudaStream_t s) {
  CountArgs a{counts, tokens, P, row_off, path, D_path, n_new, n_extra, prompt, h->cfg.V, h->ws.status};
  const int64_t most = path ? D_path : P;
  const int chunks = (int)min((int64_t)64, max((int64_t)1, (most + kLogThreads - 1) / kLogThreads));
  launch_k(count_kernel, dim3(chunks, B), dim3(kLogThreads), 0, s, a);
  return cudaGetLastError();
}

}  // namespace dt
