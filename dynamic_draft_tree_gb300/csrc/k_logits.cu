// Target rows prepared for the verify pass: penalties for repeated tokens, biases, grammar masks.
//
// Every row is read and written once. A CTA owns a chunk of the vocabulary for one request and goes
// through a group of that request's rows, so the request's counts and biases of the chunk are read once
// a group into registers. What differs from row to row is the tree path: the path tokens that fall into
// the chunk (a few of D <= 17 over V / 2048 chunks) are listed a row in shared memory before the row loop.
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

// VEC: every row starts on a 16-byte boundary; a thread's tokens are then kLogPer neighbours (one or two
// 16-byte accesses), else one token in every kLogThreads (coalesced single elements).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kLogThreads) logits_kernel(LogitsArgs a) {
  extern __shared__ char dyn[];
  const int P = a.p.P;
  int32_t* path_tok = (int32_t*)dyn;               // [P] chunk offset of a position's token, its position
  int32_t* path_pos = path_tok + P;                // [P]
  uint16_t* row_list = (uint16_t*)(path_pos + P);  // [kLogRows][P] chunk offsets of the row's path tokens
  __shared__ int n_path, n_row[kLogRows], n_bias_s;
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
  if (tid == 0) n_path = 0;
  if (tid < kLogRows) n_row[tid] = 0;
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
      const bool in = id >= v0 && id - v0 < kLogChunk;
      const float val = in ? a.p.bias_vals[(int64_t)b * a.p.n_bias + k] : 0.0f;
      for (uint32_t m = __ballot_sync(0xFFFFFFFFu, in); m; m &= m - 1) {
        if (tid == __ffs(m) - 1) bias_s[id - v0] = __fadd_rn(bias_s[id - v0], val);
        __syncwarp();
      }
    }
  }
  __syncthreads();
  const int np = n_path;
  for (int x = tid; x < np * rows; x += kLogThreads) {
    const int r = x / np, k = x - r * np, i = row0 + r, j = path_pos[k];
    const bool on = a.p.mask ? a.p.mask[((int64_t)b * P + i) * P + j] != 0 : j <= i;
    if (on) row_list[r * P + atomicAdd(&n_row[r], 1)] = (uint16_t)path_tok[k];
  }
  // a thread's counts and biases
  int cnt[kLogPer];
  float bias[kLogPer];
  uint32_t prompt = 0;
#pragma unroll
  for (int u = 0; u < kLogPer; ++u) {
    const int off = VEC ? tid * kLogPer + u : tid + u * kLogThreads;
    const int v = v0 + off;
    const int c = (a.p.counts && v < a.V) ? a.p.counts[(int64_t)b * a.V + v] : 0;
    cnt[u] = c & (DT_SEEN_PROMPT - 1);
    if (c & DT_SEEN_PROMPT) prompt |= 1u << u;
    bias[u] = with_bias ? bias_s[off] : 0.0f;
  }
  const float rep = a.p.repetition ? a.p.repetition[b] : 1.0f;
  const float freq = a.p.frequency ? a.p.frequency[b] : 0.0f;
  const float pres = a.p.presence ? a.p.presence[b] : 0.0f;
  __syncthreads();
  for (int r = 0; r < rows; ++r) {
    const int64_t row = base + row0 + r;
    const T* x = (const T*)a.logits + row * a.ld;
    T* y = (T*)a.out + row * a.ld_out;
    uint32_t allow = 0xFFu;
    if (a.p.allow) {
      const uint32_t* w = a.p.allow + row * a.p.allow_ld;
      if (VEC) {
        const int v = v0 + tid * kLogPer;
        allow = v < a.V ? (w[v >> 5] >> (v & 31)) & 0xFFu : 0u;
      } else {
        allow = 0;
#pragma unroll
        for (int u = 0; u < kLogPer; ++u) {
          const int v = v0 + tid + u * kLogThreads;
          if (v < a.V) allow |= ((w[v >> 5] >> (v & 31)) & 1u) << u;
        }
      }
    }
    T in[kLogPer];
    if (VEC && v0 + (tid + 1) * kLogPer <= a.V) {
      constexpr int kVec = (int)sizeof(T) * kLogPer / 16;
      uint4 q[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) q[k] = __ldcs((const uint4*)(x + v0 + tid * kLogPer) + k);
      memcpy(in, q, sizeof(in));
    } else {
#pragma unroll
      for (int u = 0; u < kLogPer; ++u) {
        const int v = v0 + (VEC ? tid * kLogPer + u : tid + u * kLogThreads);
        if (v < a.V) in[u] = x[v];
      }
    }
    int add[kLogPer];
#pragma unroll
    for (int u = 0; u < kLogPer; ++u) add[u] = 0;
    const int nr = n_row[r];
    for (int k = 0; k < nr; ++k) {
      const int off = row_list[r * P + k];
#pragma unroll
      for (int u = 0; u < kLogPer; ++u) add[u] += off == (VEC ? tid * kLogPer + u : tid + u * kLogThreads);
    }
    T res[kLogPer];
#pragma unroll
    for (int u = 0; u < kLogPer; ++u) {
      float f = to_f(in[u]);
      const int c = cnt[u] + add[u];
      if (c > 0 || (prompt >> u & 1)) {
        f = f > 0.0f ? __fdiv_rn(f, rep) : __fmul_rn(f, rep);
        if (c > 0) f = __fsub_rn(__fsub_rn(f, __fmul_rn(freq, (float)c)), pres);
      }
      if (with_bias) f = __fadd_rn(f, bias[u]);
      if (!(allow >> u & 1)) f = -INFINITY;
      from_f(f, res[u]);
    }
    if (VEC && v0 + (tid + 1) * kLogPer <= a.V) {
      constexpr int kVec = (int)sizeof(T) * kLogPer / 16;
      uint4 q[kVec];
      memcpy(q, res, sizeof(res));
#pragma unroll
      for (int k = 0; k < kVec; ++k) __stcs((uint4*)(y + v0 + tid * kLogPer) + k, q[k]);
    } else {
#pragma unroll
      for (int u = 0; u < kLogPer; ++u) {
        const int v = v0 + (VEC ? tid * kLogPer + u : tid + u * kLogThreads);
        if (v < a.V) y[v] = res[u];
      }
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
