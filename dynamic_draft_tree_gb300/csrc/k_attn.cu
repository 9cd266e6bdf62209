// Attention of the verify tree over a paged cache: one CTA a query row and head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dt_internal.cuh"

namespace dt {
namespace {

__device__ __forceinline__ float tof(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float tof(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(__nv_bfloat16& o, float x) { o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half& o, float x) { o = __float2half_rn(x); }

// Grid (position, head, request); warp w takes every fourth key, lane l the elements l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(128) attn_rows_kernel(dt_attn_args a, int32_t* status) {
  __shared__ float m_s[4], l_s[4], o_s[4][128];
  pdl_begin();
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = min(max(a.n_pos[b], 0), a.P);
  if (i >= n) return;
  const int64_t base = a.row_off ? (int64_t)a.row_off[b] : (int64_t)b * a.P;
  if (base < 0 || base + n > a.rows) {
    set_status(status, DT_DEV_BAD_PAGE);
    return;
  }
  int len = a.seq_len[b];
  if (len < a.shared_len || len > (int64_t)a.max_blocks * a.page) {
    set_status(status, DT_DEV_BAD_PAGE);
    len = (int)min((int64_t)max(len, a.shared_len), (int64_t)a.max_blocks * a.page);
  }
  const int kvh = h / (a.H_q / a.H_kv);
  const T* q = (const T*)a.q + (base + i) * a.q_row + h * a.q_head;
  float qf[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) qf[u] = lane + 32 * u < a.D ? tof(q[lane + 32 * u]) * a.scale : 0.0f;
  for (int t = warp; t < len + n; t += 4) {
    const T *k, *v;
    if (t < len) {
      const int e = t / a.page;
      const int id = a.block_table[(t < a.shared_len ? 0 : (int64_t)b * a.max_blocks) + e];
      if (id < 0 || id >= a.n_blocks) {
        set_status(status, DT_DEV_BAD_PAGE);
        continue;
      }
      k = (const T*)a.k_pages + id * a.k_block + (t - e * a.page) * a.k_tok + kvh * a.k_head;
      v = (const T*)a.v_pages + id * a.v_block + (t - e * a.page) * a.v_tok + kvh * a.v_head;
    } else {
      const int j = t - len;
      if (a.mask ? !a.mask[((int64_t)b * a.P + i) * a.P + j] : j > i) continue;
      k = (const T*)a.k_new + (base + j) * a.kn_row + kvh * a.kn_head;
      v = (const T*)a.v_new + (base + j) * a.vn_row + kvh * a.vn_head;
    }
    float s = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (lane + 32 * u < a.D) s += qf[u] * tof(k[lane + 32 * u]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    const float mn = fmaxf(m, s), c = m == -INFINITY ? 0.0f : __expf(m - mn), p = mn == -INFINITY ? 0.0f : __expf(s - mn);
    l = l * c + p;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (lane + 32 * u < a.D) o[u] = o[u] * c + p * tof(v[lane + 32 * u]);
    m = mn;
  }
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) o_s[warp][lane + 32 * u] = o[u];
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= a.D) return;
  const float mm = fmaxf(fmaxf(m_s[0], m_s[1]), fmaxf(m_s[2], m_s[3]));
  float ll = 0, oo = 0;
  for (int w = 0; w < 4; ++w) {
    const float c = m_s[w] == -INFINITY ? 0.0f : __expf(m_s[w] - mm);
    ll += l_s[w] * c;
    oo += o_s[w][d] * c;
  }
  put(((T*)a.out)[(base + i) * a.o_row + h * a.o_head + d], ll > 0 ? oo / ll : 0.0f);
}

}  // namespace

int64_t attn_workspace_bytes(const dt_handle* h, int B, int P, int H_q, int H_kv, int D, int shared) { return 256; }

cudaError_t launch_attention(dt_handle* h, const dt_attn_args* a, cudaStream_t s) {
  const dim3 grid(a->P, a->H_q, a->B);
  if (a->dtype == DT_BF16)
    launch_k(attn_rows_kernel<__nv_bfloat16>, grid, dim3(128), 0, s, *a, h->ws.status);
  else
    launch_k(attn_rows_kernel<__half>, grid, dim3(128), 0, s, *a, h->ws.status);
  return cudaGetLastError();
}

}  // namespace dt
