// Pages of the KV cache: reservation (block tables and slot maps), release, and the commit of KV rows
// into the pages of a slot map.
//
// Who gets which block follows from sums over the requests before: request b lacks
//   need_b = max(0, ceil((len_b + n_b) / page) - owned_b)
// blocks, and takes entries [sum_{b'<b} need, sum_{b'<=b} need) counted from the end of the free list when
// they exist. Every CTA sums the requests before its own one (three loads a request, B <= 4096), so no CTA waits
// for another; the counts that all of them read are changed by the CTA that finishes last (a ticket in the
// handle's workspace that returns to zero by itself).
#include <algorithm>

#include "dt_internal.cuh"

namespace dt {
namespace {

constexpr int kPageThreads = 256;
constexpr int kSlotsPerCta = 512;  // slots of one request that a CTA writes at a time: two independent chains a thread
// Up to this many CTAs the last one changes the counts; more of them queue up at the ticket, and a second launch is
// faster. Reserve + release, 64 requests of up to 8000 slots: 13.0 us with two launches each, 15.0 with the ticket;
// 8 requests of 9 slots: 8.2 and 8.3 us on the device, but two launches take 3 us more on the host.
constexpr int kTicketCtas = 64;


struct ReserveArgs {
  dt_block_pool pool;
  int32_t page_shift;
  int32_t B;
  const int32_t* seq_len;
  const int32_t* n_new;
  int32_t n_extra;
  int64_t* slots;
  int64_t n_slots;
  int32_t S;
  const int32_t* slot_off;
  int32_t* status;
  unsigned* ticket;  // null: the counts change in a launch of their own
};

// What request b asks for. status: DT_DEV_* bits of a request that cannot be served at all.
struct Ask {
  int32_t len, n, owned, need, status;
  int64_t want, first, room;  // blocks it should own; its first slot entry and how many it has
};

__device__ __forceinline__ Ask ask_of(const ReserveArgs& a, int b) {
  Ask r;
  r.len = a.seq_len[b];
  const int64_t n = (int64_t)a.n_new[b] + a.n_extra;
  r.owned = a.pool.n_owned[b];
  r.first = (int64_t)b * a.S;
  r.room = a.S;
  r.status = 0;
  if (a.slot_off) {
    r.first = a.slot_off[b];
    const int64_t end = a.slot_off[b + 1];
    r.room = end - r.first;
    if (r.first < 0 || r.room < 0 || end > a.n_slots) {
      r.status = DT_DEV_BAD_PAGE;
      r.room = 0;
    }
  }
  if (r.len < 0 || n < 0 || r.owned < 0 || r.owned > a.pool.max_blocks) r.status = DT_DEV_BAD_PAGE;
  r.want = ((int64_t)r.len + n + a.pool.page - 1) >> a.page_shift;
  if (!r.status && (n > min((int64_t)a.S, r.room) || r.want > a.pool.max_blocks)) r.status = DT_DEV_KV_FULL;
  r.n = r.status ? 0 : (int32_t)n;
  r.need = r.status ? 0 : (int32_t)max((int64_t)0, r.want - r.owned);
  return r;
}

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* smem) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += (int64_t)shfl_xor_u64((uint64_t)v, m);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  int64_t t = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += smem[w];
  __syncthreads();
  return t;
}

// True in every thread of the CTA that comes last: what the others read and wrote before is done.
__device__ __forceinline__ bool comes_last(unsigned* ticket, unsigned ctas) {
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicInc(ticket, ctas - 1) == ctas - 1;
    __threadfence();
  }
  __syncthreads();
  return last;
}

__device__ __forceinline__ int free_blocks(const dt_block_pool& p) { return min(max(p.free_count[0], 0), p.n_blocks); }

// One CTA: owned counts of the requests that were served, and the free count.
__device__ void reserve_counts(const ReserveArgs& a, int nfree) {
  __shared__ int64_t wsum[kPageThreads / 32];
  __shared__ int64_t taken_s;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (a.B + kPageThreads - 1) / kPageThreads, b0 = tid * per;
  if (tid == 0) taken_s = 0;
  int64_t mine = 0;
  for (int b = b0; b < min(a.B, b0 + per); ++b) mine += ask_of(a, b).need;
  int64_t inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = (int64_t)shfl_u64((uint64_t)inc, max(lane - d, 0));
    if (lane >= d) inc += o;
  }
  if (lane == 31) wsum[w] = inc;
  __syncthreads();
  int64_t upto = inc - mine;
  for (int i = 0; i < w; ++i) upto += wsum[i];
  int64_t taken = 0;
  for (int b = b0; b < min(a.B, b0 + per); ++b) {
    const Ask r = ask_of(a, b);
    upto += r.need;
    if (r.need > 0 && upto <= nfree) {
      a.pool.n_owned[b] = (int32_t)r.want;
      taken = upto;
    }
  }
  if (taken > 0) atomicMax((long long*)&taken_s, (long long)taken);
  __syncthreads();
  if (tid == 0 && taken_s > 0) a.pool.free_count[0] = nfree - (int32_t)taken_s;
}

// CTA (c, b): slots [c * kSlotsPerCta, ...) of request b, then gridDim.x * kSlotsPerCta further, and its share of the
// new table entries.
__global__ void __launch_bounds__(kPageThreads) reserve_kernel(ReserveArgs a) {
  __shared__ int64_t red[kPageThreads / 32];
  pdl_begin();
  const int b = blockIdx.y, tid = threadIdx.x;
  int64_t part = 0;
  for (int i = tid; i < b; i += kPageThreads) part += ask_of(a, i).need;
  const Ask r = ask_of(a, b);
  const int64_t pre = block_sum(part, red);
  const int nfree = free_blocks(a.pool);
  int status = r.status;
  if (!status && r.need > 0 && pre + r.need > nfree) status = DT_DEV_KV_FULL;
  if (status && blockIdx.x == 0 && tid == 0) set_status(a.status, status);
  int32_t* table = a.pool.block_table + (int64_t)b * a.pool.max_blocks;
  // the q-th block granted in this call is the q-th from the end of the free list
  auto granted = [&](int64_t e) { return a.pool.free_list[nfree - 1 - (pre + e - r.owned)]; };
  if (!status) {
    for (int64_t e = r.owned + (int64_t)blockIdx.x * kPageThreads + tid; e < r.want;
         e += (int64_t)gridDim.x * kPageThreads) {
      const int32_t id = granted(e);
      if (id < 0 || id >= a.pool.n_blocks) set_status(a.status, DT_DEV_BAD_PAGE);
      table[e] = id;
    }
  }
  const int64_t hi = min((int64_t)a.S, r.room);
  for (int64_t lo = (int64_t)blockIdx.x * kSlotsPerCta; lo < hi; lo += (int64_t)gridDim.x * kSlotsPerCta) {
#pragma unroll
    for (int u = 0; u < kSlotsPerCta / kPageThreads; ++u) {
      const int64_t j = lo + tid + u * kPageThreads;
      if (j >= hi) break;
      int64_t slot = -1;
      if (!status && j < r.n) {
        const int64_t pos = r.len + j, e = pos >> a.page_shift;
        const int32_t id = e < r.owned ? table[e] : granted(e);
        if (id >= 0 && id < a.pool.n_blocks)
          slot = ((int64_t)id << a.page_shift) + (pos & (a.pool.page - 1));
        else
          set_status(a.status, DT_DEV_BAD_PAGE);
      }
      a.slots[r.first + j] = slot;
    }
  }
  if (a.ticket && comes_last(a.ticket, gridDim.x * gridDim.y)) reserve_counts(a, nfree);
}

__global__ void __launch_bounds__(kPageThreads) reserve_counts_kernel(ReserveArgs a) {
  pdl_begin();
  reserve_counts(a, free_blocks(a.pool));
}

struct ReleaseArgs {
  dt_block_pool pool;
  int32_t page_shift;
  int32_t B;
  const int32_t* keep_len;
  int32_t* status;
  unsigned* ticket;  // null: the counts change in a launch of their own
};

// Blocks that request b keeps; `back` the ones it gives back (0 for a corrupt count).
__device__ __forceinline__ int keep_of(const ReleaseArgs& a, int b, int& back, bool& bad) {
  const int owned = a.pool.n_owned[b], keep_len = a.keep_len[b];
  bad = owned < 0 || owned > a.pool.max_blocks || keep_len < 0;
  if (bad) {
    back = 0;
    return owned;
  }
  const int keep = (int)min((int64_t)owned, ((int64_t)keep_len + a.pool.page - 1) >> a.page_shift);
  back = owned - keep;
  return keep;
}

// One CTA: owned counts and the free count after `total` blocks have come back.
__device__ void release_counts(const ReleaseArgs& a, int nfree, int64_t total) {
  for (int i = threadIdx.x; i < a.B; i += kPageThreads) {
    int back;
    bool bad;
    const int kept = keep_of(a, i, back, bad);
    if (back) a.pool.n_owned[i] = kept;
  }
  if (threadIdx.x == 0 && total > 0) a.pool.free_count[0] = (int32_t)min(nfree + total, (int64_t)a.pool.n_blocks);
}

// CTA b: the r-th block given back, counted over requests and then entries in ascending order, goes to
// place free_count + total - 1 - r: the reverse of the order in which a reservation takes them.
__global__ void __launch_bounds__(kPageThreads) release_kernel(ReleaseArgs a) {
  __shared__ int64_t red[kPageThreads / 32];
  pdl_begin();
  const int b = blockIdx.x, tid = threadIdx.x;
  int back;
  bool bad;
  int64_t before = 0, total = 0;
  for (int i = tid; i < a.B; i += kPageThreads) {
    keep_of(a, i, back, bad);
    total += back;
    if (i < b) before += back;
  }
  total = block_sum(total, red);
  before = block_sum(before, red);
  const int keep = keep_of(a, b, back, bad);
  const int nfree = free_blocks(a.pool);
  if (tid == 0 && (bad || nfree + total > a.pool.n_blocks)) set_status(a.status, DT_DEV_BAD_PAGE);
  int32_t* table = a.pool.block_table + (int64_t)b * a.pool.max_blocks;
  for (int e = tid; e < back; e += kPageThreads) {
    const int64_t at = nfree + total - 1 - (before + e);
    if (at < a.pool.n_blocks) a.pool.free_list[at] = table[keep + e];
    table[keep + e] = -1;
  }
  if (a.ticket && comes_last(a.ticket, gridDim.x)) release_counts(a, nfree, total);
}

__global__ void __launch_bounds__(kPageThreads) release_counts_kernel(ReleaseArgs a) {
  __shared__ int64_t red[kPageThreads / 32];
  pdl_begin();
  int64_t total = 0;
  for (int i = threadIdx.x; i < a.B; i += kPageThreads) {
    int back;
    bool bad;
    keep_of(a, i, back, bad);
    total += back;
  }
  release_counts(a, free_blocks(a.pool), block_sum(total, red));
}

// ------------------------------------------------------------------------------- commit --------
struct PagedCommitArgs {
  dt_kv_rows kv;
  int32_t page_shift;
  int32_t P, D_path, n_extra, S, tok_per_cta;
  const int32_t* row_off;
  const int32_t* path;
  const int32_t* n_new;
  const int64_t* slots;
  int64_t n_slots;
  const int32_t* slot_off;
  const int32_t* seq_len;
  int32_t* len_out;
  int32_t* status;
};

constexpr int kMaxTok = 64;  // tokens of a CTA

// Tokens [t0, t0 + cnt) of request b in one plane; all threads of the CTA.
__device__ __forceinline__ void commit_rows(const PagedCommitArgs& a, int b, int plane, int64_t first, int t0, int cnt,
                                            const char** src_s, char** dst_s) {
  const int tid = threadIdx.x;
  if (tid < cnt) {
    const int j = t0 + tid;
    const int64_t slot = a.slots[first + j];
    const int64_t pos = a.path ? a.path[(int64_t)b * a.D_path + j] : j;
    const int64_t row = (a.row_off ? (int64_t)a.row_off[b] : (int64_t)b * a.P) + pos;
    const char* src = nullptr;
    char* dst = nullptr;
    const int64_t n_tok = (int64_t)a.kv.n_blocks << a.page_shift;
    if (slot < 0 || slot >= n_tok) {
      if (plane == 0) set_status(a.status, DT_DEV_BAD_PAGE);
    } else if (pos < 0 || pos >= a.P || row < 0 || row >= a.kv.rows) {
      if (plane == 0) set_status(a.status, DT_DEV_BAD_TREE);
    } else {
      src = (const char*)a.kv.tmp + plane * a.kv.tmp_plane + row * a.kv.tmp_row;
      dst = (char*)a.kv.cache + plane * a.kv.cache_plane + (slot >> a.page_shift) * a.kv.cache_block +
            (slot & (a.kv.page - 1)) * a.kv.cache_tok;
    }
    src_s[tid] = src;
    dst_s[tid] = dst;
  }
  __syncthreads();
  const uint32_t hv = (uint32_t)(a.kv.head_bytes >> 4), rv = hv * (uint32_t)a.kv.heads;
  const uint32_t total = rv * (uint32_t)cnt;
  // four 16-byte loads in flight a thread before any is stored
  for (uint32_t v0 = tid; v0 < total; v0 += 4 * kPageThreads) {
    uint4 r[4];
    char* to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t v = v0 + u * kPageThreads;
      to[u] = nullptr;
      if (v < total) {
        const uint32_t t = v / rv, x = v - t * rv, hd = x / hv, c = x - hd * hv;
        const char* src = src_s[t];
        if (src) {
          r[u] = __ldcs((const uint4*)(src + hd * a.kv.tmp_head) + c);
          to[u] = dst_s[t] + hd * a.kv.cache_head + ((int64_t)c << 4);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (to[u]) *(uint4*)to[u] = r[u];
  }
}

// CTA (c, b, p): tokens [c * T, (c + 1) * T) of request b in plane p, then gridDim.x * T further.
__global__ void __launch_bounds__(kPageThreads) commit_paged_kernel(PagedCommitArgs a) {
  __shared__ const char* src_s[kMaxTok];
  __shared__ char* dst_s[kMaxTok];
  pdl_begin();
  const int b = blockIdx.y, plane = blockIdx.z, tid = threadIdx.x;
  const int64_t n64 = (int64_t)a.n_new[b] + a.n_extra;
  int64_t first = (int64_t)b * a.S, room = a.S;
  int status = 0;
  if (a.slot_off) {
    first = a.slot_off[b];
    room = (int64_t)a.slot_off[b + 1] - first;
    if (first < 0 || room < 0 || first + room > a.n_slots) status = DT_DEV_BAD_PAGE;
  }
  if (n64 < 0) status = DT_DEV_BAD_PAGE;
  if (!status && (n64 > min((int64_t)a.S, room) || (a.path && n64 > a.D_path))) status = DT_DEV_KV_FULL;
  const int n = (int)n64;
  if (!status && n > 0 && (a.slots[first] < 0 || a.slots[first + n - 1] < 0)) status = DT_DEV_KV_FULL;
  const bool lead = plane == 0 && blockIdx.x == 0 && tid == 0;
  if (lead) {
    if (status) set_status(a.status, status);
    const int32_t len = a.seq_len[b];
    a.len_out[b] = status ? len : len + n;
    if (a.kv.committed) a.kv.committed[b] = status ? 0 : n;
  }
  if (status) return;
  const int64_t begin = (int64_t)blockIdx.x * a.tok_per_cta;
  for (int64_t t0 = begin; t0 < n; t0 += (int64_t)gridDim.x * a.tok_per_cta) {
    if (t0 != begin) __syncthreads();  // the addresses of the last turn have been used
    commit_rows(a, b, plane, first, (int)t0, (int)min((int64_t)a.tok_per_cta, n - t0), src_s, dst_s);
  }
}

int shift_of(int page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

}  // namespace

// CTAs of a request that has at most S of the slots, `each` at a time. Packed slots leave S loose: four times a
// request's mean share bounds them there, and longer requests take several turns.
static int chunks_of(int S, int64_t n_slots, int B, int each, bool packed) {
  const int64_t most = ((int64_t)S + each - 1) / each;
  if (!packed) return (int)most;
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, 4 * ((n_slots + (int64_t)each * B - 1) / ((int64_t)each * B))));
}

cudaError_t launch_kv_reserve(dt_handle* h, int B, const dt_block_pool* pool, const int32_t* seq_len,
                              const int32_t* n_new, int n_extra, int64_t* slots, int64_t n_slots, int S,
                              const int32_t* slot_off, cudaStream_t s) {
  ReserveArgs a{*pool, shift_of(pool->page), B, seq_len, n_new, n_extra, slots, n_slots, S, slot_off, h->ws.status, h->ws.ticket};
  const int chunks = chunks_of(S, n_slots, B, kSlotsPerCta, slot_off != nullptr);
  if ((int64_t)chunks * B > kTicketCtas) a.ticket = nullptr;
  launch_k(reserve_kernel, dim3(chunks, B), dim3(kPageThreads), 0, s, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.ticket) return e;
  launch_k(reserve_counts_kernel, dim3(1), dim3(kPageThreads), 0, s, a);
  return cudaGetLastError();
}

cudaError_t launch_kv_release(dt_handle* h, int B, const dt_block_pool* pool, const int32_t* keep_len,
                              cudaStream_t s) {
  ReleaseArgs a{*pool, shift_of(pool->page), B, keep_len, h->ws.status, h->ws.ticket};
  if (B > kTicketCtas) a.ticket = nullptr;
  launch_k(release_kernel, dim3(B), dim3(kPageThreads), 0, s, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.ticket) return e;
  launch_k(release_counts_kernel, dim3(1), dim3(kPageThreads), 0, s, a);
  return cudaGetLastError();
}

cudaError_t launch_commit_kv_paged(dt_handle* h, int B, const dt_kv_rows* kv, int P, const int32_t* row_off,
                                   const int32_t* path, int D_path, const int32_t* n_new, int n_extra,
                                   const int64_t* slots, int64_t n_slots, int S, const int32_t* slot_off,
                                   const int32_t* seq_len, int32_t* len_out, cudaStream_t s) {
  PagedCommitArgs a;
  a.kv = *kv;
  a.page_shift = shift_of(kv->page);
  a.P = P;
  a.D_path = D_path;
  a.n_extra = n_extra;
  a.S = S;
  // about 32 KB a CTA: 8 vectors a thread
  a.tok_per_cta = (int)std::min<int64_t>(kMaxTok, std::max<int64_t>(1, 32768 / (kv->head_bytes * kv->heads)));
  a.row_off = row_off;
  a.path = path;
  a.n_new = n_new;
  a.slots = slots;
  a.n_slots = n_slots;
  a.slot_off = slot_off;
  a.seq_len = seq_len;
  a.len_out = len_out;
  a.status = h->ws.status;
  launch_k(commit_paged_kernel, dim3(chunks_of(S, n_slots, B, a.tok_per_cta, slot_off != nullptr), B, kv->planes), dim3(kPageThreads), 0,
           s, a);
  return cudaGetLastError();
}

}  // namespace dt
