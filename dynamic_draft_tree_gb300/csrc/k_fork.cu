// Requests that continue others (samples of one prompt, branches of a beam): whole pages are shared, the page that the next
// tokens go into is copied; and the release of pages that requests share.
//
// refs[x] counts the owners of block x beyond its first, so that blocks that nobody forked need no attention (0) and
// reservations and commits go on as they are. A fork at `len` tokens adds one to the counts of the len / page whole pages,
// which nobody writes again, and takes one free block for the len % page tokens of the last one.
//
// Which free block a fork takes follows from sums over the forks before it (at most one block each), as in the reservation.
// A release marks who gives what back in the upper halves of refs (sums, so that their order does not matter); the last
// giver in request order is the one that acts: it returns a block that nobody keeps, or takes the givers off the count. A
// block stands at the same place of every owner's table, so the last giver is found by a look at that place of the later
// requests. Bound by DRAM where pages are copied; else by the latency of the launches.
#include <algorithm>

#include "dt_internal.cuh"
#include "pages.cuh"

namespace dt {
namespace {

struct ForkArgs {
  dt_block_pool pool;
  dt_kv_pages kv;
  int32_t page_shift, B, n, shared_blocks, rows_per_cta;
  int32_t* refs;
  const int32_t *src, *dst, *length;
  int32_t* seq_len;
  int32_t* state;     // [n] blocks that a fork takes, or minus the status bits of one that is refused
  int32_t* status;
  unsigned* ticket;   // null: the counts change in a launch of their own
};

struct Fork {
  int32_t src, dst, len, need;
  int32_t status;  // DT_DEV_* bits of one that is refused, by itself
};

__device__ __forceinline__ Fork fork_of(const ForkArgs& a, int f) {
  Fork r{a.src[f], a.dst[f], 0, 0, 0};
  if (r.src < 0 || r.src >= a.B || r.dst < 0 || r.dst >= a.B || r.src == r.dst) {
    r.status = DT_DEV_BAD_PAGE;
    return r;
  }
  const int have = a.seq_len[r.src], owned = a.pool.n_owned[r.src];
  r.len = a.length ? a.length[f] : have;
  if (r.len < 0 || r.len > have || r.len < a.shared_blocks << a.page_shift || owned < 0 || owned > a.pool.max_blocks ||
      ((int64_t)r.len + a.pool.page - 1) >> a.page_shift > owned || a.pool.n_owned[r.dst] != a.shared_blocks)
    r.status = DT_DEV_BAD_PAGE;
  r.need = !r.status && (r.len & (a.pool.page - 1)) ? 1 : 0;
  return r;
}

// Whether an earlier fork has the same destination, or any has this one's source as its destination.
template <typename At>
__device__ __forceinline__ bool conflicts(int n, int f, int src, int dst, At dst_at) {
  bool bad = false;
  for (int j = 0; j < n; ++j) {
    const int d = dst_at(j);
    bad |= (d == dst && j < f) || d == src;
  }
  return bad;
}

__device__ __forceinline__ int state_of(const Fork& r, bool conflict) {
  const int status = r.status | (conflict ? DT_DEV_BAD_PAGE : 0);
  return status ? -status : r.need;
}

// More forks than threads: their states in a launch of their own.
__global__ void __launch_bounds__(kPageThreads) fork_state_kernel(const __grid_constant__ ForkArgs a) {
  pdl_begin();
  const int f = blockIdx.x * kPageThreads + threadIdx.x;
  if (f >= a.n) return;
  const Fork r = fork_of(a, f);
  a.state[f] = state_of(r, conflicts(a.n, f, r.src, r.dst, [&](int j) { return a.dst[j]; }));
}

// One CTA: counts of the forks that were served.
__device__ void fork_counts(const ForkArgs& a, int nfree) {
  __shared__ int64_t red[kPageThreads / 32];
  int64_t taken = 0;
  for (int f = threadIdx.x; f < a.n; f += kPageThreads) {
    const int need = __ldcg(a.state + f);
    if (need < 0) continue;
    const Fork r = fork_of(a, f);
    a.seq_len[r.dst] = r.len;
    a.pool.n_owned[r.dst] = (r.len >> a.page_shift) + need;
    taken += need;
  }
  taken = block_sum(taken, red);
  if (threadIdx.x == 0 && taken > 0) a.pool.free_count[0] = nfree - (int32_t)taken;
}

// x / d by a multiplication: exact for x d < 2^32.
struct Divide {
  uint32_t d, magic;
  __device__ __forceinline__ explicit Divide(uint32_t d_) : d(d_), magic(0xFFFFFFFFu / d_ + 1) {}
  __device__ __forceinline__ uint32_t by(uint32_t x) const { return d == 1 ? x : __umulhi(x, magic); }
};

__global__ void __launch_bounds__(kPageThreads) fork_counts_kernel(const __grid_constant__ ForkArgs a) {
  pdl_begin();
  fork_counts(a, free_blocks(a.pool));
}

// CTA (c, f): fork f's rows [c R, (c + 1) R) of the last page in all planes, then gridDim.x R further; CTA (0, f) its table.
__global__ void __launch_bounds__(kPageThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ int64_t red[kPageThreads / 32];
  __shared__ int32_t dst_s[kPageThreads];
  __shared__ int32_t mine_s;
  pdl_begin();
  const int f = blockIdx.y, tid = threadIdx.x;
  const Fork r = fork_of(a, f);
  int64_t before = 0;
  int state;
  if (a.n <= kPageThreads) {
    const Fork other = tid < a.n ? fork_of(a, tid) : Fork{};
    if (tid < a.n) dst_s[tid] = other.dst;
    __syncthreads();
    int s = 0;
    if (tid < a.n && tid <= f) s = state_of(other, conflicts(a.n, tid, other.src, other.dst, [&](int j) { return dst_s[j]; }));
    if (tid == f) mine_s = s;
    if (tid < f) before = max(s, 0);
    before = block_sum(before, red);
    state = mine_s;
  } else {
    for (int i = tid; i < f; i += kPageThreads) before += max(a.state[i], 0);
    before = block_sum(before, red);
    state = a.state[f];
  }
  const int nfree = free_blocks(a.pool);
  if (state > 0 && before + state > nfree) state = -DT_DEV_KV_FULL;
  const int full = r.len >> a.page_shift, tail = r.len & (a.pool.page - 1);
  const int32_t* from = a.pool.block_table + (int64_t)r.src * a.pool.max_blocks;
  int32_t* to = a.pool.block_table + (int64_t)r.dst * a.pool.max_blocks;
  const int block = state > 0 ? a.pool.free_list[nfree - 1 - before] : -1;  // the one that it takes
  if (blockIdx.x == 0) {
    if (state < 0) {
      if (tid == 0) set_status(a.status, -state);
    } else {
      for (int e = a.shared_blocks + tid; e < full; e += kPageThreads) {
        const int id = from[e];
        if (id < 0 || id >= a.pool.n_blocks) set_status(a.status, DT_DEV_BAD_PAGE);
        else atomicAdd(a.refs + id, 1);
        to[e] = id;
      }
      if (state > 0 && tid == 0) to[full] = block;
    }
  }
  if (state > 0) {
    const int old = from[full];
    if (old < 0 || old >= a.pool.n_blocks || block < 0 || block >= a.pool.n_blocks) {
      if (blockIdx.x == 0 && tid == 0) set_status(a.status, DT_DEV_BAD_PAGE);
    } else {
      // four 16-byte loads in flight a thread before any is stored; vectors in the order plane, token, head
      // (a row has at most 65536 of them and a CTA's turn no more, and a page has up to 2^24 rows)
      const uint32_t hv = (uint32_t)(a.kv.head_bytes >> 4), rv = hv * (uint32_t)a.kv.heads;
      const Divide by_row(rv), by_head(hv), by_plane((uint32_t)tail);
      const char* base = (const char*)a.kv.cache + (int64_t)old * a.kv.cache_block;
      const int64_t off = ((int64_t)block - old) * a.kv.cache_block;
      const int rows = tail * a.kv.planes;
      for (int row0 = blockIdx.x * a.rows_per_cta; row0 < rows; row0 += gridDim.x * a.rows_per_cta) {
        const uint32_t total = (uint32_t)min(a.rows_per_cta, rows - row0) * rv;
        for (uint32_t v0 = tid; v0 < total; v0 += 4 * kPageThreads) {
          uint4 q[4];
          char* at[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t v = v0 + u * kPageThreads;
            at[u] = nullptr;
            if (v < total) {
              const uint32_t k = by_row.by(v), x = v - k * rv, hd = by_head.by(x), c = x - hd * hv;
              const uint32_t row = (uint32_t)row0 + k, plane = by_plane.by(row), t = row - plane * (uint32_t)tail;
              const char* src = base + plane * a.kv.cache_plane + t * a.kv.cache_tok + hd * a.kv.cache_head + ((int64_t)c << 4);
              q[u] = __ldcs((const uint4*)src);
              at[u] = const_cast<char*>(src) + off;
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (at[u]) *(uint4*)at[u] = q[u];
        }
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    // read by the CTA that comes last, or by the launch behind this one; with more forks than threads the needs of others
    // are still being read here, and a fork without a page is told apart by them
    if (a.n <= kPageThreads) a.state[f] = state;
  }
  if (a.ticket && comes_last(a.ticket, gridDim.x * gridDim.y)) fork_counts(a, nfree);
}

// More forks than threads: those that found no page (the first ones took all there are).
__global__ void __launch_bounds__(kPageThreads) fork_refuse_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ int64_t red[kPageThreads / 32];
  pdl_begin();
  const int nfree = free_blocks(a.pool);
  int64_t before = 0;
  for (int f0 = 0; f0 < a.n; f0 += kPageThreads) {  // one CTA
    const int f = f0 + threadIdx.x;
    const int need = f < a.n ? max(a.state[f], 0) : 0;
    // sums up to this thread's: over the warps before, then within the warp
    int64_t inc = need;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = (int64_t)shfl_u64((uint64_t)inc, max((int)(threadIdx.x & 31) - d, 0));
      if ((int)(threadIdx.x & 31) >= d) inc += o;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 31) red[threadIdx.x >> 5] = inc;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kPageThreads / 32; ++w) {
      if (w < (int)(threadIdx.x >> 5)) inc += red[w];
      all += red[w];
    }
    if (need > 0 && before + inc > nfree) a.state[f] = -DT_DEV_KV_FULL;
    before += all;
  }
}

// ------------------------------------------------------------------------------ release ---------
struct SharedReleaseArgs {
  dt_block_pool pool;
  int32_t page_shift, B;
  int32_t* refs;
  const int32_t* keep_len;
  int32_t* count;     // [B] blocks that go back to the list through request b
  int32_t* status;
  unsigned* ticket;   // null: the free count changes in a launch of its own
};

constexpr int kGiver = 1 << 16;      // of a block's count: one who gives it back in this call (owners: lower half)
constexpr int kSettles = 1 << 30;    // of a table entry: its request takes the givers off the count; ~id: it returns the block

__device__ __forceinline__ int keep_blocks(const SharedReleaseArgs& a, int b, int& owned) {
  owned = a.pool.n_owned[b];
  const int keep_len = a.keep_len[b];
  if (owned < 0 || owned > a.pool.max_blocks || keep_len < 0) return owned = max(0, min(owned, a.pool.max_blocks));
  return (int)min((int64_t)owned, ((int64_t)keep_len + a.pool.page - 1) >> a.page_shift);
}
__device__ __forceinline__ int block_of(int entry) { return entry < 0 ? ~entry : entry & (kSettles - 1); }

// Request b gives back the block at place e.
__device__ __forceinline__ void give(const SharedReleaseArgs& a, int32_t* entry) {
  const int id = *entry;
  if (id >= 0 && id < a.pool.n_blocks) {
    atomicAdd(a.refs + id, kGiver);
  } else {
    set_status(a.status, DT_DEV_BAD_PAGE);
    *entry = a.pool.n_blocks;  // nobody's
  }
}
// After all have given: marks the entry if request b acts for its block (a later request looks through the mark); true if
// the block goes back to the list. keep_s, has_s: blocks that each request keeps and has. LOOK later requests' entries are looked at
// together: 56 samples of 8 prompts of 2000 tokens, fork and release, 59.0 us with two, 55.6 with four, 53.6 with eight, 65.7 one
// after the other; 8 samples of one prompt (one CTA) 13.6, 13.7 and 14.2.
template <int LOOK>
__device__ __forceinline__ bool mark(const SharedReleaseArgs& a, int b, int e, int32_t* entry, const int32_t* keep_s, const int32_t* has_s) {
  const int id = *entry;
  if (id >= a.pool.n_blocks) return false;
  const int refs = __ldcg(a.refs + id), extra = refs & (kGiver - 1), givers = refs >> 16;
  if (givers > extra + 1) set_status(a.status, DT_DEV_BAD_PAGE);  // given back by more than own it
  if (givers > 1) {
    const int32_t* at = a.pool.block_table + e;
    for (int o0 = b + 1; o0 < a.B; o0 += LOOK) {
      int32_t x[LOOK];
#pragma unroll
      for (int u = 0; u < LOOK; ++u) {
        const int o = min(o0 + u, a.B - 1);
        x[u] = e >= keep_s[o] && e < has_s[o] ? __ldcg(at + (int64_t)o * a.pool.max_blocks) : INT32_MAX;
      }
      bool later = false;
#pragma unroll
      for (int u = 0; u < LOOK; ++u) later |= o0 + u < a.B && block_of(x[u]) == id;
      if (later) return false;
    }
  }
  *entry = givers > extra ? ~id : id | kSettles;
  return givers > extra;
}
// The entry goes; `at`: place of the list that a block that goes back takes.
__device__ __forceinline__ void settle(const SharedReleaseArgs& a, int32_t* entry, int64_t at) {
  const int x = *entry;
  if (x < 0) {
    if (at >= 0 && at < a.pool.n_blocks) a.pool.free_list[at] = ~x;
    a.refs[~x] = 0;
  } else if (x >= kSettles) {
    const int id = x & (kSettles - 1), refs = a.refs[id];
    a.refs[id] = (refs & (kGiver - 1)) - (refs >> 16);
  }
  *entry = -1;
}
// Tokens that request b keeps inside a page that others go on owning are not its own to overwrite. (After all have given.)
__device__ __forceinline__ void check_kept(const SharedReleaseArgs& a, int b, int keep) {
  const int keep_len = a.keep_len[b];
  if (keep <= 0 || !(keep_len & (a.pool.page - 1)) || (int64_t)keep << a.page_shift <= keep_len) return;
  const int id = a.pool.block_table[(int64_t)b * a.pool.max_blocks + keep - 1];
  if (id < 0 || id >= a.pool.n_blocks) return;
  const int refs = __ldcg(a.refs + id);
  if ((refs & (kGiver - 1)) > refs >> 16) set_status(a.status, DT_DEV_BAD_PAGE);
}
__device__ __forceinline__ void check_counts(const SharedReleaseArgs& a, int b, int owned) {
  if (a.keep_len[b] < 0 || a.pool.n_owned[b] != owned) set_status(a.status, DT_DEV_BAD_PAGE);
}

// CTA b: request b gives.
__global__ void __launch_bounds__(kPageThreads) release_give_kernel(const __grid_constant__ SharedReleaseArgs a) {
  pdl_begin();
  const int b = blockIdx.x;
  int owned;
  const int keep = keep_blocks(a, b, owned);
  if (threadIdx.x == 0) check_counts(a, b, owned);
  int32_t* table = a.pool.block_table + (int64_t)b * a.pool.max_blocks;
  for (int e = keep + threadIdx.x; e < owned; e += kPageThreads) give(a, table + e);
}

// CTA b: which of them request b acts for.
__global__ void __launch_bounds__(kPageThreads) release_mark_kernel(const __grid_constant__ SharedReleaseArgs a) {
  extern __shared__ int32_t kept[];  // [B] blocks that are kept, [B] that there are
  __shared__ int64_t red[kPageThreads / 32];
  pdl_begin();
  const int b = blockIdx.x;
  for (int o = b + threadIdx.x; o < a.B; o += kPageThreads) {
    int has;
    kept[o] = keep_blocks(a, o, has);
    kept[a.B + o] = has;
  }
  __syncthreads();
  const int keep = kept[b], owned = kept[a.B + b];
  int32_t* table = a.pool.block_table + (int64_t)b * a.pool.max_blocks;
  int64_t mine = 0;
  for (int e = keep + threadIdx.x; e < owned; e += kPageThreads)
    mine += mark<8>(a, b, e, table + e, kept, kept + a.B);
  if (threadIdx.x == 0) check_kept(a, b, keep);
  mine = block_sum(mine, red);
  if (threadIdx.x == 0) a.count[b] = (int32_t)mine;
}

// CTA b: the r-th block that goes back, counted over requests and then entries in ascending order, goes to place
// free_count + total - 1 - r: the reverse of the order in which forks and reservations take them.
__global__ void __launch_bounds__(kPageThreads) release_return_kernel(const __grid_constant__ SharedReleaseArgs a) {
  __shared__ int64_t red[kPageThreads / 32];
  pdl_begin();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  int64_t before = 0, total = 0;
  for (int i = tid; i < a.B; i += kPageThreads) {
    const int c = a.count[i];
    total += c;
    if (i < b) before += c;
  }
  total = block_sum(total, red);
  before = block_sum(before, red);
  int owned;
  const int keep = keep_blocks(a, b, owned), nfree = free_blocks(a.pool);
  if (tid == 0 && nfree + total > a.pool.n_blocks) set_status(a.status, DT_DEV_BAD_PAGE);
  int32_t* table = a.pool.block_table + (int64_t)b * a.pool.max_blocks;
  for (int e0 = keep; e0 < owned; e0 += kPageThreads) {
    const int e = e0 + tid;
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, e < owned && table[e] < 0);
    __syncthreads();
    if (lane == 0) red[tid >> 5] = __popc(votes);
    __syncthreads();
    int64_t rank = before + __popc(votes & ((1u << lane) - 1));
    for (int w = 0; w < kPageThreads / 32; ++w) {
      if (w < tid >> 5) rank += red[w];
      before += red[w];
    }
    if (e < owned) settle(a, table + e, nfree + total - 1 - rank);
  }
  if (tid == 0 && keep < owned) a.pool.n_owned[b] = keep;
  if (a.ticket && comes_last(a.ticket, gridDim.x) && tid == 0) a.pool.free_count[0] = (int32_t)min(nfree + total, (int64_t)a.pool.n_blocks);
}

// Few entries: one CTA does all of it, three steps over the tables in one launch instead of three. A fork and a release, one CTA
// and three launches: tables of 2 x 16 entries 13.1 and 14.0 us, 16 x 64 12.6 and 13.9, 128 x 8 15.9 and 21.0, 32 x 64 16.8 and
// 14.2, 64 x 64 28.5 and 17.6; on the host 10.0 and 13.5 us.
constexpr int kSmallThreads = 1024;
constexpr int kSmallEntries = 1024;
__global__ void __launch_bounds__(kSmallThreads) release_small_kernel(const __grid_constant__ SharedReleaseArgs a) {
  __shared__ int32_t keep_s[kSmallEntries], has_s[kSmallEntries];
  __shared__ int32_t warps[kSmallThreads / 32];
  __shared__ int32_t total_s;
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, mb = a.pool.max_blocks, all = a.B * mb;
  const int nfree = free_blocks(a.pool);
  for (int b = tid; b < a.B; b += kSmallThreads) {
    int owned;
    keep_s[b] = keep_blocks(a, b, owned);
    has_s[b] = owned;
    check_counts(a, b, owned);
  }
  if (tid == 0) total_s = 0;
  __syncthreads();
  auto mine = [&](int i, int& b, int& e) {  // entry i of the tables, in order: whether its request gives it back
    b = i / mb;
    e = i - b * mb;
    return i < all && e >= keep_s[b] && e < has_s[b];
  };
  int b, e;
  for (int i = tid; i < all; i += kSmallThreads)
    if (mine(i, b, e)) give(a, a.pool.block_table + i);
  __threadfence();
  __syncthreads();
  int back = 0;
  for (int i = tid; i < all; i += kSmallThreads)
    if (mine(i, b, e)) back += mark<2>(a, b, e, a.pool.block_table + i, keep_s, has_s);
  for (int q = tid; q < a.B; q += kSmallThreads) check_kept(a, q, keep_s[q]);
  back = __reduce_add_sync(0xFFFFFFFFu, back);
  if (lane == 0) atomicAdd(&total_s, back);
  __threadfence();
  __syncthreads();
  const int total = total_s;
  if (tid == 0 && nfree + total > a.pool.n_blocks) set_status(a.status, DT_DEV_BAD_PAGE);
  int before = 0;
  for (int i0 = 0; i0 < all; i0 += kSmallThreads) {
    const int i = i0 + tid;
    const bool is = mine(min(i, all - 1), b, e) && i < all;
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, is && __ldcg(a.pool.block_table + i) < 0);
    __syncthreads();
    if (lane == 0) warps[tid >> 5] = __popc(votes);
    __syncthreads();
    int rank = before + __popc(votes & ((1u << lane) - 1));
    for (int w = 0; w < kSmallThreads / 32; ++w) {
      if (w < tid >> 5) rank += warps[w];
      before += warps[w];
    }
    if (is) settle(a, a.pool.block_table + i, (int64_t)nfree + total - 1 - rank);
  }
  for (int q = tid; q < a.B; q += kSmallThreads)
    if (keep_s[q] < has_s[q]) a.pool.n_owned[q] = keep_s[q];
  if (tid == 0 && total > 0) a.pool.free_count[0] = (int32_t)min((int64_t)nfree + total, (int64_t)a.pool.n_blocks);
}

__global__ void __launch_bounds__(kPageThreads) release_total_kernel(const __grid_constant__ SharedReleaseArgs a) {
  __shared__ int64_t red[kPageThreads / 32];
  pdl_begin();
  int64_t total = 0;
  for (int i = threadIdx.x; i < a.B; i += kPageThreads) total += a.count[i];
  total = block_sum(total, red);
  if (threadIdx.x == 0) a.pool.free_count[0] = (int32_t)min(free_blocks(a.pool) + total, (int64_t)a.pool.n_blocks);
}

}  // namespace

cudaError_t launch_kv_fork(dt_handle* h, int B, const dt_block_pool* pool, int32_t* refs, const dt_kv_pages* kv, int n,
                           const int32_t* src, const int32_t* dst, const int32_t* length, int32_t* seq_len, int shared_len,
                           cudaStream_t s) {
  ForkArgs a{};
  a.pool = *pool;
  a.kv = *kv;
  a.page_shift = shift_of(pool->page);
  a.B = B;
  a.n = n;
  a.shared_blocks = shared_len >> a.page_shift;
  // about 32 KB a CTA: 8 vectors a thread; a fork has up to page - 1 rows a plane
  a.rows_per_cta = (int)std::max<int64_t>(1, 32768 / (kv->head_bytes * kv->heads));
  a.refs = refs;
  a.src = src;
  a.dst = dst;
  a.length = length;
  a.seq_len = seq_len;
  a.state = h->ws.page_state;
  a.status = h->ws.status;
  const int64_t most = ((int64_t)(pool->page - 1) * kv->planes + a.rows_per_cta - 1) / a.rows_per_cta;
  const int chunks = (int)std::max<int64_t>(1, std::min<int64_t>(most, (int64_t)h->num_sms * 16 / n));
  const bool many = n > kPageThreads;
  a.ticket = !many && (int64_t)chunks * n <= kTicketCtas ? h->ws.ticket : nullptr;
  const dim3 block(kPageThreads);
  if (many) {
    launch_k(fork_state_kernel, dim3((n + kPageThreads - 1) / kPageThreads), block, 0, s, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  launch_k(fork_kernel, dim3(chunks, n), block, 0, s, a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && many) {
    launch_k(fork_refuse_kernel, dim3(1), block, 0, s, a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || a.ticket) return e;
  launch_k(fork_counts_kernel, dim3(1), block, 0, s, a);
  return cudaGetLastError();
}

cudaError_t launch_kv_release_shared(dt_handle* h, int B, const dt_block_pool* pool, int32_t* refs, const int32_t* keep_len,
                                     cudaStream_t s) {
  SharedReleaseArgs a{*pool, shift_of(pool->page), B, refs, keep_len, h->ws.page_state, h->ws.status,
                      B <= kTicketCtas ? h->ws.ticket : nullptr};
  const dim3 grid(B), block(kPageThreads);
  if ((int64_t)B * pool->max_blocks <= kSmallEntries) {
    launch_k(release_small_kernel, dim3(1), dim3(kSmallThreads), 0, s, a);
    return cudaGetLastError();
  }
  launch_k(release_give_kernel, grid, block, 0, s, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  launch_k(release_mark_kernel, grid, block, 8 * (size_t)B, s, a);  // B <= 4096: 32 KB
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  launch_k(release_return_kernel, grid, block, 0, s, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.ticket) return e;
  launch_k(release_total_kernel, dim3(1), block, 0, s, a);
  return cudaGetLastError();
}

}  // namespace dt
