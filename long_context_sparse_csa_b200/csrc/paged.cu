// Pages of the 8-bit key/value cache: the quantising append, and the copying, forking, reserving,
// freeing and compacting of pages (definitions at the calls in csa.h).
//
// The bookkeeping runs on the device, because positions and page numbers live there: a decode loop
// never reads them back.  fork and free are one pass over the table rows concerned, with integer
// atomics on the counts (their sums do not depend on the order).  reserve and compact need one order
// over all rows or all pages; they run as one cluster of 8 CTAs whose barrier separates the phases
// and whose shared memory holds the running counts, so that no scratch memory is needed.  Measured on
// the device: fork 1.7-2.3 us, free 2, reserve 8-9 (512 rows, 50,000 pages), compact 7, all bound by latency;
// the append of 16,384 tokens of 8 heads of 128 dims 25-29 us (100 MB: 3.5-4 TB/s), of one token of 64
// sequences 5.3 (with its pages' bytes in memory 10 where no scale grows, 16 where 436 of 1,024 do: their earlier codes are
// read and written in one more chain); the copy of 900 pages of 128 KB 45 us (236 MB: 5.2 TB/s).
#include <cooperative_groups.h>
#include <mutex>

#include "paged.h"

namespace csa {

namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kThreads = 1024;

__device__ int g_page_error;

__device__ __forceinline__ int tokens_of(const TokenArgs& t, int b) {
  const int n = t.n_new ? t.n_new[b] : t.Tq;
  return n < 0 ? 0 : (n > t.Tq ? t.Tq : n);
}

// Lowers a page's count unless it is zero already.
__device__ __forceinline__ void release_page(int32_t* ref, int* err) {
  int32_t old = __ldcg(ref);
  while (old > 0) {
    const int32_t seen = atomicCAS(ref, old, old - 1);
    if (seen == old) return;
    old = seen;
  }
  set_device_error(err, kErrPage);
}

// ----------------------------------------------------------------------------- append
// One CTA per (sequence, page that the call writes, KV head, keys or values): the largest finite new
// value, the page's scale, the new codes, and the earlier tokens' codes once more if the scale grew.
// Each thread holds its part of the page (NV vectors of 8 values, as they came) in registers between the
// two passes, so the new values are read once; earlier codes are read only where the scale grows.  A
// decode step (one token) is bound by latency: the values are loaded beside the page's look-up.
template <int FMT>
__device__ __forceinline__ void unpack8(const uint4* raw, float v[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
  for (int i = 0; i < (FMT == CSA_FMT_F32 ? 8 : 4); ++i) {
    if (FMT == CSA_FMT_F32) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = bf16_bits_to_f(w[i] & 0xFFFFu);
      v[2 * i + 1] = bf16_bits_to_f(w[i] >> 16);
    }
  }
}

__device__ __forceinline__ uint2 encode8(const float v[8], float f) {
  uint2 r;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * f, v[2 * i + 1] * f), __NV_SATFINITE, __NV_E4M3);
  r.x = w[0] | (w[1] << 16);
  r.y = w[2] | (w[3] << 16);
  return r;
}

template <int FMT, int NV>
__global__ void __launch_bounds__(256, FMT == CSA_FMT_F32 ? 2 : 4)
paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  __shared__ float scratch[32];
  uint32_t id = blockIdx.x;
  const int kv = id & 1;
  id >>= 1;
  const int h = id % a.Hkv;
  id /= a.Hkv;
  const int i = id % a.kmax, b = id / a.kmax;
  const int64_t start = a.tok.start[b];
  const int n = tokens_of(a.tok, b);
  if (start < 0 || n == 0) return;
  const int page = a.T.page;
  const int64_t off64 = (start & (page - 1)) - (int64_t)i * page;     // slot of token 0
  if (off64 + n <= 0) return;
  const int off = (int)off64;
  const int64_t p = (start >> a.T.page_log2) + i;
  const int lo = off > 0 ? off : 0, hi = off + n < page ? off + n : page;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int lane8 = a.D >> 3, dlog = a.D == 128 ? 4 : 3;
  // the new values are on their way before the page is looked up: they do not depend on it
  constexpr int kRaw = FMT == CSA_FMT_F32 ? 2 : 1;
  const uint8_t* src = (kv ? a.v_new : a.k_new);
  uint4 raw[NV][kRaw];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int e = u * nt + tid, slot = e >> dlog, c = (e & (lane8 - 1)) * 8;
    const size_t at = ((size_t)b * a.tok.Tq + (slot - off)) * a.kv_stride + (size_t)h * a.D + c;
#pragma unroll
    for (int w = 0; w < kRaw; ++w)
      raw[u][w] = slot >= lo && slot < hi ? __ldg(reinterpret_cast<const uint4*>(src + at * (FMT == CSA_FMT_F32 ? 4 : 2)) + w)
                                          : make_uint4(0u, 0u, 0u, 0u);
  }
  int32_t g = -1;
  if (p < a.T.cap) g = a.T.table[(size_t)b * a.T.cap + p];
  if (g < 0 || g >= a.T.n_pages || (a.T.refs && a.T.refs[g] > 1)) {
    if (tid == 0) set_device_error(a.err, kErrPage);
    return;
  }
  const size_t gh = (size_t)g * a.Hkv + h;
  float* scale_p = (kv ? a.P.vs : a.P.ks) + gh;
  uint8_t* codes = (kv ? a.P.v : a.P.k) + gh * page * a.D;
  const float old = lo > 0 ? *scale_p : 0.f;
  float amax = 0.f;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    float x[8];
    unpack8<FMT>(raw[u], x);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float ax = fabsf(x[w]);
      if (ax < INFINITY) amax = fmaxf(amax, ax);
    }
  }
  amax = block_max(amax, scratch);
  // the smallest power of two s >= 2^-126 with amax / s <= 448 = 0.875 * 2^9
  int ex = -126;
  if (amax > 0.f) {
    int e;
    const float f = frexpf(amax, &e);
    ex = f <= 0.875f ? e - 9 : e - 8;
    if (ex < -126) ex = -126;
  }
  const float need = __uint_as_float((uint32_t)(ex + 127) << 23);
  const float now = fmaxf(need, old);
  if (lo > 0 && now != old) {
    const float ratio = old / now;                   // both powers of two: exact, or far below any code
    for (int e = tid; e < lo << dlog; e += nt) {
      uint2 w = *reinterpret_cast<uint2*>(codes + (size_t)e * 8);
      float y[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        y[q] = e4m3_to_f((uint8_t)(w.x >> (8 * q)));
        y[4 + q] = e4m3_to_f((uint8_t)(w.y >> (8 * q)));
      }
      *reinterpret_cast<uint2*>(codes + (size_t)e * 8) = encode8(y, ratio);
    }
  }
  const float inv = 1.f / now;                       // a power of two: exact
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int e = u * nt + tid, slot = e >> dlog;
    if (slot >= lo && slot < hi) {
      float x[8];
      unpack8<FMT>(raw[u], x);
      *reinterpret_cast<uint2*>(codes + (size_t)e * 8) = encode8(x, inv);
    }
  }
  if (tid == 0 && now != old) *scale_p = now;        // every thread read it before the reduction's barriers
}

// ----------------------------------------------------------------------------- fork
// One CTA per pair.  A pair is taken only if its dst is no src of the call and no dst of an earlier
// pair, so no row is read and written, or written twice.
__global__ void pages_fork_kernel(const __grid_constant__ PageArgs T, const int32_t* __restrict__ src,
                                  const int32_t* __restrict__ dst, int n, int* err) {
  const int i = blockIdx.x;
  const int32_t s = src[i], d = dst[i];
  if (s == -1 && d == -1) return;
  bool clash = s < 0 || s >= T.B || d < 0 || d >= T.B;
  for (int j = threadIdx.x; j < n; j += blockDim.x) clash |= src[j] == d || (j < i && dst[j] == d);
  if (__syncthreads_or(clash)) {
    if (threadIdx.x == 0) set_device_error(err, kErrPage);
    return;
  }
  const int32_t* from = T.table + (size_t)s * T.cap;
  int32_t* to = T.table + (size_t)d * T.cap;
  for (int64_t p = threadIdx.x; p < T.cap; p += blockDim.x) {
    int32_t g = from[p];
    const int32_t was = to[p];
    if (g >= T.n_pages) {
      set_device_error(err, kErrPage);
      g = -1;
    }
    if (g < 0) g = -1;
    if (was == g) continue;
    if (g >= 0) atomicAdd(T.refs + g, 1);
    if (was >= T.n_pages) set_device_error(err, kErrPage);
    else if (was >= 0) release_page(T.refs + was, err);
    to[p] = g;
  }
}

// ----------------------------------------------------------------------------- free
__global__ void pages_free_kernel(const __grid_constant__ PageArgs T, const int64_t* __restrict__ keep,
                                  const int64_t* __restrict__ begin, int64_t first, int* err) {
  for (int b = blockIdx.y; b < T.B; b += gridDim.y) {
    const int64_t k = keep ? keep[b] : -1, w = begin ? begin[b] : -1;
    for (int64_t p = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; p < T.cap;
         p += (int64_t)gridDim.x * blockDim.x) {
      const int64_t t = p << T.page_log2;
      if (!((k >= 0 && t >= k) || (t >= first && t + T.page <= w))) continue;
      int32_t* at = T.table + (size_t)b * T.cap + p;
      const int32_t g = *at;
      if (g == -1) continue;
      if (g >= T.n_pages) set_device_error(err, kErrPage);
      else if (g >= 0) release_page(T.refs + g, err);
      *at = -1;
    }
  }
}

// ----------------------------------------------------------------------------- cluster helpers
// Exclusive prefix of v over the CTA's 1,024 threads, in thread order; *total is the CTA's sum.
__device__ __forceinline__ int block_prefix(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();
  if (lane == 31) scratch[wid] = inc;
  __syncthreads();
  int w = scratch[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += up;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, wid ? wid - 1 : 0);
  return inc - v + (wid ? before : 0);
}

__device__ __forceinline__ int block_count(int v, int* scratch) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, scratch[threadIdx.x & 31]);
}

struct ClusterCounts {
  int64_t total[2];         // over the cluster
  int64_t before[2];        // over the CTAs of lower rank
};

// Gives every CTA of the cluster the sums of (x, y) and the sums over the CTAs before it.  `box` is
// [kCluster][2] in shared memory, used for one exchange only.
__device__ __forceinline__ ClusterCounts exchange(cg::cluster_group& cl, int (*box)[2], int x, int y) {
  const unsigned rank = cl.block_rank();
  if (threadIdx.x < kCluster) {
    int* to = cl.map_shared_rank(&box[rank][0], threadIdx.x);
    to[0] = x;
    to[1] = y;
  }
  cl.sync();
  ClusterCounts c = {{0, 0}, {0, 0}};
#pragma unroll
  for (unsigned r = 0; r < kCluster; ++r)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int v = box[r][q];
      c.total[q] += v;
      if (r < rank) c.before[q] += v;
    }
  return c;
}

// This CTA's part [lo, hi) of n things, in multiples of 4.
__device__ __forceinline__ void my_slice(int64_t n, unsigned rank, int64_t* lo, int64_t* hi) {
  const int64_t per = ((n + kCluster - 1) / kCluster + 3) & ~(int64_t)3;
  *lo = per * rank < n ? per * rank : n;
  *hi = *lo + per < n ? *lo + per : n;
}

// Counts of the four pages from index g on, `fill` from index hi on.
__device__ __forceinline__ int4 load_refs4(const int32_t* refs, int64_t g, int64_t hi, int fill) {
  int4 r = make_int4(fill, fill, fill, fill);
  if (g + 3 < hi) return __ldcg(reinterpret_cast<const int4*>(refs + g));
  if (g < hi) r.x = __ldcg(refs + g);
  if (g + 1 < hi) r.y = __ldcg(refs + g + 1);
  if (g + 2 < hi) r.z = __ldcg(refs + g + 2);
  return r;
}

// ----------------------------------------------------------------------------- reserve
// Entries e = b * kmax + k: the k-th page that row b's new tokens touch.  Whether every holder of a
// page is about to write it shows when each writing entry takes one off the page's count: what is left
// are the holders that do not write.  A count of zero then becomes a mark by an atomic minimum,
// -2^30 - 1 - e, so that the highest entry keeps the page.  The entries that need a page get the marker
// kWanted in the table, and the lowest free pages go to them in entry order, listed in the cluster's
// shared memory kListPer to a CTA (in rounds where that does not hold them all).
constexpr int kListPer = 8192;
constexpr int32_t kWanted = INT32_MIN;
constexpr int32_t kMarkBase = -(1 << 30);

struct ReserveEntry {
  int32_t* at;              // table entry, null where there is nothing to write
  int64_t pos;              // first position of its page
  int64_t start;
  int b, k;
};

__device__ __forceinline__ ReserveEntry reserve_entry(const PagesReserveArgs& a, int e, bool report) {
  ReserveEntry r;
  r.b = e / a.kmax;
  r.k = e - r.b * a.kmax;
  r.at = nullptr;
  r.start = a.tok.start[r.b];
  const int n = tokens_of(a.tok, r.b);
  if (r.start < 0 || n == 0) return r;
  if (r.start > (a.T.cap << a.T.page_log2) - n) {
    if (report && r.k == 0) set_device_error(a.err, kErrPage);
    return r;
  }
  const int64_t p = (r.start >> a.T.page_log2) + r.k;
  r.pos = p << a.T.page_log2;
  if (r.pos >= r.start + n) return r;
  r.at = a.T.table + (size_t)r.b * a.T.cap + p;
  return r;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
pages_reserve_kernel(const __grid_constant__ PagesReserveArgs a) {
  __shared__ int scratch[32];
  __shared__ int box[3][kCluster][2];
  __shared__ int32_t list[kListPer];
  cg::cluster_group cl = cg::this_cluster();
  const unsigned rank = cl.block_rank();
  const int tid = threadIdx.x;
  const int total_e = a.T.B * a.kmax;                     // < 2^30 (checked on the host)
  int64_t e_lo, e_hi, g_lo, g_hi;
  my_slice(total_e, rank, &e_lo, &e_hi);
  my_slice(a.T.n_pages, rank, &g_lo, &g_hi);
  int32_t* refs = a.T.refs;

  // 1: every writing entry takes one off its page's count
  for (int64_t e = e_lo + tid; e < e_hi; e += kThreads) {
    const ReserveEntry r = reserve_entry(a, (int)e, true);
    if (r.k == 0) {
      a.copy_src[r.b] = -1;
      a.copy_dst[r.b] = -1;
    }
    if (!r.at) continue;
    const int32_t g = *r.at;
    if (g >= a.T.n_pages) set_device_error(a.err, kErrPage);
    else if (g >= 0) atomicSub(refs + g, 1);
  }
  cl.sync();
  // 2: pages that nobody else holds go to their highest entry
  for (int64_t e = e_lo + tid; e < e_hi; e += kThreads) {
    const ReserveEntry r = reserve_entry(a, (int)e, false);
    if (!r.at) continue;
    const int32_t g = *r.at;
    if (g < 0 || g >= a.T.n_pages) continue;
    if (__ldcg(refs + g) <= 0) {
      const int32_t was = atomicMin(refs + g, kMarkBase - 1 - (int32_t)e);
      if (was < 0 && was > kMarkBase) set_device_error(a.err, kErrPage);    // more entries than the count said
    }
  }
  cl.sync();
  // 3: how many pages are needed, how many are free
  int need = 0, have = 0;
  for (int64_t e = e_lo + tid; e < e_hi; e += kThreads) {
    const ReserveEntry r = reserve_entry(a, (int)e, false);
    if (!r.at) continue;
    const int32_t g = *r.at;
    if (g < a.T.n_pages) need += g < 0 || __ldcg(refs + g) != kMarkBase - 1 - (int32_t)e;
  }
  for (int64_t g = g_lo + 4 * tid; g < g_hi; g += 4 * kThreads) {
    const int4 r = load_refs4(refs, g, g_hi, 1);
    have += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  need = block_count(need, scratch);
  have = block_count(have, scratch);
  ClusterCounts c = exchange(cl, box[0], need, have);
  if (rank == 0 && tid == 0) *a.missing = c.total[0] > c.total[1] ? (int32_t)(c.total[0] - c.total[1]) : 0;
  if (c.total[0] > c.total[1]) {
    // too few: the counts are put back (marks to zero, then one per entry)
    for (int64_t e = e_lo + tid; e < e_hi; e += kThreads) {
      const ReserveEntry r = reserve_entry(a, (int)e, false);
      if (!r.at) continue;
      const int32_t g = *r.at;
      if (g >= 0 && g < a.T.n_pages && __ldcg(refs + g) == kMarkBase - 1 - (int32_t)e) refs[g] = 0;
    }
    cl.sync();
    for (int64_t e = e_lo + tid; e < e_hi; e += kThreads) {
      const ReserveEntry r = reserve_entry(a, (int)e, false);
      if (!r.at) continue;
      const int32_t g = *r.at;
      if (g >= 0 && g < a.T.n_pages) atomicAdd(refs + g, 1);
    }
    return;                                              // nobody reads another CTA's memory any more
  }
  // 4: markers in the table, the kept pages' counts
  for (int64_t e = e_lo + tid; e < e_hi; e += kThreads) {
    const ReserveEntry r = reserve_entry(a, (int)e, false);
    if (!r.at) continue;
    const int32_t g = *r.at;
    if (g >= a.T.n_pages) continue;
    if (g >= 0 && __ldcg(refs + g) == kMarkBase - 1 - (int32_t)e) {
      refs[g] = 1;                                       // another entry of g sees 1 or the mark: not its own
      continue;
    }
    if (g >= 0 && r.k == 0 && r.pos < r.start) a.copy_src[r.b] = g;
    *r.at = kWanted;
  }
  // 5: the lowest free pages, in entry order
  int64_t left = c.total[0];
  for (int round = 0; left > 0; ++round) {
    const int64_t take = left < (int64_t)kCluster * kListPer ? left : (int64_t)kCluster * kListPer;
    if (round > 0) {                                     // marked entries and free pages that are left
      need = have = 0;
      for (int64_t e = e_lo + tid; e < e_hi; e += kThreads) {
        const ReserveEntry r = reserve_entry(a, (int)e, false);
        need += r.at && *r.at == kWanted;
      }
      for (int64_t g = g_lo + 4 * tid; g < g_hi; g += 4 * kThreads) {
        const int4 r = load_refs4(refs, g, g_hi, 1);
        have += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
      }
      need = block_count(need, scratch);
      have = block_count(have, scratch);
      c = exchange(cl, box[1 + (round & 1)], need, have);
    }
    int64_t at = c.before[1];
    for (int64_t g0 = g_lo; g0 < g_hi && at < take; g0 += 4 * kThreads) {
      const int64_t g = g0 + 4 * tid;
      const int4 r = load_refs4(refs, g, g_hi, 1);
      const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
      int sum;
      int64_t k = at + block_prefix(f[0] + f[1] + f[2] + f[3], scratch, &sum);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (f[q]) {
          if (k < take) *cl.map_shared_rank(&list[k % kListPer], (unsigned)(k / kListPer)) = (int32_t)(g + q);
          ++k;
        }
      at += sum;
    }
    cl.sync();
    int64_t w = c.before[0];
    for (int64_t e0 = e_lo; e0 < e_hi && w < take; e0 += kThreads) {
      const int64_t e = e0 + tid;
      ReserveEntry r;
      r.at = nullptr;
      if (e < e_hi) r = reserve_entry(a, (int)e, false);
      const bool mine = r.at && *r.at == kWanted;
      int sum;
      const int64_t k = w + block_prefix(mine ? 1 : 0, scratch, &sum);
      if (mine && k < take) {
        const int32_t g = *cl.map_shared_rank(&list[k % kListPer], (unsigned)(k / kListPer));
        *r.at = g;
        refs[g] = 1;
        if (r.k == 0 && a.copy_src[r.b] >= 0) a.copy_dst[r.b] = g;
      }
      w += sum;
    }
    cl.sync();
    left -= take;
  }
}

// ----------------------------------------------------------------------------- compact
// With U pages in use, the pages at U and above that are in use (M of them) move, the highest first,
// into the M free pages below U, the lowest first.  Three passes over the counts: U; the ranks' sums
// over the CTAs; the lists.
__device__ __forceinline__ void rewrite_entry(const PagesCompactArgs& a, int32_t* at, int m, int32_t lowest) {
  const int32_t g = *at;
  if (g < lowest) return;
  if (g >= a.T.n_pages) {
    set_device_error(a.err, kErrPage);
    return;
  }
  int lo = 0, hi = m - 1;                                // move_src descends
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(a.move_src + mid) <= g) hi = mid;
    else lo = mid + 1;
  }
  if (__ldcg(a.move_src + lo) == g) *at = __ldcg(a.move_dst + lo);
  else set_device_error(a.err, kErrPage);                // the table names a page whose count is zero
}

// Tables up to this many entries are rewritten by the cluster itself, larger ones by a second launch
// over all SMs.
constexpr int64_t kRewriteHere = 32768;

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
pages_compact_kernel(const __grid_constant__ PagesCompactArgs a) {
  __shared__ int scratch[32];
  __shared__ int box[2][kCluster][2];
  cg::cluster_group cl = cg::this_cluster();
  const unsigned rank = cl.block_rank();
  const int tid = threadIdx.x;
  int32_t* refs = a.T.refs;
  int64_t g_lo, g_hi;
  my_slice(a.T.n_pages, rank, &g_lo, &g_hi);
  cl.sync();                                             // every CTA runs before its memory is written
  int used = 0;
  for (int64_t g = g_lo + 4 * tid; g < g_hi; g += 4 * kThreads) {
    const int4 r = load_refs4(refs, g, g_hi, 0);
    used += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  used = block_count(used, scratch);
  const int64_t U = exchange(cl, box[0], used, 0).total[0];
  int below = 0, above = 0;
  for (int64_t g = g_lo + 4 * tid; g < g_hi; g += 4 * kThreads) {
    const int4 r = load_refs4(refs, g, g_hi, 0);
    const int v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      below += g + q < g_hi && g + q < U && v[q] <= 0;
      above += g + q < g_hi && g + q >= U && v[q] > 0;
    }
  }
  below = block_count(below, scratch);
  above = block_count(above, scratch);
  const ClusterCounts c = exchange(cl, box[1], below, above);
  const int64_t M = c.total[1];
  const int m = (int)(M < a.max_moves ? M : a.max_moves);
  int64_t nb = c.before[0], na = c.before[1];
  for (int64_t g0 = g_lo; g0 < g_hi; g0 += 4 * kThreads) {
    const int64_t g = g0 + 4 * tid;
    const int4 r = load_refs4(refs, g, g_hi, 0);
    const int v[4] = {r.x, r.y, r.z, r.w};
    int fb = 0, fa = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      fb += g + q < g_hi && g + q < U && v[q] <= 0;
      fa += g + q < g_hi && g + q >= U && v[q] > 0;
    }
    int sum;
    // both ranks in one scan: at most 4,096 of each
    const int pre = block_prefix(fb | (fa << 16), scratch, &sum);
    int64_t kb = nb + (pre & 0xFFFF), ka = na + (pre >> 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (g + q < g_hi && g + q < U && v[q] <= 0) {
        if (kb < m) a.move_dst[kb] = (int32_t)(g + q);
        ++kb;
      }
      if (g + q < g_hi && g + q >= U && v[q] > 0) {
        const int64_t i = M - 1 - ka;
        if (i < m) a.move_src[i] = (int32_t)(g + q);
        ++ka;
      }
    }
    nb += sum & 0xFFFF;
    na += sum >> 16;
  }
  for (int64_t i = m + (int64_t)rank * kThreads + tid; i < a.max_moves; i += (int64_t)kCluster * kThreads) {
    a.move_src[i] = -1;
    a.move_dst[i] = -1;
  }
  if (rank == 0 && tid == 0) *a.count = m;
  cl.sync();
  for (int64_t i = (int64_t)rank * kThreads + tid; i < m; i += (int64_t)kCluster * kThreads) {
    const int32_t s = __ldcg(a.move_src + i), d = __ldcg(a.move_dst + i);
    refs[d] = refs[s];
    refs[s] = 0;
  }
  const int64_t entries = (int64_t)a.T.B * a.T.cap;
  if (entries <= kRewriteHere && m > 0) {
    const int32_t lowest = __ldcg(a.move_src + m - 1);
    for (int64_t i = (int64_t)rank * kThreads + tid; i < entries; i += (int64_t)kCluster * kThreads)
      rewrite_entry(a, a.T.table + i, m, lowest);
  }
}

__global__ void pages_rewrite_kernel(const __grid_constant__ PagesCompactArgs a) {
  const int m = *a.count;
  if (m <= 0) return;
  const int32_t lowest = a.move_src[m - 1];
  const int64_t entries = (int64_t)a.T.B * a.T.cap;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < entries; i += (int64_t)gridDim.x * blockDim.x)
    rewrite_entry(a, a.T.table + i, m, lowest);
}

// ----------------------------------------------------------------------------- copy
// Pieces of 32 KB of a page's keys or values, eight 16-byte loads in flight per thread; the CTAs walk the pieces
// of all pairs, the next piece's pages on their way while a piece is copied.  900 pages of 128 KB: 45 us (5.2
// TB/s); with pieces of 16 KB 49 us, of 4 KB (16 CTAs per SM) 50.
constexpr int kPiece = 32768;
constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = kPiece / 16 / kCopyThreads;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PagesCopyArgs a) {
  int n = a.n;
  if (a.count) {
    const int c = *a.count;
    n = c < n ? c : n;
  }
  const int per = (int)((a.page_bytes + kPiece - 1) / kPiece);
  const int64_t items = (int64_t)n * 2 * per;
  if (blockIdx.x >= items) return;
  int i = (int)(blockIdx.x / (2 * per)), r = (int)(blockIdx.x - (int64_t)i * 2 * per);
  const int step_i = (int)(gridDim.x / (2 * per)), step_r = (int)(gridDim.x - (int64_t)step_i * 2 * per);
  int32_t s = a.src[i], d = a.dst[i];
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int kv = r >= per, c = kv ? r - per : r;
    const int32_t from_page = s, to_page = d;
    i += step_i;
    r += step_r;
    if (r >= 2 * per) {
      r -= 2 * per;
      ++i;
    }
    if (it + gridDim.x < items) {
      s = a.src[i];
      d = a.dst[i];
    }
    if (from_page < 0 || to_page < 0) continue;
    if (from_page >= a.n_pages || to_page >= a.n_pages) {
      if (threadIdx.x == 0) set_device_error(a.err, kErrPage);
      continue;
    }
    uint8_t* base = kv ? a.P.v : a.P.k;
    const uint8_t* from = base + (size_t)from_page * a.page_bytes + (size_t)c * kPiece;
    uint8_t* to = base + (size_t)to_page * a.page_bytes + (size_t)c * kPiece;
    const int64_t bytes = a.page_bytes - (int64_t)c * kPiece;
    uint4 x[kCopyLoads];
#pragma unroll
    for (int u = 0; u < kCopyLoads; ++u) {
      const int o = (u * kCopyThreads + threadIdx.x) * 16;
      if (o < bytes) x[u] = *reinterpret_cast<const uint4*>(from + o);
    }
#pragma unroll
    for (int u = 0; u < kCopyLoads; ++u) {
      const int o = (u * kCopyThreads + threadIdx.x) * 16;
      if (o < bytes) *reinterpret_cast<uint4*>(to + o) = x[u];
    }
    if (c == 0) {
      float* sc = kv ? a.P.vs : a.P.ks;
      for (int h = threadIdx.x; h < a.Hkv; h += kCopyThreads)
        sc[(size_t)to_page * a.Hkv + h] = sc[(size_t)from_page * a.Hkv + h];
    }
  }
}

}  // namespace

cudaError_t page_error_word(int** p) {
  static std::mutex mu;
  static int* addr[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* q = nullptr;
    e = cudaGetSymbolAddress(&q, g_page_error);
    if (e != cudaSuccess) return e;
    addr[dev] = static_cast<int*>(q);
  }
  *p = addr[dev];
  return cudaSuccess;
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
  const int vec = a.T.page * a.D / 8;                    // 128 .. 2048 vectors of 8 values per (page, head)
  const int nv = vec >= 256 ? 8 : 4;
  const unsigned grid = (unsigned)((int64_t)a.T.B * a.kmax * a.Hkv * 2);
  const dim3 block(vec / nv);
  if (a.act_fmt == CSA_FMT_F32)
    return nv == 8 ? launch_kernel(paged_append_kernel<CSA_FMT_F32, 8>, dim3(grid), block, 0, s, 0, a)
                   : launch_kernel(paged_append_kernel<CSA_FMT_F32, 4>, dim3(grid), block, 0, s, 0, a);
  return nv == 8 ? launch_kernel(paged_append_kernel<CSA_FMT_BF16, 8>, dim3(grid), block, 0, s, 0, a)
                 : launch_kernel(paged_append_kernel<CSA_FMT_BF16, 4>, dim3(grid), block, 0, s, 0, a);
}

cudaError_t launch_pages_fork(const PageArgs& T, const int32_t* src, const int32_t* dst, int n, int* err,
                              cudaStream_t s) {
  return launch_kernel(pages_fork_kernel, dim3(n), dim3(256), 0, s, 0, T, src, dst, n, err);
}

cudaError_t launch_pages_reserve(const PagesReserveArgs& a, cudaStream_t s) {
  return launch_kernel(pages_reserve_kernel, dim3(kCluster), dim3(kThreads), 0, s, 0, a);
}

cudaError_t launch_pages_free(const PageArgs& T, const int64_t* keep, const int64_t* begin, int64_t first, int* err,
                              cudaStream_t s) {
  const int64_t gx = (T.cap + 255) / 256;
  const dim3 grid((unsigned)(gx < 1024 ? gx : 1024), (unsigned)(T.B < 4096 ? T.B : 4096));
  return launch_kernel(pages_free_kernel, grid, dim3(256), 0, s, 0, T, keep, begin, first, err);
}

cudaError_t launch_pages_compact(const PagesCompactArgs& a, cudaStream_t s) {
  cudaError_t e = launch_kernel(pages_compact_kernel, dim3(kCluster), dim3(kThreads), 0, s, 0, a);
  const int64_t entries = (int64_t)a.T.B * a.T.cap;
  if (e == cudaSuccess && entries > kRewriteHere && a.max_moves > 0) {
    const int64_t g = (entries + 1023) / 1024;
    e = launch_kernel(pages_rewrite_kernel, dim3((unsigned)(g < 2048 ? g : 2048)), dim3(256), 0, s, 0, a);
  }
  return e;
}

cudaError_t launch_pages_copy(const PagesCopyArgs& a, int num_sms, cudaStream_t s) {
  const int64_t items = (int64_t)a.n * 2 * ((a.page_bytes + kPiece - 1) / kPiece);
  const int64_t most = (int64_t)num_sms * 8;
  return launch_kernel(pages_copy_kernel, dim3((unsigned)(items < most ? items : most)), dim3(kCopyThreads),
                       0, s, 0, a);
}

}  // namespace csa
