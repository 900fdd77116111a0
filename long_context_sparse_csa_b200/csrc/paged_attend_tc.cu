// Attention over the paged 8-bit cache on tcgen05 (definition: csa_paged_attend in csa.h): blocks of
// many query rows (prompt chunks, many speculative tokens), bf16 activations.
//
// What bounds it.  With hundreds of rows per KV head the products are 4 D flops per (row, key): the
// tensor core, and beside it the exponentials (one per 4 D = 512 flops at D = 128: at 16 a clock the
// same 2,048 clocks per 256 x 128 tile that the products take).  Two groups of 128 rows work in turns:
// while one group's softmax runs, the tensor core works for the other.  Measured, 2,048 tokens of 64 heads of
// 128 dims behind 14,336: 1,248-1,288 us, 800-826 TFLOP/s (half of the bf16 peak), 5,000 clocks a tile; the tensor
// pipe is active 40 % of the time, the exponential unit 34 %, issue slots 42 %: no unit is full, the softmax
// warps' latencies and the half tiles' products (96 KB of shared memory reads each) add up.
//
// Mathematics.  S = q K^T and O += P V with M = 128 query rows, f16 operands (e4m3 codes are exact in
// f16; queries scaled per row by a power of two), f32 sums in tensor memory; P stays in tensor memory,
// over S's columns, as the A operand of the second product.  Scales and the two running maxima as in
// the warp-level kernel: O sums 2^(z + v - mw + 4) codes, z the logit in log2 units and v the log2 of the
// page's value scale; the denominator sums 2^(z - mz).  One exponential serves both: per 16 keys of a
// page the weights' sum times 2^(mw - mz - v - 4), unless that factor is beyond 2^80 (pages' scales
// very far apart), where the denominators' exponentials are taken apart and the denominator's maximum follows
// logits more than 40 above it.  O's maximum, and with it the other, moves only when some keys exceed it by
// more than 11 (then O is rescaled in tensor memory), so P stays up to 2^15 and keeps its
// 11 bits down to 2^-18 of the largest weight (2^-29 of it below that, rounded either way).
//
// Roles (640 threads): warp 0 issues q K^T, warp 2 P V; warp 1 looks up the tiles' pages and scales; warps 4-7
// and 8-11 are the two groups' softmax, a thread a row; warps 12-15 convert K tiles, warps 16-19 V tiles:
// 16-byte loads of codes, one tile ahead in registers, to f16 in the 128-byte swizzle (two stages each).
// With more than 128 rows (kPair) the groups take different rows of the same tile; otherwise the same rows of
// alternate tiles, joined at the end.  A group works through half tiles in two buffers of S: while it
// weighs one, the other's scores are computed (one buffer of whole tiles: 1,460 us against 1,434).  P lies
// over its S, so the next S there waits for the product that reads it.
#include <type_traits>

#include "paged_walk.cuh"
#include "sm100.cuh"

namespace csa {

namespace {

using namespace sm100;

constexpr int kKeys = 128;
constexpr int kThreads = 640;
constexpr int kSubs = kKeys / 16;
constexpr int kMeta = 8;                        // tiles looked up ahead, four at a time
constexpr float kShift = 4.f;                   // P = 2^(weight + kShift), at most 2^15: a margin of 11
constexpr int kRegsLaunch = 96, kRegsSoftmax = 128, kRegsConvert = 72, kRegsIssue = 80;
static_assert(256 * kRegsSoftmax + 256 * kRegsConvert + 128 * kRegsIssue <= kThreads * kRegsLaunch, "register split");

struct __align__(8) TcBars {
  uint64_t kfull[2], kfree[2], vfull[2], vfree[2];
  uint64_t qfull[2], ofree[2];
  uint64_t sfull[2][2], pfull[2][2], pvdone[2][2];      // [group][S buffer]
  uint64_t recfull, recfree;
  uint64_t mfull[kMeta], mfree[kMeta];
  uint64_t part0;                             // the first part is published (the others with their first tiles)
  uint32_t tmem_base;
};

// What the other roles need of a key tile, looked up ahead by one warp.
struct __align__(16) TileMeta {
  int32_t page[kSubs];                        // page of each 16 keys, -1: none
  float ks[kSubs], lv[kSubs];                 // key scale, log2 of the value scale
  float lv_min[2];                            // the smallest lv of each half
  int pos, h;                                 // first position, KV head
  int index;                                  // number of the tile in its part
  int whole;                                  // every row of the block sees every key
  uint32_t have;                              // bits: the 16 keys have a page
};

// The tensor core cuts its sums off instead of rounding them: one chain of products over 1,048,576 keys came out
// 6.4e-3 too small, more than bf16's half step.  So a part of more tiles than this is worked through in pieces, whose
// sums are added up rounded in the CTA's record (2,048 products: 2e-4 at most; 256 tiles take 0.7 ms, a piece's end 5 us).
constexpr int kPieceTiles = 256;

// A piece of a CTA's part of a segment.
struct Part {
  Seg s;
  int sb, part0, unit0, tiles;                // first tile of the part, of the piece; tiles of the piece
  bool last;                                  // of the part's pieces
  bool complete;                              // the last, of a part that is the whole segment
};

// Walks the parts of a CTA's run.  (units are single tiles here)
struct Parts {
  Walk w;
  int part0;
  int64_t left;
};

// Parts that the looking-up warp has published.  It is at most kMeta tiles ahead of the softmax, and the softmax
// holds the part that it ends, so that twice as many entries need no waits of their own.
constexpr int kParts = 2 * kMeta;

template <int D>
struct TcShape {
  static constexpr int kHalf = kKeys * 128;                   // 128 rows of 64 f16 values
  static constexpr int kTileBytes = kHalf * (D / 64);
  static constexpr size_t kOffK = 2 * (size_t)kTileBytes;     // after the two groups' queries
  static constexpr size_t kOffV = 4 * (size_t)kTileBytes;
  static constexpr size_t kOffCq = 6 * (size_t)kTileBytes;    // [2][128] logit factor of a row
  static constexpr size_t kOffNan = kOffCq + 2 * 128 * 4;     // [2 stages][32] NaN flags of V's rows, four to a byte
  static constexpr size_t kOffBars = kOffNan + 64;
  static constexpr size_t kOffMeta = (kOffBars + sizeof(TcBars) + 15) / 16 * 16;
  static constexpr size_t kOffParts = kOffMeta + kMeta * sizeof(TileMeta);
  static constexpr size_t kBytes = 1024 + kOffParts + kParts * sizeof(Part);
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t sw128(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The products are issued by one lane of a warp that runs as a whole (`lead`: this lane issues), so that
// descriptors and addresses stay in uniform registers: 1,654 us -> 1,460 us for the chunk of 2,048
// tokens behind 14,336, against a loop that one lane ran alone.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// D[tmem] (+)= A[smem] * B[smem]^T, f16 inputs, fp32 accumulate.
__device__ __forceinline__ void umma_ss(uint32_t lead, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

// The same with A in tensor memory: two f16 values of a row per 32-bit column.
__device__ __forceinline__ void umma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// A whole warp's look at a barrier, and its bounded wait: true for all its lanes or for none.
__device__ __forceinline__ bool warp_try(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  if (warp_try(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  bool more;
  do {
    if (warp_try(bar, parity)) return true;
    more = global_timer_ns() - t0 < kWaitLimitNs;
  } while (__all_sync(0xffffffffu, more));
  return false;
}

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void parts_start(const PagedAttendArgs& a, Parts& p, const Run& run, int row_tile) {
  walk_start(a, p.w, run, row_tile, kKeys, 1);
  p.part0 = p.w.unit;
  p.left = run.u1 - run.u0;
}

__device__ __forceinline__ bool parts_next(const PagedAttendArgs& a, Parts& p, Part& out, int row_tile) {
  if (p.left <= 0) return false;
  out.s = p.w.s;
  out.sb = p.w.sb;
  out.part0 = p.part0;
  out.unit0 = p.w.unit;
  const int rest = p.w.s.units - p.w.unit;
  const int mine = p.left < rest ? (int)p.left : rest;
  out.tiles = mine < kPieceTiles ? mine : kPieceTiles;
  out.last = out.tiles == mine;
  out.complete = p.part0 == 0 && out.tiles == rest;
  p.left -= out.tiles;
  if (p.left > 0) {
    p.w.unit += out.tiles - 1;
    walk_next(a, p.w, row_tile, kKeys, 1);
    if (out.last) p.part0 = p.w.unit;
  }
  return true;
}

// First and last position of the block's tokens.
__device__ __forceinline__ void row_span(const PagedAttendArgs& a, const Seg& s, int row_tile, int* tmin, int* tmax) {
  const int j1 = (s.rb * row_tile + row_tile - 1) / a.G;
  *tmin = s.start + s.j0;
  *tmax = s.start + (j1 < s.n ? j1 : s.n - 1);
}

__device__ __forceinline__ bool sees_all(const PagedAttendArgs& a, int pos, int tmin, int tmax) {
  return pos + kKeys - 1 <= tmin && (a.window == 0 || pos > tmax - a.window || pos + kKeys <= a.first);
}

// Bits c <= x of 32.
__device__ __forceinline__ uint32_t bits_to(int x) { return x < 0 ? 0u : (x >= 31 ? 0xffffffffu : (2u << x) - 1u); }

// kW: keys that certainly share a page's scales, 16 or 32 (32 from pages of 32 on: half the work per scale).
template <int D, bool kPair, int kW>
__global__ void __launch_bounds__(kThreads, 1) paged_attend_tc_kernel(const __grid_constant__ PagedAttendArgs a) {
  using S = TcShape<D>;
  constexpr int kRowTile = kPair ? 256 : 128;
  constexpr int kHalves = D / 64;
  extern __shared__ uint8_t tc_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tc_smem_raw) + 1023) & ~uintptr_t(1023));
  float* cqs = reinterpret_cast<float*>(sm + S::kOffCq);
  uint8_t* nans = sm + S::kOffNan;
  TcBars* bars = reinterpret_cast<TcBars*>(sm + S::kOffBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->kfull[i], 128);
      mbar_init(&bars->kfree[i], 1);
      mbar_init(&bars->vfull[i], 128);
      mbar_init(&bars->vfree[i], 1);
      mbar_init(&bars->qfull[i], 128);
      for (int u = 0; u < 2; ++u) {
        mbar_init(&bars->sfull[i][u], 1);
        mbar_init(&bars->pfull[i][u], 128);
        mbar_init(&bars->pvdone[i][u], 1);
      }
      mbar_init(&bars->ofree[i], 128);
    }
    mbar_init(&bars->recfull, 128);
    mbar_init(&bars->recfree, 128);
    mbar_init(&bars->part0, 1);
    for (int i = 0; i < kMeta; ++i) {
      mbar_init(&bars->mfull[i], kSubs);
      mbar_init(&bars->mfree[i], 18);                    // the 10 warps that copy and issue, 8 of the softmax (see below)
    }
    fence_barrier_init();
  }
  const Run run = find_run(a, kRowTile, kKeys, 1, 4);
  if (run.u0 >= run.u1) return;
  if (warp == 0) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  TileMeta* metas = reinterpret_cast<TileMeta*>(sm + S::kOffMeta);
  const int64_t run_tiles = run.u1 - run.u0;
  Part* part_ring = reinterpret_cast<Part*>(sm + S::kOffParts);

  if (warp < 4) {
    // ------------------------------------------------------------------ the products
    regs_dec<kRegsIssue>();
    if (warp == 0) {
      // S = q K^T, a half tile at a time into the group's two buffers in turns
      const uint32_t idesc = instr_desc(128, 64, 0u), lead = elect_lane();
      const uint64_t q_desc = desc_kmajor_sw128(smem_u32(sm));
      const uint64_t k_desc = desc_kmajor_sw128(smem_u32(sm + S::kOffK));
      bool ok = true;
      uint32_t cnt[2] = {0, 0}, qpar[2] = {0, 0};            // the groups' jobs so far, parity of their queries
      auto qk = [&](int g, int half, uint32_t st, bool first) {
        if (first) {
          ok = ok && warp_wait(&bars->qfull[g], qpar[g]);
          qpar[g] ^= 1u;
        }
        // the buffer's last P has been read
        const uint32_t buf = cnt[g] & 1u;
        ok = ok && warp_wait(&bars->pvdone[g][buf], ((cnt[g] >> 1) & 1u) ^ 1u);
        if (!ok) return;
        ++cnt[g];
        tc_fence_after();
        const uint64_t qd = q_desc + (uint64_t)(g * (S::kTileBytes >> 4));
        const uint64_t kd = k_desc + (uint64_t)(st * (S::kTileBytes >> 4) + half * 512u);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss(lead, tmem + g * 128u + 64u * buf, qd + (uint64_t)(h * (S::kHalf >> 4) + 2 * kk),
                    kd + (uint64_t)(h * (S::kHalf >> 4) + 2 * kk), idesc, (h | kk) ? 1u : 0u);
        commit_if(lead, &bars->sfull[g][buf]);
      };
      const uint32_t total = (uint32_t)run_tiles;
#pragma unroll 1
      for (uint32_t n = 0; n < total && ok; ++n) {
        ok = warp_wait(&bars->kfull[n & 1u], (n >> 1) & 1u);
        if (!ok) break;
        const int idx = metas[n % kMeta].index;              // the conversion has seen the entry
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->mfree[n % kMeta]);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (kPair) {
            qk(0, half, n & 1u, idx + half == 0);
            qk(1, half, n & 1u, idx + half == 0);
          } else if (idx & 1) {
            qk(1, half, n & 1u, idx < 2 && half == 0);
          } else {
            qk(0, half, n & 1u, idx < 2 && half == 0);
          }
        }
        commit_if(lead, &bars->kfree[n & 1u]);
      }
      if (!ok) set_device_error(a.err, kErrWaitTimeout);
      // nothing of this warp is in flight when tensor memory is released
      for (int g = 0; g < 2; ++g)
        if (cnt[g] > 0) warp_wait(&bars->sfull[g][(cnt[g] - 1) & 1u], ((cnt[g] - 1) >> 1) & 1u);
    } else if (warp == 2) {
      // O += P V
      const uint32_t idesc = instr_desc(128, D, 0u) | (1u << 16), lead = elect_lane();        // V: dims-major
      const uint64_t v_desc = desc_mnmajor_sw128(smem_u32(sm + S::kOffV), S::kHalf, 1024u);
      bool ok = true;
      uint32_t cnt[2] = {0, 0}, opar[2] = {0, 0};
      auto pv = [&](int g, int half, uint32_t st, bool first) {
        if (first) {                                         // O of the group's last part has been read
          ok = ok && warp_wait(&bars->ofree[g], opar[g] ^ 1u);
          opar[g] ^= 1u;
        }
        const uint32_t buf = cnt[g] & 1u;
        ok = ok && warp_wait(&bars->pfull[g][buf], (cnt[g] >> 1) & 1u);
        if (!ok) return;
        ++cnt[g];
        tc_fence_after();
        const uint64_t vd = v_desc + (uint64_t)(st * (S::kTileBytes >> 4) + half * 512u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ts(lead, tmem + 256u + (uint32_t)(g * D), tmem + g * 128u + 64u * buf + 8u * kk,
                  vd + (uint64_t)((kk * 2048) >> 4), idesc, (first && kk == 0) ? 0u : 1u);
        commit_if(lead, &bars->pvdone[g][buf]);
      };
      const uint32_t total = (uint32_t)run_tiles;
#pragma unroll 1
      for (uint32_t n = 0; n < total && ok; ++n) {
        ok = warp_wait(&bars->vfull[n & 1u], (n >> 1) & 1u);
        if (!ok) break;
        const int idx = metas[n % kMeta].index;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->mfree[n % kMeta]);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (kPair) {
            pv(0, half, n & 1u, idx + half == 0);
            pv(1, half, n & 1u, idx + half == 0);
          } else if (idx & 1) {
            pv(1, half, n & 1u, idx < 2 && half == 0);
          } else {
            pv(0, half, n & 1u, idx < 2 && half == 0);
          }
        }
        commit_if(lead, &bars->vfree[n & 1u]);
      }
      if (!ok) set_device_error(a.err, kErrWaitTimeout);
      for (int g = 0; g < 2; ++g)
        if (cnt[g] > 0) warp_wait(&bars->pvdone[g][(cnt[g] - 1) & 1u], ((cnt[g] - 1) >> 1) & 1u);
    } else if (warp == 1) {
      // ---------------------------------------------------------------- pages and scales, four tiles at a time
      bool ok = true;
      int i = 0, tmin = 0, tmax = 0, parts_so_far = 0;
      Parts walk;
      Part pt;
      parts_start(a, walk, run, kRowTile);
      pt.tiles = 0;
#pragma unroll 1
      for (int64_t n0 = 0; n0 < run_tiles; n0 += 4) {
        int pos = 0, h = 0, b = 0, limit = 0, index = 0;
        bool all = false;
#pragma unroll 1
        for (int k = 0; k < 4 && n0 + k < run_tiles; ++k, ++i) {
          if (i == pt.tiles) {
            i = 0;
            parts_next(a, walk, pt, kRowTile);
            row_span(a, pt.s, kRowTile, &tmin, &tmax);
            if (lane == 0) {
              part_ring[parts_so_far % kParts] = pt;
              if (parts_so_far == 0) mbar_arrive(&bars->part0);
            }
            ++parts_so_far;
            __syncwarp();
          }
          if ((lane >> 3) == k) {
            const int p0 = tile_pos(pt.s, pt.unit0 + i, kKeys);
            all = sees_all(a, p0, tmin, tmax);
            pos = p0;
            h = pt.s.h;
            index = i;
            b = pt.s.b;
            limit = pt.s.start + pt.s.n;
          }
        }
        __syncwarp();
        const bool mine = n0 + (lane >> 3) < run_tiles;
        const int u = lane & 7, at = pos + 16 * u;
        int32_t pg = -1;
        if (mine && at < limit) pg = a.T.table[(size_t)b * a.T.cap + (at >> a.T.page_log2)];
        if (pg >= a.T.n_pages) {
          set_device_error(a.err, kErrPage);
          pg = -1;
        }
        if (pg < 0) pg = -1;
        float ks = 0.f, vs = 1.f;
        if (pg >= 0) {
          const size_t gh = (size_t)pg * a.Hkv + h;
          ks = a.P.ks[gh];
          vs = a.P.vs[gh];
          // the codes on their way to L2: the converting warps hold one tile ahead, too little for the latency of
          // memory where few rows leave little else to do (4 tokens over 524,288 keys: 404 -> 393 us)
          const size_t code = (gh * a.T.page + (at & (a.T.page - 1))) * D;
          prefetch_l2(a.P.k + code, 16 * D);
          prefetch_l2(a.P.v + code, 16 * D);
        }
        const uint32_t have = (__ballot_sync(0xffffffffu, pg >= 0) >> (lane & 24)) & 0xFFu;
        const float lv = (float)((int)((__float_as_uint(vs) >> 23) & 255u) - 127);
        float lm = fminf(lv, __shfl_xor_sync(0xffffffffu, lv, 1));
        lm = fminf(lm, __shfl_xor_sync(0xffffffffu, lm, 2));
        const int e = (int)((n0 + (lane >> 3)) & (kMeta - 1));
        bool w = true;
        if (mine) w = mbar_wait(&bars->mfree[e], (uint32_t)(((n0 + (lane >> 3)) / kMeta) & 1) ^ 1u);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        if (mine) {
          TileMeta& m = metas[e];
          m.page[u] = pg;
          m.ks[u] = ks;
          m.lv[u] = lv;
          if ((u & 3) == 0) m.lv_min[u >> 2] = lm;
          if (u == 0) {
            m.pos = pos;
            m.h = h;
            m.index = index;
            m.whole = all && have == 0xFFu;
            m.have = have;
          }
          mbar_arrive(&bars->mfull[e]);
        }
        __syncwarp();
      }
      if (!ok) set_device_error(a.err, kErrWaitTimeout);
    }
    __syncwarp();
  } else if (warp < 12) {
    // ------------------------------------------------------------------ softmax, a thread a row
    regs_inc<kRegsSoftmax>();
    const int g = (warp - 4) >> 2, w4 = warp & 3, row = 32 * w4 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * w4) << 16);
    const uint32_t s_addr = lane_addr + (uint32_t)(g * 128), o_addr = lane_addr + 256u + (uint32_t)(g * D);
    uint8_t* Q = sm + (size_t)g * S::kTileBytes;
    bool ok = true;
    uint32_t job = 0, tile0 = 0, shared = 0;            // this group's half tiles, the CTA's tiles, segments the groups share

    // The group's queries: D / 8 lanes a row, scaled by a power of two to at most 2^15, as f16.
    auto load_q = [&](const Part& p) {
      constexpr int kLanes = D / 8, kPer = 32 / kLanes;
      const int c = lane % kLanes;
      // copied as they are, then scaled where they lie: short loops, as their code is run once a part
      int r = 32 * w4 + lane / kLanes;
      const int R = p.s.rb * kRowTile + (kPair ? g * 128 : 0) + r;
      int j = R / a.G, gr = R - j * a.G;
#pragma unroll 1
      for (int it = 0; it < 32 / kPer; ++it) {
        const bool live = j < p.s.n;
        const uint8_t* from =
            a.q + (live ? 2 * (((size_t)p.s.b * a.tok.Tq + j) * a.q_stride + (size_t)(p.s.h * a.G + gr) * D + 8 * c) : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         smem_u32(Q + (c >> 3) * S::kHalf + sw128(r, c & 7))),
                     "l"(from), "r"(live ? 16 : 0)
                     : "memory");
        r += kPer;
        for (gr += kPer; gr >= a.G; gr -= a.G) ++j;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 4
      for (int it = 0; it < 32 / kPer; ++it) {
        r = 32 * w4 + it * kPer + lane / kLanes;
        uint4* at = reinterpret_cast<uint4*>(Q + (c >> 3) * S::kHalf + sw128(r, c & 7));
        const uint4 x = *at;
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
        float f[8], am = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          f[2 * u] = bf16_bits_to_f(xw[u] & 0xFFFFu);
          f[2 * u + 1] = bf16_bits_to_f(xw[u] >> 16);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (fabsf(f[u]) < INFINITY) am = fmaxf(am, fabsf(f[u]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        // am < 2^e, e from the exponent field (a subnormal maximum counts as 2^-126)
        int k = 15 - ((int)(__float_as_uint(am) >> 23) - 126);
        k = am == 0.f ? 0 : (k > 100 ? 100 : k);
        const float up = __uint_as_float((uint32_t)(k + 127) << 23);
        if (c == 0) cqs[g * 128 + r] = __uint_as_float((uint32_t)(127 - k) << 23) * a.scale_log2;
        uint4 y;
        y.x = pack_f16x2(f[0] * up, f[1] * up);
        y.y = pack_f16x2(f[2] * up, f[3] * up);
        y.z = pack_f16x2(f[4] * up, f[5] * up);
        y.w = pack_f16x2(f[6] * up, f[7] * up);
        *at = y;
      }
      fence_proxy_async_smem();
      __syncwarp();                                      // cqs: a warp's rows are its own
      mbar_arrive(&bars->qfull[g]);
    };

    // Scores x of a half tile that the row at position t does not see become -inf, and NaN where the key's V row
    // has a NaN code.
    auto mask = [&](const TileMeta& meta, int half, uint32_t tile, int t, float* x) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int su = 4 * half + u, p0 = meta.pos + 16 * su;
        uint32_t m = bits_to(t - p0);
        if (a.window > 0) m &= ~bits_to(t - a.window - p0) | bits_to(a.first - 1 - p0);
        if (t < 0 || !((meta.have >> su) & 1u)) m = 0u;
        const uint32_t nb = *reinterpret_cast<const uint32_t*>(nans + (tile & 1) * 32 + 4 * su);
#pragma unroll
        for (int c = 0; c < 16; ++c) x[16 * u + c] = (m >> c) & 1u ? x[16 * u + c] : -INFINITY;
        if (__builtin_expect(nb != 0u, 0)) {
          const uint32_t bad = ((nb & 15u) | ((nb >> 4) & 0xF0u) | ((nb >> 8) & 0xF00u) | ((nb >> 12) & 0xF000u)) & m;
#pragma unroll
          for (int c = 0; c < 16; ++c) x[16 * u + c] = (bad >> c) & 1u ? __int_as_float(0x7fffffff) : x[16 * u + c];
        }
      }
    };

    // Per part: its tiles; then the next part's queries, while the last product runs; then its end.
    int nparts = 0;                                      // parts so far
    float mw = kNone, mz = kNone, l = 0.f, cq = 0.f;
    int jobs = 0, j = 0, gr = 0, t = -1;
    // The end of the part `cur`: its answer, or its record.
    auto finish = [&](const Part& cur) {
      // ---------------------------------------------------------------- the part's end
      const int seg = cur.sb * a.Hkv + cur.s.h;
      if (g == 0 && row == 0 && cur.part0 == 0 && cur.last) {
        int2 who = make_int2(0, 0);
        if (!cur.complete) {
          const int64_t end = run.u1 + (cur.s.units - cur.unit0 - cur.tiles);  // one behind the segment's last unit
          who = make_int2((int)blockIdx.x, (int)((end * run.ctas - 1) / run.total));
        }
        a.info[seg] = who;
      }
      // A whole segment is answered here.  With the same rows in both groups, group 1 hands its share to
      // group 0 through the CTA's record.
      const bool joined = cur.unit0 > cur.part0;         // the record holds the part's earlier pieces
      const bool both = !kPair && cur.complete && (cur.tiles > 1 || joined);
      const bool direct = cur.complete && (kPair || g == 0);
      if (!kPair && cur.complete && g == 1 && !both) return true;
      float* rec = a.part + (((size_t)blockIdx.x * 2 + (cur.part0 == 0 ? 1 : 0)) * (kPair ? 1 : 2) + (kPair ? 0 : g)) *
                                record_floats(kRowTile, D);
      const int rr = (kPair ? g * 128 : 0) + row;
      const bool live = j < cur.s.n;
      const int head = cur.s.h * a.G + gr;
      if (jobs > 0 && !warp_wait(&bars->pvdone[g][(job - 1) & 1u], ((job - 1) >> 1) & 1u)) return false;
      tc_fence_after();
      const float* other = rec + record_floats(kRowTile, D);                 // group 1's record, for group 0
      // the record of the last shared segment has been read
      if (!kPair && g == 1 && !warp_wait(&bars->recfree, (shared & 1u) ^ 1u)) return false;
      if (both && g == 0 && !warp_wait(&bars->recfull, shared & 1u)) return false;
      float f = 1.f, f0 = 0.f;
      if (joined && live) {                              // rare: the earlier pieces join O, its maxima and denominator
        const float w0 = rec[(size_t)kRowTile * D + rr], z0 = rec[(size_t)kRowTile * (D + 1) + rr];
        const float W = fmaxf(mw, w0), Z = fmaxf(mz, z0);
        l = l * exp2f(mz - Z) + rec[(size_t)kRowTile * (D + 2) + rr] * exp2f(z0 - Z);
        f = exp2f(mw - W);
        f0 = exp2f(w0 - W);
        mw = W;
        mz = Z;
      }
      if (joined) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          __syncwarp();
          tmem_ld_32x32b_x16(o_addr + (uint32_t)c, o);
          tmem_wait_ld();
          uint32_t ow[16];
#pragma unroll
          for (int q = 0; q < 16; q += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live) x = *reinterpret_cast<const float4*>(rec + (size_t)rr * D + c + q);
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) ow[q + e] = __float_as_uint(fmaf(xs[e], f0, jobs > 0 ? o[q + e] * f : 0.f));
          }
          tmem_st_32x32b_x16(o_addr + (uint32_t)c, ow);
        }
        tmem_wait_st();
      }
      float f1 = 0.f, last = 1.f;
      f = 1.f;
      if (direct && live) {                              // O relative to mw (and 2^kShift), the denominator to mz
        float W = mw, Z = mz, den = l;
        if (both) {
          const float w1 = other[(size_t)kRowTile * D + rr], z1 = other[(size_t)kRowTile * (D + 1) + rr];
          W = fmaxf(mw, w1);
          Z = fmaxf(mz, z1);
          den = l * exp2f(mz - Z) + other[(size_t)kRowTile * (D + 2) + rr] * exp2f(z1 - Z);
          f1 = exp2f(w1 - W);
        }
        const float2 top = answer_factors(W, Z, den, a.sinks, head, kShift);
        f = exp2f(mw - W) * top.x;
        f1 *= top.x;
        last = top.y;
      }
      uint8_t* out = a.out + 2 * ((((size_t)cur.s.b * a.tok.Tq + j) * a.H + head) * D);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        __syncwarp();
        if (jobs > 0 || joined) {
          tmem_ld_32x32b_x32(o_addr + (uint32_t)c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] = 0.f;
        }
        if (direct && live) {
#pragma unroll
          for (int q = 0; q < 32; q += 8) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = o[q + e] * f;
            if (both) {
              const float4 x0 = *reinterpret_cast<const float4*>(other + (size_t)rr * D + c + q);
              const float4 x1 = *reinterpret_cast<const float4*>(other + (size_t)rr * D + c + q + 4);
              v[0] = fmaf(x0.x, f1, v[0]); v[1] = fmaf(x0.y, f1, v[1]); v[2] = fmaf(x0.z, f1, v[2]); v[3] = fmaf(x0.w, f1, v[3]);
              v[4] = fmaf(x1.x, f1, v[4]); v[5] = fmaf(x1.y, f1, v[5]); v[6] = fmaf(x1.z, f1, v[6]); v[7] = fmaf(x1.w, f1, v[7]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= last;
            uint4 y;
            y.x = (uint32_t)f_to_bf16_bits(v[0]) | ((uint32_t)f_to_bf16_bits(v[1]) << 16);
            y.y = (uint32_t)f_to_bf16_bits(v[2]) | ((uint32_t)f_to_bf16_bits(v[3]) << 16);
            y.z = (uint32_t)f_to_bf16_bits(v[4]) | ((uint32_t)f_to_bf16_bits(v[5]) << 16);
            y.w = (uint32_t)f_to_bf16_bits(v[6]) | ((uint32_t)f_to_bf16_bits(v[7]) << 16);
            *reinterpret_cast<uint4*>(out + 2 * (c + q)) = y;
          }
        } else if (live) {
#pragma unroll
          for (int q = 0; q < 32; q += 4)
            *reinterpret_cast<float4*>(rec + (size_t)rr * D + c + q) = make_float4(o[q], o[q + 1], o[q + 2], o[q + 3]);
        }
      }
      if (jobs > 0) {
        tc_fence_before();
        mbar_arrive(&bars->ofree[g]);
      }
      if (!direct && live) {
        rec[(size_t)kRowTile * D + rr] = mw;
        rec[(size_t)kRowTile * (D + 1) + rr] = mz;
        rec[(size_t)kRowTile * (D + 2) + rr] = l;
      }
      if (both) {
        __threadfence_block();
        mbar_arrive(g == 1 ? &bars->recfull : &bars->recfree);
        ++shared;
      }
      return true;
    };

    bool any = false;
#pragma unroll 1
    for (;;) {
      const bool more = tile0 < (uint32_t)run_tiles;
      const Part& cur = part_ring[nparts % kParts];      // published with its first tile
      if (more && !(nparts == 0 ? warp_wait(&bars->part0, 0u) : warp_wait(&bars->mfull[tile0 % kMeta], (tile0 / kMeta) & 1u))) {
        ok = false;
        break;
      }
      if (more && (kPair || cur.tiles > g)) load_q(cur);
      if (any && !finish(part_ring[(nparts - 1) % kParts])) { ok = false; break; }
      if (!more) break;
      any = true;
      ++nparts;
      // Eight softmax warps let go of every tile's entry: both groups' of a tile that both work on and of a part's
      // first tile, which both wait for; else the group's own warps twice.  So an entry that a group waits for is not
      // published again before it has waited, and neither group falls a ring behind the other.
      if (!kPair && g == 1 && lane == 0) mbar_arrive(&bars->mfree[tile0 % kMeta]);
      jobs = kPair ? cur.tiles : (cur.tiles - g + 1) / 2;
      mw = mz = kNone;
      l = 0.f;
      const int R = cur.s.rb * kRowTile + (kPair ? g * 128 : 0) + row;
      j = R / a.G;
      gr = R - j * a.G;
      t = j < cur.s.n ? cur.s.start + j : -1;
      cq = cqs[g * 128 + row];
      // a warp without live rows only keeps the barriers going: what it leaves in its rows of P stays in theirs of O
      const bool idle = __all_sync(0xffffffffu, j >= cur.s.n);
      // A half tile a step, in a short loop without rare cases: a wait that has to be waited for, keys that some row
      // does not see, P out of its range and scales far apart leave the loop, are dealt with below it, and
      // the step is taken up again.  (With those cases inside, the loop ran a quarter slower.)
      // P is formed against the present maxima; where that leaves P's range (a sum above 60,000: a part's first keys,
      // a new maximum), the maxima move.  So no maxima are taken of the scores before the exponentials, and none
      // at all for most tiles.
      constexpr int kU = 64 / kW;                        // scales of a half tile
      const int steps = 2 * jobs;
      int c = 0;
      bool seen = false, again = false;                  // the half tile's scores are there; its range has been seen to
      bool over = false;
      // The step's P over its scores, and its share of the denominator; true (and nothing done) where P leaves its range.
      auto step = [&](auto masked, uint32_t tile, uint32_t sb, const TileMeta& meta) {
        float x[64], fs[kU], ls[kU], sums[kU];         // scores; logit factor, log2 of the value scale, sum per kW keys
        uint32_t p[32];
        __syncwarp();
        tmem_ld_32x32b_x32(sb, x);
        tmem_ld_32x32b_x32(sb + 32u, x + 32);
        const int u0 = 4 * (c & 1);
#pragma unroll
        for (int v = 0; v < kU; ++v) {
          fs[v] = fmaxf(fminf(meta.ks[u0 + v * (kW / 16)] * cq, 3.0e38f), 1.2e-38f);
          ls[v] = meta.lv[u0 + v * (kW / 16)];
        }
        const float back0 = mw - mz - kShift;
        const bool far = back0 - meta.lv_min[c & 1] > 80.f;
        tmem_wait_ld();
        if (decltype(masked)::value) mask(meta, c & 1, tile, t, x);
        over = false;
#pragma unroll
        for (int v = 0; v < kU; ++v) {
          const float* xs = x + kW * v;
          const float b = ls[v] - mw + kShift;
          float2 s0 = make_float2(0.f, 0.f), s1 = s0;
          const float2 f2 = make_float2(fs[v], fs[v]), b2 = make_float2(b, b);
#pragma unroll
          for (int q = 0; q < kW; q += 4) {
            float2 y0 = fma2(make_float2(xs[q], xs[q + 1]), f2, b2);
            float2 y1 = fma2(make_float2(xs[q + 2], xs[q + 3]), f2, b2);
            y0.x = ex2(y0.x); y0.y = ex2(y0.y); y1.x = ex2(y1.x); y1.y = ex2(y1.y);
            s0 = add2(s0, y0);
            s1 = add2(s1, y1);
            p[(kW * v + q) / 2] = pack_f16x2(y0.x, y0.y);
            p[(kW * v + q) / 2 + 1] = pack_f16x2(y1.x, y1.y);
          }
          s0 = add2(s0, s1);
          sums[v] = s0.x + s0.y;
          over |= sums[v] > 60000.f;
        }
        if (__any_sync(0xffffffffu, over || far) && !again) return true;
#pragma unroll
        for (int v = 0; v < kU; ++v) {
          const float back = back0 - ls[v];
          if (!(back > 80.f)) l = fmaf(sums[v], ex2(back), l);
        }
        tmem_st_32x32b_x16(sb, p);
        tmem_st_32x32b_x16(sb + 16u, p + 16);
        tmem_wait_st();
        return false;
      };
      for (;;) {
        enum { kDone, kNoMeta, kNoScores, kHidden, kRange } why;
#pragma unroll 1
        for (;;) {
          if (c == steps) { why = kDone; break; }
          const uint32_t tile = tile0 + (uint32_t)(kPair ? c >> 1 : 2 * (c >> 1) + g), buf = job & 1u;
          const uint32_t sb = s_addr + 64u * buf;
          const TileMeta& meta = metas[tile % kMeta];
          if (!seen) {
            if ((c & 1) == 0 && !warp_try(&bars->mfull[tile % kMeta], (tile / kMeta) & 1u)) { why = kNoMeta; break; }
            if (!warp_try(&bars->sfull[g][buf], (job >> 1) & 1u)) { why = kNoScores; break; }
            tc_fence_after();
            if (!meta.whole && !idle) { why = kHidden; break; }
          }
          if (!idle && ((c == 0 && !again) || step(std::false_type(), tile, sb, meta))) { why = kRange; break; }
          tc_fence_before();
          mbar_arrive(&bars->pfull[g][buf]);
          if ((c & 1) && lane == 0) mbar_arrive_n(&bars->mfree[tile % kMeta], kPair || tile == tile0 ? 1u : 2u);
          seen = again = false;
          ++job;
          ++c;
        }
        if (why == kDone) break;
        const uint32_t tile = tile0 + (uint32_t)(kPair ? c >> 1 : 2 * (c >> 1) + g), buf = job & 1u;
        const uint32_t sb = s_addr + 64u * buf;
        const TileMeta& meta = metas[tile % kMeta];
        if (why == kNoMeta) {
          ok = warp_wait(&bars->mfull[tile % kMeta], (tile / kMeta) & 1u);
        } else if (why == kNoScores) {
          ok = warp_wait(&bars->sfull[g][buf], (job >> 1) & 1u);
        } else if (why == kHidden) {
          ok = warp_wait(&bars->vfull[tile & 1], (tile >> 1) & 1u);            // the NaN flags
          if (!ok) break;
          if (c > 0 && !step(std::true_type(), tile, sb, meta)) {
            tc_fence_before();
            mbar_arrive(&bars->pfull[g][buf]);
            if ((c & 1) && lane == 0) mbar_arrive_n(&bars->mfree[tile % kMeta], kPair || tile == tile0 ? 1u : 2u);
            ++job;
            ++c;
            continue;
          }
          float x[64];                                   // out of range: the masked scores stay, and the maxima move
          tmem_ld_32x32b_x32(sb, x);
          tmem_ld_32x32b_x32(sb + 32u, x + 32);
          tmem_wait_ld();
          mask(meta, c & 1, tile, t, x);
          tmem_st_32x32b_x32(sb, x);
          tmem_st_32x32b_x32(sb + 32u, x + 32);
          tmem_wait_st();
          why = kRange;
        }
        if (why == kRange) {
          const int u0 = 4 * (c & 1);
          const bool far = mw - mz - kShift - meta.lv_min[c & 1] > 80.f;
          if (c == 0 || __any_sync(0xffffffffu, over || far)) {  // a part's first keys: no maxima yet
            float cz = -INFINITY, cw = -INFINITY;
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
              float y[16];
              __syncwarp();
              tmem_ld_32x32b_x16(sb + 16u * u, y);
              tmem_wait_ld();
              float m16 = y[0];
#pragma unroll
              for (int q = 1; q < 16; ++q) m16 = fmaxf(m16, y[q]);
              const float zt = m16 * fmaxf(fminf(meta.ks[u0 + u] * cq, 3.0e38f), 1.2e-38f);
              cz = fmaxf(cz, zt);
              cw = fmaxf(cw, zt + meta.lv[u0 + u]);
            }
            // A maximum moves where a key exceeds it by more than 11; the others' P fit as they are.  The denominator's
            // moves by itself where a key's logit exceeds it by more than 40 (its value's scale is as much smaller):
            // the weights' sums then stay below 2^(80 + 16) a unit of keys, those taken apart below 2^40 a key.
            const bool move = cw > mw + 11.f;
            const float nw = move ? cw : mw, nz = move || cz > mz + 40.f ? fmaxf(mz, cz) : mz, al = ex2(mw - nw);
            const float down = ex2(0.5f * (mz - nz));    // in two steps: l may be 2^100 where the factor is 2^-130
            l = l * down * down;
            mw = nw;
            mz = nz;
            if (c > 0 && __any_sync(0xffffffffu, move)) {        // O, once the group's last product is complete
              ok = warp_wait(&bars->pvdone[g][(job - 1) & 1u], ((job - 1) >> 1) & 1u);
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < D; q += 16) {
                float o[16];
                tmem_ld_32x32b_x16(o_addr + (uint32_t)q, o);
                tmem_wait_ld();
                uint32_t ow[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e] * al);
                tmem_st_32x32b_x16(o_addr + (uint32_t)q, ow);
              }
              tmem_wait_st();
            }
          }
          // denominators whose factor is out of range: their exponentials apart
          const float back0 = mw - mz - kShift;
#pragma unroll 1
          for (int u = 0; u < 4; ++u) {
            float y[16];
            __syncwarp();
            tmem_ld_32x32b_x16(sb + 16u * u, y);
            tmem_wait_ld();
            const float fq = fmaxf(fminf(meta.ks[u0 + u] * cq, 3.0e38f), 1.2e-38f);
            if (back0 - meta.lv[u0 + u] > 80.f) {
#pragma unroll
              for (int q = 0; q < 16; ++q) l += ex2(y[q] * fq - mz);
            }
          }
          __syncwarp();
          seen = again = true;
        }
        if (!ok) break;
      }
      tile0 += (uint32_t)cur.tiles;
      if (!ok) break;
    }
    if (!ok) set_device_error(a.err, kErrWaitTimeout);
  } else {
    // ------------------------------------------------------------------ conversion of K or V tiles
    regs_dec<kRegsConvert>();
    const bool is_v = warp >= 16;
    const int w = warp & 3;
    constexpr int kLanes = D / 16, kRowsPer = 32 / kLanes;    // lanes a row, rows a load of the warp
    constexpr int kLoads = kSubs * 16 / (4 * kRowsPer);       // loads a thread and tile
    const int c = lane % kLanes, r0 = w * kRowsPer + lane / kLanes;
    uint8_t* tiles = sm + (is_v ? S::kOffV : S::kOffK);
    uint64_t* full = is_v ? bars->vfull : bars->kfull;
    uint64_t* freeb = is_v ? bars->vfree : bars->kfree;
    const uint8_t* pool = is_v ? a.P.v : a.P.k;
    bool ok = true;
    uint4 x[kLoads];
    uint32_t have = 0, tile = 0;
    const uint32_t total = (uint32_t)run_tiles;
    const uint8_t* lane_base = pool + 16 * c;
    const size_t per_head = (size_t)a.T.page * D, per_page = per_head * a.Hkv;
    const int inside = a.T.page - 1;
    bool loaded = false, clean = false;                       // x holds the tile's codes; without NaN codes, where it matters
    for (;;) {
      enum { kDone, kNoMeta, kNoRoom, kMasked } why;          // as above: the loop without its rare cases
#pragma unroll 1
      for (;;) {
        if (!loaded) {
          if (!warp_try(&bars->mfull[tile % kMeta], (tile / kMeta) & 1u)) { why = kNoMeta; break; }
          const TileMeta& m = metas[tile % kMeta];
          clean = !is_v || m.whole;
          have = m.have;
          int32_t pg[kSubs];
          *reinterpret_cast<int4*>(pg) = *reinterpret_cast<const int4*>(m.page);
          *reinterpret_cast<int4*>(pg + 4) = *reinterpret_cast<const int4*>(m.page + 4);
          const uint8_t* base = lane_base + m.h * per_head;
          const int at = m.pos + r0;
#pragma unroll
          for (int it = 0; it < kLoads; ++it) {
            // rows without a page read page 0 (V's are cleared below, K's scores hidden)
            const int r = it * 4 * kRowsPer;
            const int32_t p0 = pg[r >> 4], p1 = pg[(r >> 4) + (kRowsPer == 8 ? 1 : 0)];
            const int32_t p = kRowsPer == 8 && w >= 2 ? p1 : p0;
            x[it] = *reinterpret_cast<const uint4*>(base + (size_t)(p < 0 ? 0 : p) * per_page + (size_t)((at + r) & inside) * D);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->mfree[tile % kMeta]);
          loaded = true;
        }
        if (!warp_try(&freeb[tile & 1], ((tile >> 1) & 1u) ^ 1u)) { why = kNoRoom; break; }
        if (!clean) { why = kMasked; break; }
        uint8_t* dst = tiles + (tile & 1) * S::kTileBytes;
#pragma unroll
        for (int it = 0; it < kLoads; ++it) {
          const int r = it * 4 * kRowsPer + r0;
          const uint32_t xw[4] = {x[it].x, x[it].y, x[it].z, x[it].w};
          uint4 y0, y1;
          e4m3x4_f16(xw[0], y0.x, y0.y);
          e4m3x4_f16(xw[1], y0.z, y0.w);
          e4m3x4_f16(xw[2], y1.x, y1.y);
          e4m3x4_f16(xw[3], y1.z, y1.w);
          // the two 16-byte pieces, the second first in the upper half, so that a row's lanes fall on different banks
          uint8_t* at = dst + (c >> 2) * S::kHalf;
          const int jx = (c & 3) * 2, up = (c >> 2) & 1;
          *reinterpret_cast<uint4*>(at + sw128(r, jx + up)) = up ? y1 : y0;
          *reinterpret_cast<uint4*>(at + sw128(r, jx + (up ^ 1))) = up ? y0 : y1;
        }
        fence_proxy_async_smem();
        mbar_arrive(&full[tile & 1]);
        loaded = false;
        if (++tile == total) { why = kDone; break; }
      }
      if (why == kDone) break;
      if (why == kNoMeta) {
        ok = warp_wait(&bars->mfull[tile % kMeta], (tile / kMeta) & 1u);
      } else if (why == kNoRoom) {
        ok = warp_wait(&freeb[tile & 1], ((tile >> 1) & 1u) ^ 1u);
      } else {
        // some row does not see some key: NaN codes become 0 and are flagged for the rows that do
#pragma unroll
        for (int it = 0; it < kLoads; ++it) {
          if (!((have >> ((it * 4 * kRowsPer + r0) >> 4)) & 1u)) x[it] = make_uint4(0u, 0u, 0u, 0u);
          uint32_t xw[4] = {x[it].x, x[it].y, x[it].z, x[it].w};
          uint32_t any = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t nb = nan_bytes(xw[q]);
            any |= nb;
            xw[q] &= ~((nb >> 7) * 0xFFu);
          }
          x[it] = make_uint4(xw[0], xw[1], xw[2], xw[3]);
          const uint32_t bal = __ballot_sync(0xffffffffu, any != 0);
          // four rows to a byte
          if (lane < kRowsPer / 4) {
            uint32_t fl = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              fl |= ((bal >> ((4 * lane + q) * kLanes)) & ((1u << kLanes) - 1u)) ? 1u << q : 0u;
            nans[(tile & 1) * 32 + (it * 4 * kRowsPer + w * kRowsPer) / 4 + lane] = (uint8_t)fl;
          }
          __syncwarp();
        }
        clean = true;
      }
      if (!ok) break;
    }
    if (!ok) set_device_error(a.err, kErrWaitTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D, bool kPair, int kW>
cudaError_t launch_tc_as(const PagedAttendArgs& a, bool join_only, cudaStream_t s) {
  auto kernel = paged_attend_tc_kernel<D, kPair, kW>;
  // the warps' register split draws on what the block was launched with: looked at once
  static const int regs = [&] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, kernel) == cudaSuccess ? attr.numRegs : 0;
  }();
  if (regs < kRegsLaunch) return cudaErrorLaunchOutOfResources;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), TcShape<D>::kBytes);
  if (e == cudaSuccess && !join_only) e = launch_kernel(kernel, dim3(a.ctas), dim3(kThreads), TcShape<D>::kBytes, s, 0, a);
  if (e == cudaSuccess)
    e = launch_combine<D>(a, CombineShape{kPair ? 256 : 128, kKeys, 1, kPair ? 1 : 2, kShift}, s);
  return e;
}

template <int D, bool kPair>
cudaError_t launch_tc(const PagedAttendArgs& a, bool join_only, cudaStream_t s) {
  return a.T.page == 16 ? launch_tc_as<D, kPair, 16>(a, join_only, s) : launch_tc_as<D, kPair, 32>(a, join_only, s);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Which kernel: the warp-level one for float32 activations and up to 16 query rows per KV head, tcgen05 above.
PagedPlan paged_plan(int act_fmt, int B, int G, int Hkv, int D, int Tq, int num_sms) {
  PagedPlan p;
  const int64_t rows = (int64_t)Tq * G;
  p.path = act_fmt == CSA_FMT_F32 || rows <= 16 ? 1 : 2;
  p.row_tile = p.path == 1 ? (rows <= 8 ? 8 : 16) : (rows <= 128 ? 128 : 256);
  p.rb_max = (int)((rows + p.row_tile - 1) / p.row_tile);
  p.ctas = num_sms;
  size_t off = 256;                                           // the error word
  p.info = off;
  off = up256(off + (size_t)B * p.rb_max * Hkv * sizeof(int2));
  p.part = off;
  p.total = up256(off + (size_t)p.ctas * 2 * record_floats(p.path == 1 ? p.row_tile : 256, D) * 4);
  return p;
}

cudaError_t launch_paged_attend(const PagedAttendArgs& a, const PagedPlan& p, bool join_only, cudaStream_t s) {
  if (p.path == 1) return launch_paged_attend_warp(a, p.row_tile, join_only, s);
  if (a.D == 128) return p.row_tile == 256 ? launch_tc<128, true>(a, join_only, s) : launch_tc<128, false>(a, join_only, s);
  return p.row_tile == 256 ? launch_tc<64, true>(a, join_only, s) : launch_tc<64, false>(a, join_only, s);
}

}  // namespace csa
