// Attention over the paged 8-bit cache, warp-level tensor-core path (definition: csa_paged_attend in
// csa.h).  Serves short query blocks (decode, a few speculative tokens) and float32 activations.
//
// What bounds it.  A decode step reads 2 D bytes per key and KV head and does 4 D G flops with them
// (G query heads of the group): at G = 8 that is 16 flops a byte, so memory bounds it.  The design
// keeps bytes in flight: 8 or 12 warps per SM, each with its own ring of 32-key tiles that TMA fills.
// Measured, 64 heads on 8 KV heads of 128 dims: 1,048,576 keys in 337-368 us (5.8-6.4 TB/s, 0.89-0.97 of the
// measured copy rate, from card to card), 8 sequences of up to 131,072 in 269-272 us; about 640 instructions per tile and warp,
// half of them code conversions and byte permutes, leave little of the clock unused.
//
// Work.  A segment is one (sequence, block of query rows, KV head); a row is (token, head of the
// group).  Its visible keys are cut into tiles of 32 (positions in multiples of 32; with a window, the
// tiles of the first tokens and then those from the window's start), as many tiles as warps make a unit, and all
// segments' units in order are dealt to the CTAs in equal runs.  A warp walks its tile of each unit of its
// CTA's run without waiting for the other warps, so copies run ahead over segment borders.  Where a
// segment ends the CTA merges its warps; a segment cut between CTAs leaves records that a second
// kernel merges.  Which CTA did what depends on the lengths alone, so results do not change from run
// to run.
//
// Mathematics.  The keys are the M dimension of the products, the query rows the N:
//   S^T[key][row] = sum_d K[key][d] q[row][d],  O^T[d][row] += sum_key V[key][d] P[key][row]
// (mma.m16n8k16, f16 inputs, f32 sums), so a group of 8 heads fills the instruction.  e4m3 codes are
// exact in f16.  Queries are scaled per row by a power of two to at most 2^15 and rounded to f16 (exact
// for bf16 values down to 2^-32 of the row's largest); float32 queries are the sum of three f16 terms.
// A lane's 16-byte pieces of K and V need no shuffles: dims are permuted alike in K and q, and V's
// fragment takes the bytes of two keys by byte permutes.
// The scale of V's page is folded into the exponent: with z the logit in log2 units and v the log2 of
// the scale, O sums 2^(z + v - mw), mw the running maximum of z + v, and the denominator sums
// 2^(z - mz) with its own running maximum mz; both exponentials are cheap here, and neither can lose
// the other's range however much the pages' scales differ.
// P, relative to the largest probability times value scale, is f16 (11 bits): scaled by 2^7, with maxima that move only when a tile exceeds them by more than
// 8, or (float32) by 2^15 with exact maxima and a second f16 term.  Rounding P is unbiased and f16
// keeps all 11 bits down to 2^-21 (2^-29) of the largest weight.
#include <cudaTypedefs.h>
#include <limits.h>
#include <mutex>

#include "paged_walk.cuh"
#include "sm100.cuh"

namespace csa {

namespace {

using namespace sm100;

constexpr int kTile = 32;                     // keys per warp step
constexpr int kSub = 16;                      // keys per TMA box: within one page
// A warp's steps between two times that its sums go to the CTA's record: the tensor core cuts its sums off instead of
// rounding them (one chain over 8,388,608 keys shared by 12 warps came out 6e-3 too small, more than bf16's half
// step), the record is added up rounded.  Two products a step: 2e-4 at most.
constexpr int kPieceSteps = 1024;

struct Meta {                                 // one 16-key half of a ring stage
  float ks, vs;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mma_f16(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) {
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}

// 2^x: the hardware approximation (relative error about 2^-22, below half of P's rounding) for bf16
// activations, the correctly scaled function for float32.
template <bool F32>
__device__ __forceinline__ float exp2_of(float x) {
  if (F32) return exp2f(x);
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, int NT, bool F32>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTerms = F32 ? 3 : 1;
  // Warps and merge buffers: as many as registers (O takes D/16 x NT x 4 of them) and shared memory allow.  1 M keys
  // of 8 heads with 12 warps 387 us, with 8 447 us; 524,288 keys and 16 rows of 128 dims with 8 251 us, with 12
  // (which spill) 473 us.
  static constexpr int kWarps = F32 || NT * D > 128 ? 8 : 12;
  static constexpr int kBufs = NT * D > 128 ? 2 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr bool kQRegs = NT == 1 && !F32;             // query fragments stay in registers
  static constexpr int kWords = D / 16;                       // k-steps of K q: one 32-bit word of codes per lane
  static constexpr int kStageBytes = 2 * kTile * D;           // keys, then values
  static constexpr int kQBytes = kTerms * NT * kWords * 32 * 8;
  static constexpr int kMergeBytes = kBufs * kRows * D * 4;
  static constexpr int kFixed = kQBytes + kMergeBytes + kRows * 4 + 3 * kWarps * kRows * 4;
  static constexpr int kFree = 227 * 1024 - 1024 - 1024 - kFixed;
  static constexpr int kFit = kFree / (kWarps * (kStageBytes + 2 * (int)sizeof(Meta) + 8));
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static_assert(kStages >= 2, "ring");
  // offsets from a 1024-byte boundary
  static constexpr size_t kOffQ = (size_t)kWarps * kStages * kStageBytes;
  static constexpr size_t kOffMerge = kOffQ + kQBytes;
  static constexpr size_t kOffCq = kOffMerge + kMergeBytes;   // [rows] logit factor of a row
  static constexpr size_t kOffStat = kOffCq + kRows * 4;      // [3][warps][rows]: mw, mz, l
  static constexpr size_t kOffMeta = kOffStat + 3 * kWarps * kRows * 4;
  static constexpr size_t kOffBar = (kOffMeta + (size_t)kWarps * kStages * 2 * sizeof(Meta) + 7) / 8 * 8;
  static constexpr size_t kBytes = 1024 + kOffBar + (size_t)kWarps * kStages * 8;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(Shape<D, NT, F32>::kThreads, 1)
paged_attend_kernel(const __grid_constant__ PagedAttendArgs a, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<D, NT, F32>;
  constexpr int kRows = S::kRows, kTerms = S::kTerms, kWords = S::kWords, kStages = S::kStages, kWarps = S::kWarps;
  constexpr float kShift = F32 ? 15.f : 7.f;                  // P = 2^(weight + kShift)
  constexpr float kMargin = F32 ? 0.f : 8.f;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  uint2* qf = reinterpret_cast<uint2*>(sm + S::kOffQ);        // [terms][NT][words][32 lanes]
  float* merge = reinterpret_cast<float*>(sm + S::kOffMerge); // [kBufs][rows][D]
  float* cq = reinterpret_cast<float*>(sm + S::kOffCq);
  float* stat = reinterpret_cast<float*>(sm + S::kOffStat);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = sm + (size_t)warp * kStages * S::kStageBytes;
  Meta* meta = reinterpret_cast<Meta*>(sm + S::kOffMeta) + warp * kStages * 2;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kOffBar) + warp * kStages;

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars[i], 3);  // one arrival with the bytes, two of the scales
    fence_barrier_init();
  }
  const Run run = find_run(a, kRows, kTile, kWarps, 1);
  if (run.u0 >= run.u1) return;
  const int steps = (int)(run.u1 - run.u0);

  bool ok = true;
  // ------------------------------------------------------------------ the warp's copies
  // Lanes 0 and 1 each look after one 16-key half of a tile: its page, its two boxes, its two scales.
  // The page of the next tile to be copied is loaded one step ahead.
  Walk pw;                                                    // unit whose tile is copied next
  walk_start(a, pw, run, kRows, kTile, kWarps);
  int issued = 0;
  int32_t page_next = -1;
  auto load_page = [&]() {
    page_next = -1;
    const int i = pw.unit * kWarps + warp;
    if (lane < 2 && i < pw.s.tiles) {
      const int pos = tile_pos(pw.s, i, kTile) + kSub * lane;
      if (pos < pw.s.start + pw.s.n) {                        // at most n_max: inside the table's row
        const int32_t pg = a.T.table[(size_t)pw.s.b * a.T.cap + (pos >> a.T.page_log2)];
        if (pg < a.T.n_pages) page_next = pg < 0 ? -1 : pg;
        else set_device_error(a.err, kErrPage);
      }
    }
  };
  uint32_t have_bits = 0;                                     // two bits per stage: halves that were copied
  auto issue = [&]() {
    const int st = issued % kStages;
    uint8_t* kd = ring + (size_t)st * S::kStageBytes;
    const bool mine = lane < 2 && page_next >= 0;
    const uint32_t have = __ballot_sync(0xffffffffu, mine) & 3u;
    have_bits = (have_bits & ~(3u << (2 * st))) | (have << (2 * st));
    if (lane == 0) mbar_arrive_expect_tx(&bars[st], (uint32_t)__popc(have) * (2 * kSub * D));
    __syncwarp();
    if (lane < 2) {
      if (mine) {
        const int i = pw.unit * kWarps + warp;
        const int pos = tile_pos(pw.s, i, kTile) + kSub * lane;
        const int y = pw.s.h * a.T.page + (pos & (a.T.page - 1));
        tma_load_3d(kd + lane * kSub * D, &kmap, &bars[st], 0, y, page_next);
        tma_load_3d(kd + kTile * D + lane * kSub * D, &vmap, &bars[st], 0, y, page_next);
        const size_t gh = (size_t)page_next * a.Hkv + pw.s.h;
        cp_async4(&meta[2 * st + lane].ks, a.P.ks + gh);
        cp_async4(&meta[2 * st + lane].vs, a.P.vs + gh);
      }
      cp_async_arrive(&bars[st]);
    }
    ++issued;
    if (issued < steps) {
      walk_next(a, pw, kRows, kTile, kWarps);
      load_page();
    }
  };
  __syncwarp();
  load_page();
  for (int i = 0; i < kStages && i < steps; ++i) issue();

  // ------------------------------------------------------------------ the walk
  Walk cw;
  walk_start(a, cw, run, kRows, kTile, kWarps);
  float o[D / 16][NT][4];
  float mw[NT][2], mz[NT][2], l[NT][2];
  int tq[NT][2];                                              // positions of this lane's rows, -1: no such row
  bool fresh = true;                                          // a piece of a segment begins
  int seg_unit0 = cw.unit;                                    // first unit of the segment's part
  int tmin = 0, tmax = 0;
  uint2 qr[S::kQRegs ? kWords : 1];
  for (int step = 0; step < steps; ++step) {
    if (fresh) {
      fresh = false;
      // the block's queries as f16 fragments: warp w takes rows w, w + kWarps, ...; a lane D / 32 dims
      __syncthreads();
      for (int r = warp; r < kRows; r += kWarps) {
        const int R = cw.s.rb * kRows + r, j = R / a.G, gr = R - j * a.G;
        float x[D / 32];
        const bool live = j < cw.s.n;
        if (live) {
          const size_t at = ((size_t)cw.s.b * a.tok.Tq + j) * a.q_stride + (size_t)(cw.s.h * a.G + gr) * D + lane * (D / 32);
          if (F32) {
#pragma unroll
            for (int u = 0; u < D / 32; ++u) x[u] = reinterpret_cast<const float*>(a.q)[at + u];
          } else {
#pragma unroll
            for (int u = 0; u < D / 32; u += 2) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(a.q + 2 * (at + u));
              x[u] = bf16_bits_to_f(w & 0xFFFFu);
              x[u + 1] = bf16_bits_to_f(w >> 16);
            }
          }
        } else {
#pragma unroll
          for (int u = 0; u < D / 32; ++u) x[u] = 0.f;
        }
        float am = 0.f;
#pragma unroll
        for (int u = 0; u < D / 32; ++u)
          if (fabsf(x[u]) < INFINITY) am = fmaxf(am, fabsf(x[u]));
        am = warp_max(am);
        int e = 0;
        if (am > 0.f) frexpf(am, &e);                         // am < 2^e
        int k = 15 - e;                                       // am 2^k in [2^14, 2^15)
        k = k > 100 ? 100 : k;
        if (am == 0.f) k = 0;
        const float up = ldexpf(1.f, k);
        if (lane == 0) cq[r] = ldexpf(1.f, -k) * a.scale_log2;
        // dims lane * D/32 + u: fragment word w = 4 dims, of lane column tt
        const int d0 = lane * (D / 32);
#pragma unroll
        for (int u = 0; u < D / 32; u += 2) {
          const int d = d0 + u;
          const int chunk = d >> 4, tt = D == 128 ? chunk >> 1 : chunk;
          const int w = (D == 128 ? (chunk & 1) * 4 : 0) + ((d >> 2) & 3);
          float y0 = x[u] * up, y1 = x[u + 1] * up;
#pragma unroll
          for (int c = 0; c < kTerms; ++c) {
            const uint32_t h2 = pack_f16x2(y0, y1);
            uint32_t* dst = reinterpret_cast<uint32_t*>(&qf[((c * NT + (r >> 3)) * kWords + w) * 32 + (r & 7) * 4 + tt]);
            dst[(d >> 1) & 1] = h2;
            const float2 b = unpack_f16x2(h2);
            y0 -= b.x;
            y1 -= b.y;
          }
        }
      }
      __syncthreads();
      if (S::kQRegs) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) qr[S::kQRegs ? w : 0] = qf[w * 32 + lane];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int R = cw.s.rb * kRows + 8 * n + 2 * t + e, j = R / a.G;
          tq[n][e] = j < cw.s.n ? cw.s.start + j : -1;
          mw[n][e] = mz[n][e] = kNone;
          l[n][e] = 0.f;
        }
      tmin = cw.s.start + cw.s.j0;
      {
        const int j1 = (cw.s.rb * kRows + kRows - 1) / a.G;
        tmax = cw.s.start + (j1 < cw.s.n ? j1 : cw.s.n - 1);
      }
#pragma unroll
      for (int m = 0; m < D / 16; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[m][n][e] = 0.f;
    }
    const int st = step % kStages;
    const uint32_t have = (have_bits >> (2 * st)) & 3u;
    if (ok && !__all_sync(0xffffffffu, mbar_wait(&bars[st], (uint32_t)(step / kStages) & 1u))) {
      ok = false;
      set_device_error(a.err, kErrWaitTimeout);
    }
    const int ti = cw.unit * kWarps + warp;
    if (have) {
      const uint8_t* kt = ring + (size_t)st * S::kStageBytes;
      const uint8_t* vt = kt + kTile * D;
      const int pos = tile_pos(cw.s, ti, kTile);
      // every row sees every key of the tile?
      const bool whole = have == 3u && pos + kTile - 1 <= tmin &&
                         (a.window == 0 || pos > tmax - a.window || pos + kTile <= a.first);
      float z[2][NT][4];
      float lv[2];
      // S^T, scaled: z = logit (log2 units)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float acc[2][NT][4];                                  // two chains: even and odd words, or the large and small terms
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][n][e] = 0.f;
        // rows of the boxes are swizzled: 16-byte piece c of row r lies at c ^ (r & 7) (128-byte rows),
        // c ^ ((r >> 1) & 3) (64-byte rows)
        const int r0 = s * kSub + g, r1 = r0 + 8;
        uint4 w0[D / 64], w1[D / 64];
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int piece = D == 128 ? 2 * t + c : t;
          const int x0 = D == 128 ? piece ^ (r0 & 7) : piece ^ ((r0 >> 1) & 3);
          const int x1 = D == 128 ? piece ^ (r1 & 7) : piece ^ ((r1 >> 1) & 3);
          w0[c] = *reinterpret_cast<const uint4*>(kt + r0 * D + 16 * x0);
          w1[c] = *reinterpret_cast<const uint4*>(kt + r1 * D + 16 * x1);
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const uint32_t a0 = reinterpret_cast<const uint32_t*>(w0)[w], a1 = reinterpret_cast<const uint32_t*>(w1)[w];
          uint32_t fr[4];
          e4m3x4_f16(a0, fr[0], fr[2]);
          e4m3x4_f16(a1, fr[1], fr[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = kTerms - 1; c >= 0; --c) {           // the small terms apart from the large one
              const uint2 b = S::kQRegs ? qr[S::kQRegs ? w : 0] : qf[((c * NT + n) * kWords + w) * 32 + lane];
              mma_f16(acc[F32 ? (c > 0) : (w & 1)][n], fr, b.x, b.y);
            }
          }
        }
        const float ks = meta[2 * st + s].ks;
        lv[s] = (float)((int)((__float_as_uint(meta[2 * st + s].vs) >> 23) & 255u) - 127);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 c2 = *reinterpret_cast<const float2*>(&cq[8 * n + 2 * t]);
          const float f0 = fminf(ks * c2.x, 3.0e38f), f1 = fminf(ks * c2.y, 3.0e38f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            z[s][n][e] = (acc[0][n][e] + acc[1][n][e]) * ((e & 1) ? f1 : f0);
          }
        }
      }
      // values of this lane's four keys per half: 2t, 2t + 1, 2t + 8, 2t + 9; D / 8 dims
      constexpr int kVW = D / 32;                             // 32-bit words per key
      uint32_t vw[2][4][kVW];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = s * kSub + 2 * t + (q & 1) + 8 * (q >> 1);
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(vt + r * D + 16 * (g ^ (r & 7)));
            vw[s][q][0] = x.x; vw[s][q][1] = x.y; vw[s][q][kVW - 2] = x.z; vw[s][q][kVW - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(vt + r * D + 16 * ((g >> 1) ^ ((r >> 1) & 3)) + 8 * (g & 1));
            vw[s][q][0] = x.x; vw[s][q][1] = x.y;
          }
        }
      if (!whole) {
        // Some row does not see some key: its value must not enter by 0 * NaN.  NaN codes of V become
        // 0, and the logit of a key that had one becomes NaN, for the rows that see it.
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t bal[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < kVW; ++w) {
              const uint32_t nb = nan_bytes(vw[s][q][w]);
              any |= nb;
              vw[s][q][w] &= ~((nb >> 7) * 0xFFu);
            }
            bal[q] = __ballot_sync(0xffffffffu, any != 0);
          }
          const uint32_t col = 0x11111111u << (g >> 1);       // lanes that hold key g's values
          const bool bad0 = ((g & 1) ? bal[1] : bal[0]) & col, bad1 = ((g & 1) ? bal[3] : bal[2]) & col;
          const bool here = (have >> s) & 1u;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = pos + s * kSub + g + 8 * (e >> 1), tr = tq[n][e & 1];
              const bool see = here && i <= tr && (a.window == 0 || i > tr - a.window || i < a.first);
              const bool bad = (e >> 1) ? bad1 : bad0;
              z[s][n][e] = see ? (bad ? __int_as_float(0x7fffffff) : z[s][n][e]) : -INFINITY;
            }
        }
      }
      // running maxima
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY, topw = -INFINITY;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const float h = fmaxf(z[s][n][e], z[s][n][e + 2]);
            top = fmaxf(top, h);
            topw = fmaxf(topw, h + lv[s]);
          }
          over |= topw > mw[n][e] + kMargin || top > mz[n][e] + 40.f;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float nz = kNone, nw = kNone;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const float h = fmaxf(z[s][n][e], z[s][n][e + 2]);
              nz = fmaxf(nz, h);
              nw = fmaxf(nw, h + lv[s]);
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              nz = fmaxf(nz, __shfl_xor_sync(0xffffffffu, nz, d));
              nw = fmaxf(nw, __shfl_xor_sync(0xffffffffu, nw, d));
            }
            nz = fmaxf(nz, mz[n][e]);
            nw = fmaxf(nw, mw[n][e]);
            l[n][e] *= exp2_of<F32>(mz[n][e] - nz);
            const float al = exp2_of<F32>(mw[n][e] - nw);
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
              o[m][n][e] *= al;
              o[m][n][e + 2] *= al;
            }
            mz[n][e] = nz;
            mw[n][e] = nw;
          }
      }
      // P (f16, transposed to [row][key] pairs) and the denominators
      uint32_t p[2][F32 ? 2 : 1][NT][2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[n][e & 1] += exp2_of<F32>(z[s][n][e] - mz[n][e & 1]);
            y[e] = exp2_of<F32>(z[s][n][e] + (lv[s] - mw[n][e & 1] + kShift));
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t hi = pack_f16x2(y[2 * hf], y[2 * hf + 1]);
            p[s][0][n][hf] = transpose8x8(hi);
            if (F32) {
              const float2 b = unpack_f16x2(hi);
              p[s][F32 ? 1 : 0][n][hf] = transpose8x8(pack_f16x2(y[2 * hf] - b.x, y[2 * hf + 1] - b.y));
            }
          }
        }
      // O^T += V^T P^T.  float32: the tile's sums are formed apart and added to O rounded to nearest,
      // so that the tensor core's truncation does not add up over a long sequence.
#pragma unroll
      for (int m = 0; m < D / 16; ++m) {
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[n][e] = F32 ? 0.f : o[m][n][e];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          // dims 2 m and 2 m + 1 of this lane's run: bytes (2 m) & 3 and the next of word m / 2
          const uint32_t sel = (m & 1) ? 0x7362u : 0x5140u;
          const uint32_t x = __byte_perm(vw[s][0][m >> 1], vw[s][1][m >> 1], sel);
          const uint32_t y = __byte_perm(vw[s][2][m >> 1], vw[s][3][m >> 1], sel);
          uint32_t fr[4];
          e4m3x4_f16(x, fr[0], fr[1]);
          e4m3x4_f16(y, fr[2], fr[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (F32) mma_f16(acc[n], fr, p[s][F32 ? 1 : 0][n][0], p[s][F32 ? 1 : 0][n][1]);
            mma_f16(acc[n], fr, p[s][0][n][0], p[s][0][n][1]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[m][n][e] = F32 ? o[m][n][e] + acc[n][e] : acc[n][e];
      }
    }
    __syncwarp();                                             // the stage has been read by every lane
    if (issued < steps && ok) issue();

    // ---------------------------------------------------------------- the segment's end (for this CTA), or a piece's
    const bool last_unit = cw.unit + 1 == cw.s.units;
    if (!last_unit && step + 1 < steps && (step + 1) % kPieceSteps != 0) {
      ++cw.unit;
      continue;
    }
    // denominators over the lanes that share a row, then the warps' statistics
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
        if (g == 0) {
          const int r = 8 * n + 2 * t + e;
          stat[(0 * kWarps + warp) * kRows + r] = mw[n][e];
          stat[(1 * kWarps + warp) * kRows + r] = mz[n][e];
          stat[(2 * kWarps + warp) * kRows + r] = l[n][e];
        }
      }
    __syncthreads();
    // O relative to the CTA's maximum, kBufs warps at a time: the first leave theirs, the others add to it
#pragma unroll 1
    for (int turn = 0; turn < kWarps / S::kBufs; ++turn) {
      if (warp / S::kBufs == turn) {
        float* mb = merge + (size_t)(warp % S::kBufs) * kRows * D;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            float top = kNone;
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w * kRows + r]);
            const float f = exp2f(mw[n][e] - top);
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
              // dims of this lane: g * D/8 + 2 m (+1)
              float2* at = reinterpret_cast<float2*>(mb + (size_t)r * D + g * (D / 8) + 2 * m);
              float2 v = make_float2(o[m][n][e] * f, o[m][n][e + 2] * f);
              if (turn > 0) {
                const float2 b = *at;
                v.x += b.x;
                v.y += b.y;
              }
              *at = v;
            }
          }
      }
      __syncthreads();
    }
    const bool complete = seg_unit0 == 0 && last_unit;
    const bool joined = step % kPieceSteps < cw.unit - seg_unit0;    // the record holds the part's earlier pieces
    const int seg = cw.sb * a.Hkv + cw.s.h;
    float* rec = a.part + ((size_t)blockIdx.x * 2 + (seg_unit0 == 0 ? 1 : 0)) * record_floats(kRows, D);
    // A row's maxima and denominator over the warps and, with earlier pieces, the record; factors of both O.
    auto row_stats = [&](int r, float& W, float& Z, float& L, float& f, float& f0) {
      W = Z = kNone;
      L = f0 = 0.f;
      f = 1.f;
      for (int w = 0; w < kWarps; ++w) {
        W = fmaxf(W, stat[(0 * kWarps + w) * kRows + r]);
        Z = fmaxf(Z, stat[(1 * kWarps + w) * kRows + r]);
      }
      const float top = W;
      float z0 = kNone;
      if (joined) {
        const float w0 = rec[(size_t)kRows * D + r];
        z0 = rec[(size_t)kRows * (D + 1) + r];
        W = fmaxf(W, w0);
        Z = fmaxf(Z, z0);
        f = exp2f(top - W);
        f0 = exp2f(w0 - W);
      }
      for (int w = 0; w < kWarps; ++w)
        L += stat[(2 * kWarps + w) * kRows + r] * exp2f(stat[(1 * kWarps + w) * kRows + r] - Z);
      if (joined) L += rec[(size_t)kRows * (D + 2) + r] * exp2f(z0 - Z);
    };
    for (int i = tid; i < kRows * (D / 4); i += S::kThreads) {
      const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
      const int R = cw.s.rb * kRows + r, j = R / a.G, gr = R - j * a.G;
      if (j >= cw.s.n) continue;
      float W, Z, L, f, f0;
      row_stats(r, W, Z, L, f, f0);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < S::kBufs; ++q) {
        const float4 b = *reinterpret_cast<const float4*>(merge + ((size_t)q * kRows + r) * D + c);
        v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
      }
      if (joined) {
        const float4 b = *reinterpret_cast<const float4*>(rec + (size_t)r * D + c);
        v.x = fmaf(b.x, f0, v.x * f); v.y = fmaf(b.y, f0, v.y * f); v.z = fmaf(b.z, f0, v.z * f); v.w = fmaf(b.w, f0, v.w * f);
      }
      if (complete) {
        const int head = cw.s.h * a.G + gr;
        const float2 x = answer_factors(W, Z, L, a.sinks, head, kShift);
        const float out[4] = {v.x * x.x * x.y, v.y * x.x * x.y, v.z * x.x * x.y, v.w * x.x * x.y};
        const size_t at = (((size_t)cw.s.b * a.tok.Tq + j) * a.H + head) * D + c;
        store_act4(a.out + at * (F32 ? 4 : 2), F32 ? CSA_FMT_F32 : CSA_FMT_BF16, 0, out);
      } else {
        *reinterpret_cast<float4*>(rec + (size_t)r * D + c) = v;
      }
    }
    if (!complete) {
      float W, Z, L, f, f0;
      if (tid < kRows) row_stats(tid, W, Z, L, f, f0);
      if (joined) __syncthreads();                            // every thread has read the record's statistics
      if (tid < kRows) {
        rec[(size_t)kRows * D + tid] = W;
        rec[(size_t)kRows * (D + 1) + tid] = Z;
        rec[(size_t)kRows * (D + 2) + tid] = L;
      }
    }
    if (seg_unit0 == 0 && tid == 0 && (last_unit || step + 1 == steps)) {
      // the CTA with the segment's first unit names the CTAs that share it: this one to the one that
      // has the segment's last unit
      int2 who = make_int2(0, 0);
      if (!complete) {
        const int64_t end = run.u1 + (cw.s.units - 1 - cw.unit);     // one behind the segment's last unit
        who = make_int2((int)blockIdx.x, (int)((end * run.ctas - 1) / run.total));
      }
      a.info[seg] = who;
    }
    __syncthreads();                                          // merge and stat are free again
    if (step + 1 < steps) {
      walk_next(a, cw, kRows, kTile, kWarps);
      fresh = true;
      if (last_unit) seg_unit0 = 0;
    }
  }
  if (!ok) {
    // give the copies in flight time to land before the CTA's memory is handed on
    for (int i = 0; i < kStages && i < issued; ++i) mbar_wait(&bars[i], (uint32_t)((issued - 1 - i) / kStages) & 1u);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Codes as [n_pages][Hkv * page][D] bytes, read in boxes of `rows` rows of one page and head, swizzled
// so that equal 16-byte columns of neighbouring rows fall on different banks.
bool make_pool_map(CUtensorMap* m, const void* base, const PagedAttendArgs& a, int rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t D = (cuuint64_t)a.D, per = (cuuint64_t)a.Hkv * a.T.page;
  cuuint64_t dims[3] = {D, per, (cuuint64_t)a.T.n_pages};
  cuuint64_t strides[2] = {D, per * D};
  cuuint32_t box[3] = {(cuuint32_t)a.D, (cuuint32_t)rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, a.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, bool F32>
cudaError_t launch_warp_path(const PagedAttendArgs& a, bool join_only, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (!join_only) {
    CUtensorMap km, vm;
    if (!make_pool_map(&km, a.P.k, a, kSub) || !make_pool_map(&vm, a.P.v, a, kSub)) return cudaErrorInvalidValue;
    auto kernel = paged_attend_kernel<D, NT, F32>;
    e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), Shape<D, NT, F32>::kBytes);
    if (e == cudaSuccess)
      e = launch_kernel(kernel, dim3(a.ctas), dim3(Shape<D, NT, F32>::kThreads), Shape<D, NT, F32>::kBytes, s, 0, a, km, vm);
  }
  if (e == cudaSuccess) e = launch_combine<D>(a, CombineShape{8 * NT, kTile, Shape<D, NT, F32>::kWarps, 1, F32 ? 15.f : 7.f}, s);
  return e;
}

}  // namespace

cudaError_t launch_paged_attend_warp(const PagedAttendArgs& a, int row_tile, bool join_only, cudaStream_t s) {
  const bool f32 = a.act_fmt == CSA_FMT_F32;
  if (a.D == 128) {
    if (f32) return row_tile == 8 ? launch_warp_path<128, 1, true>(a, join_only, s) : launch_warp_path<128, 2, true>(a, join_only, s);
    return row_tile == 8 ? launch_warp_path<128, 1, false>(a, join_only, s) : launch_warp_path<128, 2, false>(a, join_only, s);
  }
  if (f32) return row_tile == 8 ? launch_warp_path<64, 1, true>(a, join_only, s) : launch_warp_path<64, 2, true>(a, join_only, s);
  return row_tile == 8 ? launch_warp_path<64, 1, false>(a, join_only, s) : launch_warp_path<64, 2, false>(a, join_only, s);
}

}  // namespace csa
