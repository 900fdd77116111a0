// Shared by the two kernels of csa_paged_attend: how the work is cut and dealt, and how cut segments
// are joined.
//
// A segment is one (sequence, block of query rows, KV head); a row is (token, head of the group).  Its
// visible keys lie in tiles of a fixed number of positions; some tiles make a unit, and all segments'
// units in order are dealt to the CTAs in equal runs.  A segment cut between CTAs leaves records (O,
// its two running maxima, the denominator) that the combine kernel joins.  The cut depends on the
// lengths alone, so results do not change from run to run.
#pragma once

#include <cuda_fp16.h>

#include "paged.h"

namespace csa {

namespace {

constexpr float kNone = -3.0e38f;             // a running maximum before any key: finite, below every logit

// Four e4m3 codes as two pairs of f16 values, exactly; NaN codes become NaN.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// NaN codes of four e4m3 bytes as a mask of 0x80 bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// One segment's tiles: [0, ta) and [tb, te) in units of 32 positions.
struct Seg {
  int b, rb, h;
  int j0, n;                                  // first token of the block, tokens of the sequence answered
  int start;
  int ta, tb, te, tiles, units;
};

__device__ __forceinline__ int answered(const PagedAttendArgs& a, int b, int* start) {
  const int64_t s = a.tok.start[b];
  int n = a.tok.n_new ? a.tok.n_new[b] : a.tok.Tq;
  n = n < 0 ? 0 : (n > a.tok.Tq ? a.tok.Tq : n);
  if (s < 0 || s >= a.n_max) n = 0;
  else if (s + n > a.n_max) n = (int)(a.n_max - s);
  *start = n ? (int)s : 0;
  return n;
}

// Fills the tile range of block rb (`tile` keys to a tile, `per` tiles to a unit).
__device__ __forceinline__ void seg_range(const PagedAttendArgs& a, Seg& s, int row_tile, int tile, int per) {
  const int r0 = s.rb * row_tile;
  s.j0 = r0 / a.G;
  if (s.j0 >= s.n) {
    s.ta = s.tb = s.te = s.tiles = s.units = 0;
    return;
  }
  int j1 = (r0 + row_tile - 1) / a.G;
  j1 = j1 < s.n ? j1 : s.n - 1;
  const int end = s.start + j1 + 1;
  int lo = 0, fa = 0;
  if (a.window > 0) {
    lo = s.start + s.j0 + 1 - a.window;
    lo = lo > 0 ? lo : 0;
    fa = a.first < lo ? a.first : lo;
  }
  s.ta = (fa + tile - 1) / tile;
  s.tb = lo / tile > s.ta ? lo / tile : s.ta;
  s.te = (end + tile - 1) / tile;
  if (s.tb > s.te) s.tb = s.te;
  s.tiles = s.ta + s.te - s.tb;
  s.units = (s.tiles + per - 1) / per;
}

__device__ __forceinline__ void seg_load(const PagedAttendArgs& a, Seg& s, int sb, int row_tile, int tile, int per) {
  s.b = sb / a.rb_max;
  s.rb = sb - s.b * a.rb_max;
  s.n = answered(a, s.b, &s.start);
  seg_range(a, s, row_tile, tile, per);
}

// This CTA's run of units [u0, u1) of all segments' units, and where it begins.
struct Run {
  int64_t u0, u1, total;
  int sb, h, unit;                            // (sequence, block), KV head and unit of the segment that hold u0
  int ctas;                                   // CTAs with work: no more than units
};

// Runs are equal numbers of units, or, where that makes the longest run at most `slack` units longer, whole segments:
// those leave no records to write and join.  Every warp finds the run for itself (a lane takes every 32nd part of the
// (sequence, block)s): with one scan over the whole CTA, its barriers and shared memory, this took 4 us of a
// kernel's start.
__device__ __forceinline__ Run find_run(const PagedAttendArgs& a, int row_tile, int tile, int per, int slack) {
  const int lane = threadIdx.x & 31;
  const int n = a.T.B * a.rb_max;
  const int each = (n + 31) >> 5;
  int64_t sum = 0;
  int cnt = 0, most = 0;
#pragma unroll 1
  for (int i = lane * each; i < (lane + 1) * each && i < n; ++i) {
    Seg s;
    seg_load(a, s, i, row_tile, tile, per);
    sum += s.units;
    cnt += s.units > 0;
    most = s.units > most ? s.units : most;
    // segments without work: nothing to join (the others' entries are written by whoever begins them)
    if (s.units == 0 && blockIdx.x == 0 && threadIdx.x < 32)
      for (int h = 0; h < a.Hkv; ++h) a.info[i * a.Hkv + h] = make_int2(0, 0);
  }
  sum *= a.Hkv;
  cnt *= a.Hkv;
  int64_t at = sum;
  int atc = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, at, o);
    const int upc = __shfl_up_sync(0xffffffffu, atc, o);
    if (lane >= o) {
      at += up;
      atc += upc;
    }
  }
  Run r;
  r.total = __shfl_sync(0xffffffffu, at, 31);
  const int segs = __shfl_sync(0xffffffffu, atc, 31);
  most = __reduce_max_sync(0xffffffffu, most);
  at -= sum;
  atc -= cnt;
  r.u0 = r.u1 = 0;
  r.sb = r.h = r.unit = 0;
  // units of a CTA, rounded down
  const int64_t share = r.total >> 32 ? r.total / a.ctas : (int64_t)((uint32_t)r.total / (uint32_t)a.ctas);
  const bool whole =
      (int64_t)(((uint32_t)segs + a.ctas - 1) / a.ctas) * most <= share + (r.total > share * a.ctas) + slack;
  const int64_t things = whole ? segs : r.total;
  r.ctas = things < a.ctas ? (int)things : a.ctas;
  if ((int)blockIdx.x >= r.ctas) return r;
  // things * c / ctas, without a wide division
  const int64_t each_q = whole ? (int64_t)((uint32_t)segs / (uint32_t)r.ctas) : (r.total < a.ctas ? 1 : share);
  const uint32_t each_r = (uint32_t)(things - each_q * r.ctas);
  const int64_t mine = whole ? atc : at, count = whole ? cnt : sum;
#pragma unroll 1
  for (int end = 0; end < 2; ++end) {
    const int64_t t = each_q * (blockIdx.x + end) + each_r * (blockIdx.x + end) / (uint32_t)r.ctas;
    if (t >= things) {                                        // only the last run's end
      r.u1 = r.total;
      break;
    }
    // the lane whose (sequence, block)s hold it
    const bool here = t >= mine && t < mine + count;
    int64_t u = at, k = mine;                                 // units and things before (sequence, block) i
    int i = lane * each, units = 0;
    if (here) {
#pragma unroll 1
      for (;; ++i) {
        Seg s;
        seg_load(a, s, i, row_tile, tile, per);
        units = s.units;
        const int64_t us = (int64_t)units * a.Hkv, ks = whole ? (units > 0 ? a.Hkv : 0) : us;
        if (t < k + ks) break;
        u += us;
        k += ks;
      }
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    i = __shfl_sync(0xffffffffu, i, from);
    units = __shfl_sync(0xffffffffu, units, from);
    u = __shfl_sync(0xffffffffu, u, from);
    k = t - __shfl_sync(0xffffffffu, k, from);                // things into it
    const int h = whole ? (int)k : (int)(k >> 32 ? k / units : (int64_t)((uint32_t)k / (uint32_t)units));
    const int unit = whole ? 0 : (int)(k - (int64_t)h * units);
    u += (int64_t)h * units + unit;
    if (end == 0) {
      r.u0 = u;
      r.sb = i;
      r.h = h;
      r.unit = unit;
    } else {
      r.u1 = u;
    }
  }
  return r;
}

// Position of a walk over the units of a run.
struct Walk {
  Seg s;
  int sb;
  int unit;                                   // of the segment
};

__device__ __forceinline__ void walk_start(const PagedAttendArgs& a, Walk& w, const Run& r, int row_tile, int tile,
                                           int per) {
  w.sb = r.sb;
  seg_load(a, w.s, w.sb, row_tile, tile, per);
  w.s.h = r.h;
  w.unit = r.unit;
}

__device__ __forceinline__ void walk_next(const PagedAttendArgs& a, Walk& w, int row_tile, int tile, int per) {
  if (++w.unit < w.s.units) return;
  w.unit = 0;
  if (++w.s.h < a.Hkv) return;
  w.s.h = 0;
  const int n = a.T.B * a.rb_max;
  do {
    ++w.sb;
    if (w.sb >= n) return;                    // only behind the last unit
    seg_load(a, w.s, w.sb, row_tile, tile, per);
  } while (w.s.units == 0);
}

__device__ __forceinline__ int tile_pos(const Seg& s, int i, int tile) {
  return (i < s.ta ? i : s.tb + (i - s.ta)) * tile;
}

// The factors that turn O, which is relative to its running maximum W and scaled by 2^shift, into the answer O * x * y:
// 2^(W - Z - shift) over the denominator L (relative to Z) with the sink's term.  A sink above Z becomes the reference, so
// that weights far below its own keep their ratio to it.  y is about the root of 2^(W - Z), a power of two: one factor
// would lose its digits below 2^-126 where all values' scales are near 2^-126.  0 for a row that saw nothing.
__device__ __forceinline__ float2 answer_factors(float W, float Z, float L, const float* sinks, int head, float shift) {
  if (Z == kNone && L == 0.f) return make_float2(0.f, 0.f);
  if (sinks) {
    const float s = sinks[head] * kLog2e, ref = fmaxf(Z, fminf(s, -kNone));
    L = L * exp2f(Z - ref) + exp2f(s - ref);
    Z = ref;
  }
  const float e = rintf(fminf(fmaxf(0.5f * (W - Z), -126.f), 126.f));
  return make_float2(exp2f(W - Z - e - shift) / L, __uint_as_float((uint32_t)((int)e + 127) << 23));
}

// Floats of one partial record: O [rows][D], then mw, mz, l per row.
__host__ __device__ constexpr size_t record_floats(int rows, int D) { return (size_t)rows * (D + 3); }

// Record `slot` of CTA q: its first segment may have begun before it (slot 0), its last may end after it
// (slot 1); a segment that begins in it is slot 1.
struct CombineShape {
  int rows, tile, per;                        // rows of a block, keys of a tile, tiles of a unit
  int groups;                                 // records of a part
  float shift;                                // O is scaled by 2^shift
};

// Joins the records of the segments that were cut: blockIdx.x is the segment, and the blocks of y share its
// rows, 1024 / D at a time.
template <int D>
__global__ void __launch_bounds__(256) paged_combine_kernel(const __grid_constant__ PagedAttendArgs a,
                                                            const __grid_constant__ CombineShape cs) {
  constexpr int kPass = 1024 / D;
  const int seg = blockIdx.x, rows = cs.rows;
  const int2 who = a.info[seg];
  if (who.x >= who.y) return;                                 // one CTA had all of it, or there was nothing
  if (who.x < 0 || who.y >= a.ctas) return;                   // never written: a wait gave up, and was reported
  Seg s;
  seg_load(a, s, seg / a.Hkv, rows, cs.tile, cs.per);
  s.h = seg % a.Hkv;
  const size_t floats = record_floats(rows, D);
  const int c = (threadIdx.x % (D / 4)) * 4;
  for (int r = blockIdx.y * kPass + threadIdx.x / (D / 4); r < rows; r += gridDim.y * kPass) {
    const int R = s.rb * rows + r, j = R / a.G, gr = R - j * a.G;
    if (j >= s.n) break;
    // records first .. last of the segment, `groups` to a CTA; CTA who.x's are its second ones
    const float* first = a.part + ((size_t)who.x * 2 + 1) * cs.groups * floats + r;
    const float* rest = a.part + (size_t)(who.x + 1) * 2 * cs.groups * floats + r;
    float W = kNone, Z = kNone, L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float* rec) {
      const float4 x = *reinterpret_cast<const float4*>(rec + (size_t)r * (D - 1) + c);
      const float w = rec[(size_t)rows * D], z = rec[(size_t)rows * (D + 1)], l = rec[(size_t)rows * (D + 2)];
      const float nw = fmaxf(W, w), nz = fmaxf(Z, z), f = exp2f(W - nw), f1 = exp2f(w - nw);
      L = L * exp2f(Z - nz) + l * exp2f(z - nz);
      v.x = v.x * f + x.x * f1; v.y = v.y * f + x.y * f1; v.z = v.z * f + x.z * f1; v.w = v.w * f + x.w * f1;
      W = nw;
      Z = nz;
    };
#pragma unroll 1
    for (int g = 0; g < cs.groups; ++g) {
      add(first + g * floats);
#pragma unroll 2
      for (int q = 0; q < who.y - who.x; ++q) add(rest + ((size_t)q * 2 * cs.groups + g) * floats);
    }
    const int head = s.h * a.G + gr;
    const float2 f = answer_factors(W, Z, L, a.sinks, head, cs.shift);
    const float out[4] = {v.x * f.x * f.y, v.y * f.x * f.y, v.z * f.x * f.y, v.w * f.x * f.y};
    const size_t at = (((size_t)s.b * a.tok.Tq + j) * a.H + head) * D + c;
    store_act4(a.out + at * act_bytes(a.act_fmt), a.act_fmt, 0, out);
  }
}

template <int D>
cudaError_t launch_combine(const PagedAttendArgs& a, const CombineShape& cs, cudaStream_t s) {
  const int passes = (cs.rows + 1024 / D - 1) / (1024 / D);
  return launch_kernel(paged_combine_kernel<D>, dim3((unsigned)(a.T.B * a.rb_max * a.Hkv), passes > 8 ? passes / 2 : passes),
                       dim3(256), 0, s, 0, a, cs);
}

}  // namespace
}  // namespace csa
