// Launch-argument structs and launchers of the paged 8-bit key/value cache (internal).
#pragma once

#include "kernels.h"

namespace csa {

// Device address, on the current device, of the word where the paged calls without a workspace report (kErrPage).  Apart
// from the library's other word, which every csa_device_error reads and clears: it would take these reports from whoever
// made the call.
cudaError_t page_error_word(int** p);

struct PageArgs {
  int32_t* table;           // [B][cap]
  int32_t* refs;            // [n_pages]; null only where a call allows it
  int64_t cap, n_pages;
  int B, page, page_log2;
};

struct PoolArgs {
  uint8_t* k;               // [n_pages][Hkv][page][D] e4m3
  uint8_t* v;
  float* ks;                // [n_pages][Hkv]
  float* vs;
};

// New tokens of sequence b: positions [start, start + n), none when start is negative.
struct TokenArgs {
  const int64_t* start;     // [B]
  const int32_t* n_new;     // [B] or null (all Tq)
  int Tq;
};

// Positions a row's new tokens can touch: at most this many pages.
inline int64_t pages_touched_max(int Tq, int page) { return ((int64_t)Tq + page - 2) / page + 1; }

struct PagedAppendArgs {
  PageArgs T;
  PoolArgs P;
  TokenArgs tok;
  int Hkv, D, act_fmt;
  const uint8_t* k_new;
  const uint8_t* v_new;
  int64_t kv_stride;        // elements between tokens
  int kmax;                 // pages_touched_max
  int* err;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s);

cudaError_t launch_pages_fork(const PageArgs& T, const int32_t* src, const int32_t* dst, int n, int* err,
                              cudaStream_t s);

struct PagesReserveArgs {
  PageArgs T;
  TokenArgs tok;
  int kmax;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* missing;
  int* err;
};
cudaError_t launch_pages_reserve(const PagesReserveArgs& a, cudaStream_t s);

cudaError_t launch_pages_free(const PageArgs& T, const int64_t* keep, const int64_t* begin, int64_t first, int* err,
                              cudaStream_t s);

struct PagesCompactArgs {
  PageArgs T;
  int max_moves;
  int32_t* move_src;
  int32_t* move_dst;
  int32_t* count;
  int* err;
};
cudaError_t launch_pages_compact(const PagesCompactArgs& a, cudaStream_t s);

struct PagesCopyArgs {
  PoolArgs P;
  int64_t n_pages;
  int64_t page_bytes;       // Hkv * page * D
  int Hkv;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;     // or null
  int n;
  int* err;
};
cudaError_t launch_pages_copy(const PagesCopyArgs& a, int num_sms, cudaStream_t s);

struct PagedAttendArgs {
  PageArgs T;
  PoolArgs P;
  TokenArgs tok;
  int H, Hkv, G, D, act_fmt, window, first;
  float scale_log2;         // logit scale * log2(e)
  int n_max;
  const uint8_t* q;
  int64_t q_stride;         // elements between tokens
  const float* sinks;       // [H] or null
  uint8_t* out;             // [B][Tq][H][D]
  int* err;
  // split work (see paged_attend.cu)
  int rb_max;               // row blocks per (sequence, KV head) at most
  int ctas;
  int2* info;               // [B * rb_max * Hkv] first and last CTA of a cut segment, written by every call
  float* part;              // [ctas][2] records
};
struct PagedPlan {
  int path;                 // 1: warp-level kernel, 2: tcgen05 kernel
  int row_tile;             // query rows (token, head of the group) per block
  int rb_max, ctas;
  size_t info, part, total;
};
PagedPlan paged_plan(int act_fmt, int B, int G, int Hkv, int D, int Tq, int num_sms);
// row_tile: 8 or 16
cudaError_t launch_paged_attend_warp(const PagedAttendArgs& a, int row_tile, bool join_only, cudaStream_t s);
// join_only: only the kernel that joins cut segments, over what the workspace holds (test aid)
cudaError_t launch_paged_attend(const PagedAttendArgs& a, const PagedPlan& p, bool join_only, cudaStream_t s);

}  // namespace csa
