// paged_common.cuh -- what the kernels of attention over a paged cache share: arguments,
// sequences, and the warp that turns tiles of keys into rows of the cache.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace paged {

constexpr int kTile = 128;  // keys per tile
constexpr uint32_t kNoRow = 0xFFFFFFFFu;  // past the sequence's end

struct PagedArgs {
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const __nv_bfloat16* q;
  long long q_stride;  // elements between tokens
  __nv_bfloat16* o;
  float* lse;
  long long lse_head, lse_row;  // strides of lse
  const int32_t* cu_q;          // null: one token per sequence
  const int32_t* table;
  const int32_t* seqlens;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  int* status;
  int B, Hq, Hkv, G;
  int team, teams, sets;  // CTAs (key heads, or pairs of them when d = 64) of a team, teams, teams' worths of heads
  int total_q, max_q, max_k;
  int num_pages, page_size, max_pages;
  uint32_t page_mul, page_shift;    // division by page_size
  uint32_t group_mul, group_shift;  // and by G
  long long scale_bytes;          // of k_scales, v_scales
  // sequences of min_rows to max_rows rows (new tokens times G) are this kernel's
  int min_rows, max_rows;
  int causal;
  float scale_log2;
  // partial states, for N rows a unit
  int4* meta;       // [CTAs]: parts of the unit that begins in this CTA and ends in a later one
  int* part_rows;   // [CTAs, N] its rows' output rows (-1: none)
  float* part_m;    // [2 CTAs, N] reference, log2 units
  float* part_l;    // [2 CTAs, N] sum of the unrounded weights
  float* part_lr;   // [2 CTAs, N] the sum that divides O
  float* part_o;    // [2 CTAs, ...] O, N rows of 128 or d dims
  unsigned long long timeout_ns;
};

// Bounded waits, false also when another role of the CTA has given up.  A phase that is
// complete at the first look costs no more than that look (every lane's, so that nothing
// has to be handed over).
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity, unsigned long long timeout_ns,
                                            volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, timeout_ns) && !*abort_flag;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned long long timeout_ns,
                                          volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  bool ok = true;
  if (lane_id() == 0) ok = mbar_wait(bar, parity, timeout_ns) && !*abort_flag;
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// Sequence b: new tokens (at most max_q of them), keys and first packed row; nq = -1 when its
// offsets do not fit, 0 when it is not this kernel's.  lk0: how many keys are there before
// the new tokens (fewer than none when there are more tokens than keys), whether or not all
// the tokens are attended: token i sees keys 0 .. lk0 + i.
struct SeqInfo {
  int nq, lk, qoff, lk0;
};
__device__ __forceinline__ SeqInfo seq_info(const PagedArgs& a, int b) {
  SeqInfo s;
  s.lk = max(0, min(a.seqlens[b], a.max_k));
  if (a.cu_q == nullptr) {
    s.nq = 1;
    s.qoff = b;
    s.lk0 = s.lk - 1;
    return s;
  }
  s.qoff = a.cu_q[b];
  const int end = a.cu_q[b + 1];
  if (s.qoff < 0 || end < s.qoff || end > a.total_q) {
    s.nq = -1;
    return s;
  }
  s.lk0 = s.lk - (end - s.qoff);
  s.nq = min(end - s.qoff, a.max_q);
  if (s.nq * a.G < a.min_rows || s.nq * a.G > a.max_rows) s.nq = 0;  // another kernel's
  return s;
}

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// Invariant Integers using Multiplication", 1994): s = ceil(log2 d), m = floor(2^32 (2^s - d)
// / d) + 1, n / d = (hi(m n) + n) >> s.
__device__ __forceinline__ int page_index(const PagedArgs& a, int n) {
  return (int)((__umulhi(a.page_mul, (uint32_t)n) + (uint32_t)n) >> a.page_shift);
}
__device__ __forceinline__ int token_of_row(const PagedArgs& a, int n) {
  return (int)((__umulhi(a.group_mul, (uint32_t)n) + (uint32_t)n) >> a.group_shift);
}

__device__ __forceinline__ float redux_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// A ring of tiles in shared memory, written by the lookup warp: the rows of the flattened
// pages that hold the tile's keys (kNoRow past the sequence's end), the key head (or pair of
// heads), -1 after the last tile, and in 8 bits per key the words that hold its K and V
// scale bytes, one each, or two each (K, K, V, V) when the heads of a pair may lie in
// different words.  Rows and head arrive on `full`, once; the words, which are a trip to
// memory later, on `scaled`, once a lane.  (The two may be one barrier of 33 arrivals.)
// The readers arrive on `empty`.
struct PageRing {
  uint32_t* rows;
  volatile int* tile;
  uint32_t scales;  // shared-memory address
  uint64_t* full;
  uint64_t* scaled;
  uint64_t* empty;
};

// Run by one warp.  next(b, head, t0, t1, lk): the next stretch of tiles, false at the end.
// A page outside the cache is recorded and read as page 0.  The pages of a tile are loaded
// while the one before is written out.  Returns false when a wait gave up.
template <int kRing, bool kQ8, bool kPair, class Next>
__device__ __forceinline__ bool look_up_pages(const PagedArgs& a, const PageRing& ring, volatile int* abort_flag, Next next) {
  const int lane = lane_id();
  uint32_t c = 0;
  bool ok = true;
  auto publish = [&](const int(&page)[4], int key0, int lk, int head) {
    const uint32_t at = c % kRing;
    ok = warp_wait(ring.empty + at, ((c / kRing) & 1) ^ 1, a.timeout_ns, abort_flag);
    if (!ok) return;
    uint32_t row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key0 + lane + 32 * i;
      int pg = page[i];
      if (pg < 0 || pg >= a.num_pages) {  // never read outside the cache
        atomicExch(a.status, kStatusBadArg);
        pg = 0;
      }
      row[i] = key < lk ? (uint32_t)(pg * a.page_size + (key - page_index(a, key) * a.page_size)) : kNoRow;
      ring.rows[at * kTile + lane + 32 * i] = row[i];
    }
    if (lane == 0) ring.tile[at] = head;
    mbar_arrive_warp(ring.full + at);
    if constexpr (kQ8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (row[i] != kNoRow) {
          constexpr int kWords = kPair ? 2 : 1;
          // the words that hold the key's scale bytes (never past the arrays' ends)
          const uint32_t to = ring.scales + (at * kTile + lane + 32 * i) * 8 * kWords;
          const long long o = ((long long)row[i] * a.Hkv + (kPair ? 2 : 1) * head) & ~3LL;
          const int n0 = (int)min(4LL, a.scale_bytes - o), n1 = (int)max(0LL, min(4LL, a.scale_bytes - o - 4));
          cp_async4(to, a.k_scales + o, n0);
          cp_async4(to + 4 * kWords, a.v_scales + o, n0);
          if constexpr (kPair) {
            cp_async4(to + 4, a.k_scales + (n1 ? o + 4 : o), n1);
            cp_async4(to + 12, a.v_scales + (n1 ? o + 4 : o), n1);
          }
        }
      }
      cp_async_arrive(ring.scaled + at);
    }
    ++c;
  };
  int b, head, t0, t1, lk;
  while (ok && next(b, head, t0, t1, lk)) {
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    int page[4], ahead[4];
    auto look_up = [&](int t, int(&x)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = t * kTile + lane + 32 * i;
        x[i] = t < t1 && key < lk ? __ldg(table + page_index(a, key)) : 0;
      }
    };
    look_up(t0, ahead);
#pragma unroll 1
    for (int t = t0; ok && t < t1; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) page[i] = ahead[i];
      look_up(t + 1, ahead);
      publish(page, t * kTile, lk, head);
    }
  }
  if (ok) {
    const int none[4] = {0, 0, 0, 0};
    publish(none, 0, 0, -1);
  }
  if constexpr (kQ8) cp_async_wait_all();
  return ok;
}

// Programmatic dependent launch: the second kernel's blocks start when every block of the
// first has called grid_dependents_launch or ended, and wait for all of its writes.
__device__ __forceinline__ void grid_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ----------------------------------------------------------------------------- host side

// Launches a kernel that calls grid_dependency_wait before it touches memory, behind the
// stream's last one, whose end its own start overlaps.
inline cudaError_t launch_dependent(void (*kernel)(const PagedArgs), dim3 grid, int threads, size_t smem,
                                    cudaStream_t stream, const PagedArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
  const cudaError_t last = cudaGetLastError();  // consumed, or the next launch would report it
  return err != cudaSuccess ? err : last;
}

inline PagedArgs paged_args(const PagedLaunch& L) {
  PagedArgs a{};
  a.k_pages = static_cast<const uint8_t*>(L.k_pages);
  a.v_pages = static_cast<const uint8_t*>(L.v_pages);
  a.q = static_cast<const __nv_bfloat16*>(L.q);
  a.q_stride = L.q_stride;
  a.o = static_cast<__nv_bfloat16*>(L.o);
  a.lse = L.lse;
  a.lse_head = L.lse_head;
  a.lse_row = L.lse_row;
  a.cu_q = L.cu_q;
  a.table = L.table;
  a.seqlens = L.seqlens;
  a.k_scales = L.k_scales;
  a.v_scales = L.v_scales;
  a.status = static_cast<int*>(L.workspace);
  a.B = L.B;
  a.Hq = L.Hq;
  a.Hkv = L.Hkv;
  a.G = L.Hq / L.Hkv;
  a.total_q = L.total_q;
  a.max_q = L.max_q;
  a.max_k = L.max_k;
  a.num_pages = L.num_pages;
  a.page_size = L.page_size;
  auto divide_by = [](unsigned d, uint32_t& mul, uint32_t& shift) {
    shift = 0;
    while ((1ull << shift) < d) ++shift;
    mul = (uint32_t)((((1ull << shift) - d) << 32) / d + 1);
  };
  divide_by(L.page_size, a.page_mul, a.page_shift);
  divide_by(a.G, a.group_mul, a.group_shift);
  a.max_pages = L.max_pages;
  a.scale_bytes = (long long)L.num_pages * L.page_size * L.Hkv;
  a.causal = L.causal;
  a.scale_log2 = L.scale * 1.4426950408889634f;
  a.timeout_ns = L.timeout_ns;
  return a;
}

// Partial states of `ctas` CTAs, n rows of d dims a unit, behind the status word.
struct PagedCarve {
  size_t meta, rows, m, l, lr, o, bytes;
  void place(PagedArgs& a, void* workspace) const {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.meta = reinterpret_cast<int4*>(ws + meta);
    a.part_rows = reinterpret_cast<int*>(ws + rows);
    a.part_m = reinterpret_cast<float*>(ws + m);
    a.part_l = reinterpret_cast<float*>(ws + l);
    a.part_lr = reinterpret_cast<float*>(ws + lr);
    a.part_o = reinterpret_cast<float*>(ws + o);
  }
};
inline PagedCarve paged_carve(int ctas, int n, int d) {
  PagedCarve c;
  size_t at = kStatusBytes;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += (bytes + 255) & ~size_t(255);
    return x;
  };
  c.meta = take(sizeof(int4) * ctas);
  c.rows = take(sizeof(int) * ctas * n);
  c.m = take(sizeof(float) * 2 * ctas * n);
  c.l = take(sizeof(float) * 2 * ctas * n);
  c.lr = take(sizeof(float) * 2 * ctas * n);
  c.o = take(sizeof(float) * 2 * ctas * n * d);
  c.bytes = at;
  return c;
}

}  // namespace paged

}  // namespace fa
