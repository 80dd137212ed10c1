// cache_sm100.cu -- writing new keys and values into a paged cache, and reading a
// paged cache back, in bf16 or in 8 bits (B200, sm_100a).
//
// The 8 bit form of a row x (one token's slice of one key head, d values): with a
// the largest magnitude among its finite values,
//     e    = the smallest whole number in [-60, 60] with a <= 448 * 2^e,
//     code = the e4m3 value nearest x * 2^-e (ties to even; magnitudes over 448 to
//            448; infinities and NaN to NaN),
// stored as d code bytes and the scale byte e + 127; a code c stands for c * 2^e.
//  * The scale is a power of two: e4m3 is a floating format, so a finer scale would
//    win no relative precision (a code is off by at most 2^-4 of its value either
//    way), while c * 2^e is always a bf16 number (4 significant bits, exponents -69 to
//    68), so reading back rounds nothing and the attention kernels can apply the
//    scale exactly wherever it is cheapest.
//  * |e| <= 60 keeps the ratio of two rows' scales under 2^126, so an attention
//    kernel may carry the value scales inside its fp32 softmax weights.  Values over
//    448 * 2^60 saturate; below 2^-69 they lose bits, as subnormals do.
//
// Both kernels move each byte once and do next to nothing with it: they are bound
// by HBM for large calls and by the latency of three dependent loads (offsets, page
// table, then the stores; the rows themselves are loaded meanwhile) for small ones.
// A CTA takes a run of packed rows.  Its threads look at all sequences' offsets at
// once, each marking the rows that its sequence has in the run, which takes one
// round trip where a binary search per row takes log2 B; then one thread per row
// reads the page table.  Each thread moves 16 values (32 bytes of bf16, 16 of
// e4m3), so a row's maximum needs D / 16 neighbouring lanes.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kMaxRows = 128;  // packed rows per CTA

struct CacheArgs {
  const int32_t* cu;       // [B + 1] offsets of the packed rows
  const int32_t* seqlens;  // write: [B] keys per sequence after the write; null: sequences start at key 0
  const int32_t* table;    // [B, max_pages]
  int* status;
  int B, total, H, rows;   // rows: packed rows per CTA
  int num_pages, page_size, max_pages;
  long long k_stride, v_stride;  // write: elements between packed rows
};

// Cache row (page * page_size + place in it) of each of this CTA's packed rows r0 ..
// r0 + nr - 1, -1 for a row that no sequence has or whose page is not in the cache.
__device__ __forceinline__ void map_rows(const CacheArgs& a, int r0, int nr, long long* slot, int* seq, int* pos) {
  for (int r = threadIdx.x; r < nr; r += kCacheThreads) seq[r] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += kCacheThreads) {
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    int base = 0;
    bool bad = c0 < 0 || c1 < c0 || c1 > a.total;
    if (a.seqlens != nullptr && !bad) {
      base = a.seqlens[b] - (c1 - c0);  // position of the sequence's first new row
      bad = a.seqlens[b] < 0 || base < 0;
    }
    if (!bad) bad = (long long)base + (c1 - c0) > (long long)a.max_pages * a.page_size;
    if (bad) {
      if (blockIdx.x == 0) atomicExch(a.status, kStatusBadArg);
      continue;
    }
    for (int r = max(c0, r0); r < min(c1, r0 + nr); ++r) {
      seq[r - r0] = b;
      pos[r - r0] = base + (r - c0);
    }
  }
  __syncthreads();
  for (int r = threadIdx.x; r < nr; r += kCacheThreads) {
    long long s = -1;
    if (seq[r] >= 0) {
      const int page = a.table[(size_t)seq[r] * a.max_pages + pos[r] / a.page_size];
      if (page < 0 || page >= a.num_pages)
        atomicExch(a.status, kStatusBadArg);
      else
        s = (long long)page * a.page_size + pos[r] % a.page_size;
    }
    slot[r] = s;
  }
  __syncthreads();
}

// Two bf16 values, scaled by a power of two, to two e4m3 codes (an infinity becomes
// the NaN that satfinite leaves alone).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, float f) {
  float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
  if ((w & 0x00007FFFu) >= 0x00007F80u) lo = __uint_as_float(0x7FC00000u);
  if ((w & 0x7FFF0000u) >= 0x7F800000u) hi = __uint_as_float(0x7FC00000u);
  return __nv_cvt_float2_to_fp8x2(make_float2(lo * f, hi * f), __NV_SATFINITE, __NV_E4M3);
}

// Larger magnitude of each half, infinities and NaN left out.
__device__ __forceinline__ uint32_t max_finite2(uint32_t m, uint32_t w) {
  w &= 0x7FFF7FFFu;
  if ((w & 0xFFFFu) >= 0x7F80u) w &= 0xFFFF0000u;
  if ((w >> 16) >= 0x7F80u) w &= 0x0000FFFFu;
  return __vmaxu2(m, w);
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(kCacheThreads)
    cache_write_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v, uint8_t* k_pages,
                       uint8_t* v_pages, uint8_t* k_scales, uint8_t* v_scales, const CacheArgs a) {
  constexpr int kLanes = D / 16;  // lanes per (row, head)
  __shared__ long long slot[kMaxRows];
  __shared__ int seq[kMaxRows], pos[kMaxRows];
  const int r0 = blockIdx.x * a.rows, nr = min(a.rows, a.total - r0);
  const int per_row = a.H * kLanes, n = nr * per_row;
  // Whole warps run every trip, so that the maximum's shuffles have all lanes.  A trip loads
  // both tensors' values, and the next trip's before it uses them; the first trip's loads
  // cover the rows' look-up.
  auto load = [&](int c, uint4(&x)[4]) {
    if (c >= n) return;
    const int r = c / per_row, part = c - r * per_row;  // part: head * kLanes + lane of it
    const uint4* ks = reinterpret_cast<const uint4*>(k + (r0 + r) * a.k_stride) + 2 * part;
    const uint4* vs = reinterpret_cast<const uint4*>(v + (r0 + r) * a.v_stride) + 2 * part;
    x[0] = __ldcs(ks), x[1] = __ldcs(ks + 1), x[2] = __ldcs(vs), x[3] = __ldcs(vs + 1);
  };
  uint4 ahead[4] = {};
  load(threadIdx.x, ahead);
  map_rows(a, r0, nr, slot, seq, pos);
  for (int c0 = threadIdx.x & ~31; c0 < n; c0 += kCacheThreads) {
    const int c = c0 + lane_id();
    const int r = min(c, n - 1) / per_row, part = min(c, n - 1) - r * per_row;
    const long long s = c < n ? slot[r] : -1;
    uint4 now[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) now[i] = ahead[i];
    load(c + kCacheThreads, ahead);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4 x = now[2 * kv], y = now[2 * kv + 1];
      if constexpr (kQ8) {
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        m = max(m & 0xFFFFu, m >> 16);
        if (m >= 0x7F80u) {  // an infinity or NaN among them: left out
          m = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = max_finite2(m, w[i]);
          m = max(m & 0xFFFFu, m >> 16);
        }
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        // a = 1.f * 2^(E - 127) <= 1.75 * 2^(8 + e), f the 7 mantissa bits of the bf16 m
        const int e = min(60, max(-60, (int)(m >> 7) - 127 - ((m & 127u) <= 96u ? 8 : 7)));
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = e4m3_pair(w[2 * i], f) | (e4m3_pair(w[2 * i + 1], f) << 16);
        if (s >= 0) {
          reinterpret_cast<uint4*>((kv ? v_pages : k_pages) + (size_t)s * a.H * D)[part] = make_uint4(q[0], q[1], q[2], q[3]);
          if (part % kLanes == 0) (kv ? v_scales : k_scales)[(size_t)s * a.H + part / kLanes] = (uint8_t)(e + 127);
        }
      } else if (s >= 0) {
        uint4* dst = reinterpret_cast<uint4*>((kv ? v_pages : k_pages) + (size_t)s * a.H * D * 2) + 2 * part;
        dst[0] = x;
        dst[1] = y;
      }
    }
  }
}

// Four codes times 2^e as bf16 (exact): two words.
__device__ __forceinline__ uint2 bf16_of_codes(uint32_t q, float f) {
  const __half2 a = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q & 0xFFFFu), __NV_E4M3));
  const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> 16), __NV_E4M3));
  const float2 x = __half22float2(a), y = __half22float2(b);
  return make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(y.x * f, y.y * f));
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(const uint8_t* __restrict__ k_pages, const uint8_t* __restrict__ v_pages,
                      const uint8_t* __restrict__ k_scales, const uint8_t* __restrict__ v_scales, __nv_bfloat16* k,
                      __nv_bfloat16* v, const CacheArgs a) {
  constexpr int kLanes = D / 16;
  __shared__ long long slot[kMaxRows];
  __shared__ int seq[kMaxRows], pos[kMaxRows];
  const int r0 = blockIdx.x * a.rows, nr = min(a.rows, a.total - r0);
  map_rows(a, r0, nr, slot, seq, pos);
  const int per_row = a.H * kLanes, n = nr * per_row;
  for (int c = threadIdx.x; c < n; c += kCacheThreads) {
    const int r = c / per_row, part = c - r * per_row;
    const long long s = slot[r];
    if (s < 0) continue;
    if constexpr (kQ8) {
      // both tensors' loads first
      const size_t at = (size_t)s * a.H * D / 16 + part, row = (size_t)s * a.H + part / kLanes;
      const uint4 q[2] = {__ldcs(reinterpret_cast<const uint4*>(k_pages) + at), __ldcs(reinterpret_cast<const uint4*>(v_pages) + at)};
      const uint32_t e[2] = {__ldg(k_scales + row), __ldg(v_scales + row)};
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint4* dst = reinterpret_cast<uint4*>((kv ? v : k) + (size_t)(r0 + r) * a.H * D) + 2 * part;
        const float f = __uint_as_float(e[kv] << 23);
        const uint2 w0 = bf16_of_codes(q[kv].x, f), w1 = bf16_of_codes(q[kv].y, f), w2 = bf16_of_codes(q[kv].z, f),
                    w3 = bf16_of_codes(q[kv].w, f);
        __stcs(dst, make_uint4(w0.x, w0.y, w1.x, w1.y));
        __stcs(dst + 1, make_uint4(w2.x, w2.y, w3.x, w3.y));
      }
    } else {
      const size_t at = (size_t)s * a.H * D / 8 + 2 * part;
      const uint4* ks = reinterpret_cast<const uint4*>(k_pages) + at;
      const uint4* vs = reinterpret_cast<const uint4*>(v_pages) + at;
      const uint4 x[4] = {__ldcs(ks), __ldcs(ks + 1), __ldcs(vs), __ldcs(vs + 1)};
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint4* dst = reinterpret_cast<uint4*>((kv ? v : k) + (size_t)(r0 + r) * a.H * D) + 2 * part;
        __stcs(dst, x[2 * kv]);
        __stcs(dst + 1, x[2 * kv + 1]);
      }
    }
  }
}

// Rows per CTA: about `trips` chunks of 16 values per thread and tensor (each CTA looks its
// rows up once), fewer where that would leave SMs without a CTA.  Measured: 8192 tokens
// written with 2, 4, 8 and 16 trips 45.1, 42.4, 41.9 and 45.1 us; 16 sequences read with 2,
// 4 and 8 141.7, 143.1 and 148.8 us.
int rows_per_cta(int total, int H, int d, int trips) {
  const int per_row = H * (d / 16);
  const int full = std::max(1, trips * kCacheThreads / per_row);
  const int spread = std::max(1, total / (2 * num_sms()));
  return std::min({full, spread, kMaxRows});
}

template <int D, bool kQ8>
fa_status launch_cache_impl(const CacheLaunch& L, CacheArgs& a, unsigned grid, cudaStream_t stream) {
  if (L.write)
    cache_write_kernel<D, kQ8><<<grid, kCacheThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(L.k), static_cast<const __nv_bfloat16*>(L.v), static_cast<uint8_t*>(L.k_pages),
        static_cast<uint8_t*>(L.v_pages), L.k_scales, L.v_scales, a);
  else
    cache_read_kernel<D, kQ8><<<grid, kCacheThreads, 0, stream>>>(
        static_cast<const uint8_t*>(L.k_pages), static_cast<const uint8_t*>(L.v_pages), L.k_scales, L.v_scales,
        static_cast<__nv_bfloat16*>(L.k), static_cast<__nv_bfloat16*>(L.v), a);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

fa_status launch_cache(const CacheLaunch& L, cudaStream_t stream) {
  CacheArgs a;
  a.cu = L.cu;
  a.seqlens = L.write ? L.seqlens : nullptr;
  a.table = L.table;
  a.status = L.status;
  a.B = L.B;
  a.total = L.total;
  a.H = L.H;
  a.rows = rows_per_cta(L.total, L.H, L.d, L.write ? 8 : 2);
  a.num_pages = L.num_pages;
  a.page_size = L.page_size;
  a.max_pages = L.max_pages;
  a.k_stride = L.k_stride;
  a.v_stride = L.v_stride;
  const unsigned grid = (unsigned)((L.total + a.rows - 1) / a.rows);
  const int id = L.write ? kKCacheWrite : kKCacheRead;
  prof_before(stream, id);
  fa_status st;
  if (L.d == 64)
    st = L.q8 ? launch_cache_impl<64, true>(L, a, grid, stream) : launch_cache_impl<64, false>(L, a, grid, stream);
  else
    st = L.q8 ? launch_cache_impl<128, true>(L, a, grid, stream) : launch_cache_impl<128, false>(L, a, grid, stream);
  prof_after(stream, id);
  return st;
}

}  // namespace fa
