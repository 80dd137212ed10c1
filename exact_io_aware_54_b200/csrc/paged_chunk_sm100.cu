// paged_chunk_sm100.cu -- attention of many new rows per sequence over a paged key/value
// cache in bf16 or 8 bits (B200, sm_100a): a prompt, or a later piece of one.
//
// The computation is that of paged_sm100.cu.  A unit is (sequence, key head, 256 rows), a
// row being (token, query head of the key head's group): G query heads share every key
// tile that is loaded, and a piece of 64 tokens with G = 4 fills a unit.  With this many
// rows per key the tensor cores and the exponentials are the floor, as in the dense
// forward, whose inner loop this is (fwd_sm100.cu, d = 128: scores and weights in tensor
// memory, two 128-row tiles that take turns, P V in two halves, lazy rescale).  What differs:
//
//  * Rows.  The softmax threads load their own row of Q (any token stride, any G) into the
//    swizzled tile and store their own row of O; a row's limit follows from its token.
//  * Keys.  Pages are looked up by the warp of paged_common.cuh; loader warps fill
//    the K and V tiles, each its keys of every tile.  bf16: 16-byte asynchronous copies.
//    8 bit: each lane loads 16 codes, multiplies by the row's scale and stores 16 bf16
//    values, all of the tile times 2^-60, which the softmax scale and the final 1 / l make
//    up for.  A code times its power of two is a bf16 number, so the softmax warps, which
//    bound the kernel, have nothing to add.  The conversion is integer shifts and one bf16
//    multiplication per pair of codes (dequantise2).
//  * Work split: the line of all units' tiles, causal ones counted, is cut into equal
//    parts, one per CTA (one CTA per SM).  A unit cut by a border leaves fp32 partial
//    states of its 256 rows, two at most per CTA, which a second kernel joins in order.
//    512 tokens over 16K keys (8 key heads, G = 4) are 64 units for 148 CTAs.
//  * Weights are rounded to bf16, the tensor cores' operand, and O is divided by the sum of
//    the rounded ones, as in the dense forward; lse comes from the unrounded sum.
//  * What it measures: 8192 causal tokens over themselves (32 heads of 128, bf16) 630 to
//    660 us inside a graph, by the clock under the power limit, and 690 as a call: 790 to 870
//    TFLOP/s.  The chain from scores to weights to the next scores bounds it, as it does the
//    dense forward (3600 of a tile's 4360 cycles; the products take 2100), which takes 575 us
//    for the same work.  16 ragged sequences of 64-wide heads 150 us a call.  512 tokens
//    over 16K keys (8 key heads), 8 bit: 204 us, where the conversion of the tiles by the
//    loader warps bounds it (6000 cycles a tile); of 64-wide heads 147 us.
//  * Warp roles (512 threads): 0 MMA issuer, 1 page lookup, 4-7 loaders (8 bits, d = 128:
//    2-7), 8-11 and 12-15 the softmax groups of the two row tiles.
#include "paged_common.cuh"

namespace fa {

using namespace paged;

namespace {

constexpr int kThreads = 512;
// registers per thread of the four warpgroups, out of 4 x 128
template <bool kQ8>
constexpr uint32_t kRegsIssue = kQ8 ? 72 : 88;
template <bool kQ8>
constexpr uint32_t kRegsLoad = kQ8 ? 72 : 56;
constexpr uint32_t kRegsSoftmax = 184;
static_assert(kRegsIssue<true> + kRegsLoad<true> + 2 * kRegsSoftmax <= 4 * 128 &&
                  kRegsIssue<false> + kRegsLoad<false> + 2 * kRegsSoftmax <= 4 * 128,
              "register split exceeds the launch budget");
// Loader warps, up to warp 7.  Converting 8 bit tiles of 128-wide heads is what bounds the
// kernel, so the two warps beside the MMA issuer and the page lookup help.
template <int D, bool kQ8>
constexpr int kLoaders = kQ8 && D == 128 ? 6 : 4;
constexpr uint32_t kTmemCols = 512;
constexpr int kUnitRows = 256;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kTwo60 = 1152921504606846976.f;
__host__ __device__ constexpr uint32_t tm_s(int t) { return t * 128u; }
template <int D>
__host__ __device__ constexpr uint32_t tm_o(int t) {
  return 256u + t * (uint32_t)D;
}

template <int D>
struct ChunkLayout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kBoxBytes = 128 * 128;  // a 64-column (128-byte) block of a tile's rows
  static constexpr int kStages = D == 64 ? 8 : 4;
  static constexpr int kRing = 8;               // tiles that the page lookup may be ahead
  static constexpr int kOffSlots = 2 * kTileBytes;  // behind the two Q tiles
  static constexpr int kOffScales = kOffSlots + kStages * kTileBytes;
  static constexpr int kOffRows = kOffScales + kRing * kTile * 8;
  static constexpr int kOffTile = kOffRows + kRing * kTile * 4;
  static constexpr int kOffBar = kOffTile + kRing * 4;
  static constexpr int kPieces = 4;  // pieces that the page lookup may be ahead
  // kv_full[S], kv_empty[S], rows_full[R], rows_empty[R], q_full[2], s_full[2], p_half[2], p_full[2], o_done[2],
  // piece_full[P], piece_empty[P]
  static constexpr int kNumBars = 2 * kStages + 2 * kRing + 10 + 2 * kPieces;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kPieceBytes = 64;
  static constexpr int kOffPieces = (kOffMisc + 8 + 15) & ~15;
  static constexpr int kOffCodes = kOffPieces + kPieces * kPieceBytes;  // 8 bit: the loaders' codes, 128 keys of d
  static constexpr int kSmemBytes = kOffCodes + kTile * D + 1024;   // + alignment slack
  static_assert(kSmemBytes <= 232448, "shared memory of one SM");
};

// This CTA's stretch [pos, end) of the line of tiles: it begins t into what unit `unit` of
// head hk of sequence b counts.
struct Work {
  long long pos, end, total;
  int b, hk, unit, t;
  int ctas;  // CTAs that have a stretch
};

// Keys that rows up to `row` of a unit's sequence see, and the tiles of them (one, fully
// masked, when there are none).
__device__ __forceinline__ int keys_of(const PagedArgs& a, const SeqInfo& s, int row) {
  if (!a.causal) return s.lk;
  const int token = min(token_of_row(a, row), s.nq - 1);
  return max(0, min(s.lk, s.lk0 + token + 1));
}
__device__ __forceinline__ int tiles_of(int keys) { return max(1, (keys + kTile - 1) / kTile); }
__device__ __forceinline__ int units_of(const PagedArgs& a, int nq) {
  return nq <= 0 ? 0 : (nq * a.G + kUnitRows - 1) / kUnitRows;
}
// A unit's start and end (Q in, O out, the pipeline filled and drained) take about as long as
// two or three tiles, so each unit counts kUnitCost tiles more, at its beginning: without
// them the CTAs of many short units (a prompt's first rows) came 13% after the mean.  (1, 2, 3
// and 4: 165, 146, 147 and 144 us for 16 ragged sequences of 64-wide heads, 617 to 652 us for
// 8192 tokens without an order.  Counting a tile of a unit with up to 128 rows four fifths of
// another won 2% of the ragged sequences.)
constexpr int kUnitCost = 3;
// Tiles of unit u of a key head, and what it counts.
__device__ __forceinline__ int unit_tiles(const PagedArgs& a, const SeqInfo& s, int u) {
  return tiles_of(keys_of(a, s, u * kUnitRows + kUnitRows - 1));
}
__device__ __forceinline__ int unit_cost(const PagedArgs& a, const SeqInfo& s, int u) {
  return unit_tiles(a, s, u) + kUnitCost;
}
struct Piece {
  int b, hk, unit, t0, t1, tiles;  // tiles t0 .. t1 - 1 of the unit's
  int parts;                       // 0: the whole unit; else, where it begins the unit: parts that it is cut into
  SeqInfo s;
};
__device__ __forceinline__ bool next_piece(const PagedArgs& a, Work& w, Piece& p) {
  while (w.pos < w.end) {
    p.s = seq_info(a, w.b);
    if (w.hk >= a.Hkv || p.s.nq <= 0) {  // past the sequence's last head, or no rows: the next sequence
      if (++w.b >= a.B) return false;
      w.hk = w.unit = w.t = 0;
      continue;
    }
    p.b = w.b;
    p.hk = w.hk;
    p.unit = w.unit;
    p.tiles = unit_tiles(a, p.s, w.unit);
    const int cost = p.tiles + kUnitCost, c0 = w.t, c1 = (int)min((long long)cost, c0 + (w.end - w.pos));
    p.t0 = max(0, c0 - kUnitCost);
    p.t1 = max(0, c1 - kUnitCost);
    w.pos += c1 - c0;
    // the CTA that has the end of the unit's cost, counted from this one
    p.parts = c1 < cost || p.t0 > 0 ? (int)(((w.pos + cost - c1) * w.ctas - 1) / w.total) - (int)blockIdx.x + 1 : 0;
    w.t = c1;
    if (c1 == cost) {
      w.t = 0;
      if (++w.unit == units_of(a, p.s.nq)) {
        w.unit = 0;
        ++w.hk;
      }
    }
    if (p.t1 > p.t0) return true;  // else only of what the unit counts more: the next CTA begins it
  }
  return false;
}

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// Run by one warp: the line's length and where this CTA's stretch begins.  The lanes take
// the sequences, each walking its units (some 30 cycles each), or, where chunks are long,
// the units of one sequence after the other (some 700 cycles each sequence).
__device__ __forceinline__ Work find_work(const PagedArgs& a) {
  const int lane = lane_id();
  Work w;
  // what one key head counts: by the whole warp
  auto head_cost = [&](const SeqInfo& s) {
    int n = 0;
    const int units = units_of(a, s.nq);
    for (int u = lane; u < units; u += 32) n += unit_cost(a, s, u);
    return warp_sum(n);
  };
  // the same by one lane
  auto cost_alone = [&](const SeqInfo& s) {
    int n = 0;
    const int units = units_of(a, s.nq);
    for (int u = 0; u < units; ++u) n += unit_cost(a, s, u);
    return n;
  };
  const bool by_units = units_of(a, a.max_q) > 24 * a.B;
  auto info = [&](int b) {
    const SeqInfo s = seq_info(a, b);
    if (s.nq < 0 && blockIdx.x == 0) atomicExch(a.status, kStatusBadArg);
    return s;
  };
  long long total = 0;
  if (by_units) {
    for (int b = 0; b < a.B; ++b) total += (long long)head_cost(info(b)) * a.Hkv;
  } else {
    for (int b = lane; b < a.B; b += 32) total += (long long)cost_alone(info(b)) * a.Hkv;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  }
  w.total = total;
  w.ctas = (int)min((long long)gridDim.x, total);
  w.b = w.hk = w.unit = w.t = 0;
  w.pos = w.end = 0;
  if ((int)blockIdx.x >= w.ctas) return w;
  w.pos = total * blockIdx.x / w.ctas;
  w.end = total * (blockIdx.x + 1) / w.ctas;
  // the sequence
  long long before = 0;
  int per_head = 0;
  if (by_units) {
    for (;; ++w.b) {
      per_head = head_cost(seq_info(a, w.b));
      if (before + (long long)per_head * a.Hkv > w.pos) break;
      before += (long long)per_head * a.Hkv;
    }
  } else {
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int alone = b0 + lane < a.B ? cost_alone(seq_info(a, b0 + lane)) : 0;
      const long long mine = (long long)alone * a.Hkv;
      long long upto = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + upto > w.pos);
      if (hit != 0) {
        const int src = __ffs(hit) - 1;
        w.b = b0 + src;
        before += __shfl_sync(0xffffffffu, upto - mine, src);
        per_head = __shfl_sync(0xffffffffu, alone, src);
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  // the head, then the unit
  const SeqInfo s = seq_info(a, w.b);
  int rest = (int)(w.pos - before);
  w.hk = rest / per_head;
  rest -= w.hk * per_head;
  const int units = units_of(a, s.nq);
  for (int u0 = 0; u0 < units; u0 += 32) {
    const int mine = u0 + lane < units ? unit_cost(a, s, u0 + lane) : 0;
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, upto > rest);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      w.unit = u0 + src;
      w.t = rest - __shfl_sync(0xffffffffu, upto - mine, src);
      break;
    }
    rest -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return w;
}

// S = Q K^T, 128 x 128: as in the dense forward.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, SDesc q, SDesc k) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 2;  // 16-byte units
    umma_ss(d_tmem, sdesc_at(q, off), sdesc_at(k, off), idesc, kk > 0 ? 1u : 0u);
  }
}
// O (+)= P V for keys 64 half .. 64 half + 63, P bf16 in tensor memory.
template <int D>
__device__ __forceinline__ void issue_pv_half(uint32_t o_tmem, uint32_t p_tmem, SDesc v, bool accumulate, int half) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, D, false, true);
#pragma unroll
  for (int k4 = 0; k4 < 4; ++k4) {
    const int kk = 4 * half + k4;
    umma_ts(o_tmem, p_tmem + kk * 8, sdesc_at(v, kk * 128), idesc, (accumulate || kk > 0) ? 1u : 0u);
  }
}

// Two e4m3 codes times 2^e as bf16, times 2^-60, from t with the codes in its high bytes
// (bits 8-15 and 24-31) and f = 2^(e + 60) twice.  A code's 7 magnitude bits, moved down by
// 4, are a bf16 number 2^120 too small, subnormal codes included, so one exact
// multiplication is left: by 2^(e + 120), of which bf16 holds 2^(e + 60) for every e in
// [-60, 60].  (The smallest product, 2^-9 of the lowest scale, is 2^-129: a bf16 subnormal,
// still exact.)
// m: the magnitudes moved down; 0x7F0 tells of a NaN (code 127), which comes out as a number.
__device__ __forceinline__ uint32_t dequantise2(uint32_t t, uint32_t f, uint32_t& m) {
  m = (t >> 4) & 0x07F007F0u;
  const uint32_t x = (t & 0x80008000u) | m;
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(f));
  return y;
}
// Four codes; top: the largest m so far in either half.
__device__ __forceinline__ uint2 dequantise4(uint32_t q, uint32_t f, uint32_t& top) {
  uint32_t m0, m1;
  const uint2 y = make_uint2(dequantise2(__byte_perm(q, 0, 0x1404), f, m0), dequantise2(__byte_perm(q, 0, 0x3424), f, m1));
  top = __vimax3_u16x2(top, m0, m1);
  return y;
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(const __grid_constant__ PagedArgs a) {
  using L = ChunkLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* kv_empty = kv_full + L::kStages;
  uint64_t* rows_full = kv_empty + L::kStages;
  uint64_t* rows_empty = rows_full + L::kRing;
  uint64_t* q_full = rows_empty + L::kRing;
  uint64_t* s_full = q_full + 2;
  uint64_t* p_half = q_full + 4;
  uint64_t* p_full = q_full + 6;
  uint64_t* o_done = q_full + 8;
  uint64_t* piece_full = q_full + 10;
  uint64_t* piece_empty = piece_full + L::kPieces;
  uint32_t* ring_rows = reinterpret_cast<uint32_t*>(smem + L::kOffRows);
  volatile int* ring_tile = reinterpret_cast<volatile int*>(smem + L::kOffTile);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  const uint32_t warp = warp_id(), lane = lane_id();
  // The lookup warp walks the line and publishes each piece to the MMA issuer and the softmax
  // warps (tiles = 0 after the last); one copy of the walk keeps the kernel's code small.
  static_assert(sizeof(Piece) <= L::kPieceBytes, "a piece fits");
  auto piece_at = [&](uint32_t n) { return reinterpret_cast<Piece*>(smem + L::kOffPieces + n % L::kPieces * L::kPieceBytes); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(kv_full + s, kQ8 ? kLoaders<D, kQ8> : 128);  // a loader warp, or each copying lane
      mbar_init(kv_empty + s, 1);
    }
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(rows_full + i, kQ8 ? 33 : 1);
      mbar_init(rows_empty + i, kLoaders<D, kQ8>);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full + t, 4);
      mbar_init(s_full + t, 1);
      mbar_init(p_half + t, 4);
      mbar_init(p_full + t, 4);
      mbar_init(o_done + t, 1);
    }
    for (int i = 0; i < L::kPieces; ++i) {
      mbar_init(piece_full + i, 1);
      mbar_init(piece_empty + i, 9);
    }
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  // up to here the kernel before may still run
  grid_dependency_wait();
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto give_up = [&]() {
    *abort_flag = 1;
    atomicCAS(a.status, 0, kStatusTimeout);
  };

  // ------------------------------------------------------------------ loaders
  auto load_tiles = [&]() {
    constexpr int kChunks = D * (kQ8 ? 1 : 2) / 16;  // 16-byte pieces of a cache row's slice
    constexpr int kKeys = 32 / kChunks;              // keys per step of the warp
    // steps of the warps past 3, and of 2 and 3 if they load
    constexpr int kMost = kLoaders<D, kQ8> == 6 ? 24 / kKeys : 32 / kKeys, kFew = kLoaders<D, kQ8> == 6 ? 16 / kKeys : kMost;
    const int steps = warp < 4 ? kFew : kMost;
    const uint32_t row_bytes = (uint32_t)a.Hkv * D * (kQ8 ? 1 : 2);
    const int chunk = lane % kChunks, sub = lane / kChunks, first = kTile - (warp < 4 ? 4 * kMost + (4 - (int)warp) * kFew : (8 - (int)warp) * kMost) * kKeys;
    const uint32_t ring = smem_u32(ring_rows), words = smem_u32(smem + L::kOffScales);
    bool ok = true;
    // head of tile c, -1 after the last; row of key first + i kKeys + sub
    auto head_of = [&](uint32_t c) {
      ok = warp_wait(rows_full + c % L::kRing, (c / L::kRing) & 1, a.timeout_ns, abort_flag);
      return ok ? ring_tile[c % L::kRing] : -1;
    };
    auto row_of = [&](uint32_t c, int i) { return ld_shared_u32(ring + ((c % L::kRing) * kTile + first + i * kKeys + sub) * 4); };
    auto tile_of = [&](uint32_t g) { return smem_u32(smem + L::kOffSlots + (g % L::kStages) * L::kTileBytes); };
    auto wait_empty = [&](uint32_t g) {
      ok = warp_wait(kv_empty + g % L::kStages, ((g / L::kStages) & 1) ^ 1, a.timeout_ns, abort_flag);
      return ok;
    };
    int hk = head_of(0);
    if constexpr (kQ8) {
      // Slot after slot (K, V of tile 0, K of tile 1, ..).  Each lane's 16 codes of a step
      // come by an asynchronous copy to a place that only it reads, a slot ahead: no
      // registers held, and the loop stays at one step's instructions.  (Unrolled over a
      // slot or more, loads in registers, the loaders and the softmax together outgrew
      // the instruction cache: 8192 tokens 1190 us.)
      constexpr int kTogether = 2;  // steps converted side by side (one: 981 us; four: as two)
      const uint32_t codes = smem_u32(smem + L::kOffCodes) + (first * D) + lane * 16;
      auto copy = [&](uint32_t g, int head, int i) {
        const uint32_t row = row_of(g >> 1, i);
        const uint8_t* src = (g & 1 ? a.v_pages : a.k_pages) + (size_t)head * D + chunk * 16;
        cp_async16_or_zero(codes + i * 512, src + (uint64_t)(row != kNoRow ? row : 0u) * row_bytes, row != kNoRow);
      };
      if (hk >= 0) {
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
          copy(0, hk, i);
          cp_async_commit();
        }
      }
#pragma unroll 1
      for (uint32_t g = 0; hk >= 0; ++g) {
        const int next = g & 1 ? head_of((g >> 1) + 1) : hk;
        if (!ok || !wait_empty(g)) break;
        const uint32_t tile = tile_of(g) + (chunk >> 2) * L::kBoxBytes;
        const uint32_t word_at = words + (((g >> 1) % L::kRing) * kTile + first + sub) * 8 + (g & 1) * 4;
#pragma unroll 1
        for (int i0 = 0; i0 < steps; i0 += kTogether) {
          uint32_t row[kTogether], word[kTogether];
          uint4 x[kTogether];
          if (warp < 4)
            cp_async_wait<kFew - kTogether>();
          else
            cp_async_wait<kMost - kTogether>();
#pragma unroll
          for (int j = 0; j < kTogether; ++j) {
            row[j] = row_of(g >> 1, i0 + j);
            word[j] = ld_shared_u32(word_at + (i0 + j) * kKeys * 8);
            ld_shared_v4(codes + (i0 + j) * 512, x[j].x, x[j].y, x[j].z, x[j].w);
          }
#pragma unroll
          for (int j = 0; j < kTogether; ++j) {
            const int key = first + (i0 + j) * kKeys + sub;
            const uint32_t cut = ((row[j] * (uint32_t)a.Hkv + hk) & 3u) * 8;
            // past the sequence's end the codes are zeros, and the word holds anything
            const uint32_t f = row[j] != kNoRow ? ((((word[j] >> cut) & 0xFFu) + 60u) << 7) * 0x00010001u : 0u;
            uint32_t top = 0;
            const uint2 w0 = dequantise4(x[j].x, f, top), w1 = dequantise4(x[j].y, f, top),
                        w2 = dequantise4(x[j].z, f, top), w3 = dequantise4(x[j].w, f, top);
            const uint32_t to = tile + key * 128, c2 = 2 * (chunk & 3);  // 16-byte chunks of the bf16 row: c2 and c2 + 1
            st_shared_v4(to + ((c2 ^ (key & 7)) << 4), w0.x, w0.y, w1.x, w1.y);
            st_shared_v4(to + (((c2 + 1) ^ (key & 7)) << 4), w2.x, w2.y, w3.x, w3.y);
            if (((top + 0x00100010u) & 0x08000800u) != 0) {  // NaN among the 16: once more, one by one
#pragma unroll 1
              for (int i = 0; i < 16; ++i)
                if ((ld_shared_u8(codes + (i0 + j) * 512 + i) & 0x7F) == 0x7F)
                  st_shared_u16(to + (((c2 + i / 8) ^ (key & 7)) << 4) + (i % 8) * 2, 0x7FC0);
            }
          }
#pragma unroll
          for (int j = 0; j < kTogether; ++j) {
            if (next >= 0) copy(g + 1, next, i0 + j);  // (the codes have been read: they were used above)
            cp_async_commit();
          }
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(kv_full + g % L::kStages);
        if (g & 1) mbar_arrive_warp(rows_empty + (g >> 1) % L::kRing);
        hk = next;
      }
    } else {
      // Landed copies arrive by themselves, and the MMA issuer fences them: with four slots
      // a hand-over by the loaders comes too late (8192 tokens of 64-wide heads 311, not 298 us).
#pragma unroll 1
      for (uint32_t g = 0; hk >= 0; ++g) {
        const uint8_t* src = (g & 1 ? a.v_pages : a.k_pages) + (size_t)hk * D * 2 + chunk * 16;
        if (!wait_empty(g)) break;
        const uint32_t tile = tile_of(g) + (chunk >> 3) * L::kBoxBytes;
#pragma unroll 1
        for (int i0 = 0; i0 < kMost; i0 += 8) {
          uint32_t rw[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) rw[i] = row_of(g >> 1, i0 + i);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int key = first + (i0 + i) * kKeys + sub;
            const bool have = rw[i] != kNoRow;
            cp_async16_or_zero(tile + key * 128 + (((chunk & 7) ^ (key & 7)) << 4), src + (uint64_t)(have ? rw[i] : 0u) * row_bytes, have);
          }
        }
        cp_async_arrive(kv_full + g % L::kStages);
        if (g & 1) {
          mbar_arrive_warp(rows_empty + (g >> 1) % L::kRing);
          hk = head_of((g >> 1) + 1);
        }
      }
    }
    if (!ok && lane == 0) give_up();
    cp_async_wait_all();
  };

  if (warp < (kQ8 ? 8 : 4)) {
    regs_dec<kRegsIssue<kQ8>>();
    if (warp == 1) {
      // ------------------------------------------------------------------ page lookup
      const PageRing ring{ring_rows, ring_tile, smem_u32(smem + L::kOffScales), rows_full, rows_full, rows_empty};
      Work w = find_work(a);
      uint32_t n = 0;
      bool fine = true;
      auto publish = [&](const Piece& p) {
        fine = warp_wait(piece_empty + n % L::kPieces, ((n / L::kPieces) & 1) ^ 1, a.timeout_ns, abort_flag);
        if (!fine) return;
        if (lane == 0) *piece_at(n) = p;
        mbar_arrive_warp(piece_full + n % L::kPieces);
        ++n;
        // its rows of Q into L2, some tiles before they are wanted
        const int rows = p.tiles == 0 ? 0 : min(kUnitRows, p.s.nq * a.G - p.unit * kUnitRows);
#pragma unroll 1
        for (int i = lane; i < rows; i += 32) {
          const int row = p.unit * kUnitRows + i, token = token_of_row(a, row);
          const __nv_bfloat16* from = a.q + (long long)(p.s.qoff + token) * a.q_stride + (long long)(p.hk * a.G + row - token * a.G) * D;
          prefetch_l2(from);
          if (D == 128) prefetch_l2(from + 64);
        }
      };
      bool ok = look_up_pages<L::kRing, kQ8, false>(a, ring, abort_flag, [&](int& b, int& hk, int& t0, int& t1, int& lk) {
        Piece p;
        const bool more = next_piece(a, w, p);
        if (!more) p.tiles = 0;
        publish(p);
        b = p.b, hk = p.hk, t0 = p.t0, t1 = p.t1, lk = p.s.lk;
        return more && fine;
      });
      ok = ok && fine;
      if (!ok && lane == 0) give_up();
    } else if (warp == 0 && elect_one()) {
      // ------------------------------------------------------------------ MMA issuer
      const uint32_t base = smem_u32(smem);
      const SDesc q_desc[2] = {sdesc_make(base, 16, 1024), sdesc_make(base + L::kTileBytes, 16, 1024)};
      const SDesc ring_k = sdesc_make(base + L::kOffSlots, 16, 1024);            // K tiles, K-major
      const SDesc ring_v = sdesc_make(base + L::kOffSlots, L::kBoxBytes, 1024);  // V tiles, MN-major
      constexpr uint32_t kSlot16 = L::kTileBytes / 16;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !thread_wait(bar, parity, a.timeout_ns, abort_flag)) {
          give_up();
          ok = false;
        }
        return ok;
      };
      uint32_t g = 0, q_cnt[2] = {0, 0}, p_cnt[2] = {0, 0};
      auto slot_ready = [&](uint32_t i) {
        if (!wait(kv_full + i % L::kStages, (i / L::kStages) & 1)) return false;
        if constexpr (!kQ8) fence_proxy_async_smem();  // the loaders' copies, before the tensor core reads them
        tc_fence_after();
        return true;
      };
      for (uint32_t n = 0; wait(piece_full + n % L::kPieces, (n / L::kPieces) & 1); ++n) {
        const Piece& p = *piece_at(n);
        if (p.tiles == 0) break;
        const int t0 = p.t0, t1 = p.t1;
        // tiles of the unit that each row tile needs; the second may have no row
        const int rows = p.s.nq * a.G - p.unit * kUnitRows;
        const int nt[2] = {min(t1, tiles_of(keys_of(a, p.s, p.unit * kUnitRows + 127))), rows > 128 ? t1 : t0};
        bool have[2] = {t0 < nt[0], t0 < nt[1]};
        if (!slot_ready(g)) break;
        {
          const SDesc k = SDesc{ring_k.lo + (g % L::kStages) * kSlot16, ring_k.hi};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 0 || rows > 128) {
              if (!wait(q_full + t, q_cnt[t]++ & 1)) break;
              tc_fence_after();
              if (!have[t]) umma_commit(o_done + t);  // nothing to do for it
            }
            if (have[t]) {
              issue_qk<D>(tmem + tm_s(t), q_desc[t], k);
              umma_commit(s_full + t);
            }
          }
          if (!ok) break;
          umma_commit(kv_empty + g % L::kStages);
          ++g;
        }
        for (int j = t0; j < t1 && ok; ++j) {
          const uint32_t gv = g++, slot_v = gv % L::kStages;
          if (!slot_ready(gv)) break;
          const SDesc v = SDesc{ring_v.lo + slot_v * kSlot16, ring_v.hi};
          const bool more = j + 1 < t1;
          // the next K as well, before the weights are waited for: off the chain of a tile
          // from its weights to its next scores
          if (more && !slot_ready(g)) break;
          const SDesc k = SDesc{ring_k.lo + (g % L::kStages) * kSlot16, ring_k.hi};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (j < nt[t]) {
              if (!wait(p_half + t, p_cnt[t] & 1)) break;
              tc_fence_after();
              issue_pv_half<D>(tmem + tm_o<D>(t), tmem + tm_s(t), v, j > t0, 0);
              if (!wait(p_full + t, p_cnt[t] & 1)) break;
              tc_fence_after();
              ++p_cnt[t];
              issue_pv_half<D>(tmem + tm_o<D>(t), tmem + tm_s(t), v, true, 1);
              // a row tile's end and its next beginning overlap the other's last tile
              if (j + 1 == nt[t]) umma_commit(o_done + t);
            }
            if (more && j + 1 < nt[t]) {
              issue_qk<D>(tmem + tm_s(t), q_desc[t], k);
              umma_commit(s_full + t);
            }
          }
          if (!ok) break;
          umma_commit(kv_empty + slot_v);
          if (more) {
            umma_commit(kv_empty + g % L::kStages);
            ++g;
          }
        }
        if (!ok) break;
        mbar_arrive(piece_empty + n % L::kPieces);
      }
    } else if (kQ8 && warp != 0 && warp >= 8 - kLoaders<D, kQ8>) {
      load_tiles();
    }
  } else if (!kQ8 && warp < 8) {
    regs_dec<kRegsLoad<kQ8>>();
    load_tiles();
  } else {
    regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax groups
    const int t = (warp - 8) >> 2;
    const uint32_t quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile
    const uint32_t lanes = (quarter * 32) << 16;
    const uint32_t tS = tmem + lanes + tm_s(t), tO = tmem + lanes + tm_o<D>(t);
    const float scale_log2 = a.scale_log2 * (kQ8 ? kTwo60 : 1.f);  // the 8 bit tiles are 2^-60 of their values
    uint32_t s_cnt = 0, items = 0;
    for (uint32_t n = 0;; ++n) {
      if (!warp_wait(piece_full + n % L::kPieces, (n / L::kPieces) & 1, a.timeout_ns, abort_flag)) {
        if (lane == 0) give_up();
        break;
      }
      const Piece& p = *piece_at(n);
      if (p.tiles == 0) break;
      const int row0 = p.unit * kUnitRows + t * 128;
      const int rows = p.s.nq * a.G - row0;  // of this tile
      if (rows <= 0) {                       // (the second tile of a short unit)
        mbar_arrive_warp(piece_empty + n % L::kPieces);
        continue;
      }
      const int row = row0 + r, token = token_of_row(a, row), head = p.hk * a.G + (row - token * a.G);
      const bool mine = r < rows;
      // Q: every MMA that read the tile has completed (o_done of the piece before).  The
      // warp moves its 32 rows together, D / 8 lanes to a row, so that its loads are whole rows.
      constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;
      const uint32_t q_tile = smem_u32(smem) + t * L::kTileBytes;
      {
        const long long from = mine ? (long long)(p.s.qoff + token) * a.q_stride + (long long)head * D : -1;
        const int chunk = lane % kLanes, sub = lane / kLanes;
#pragma unroll 4
        for (int i = 0; i < 32; i += kRowsAtOnce) {
          const long long src = __shfl_sync(0xffffffffu, from, i + sub);
          const int rr = quarter * 32 + i + sub;
          cp_async16_or_zero(q_tile + (chunk >> 3) * L::kBoxBytes + rr * 128 + (((chunk & 7) ^ (rr & 7)) << 4),
                             a.q + (src >= 0 ? src : 0) + chunk * 8, src >= 0);
        }
        cp_async_wait_all();
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(q_full + t);

      const int lim = mine ? keys_of(a, p.s, row) : 0;
      const int first_lim = keys_of(a, p.s, row0);  // the fewest keys that a row of the tile sees
      const int nt = min(p.t1, tiles_of(keys_of(a, p.s, row0 + 127)));
      float m2 = -INFINITY, l = 0.f, le = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int j = p.t0; j < nt; ++j) {
        if (!warp_wait(s_full + t, s_cnt & 1, a.timeout_ns, abort_flag)) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(tS + i * 32, s[i]);
        tmem_ld_wait(s[0]);
        reg_pin(s[1]);
        reg_pin(s[2]);
        reg_pin(s[3]);
        const int kbase = j * kTile;
        if (kbase + kTile > first_lim) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (kbase + i * 32 + c >= lim) s[i][c] = __float_as_uint(-INFINITY);
        }
        float mxv[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 32; c += 2)
            mxv[i] = fmax3(mxv[i], __uint_as_float(s[i][c]), __uint_as_float(s[i][c + 1]));
        const float m_tile = fmaxf(fmaxf(mxv[0], mxv[1]), fmaxf(mxv[2], mxv[3])) * scale_log2;
        const bool need = (m2 == -INFINITY) || (m_tile > m2 + kRescaleThreshold);
        const float m_use = need ? fmaxf(m2, m_tile) : m2;
        const float alpha = (m2 == -INFINITY) ? 0.f : ex2(m2 - m_use);
        const float m_ref = (m_use == -INFINITY) ? 0.f : m_use;
        const float2 sc2 = make_float2(scale_log2, scale_log2), nm2 = make_float2(-m_ref, -m_ref);
        float2 ex0 = make_float2(0.f, 0.f), ex1 = ex0, rd0 = ex0, rd1 = ex0;  // unrounded and bf16 sums
        auto exp_half = [&](int hf, uint32_t(&pk)[32]) {
#pragma unroll
          for (int ii = 0; ii < 2; ++ii) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const uint32_t* sr = s[hf * 2 + ii];
              const float2 x0 = ffma2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sc2, nm2);
              const float2 x1 = ffma2(make_float2(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), sc2, nm2);
              const float2 p0 = make_float2(ex2(x0.x), ex2(x0.y));
              // a sixteenth of the exponentials on the FMA pipes, as in the dense forward
              const float2 p1 = ((c >> 2) % 8 == 7) ? exp2_fma2(x1) : make_float2(ex2(x1.x), ex2(x1.y));
              const uint32_t k0 = pack_bf16x2(p0.x, p0.y), k1 = pack_bf16x2(p1.x, p1.y);
              pk[ii * 16 + (c >> 1)] = k0;
              pk[ii * 16 + (c >> 1) + 1] = k1;
              ex0 = fadd2(ex0, p0);
              ex1 = fadd2(ex1, p1);
              acc_bf16x2(rd0, k0);
              acc_bf16x2(rd1, k1);
            }
          }
        };
        // the previous P V of this tile has completed: the scores just read were issued
        // after it, and tcgen05 operations complete in order
        if (j > p.t0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + cc * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tmem_st32(tO + cc * 32, o);
          }
        }
        uint32_t pk[32];
        exp_half(0, pk);
        tmem_st32(tS, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(p_half + t);
        exp_half(1, pk);
        tmem_st32(tS + 32, pk);
        l = l * alpha + ((rd0.x + rd0.y) + (rd1.x + rd1.y));
        le = le * alpha + ((ex0.x + ex0.y) + (ex1.x + ex1.y));
        m2 = m_use;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(p_full + t);
        ++s_cnt;
      }
      if (!ok) break;
      // ---- epilogue
      if (!warp_wait(o_done + t, items & 1, a.timeout_ns, abort_flag)) {
        if (lane == 0) give_up();
        break;
      }
      ++items;
      tc_fence_after();
      const bool whole = p.parts == 0;
      const int again = p.unit * kUnitRows + t * 128 + r;  // worked out again rather than kept
      const int out_token = p.s.qoff + token_of_row(a, again);
      const int out_head = p.hk * a.G + (again - token_of_row(a, again) * a.G);
      const int out_row = mine ? out_token * a.Hq + out_head : -1;
      if (whole) {
        const float inv = ((l > 0.f) ? 1.f / l : (l == 0.f ? 0.f : l)) * (kQ8 ? kTwo60 : 1.f);
        const bool none = l == 0.f;  // every key hidden: O = 0, whatever V holds
        // through the Q tile, whose readers are done, so that the warp stores whole rows
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(tO + cc * 32, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const float* f = reinterpret_cast<const float*>(o) + q4 * 8;
            uint4 x = make_uint4(pack_bf16x2(f[0] * inv, f[1] * inv), pack_bf16x2(f[2] * inv, f[3] * inv),
                                 pack_bf16x2(f[4] * inv, f[5] * inv), pack_bf16x2(f[6] * inv, f[7] * inv));
            if (none) x = make_uint4(0, 0, 0, 0);
            const int chunk = (cc & 1) * 4 + q4;
            st_shared_v4(q_tile + (cc >> 1) * L::kBoxBytes + r * 128 + ((chunk ^ (r & 7)) << 4), x.x, x.y, x.z, x.w);
          }
        }
        __syncwarp();
        const int chunk = lane % kLanes, sub = lane / kLanes;
#pragma unroll 4
        for (int i = 0; i < 32; i += kRowsAtOnce) {
          const int rr = quarter * 32 + i + sub;
          const int to = __shfl_sync(0xffffffffu, out_row, i + sub);
          uint4 x;
          ld_shared_v4(q_tile + (chunk >> 3) * L::kBoxBytes + rr * 128 + (((chunk & 7) ^ (rr & 7)) << 4), x.x, x.y, x.z, x.w);
          if (to >= 0) reinterpret_cast<uint4*>(a.o + (size_t)to * D)[chunk] = x;
        }
        __syncwarp();
        if (mine)
          a.lse[out_token * a.lse_row + out_head * a.lse_head] =
              le == 0.f ? -INFINITY : (m2 + __log2f(le)) * 0.69314718055994530942f;
      } else {
        // slot 0: goes on with a unit begun before; slot 1: a unit begun here.  O as
        // [d / 4][128 rows] of float4, so that a warp's stores are contiguous
        const size_t slot = 2 * (size_t)blockIdx.x + (p.t0 == 0 ? 1 : 0);
        float4* dst = reinterpret_cast<float4*>(a.part_o) + (slot * 2 + t) * (D / 4) * 128 + r;
        if (p.t0 < nt) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + cc * 32, o);
            tmem_ld_wait(o);
            const float* f = reinterpret_cast<const float*>(o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[(cc * 8 + i) * 128] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
          }
        }
        const size_t at = slot * kUnitRows + t * 128 + r;
        a.part_m[at] = m2;
        a.part_l[at] = le;
        a.part_lr[at] = l;
        if (p.t0 == 0) {
          a.part_rows[(size_t)blockIdx.x * kUnitRows + t * 128 + r] = out_row;
          if (t == 0 && r == 0) a.meta[blockIdx.x] = make_int4(p.parts, rows > 128 ? 2 : 1, 0, 0);
        }
      }
      mbar_arrive_warp(piece_empty + n % L::kPieces);
      tc_fence_before();  // O is read before the next piece's products overwrite it (q_full orders them)
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) grid_dependents_launch();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partial states of the unit that begins in attention CTA blockIdx.x: 128 rows
// (blockIdx.y of the unit), 32 dims (blockIdx.z), a thread per row.
template <int D>
__global__ void __launch_bounds__(128) paged_chunk_merge_kernel(const PagedArgs a) {
  grid_dependency_wait();  // launched while the attention kernel still runs
  grid_dependents_launch();
  const int cta = blockIdx.x, t = blockIdx.y, r = threadIdx.x;
  const int4 meta = a.meta[cta];
  const int parts = meta.x;
  if (parts == 0 || t >= meta.y) return;
  const int row = a.part_rows[(size_t)cta * kUnitRows + t * 128 + r];
  auto slot = [&](int i) { return 2 * (size_t)(cta + i) + (i == 0 ? 1 : 0); };
  float M = -INFINITY;
  for (int i = 0; i < parts; ++i) {
    const size_t at = slot(i) * kUnitRows + t * 128 + r;
    if (a.part_l[at] != 0.f) M = fmaxf(M, a.part_m[at]);
  }
  float acc[32], l = 0.f, lr = 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) acc[e] = 0.f;
  for (int i = 0; i < parts; ++i) {
    const size_t at = slot(i) * kUnitRows + t * 128 + r;
    const float pl = a.part_l[at];
    if (pl == 0.f) continue;  // no key in this part: its O was not written
    const float wt = ex2(a.part_m[at] - M);
    l = fmaf(wt, pl, l);
    lr = fmaf(wt, a.part_lr[at], lr);
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + (slot(i) * 2 + t) * (D / 4) * 128 + blockIdx.z * 8 * 128 + r;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float4 x = src[e * 128];
      acc[4 * e] = fmaf(wt, x.x, acc[4 * e]);
      acc[4 * e + 1] = fmaf(wt, x.y, acc[4 * e + 1]);
      acc[4 * e + 2] = fmaf(wt, x.z, acc[4 * e + 2]);
      acc[4 * e + 3] = fmaf(wt, x.w, acc[4 * e + 3]);
    }
  }
  if (row < 0) return;
  const float inv = (lr > 0.f ? 1.f / lr : (lr == 0.f ? 0.f : lr)) * (a.k_scales != nullptr ? kTwo60 : 1.f);
  uint4* dst = reinterpret_cast<uint4*>(a.o + (size_t)row * D + blockIdx.z * 32);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* f = acc + 8 * i;
    dst[i] = make_uint4(pack_bf16x2(f[0] * inv, f[1] * inv), pack_bf16x2(f[2] * inv, f[3] * inv),
                        pack_bf16x2(f[4] * inv, f[5] * inv), pack_bf16x2(f[6] * inv, f[7] * inv));
  }
  if (blockIdx.z == 0) {
    const int token = row / a.Hq, head = row - token * a.Hq;
    a.lse[token * a.lse_row + head * a.lse_head] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.69314718055994530942f;
  }
}

template <int D, bool kQ8>
fa_status launch_chunk_impl(const PagedLaunch& L0, cudaStream_t stream) {
  using L = ChunkLayout<D>;
  static PerDeviceOnce attr_once;
  if (!attr_once.run([] {
        return cudaFuncSetAttribute(paged_chunk_kernel<D, kQ8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    L::kSmemBytes) == cudaSuccess;
      }))
    return FA_ERR_CUDA;
  const int ctas = num_sms();
  PagedArgs a = paged_args(L0);
  paged_carve(ctas, kUnitRows, D).place(a, L0.workspace);
  a.min_rows = L0.few_rows + 1;
  a.max_rows = 0x7fffffff;
  prof_before(stream, kKPagedChunk);
  cudaError_t err = launch_dependent(paged_chunk_kernel<D, kQ8>, dim3(ctas), kThreads, L::kSmemBytes, stream, a);
  prof_after(stream, kKPagedChunk);
  if (err != cudaSuccess) return FA_ERR_CUDA;
  if (L0.max_k <= kTile) return FA_OK;  // units of one tile are never split
  prof_before(stream, kKPagedChunkMerge);
  err = launch_dependent(paged_chunk_merge_kernel<D>, dim3(ctas, 2, D / 32), 128, 0, stream, a);
  prof_after(stream, kKPagedChunkMerge);
  return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

size_t paged_chunk_workspace(int d) { return paged_carve(num_sms(), kUnitRows, d).bytes; }

fa_status launch_paged_chunk(const PagedLaunch& L, cudaStream_t stream) {
  const bool q8 = L.k_scales != nullptr;
  if (L.d == 64) return q8 ? launch_chunk_impl<64, true>(L, stream) : launch_chunk_impl<64, false>(L, stream);
  return q8 ? launch_chunk_impl<128, true>(L, stream) : launch_chunk_impl<128, false>(L, stream);
}

}  // namespace fa
