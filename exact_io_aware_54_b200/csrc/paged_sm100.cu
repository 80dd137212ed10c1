// paged_sm100.cu -- attention of few new rows per sequence over a paged key/value
// cache in bf16 or 8 bits (B200, sm_100a).
//
// What it computes: sequence b has n_b new query tokens (its last ones) and L_b keys
// in pages; query head h reads key head h / G, G = Hq / Hkv.  For every new token i
//     x_ij = scale * q_i . k_j,  j <= L_b - n_b + i (causal) or j < L_b,
//     o_i  = sum_j softmax_j(x_ij) v_j,   lse_i = ln sum_j exp(x_ij).
// The G query heads of a key head share its keys, so the n_b G rows (token, head of
// the group) of one (sequence, key head) are one problem: every key is read once
// for all of them.  With few rows the cache's bytes are the floor; the tensor cores
// do the arithmetic because G rows per key are too much of it for the FMA pipes at
// the rate at which 8 bit keys arrive.
//
// B200 design
//  * Transposed products.  A tile of 128 keys is the M side: S^T [128 keys, N rows] =
//    K Q^T and O^T [128 dims, N rows] += V^T P^T, with N = 16 or 32 rows, so a
//    tile of few rows does not pay for 128.  Lane of tensor memory = key (then
//    dim), column = row: a softmax thread owns one key and N scores.
//  * 8 bit cache without conversion.  K and V tiles stay e4m3 in shared memory and are
//    multiplied by kind::f8f6f4 MMAs.  The bf16 row of Q is split into two e4m3
//    pieces, q = q1 + q2 / 32: four significant bits each make bf16's eight, exact but
//    for elements under 2^-14 of the row's largest, off by at most 2^-22 of it (half of
//    e4m3's subnormal step, 32 times down).  A weight is an fp16 number cut into three e5m2 pieces (three
//    significant bits each, e5m2 being the upper byte of fp16), p = p1 + p2 / 8 + p3 / 64,
//    off by at most 2^-9 + 2^-11 of p, or 2^-36 of the row's largest weight: many weak keys
//    beside a strong one count as they do in bf16 weights.  (Two e4m3 pieces lose weights
//    under 2^-17 of the largest, of which a long cache has enough to matter.)  The pieces of
//    a row are columns of the product, added up when they are read: an MMA costs the same
//    for 32 or 64 columns as for 16, so another pass over the tile would cost as much again.
//    The key scales multiply the scores in fp32; the value scales 2^e_j are carried
//    in the weights: with y_j = x_j log2(e) + e_j the weight is 2^(y_j - m), m the
//    running maximum of y, and the sum takes it times 2^-e_j.
//  * d = 64 runs two key heads side by side as one of 128 dims: the rows of the first
//    head have zeros in the second's dims and the other way round, and each keeps
//    its own half of O^T.  Half of the product is wasted; the bytes are the floor.
//  * Tiles of the cache come by 16-byte asynchronous copies, a warp for K and one for V,
//    each row from wherever its page is, so any page size costs the same; rows past the
//    sequence's end are filled with zeros (stale shared memory could hold NaN, which a
//    weight of zero does not remove).  A TMA box costs its issuer some 260 cycles whatever its
//    size: pages of 16 keys make 16 of a K and V tile, 4200 cycles where its bytes take 1400.
//  * The running maximum moves only when some key exceeds it by more than a
//    threshold: a tile costs one barrier that ORs "does any of my scores exceed",
//    and the reduction across the 128 keys happens only then.  The l sums stay per
//    thread until the end.  bf16 keeps two: of the weights as the product takes them
//    (divides O) and of the unrounded ones (gives lse).  8 bit divides O by the
//    unrounded sum: its weights carry the value scales, so that a key of quiet values
//    may round to nothing in the product and still count fully in the sum.
//  * Work split: CTAs come in teams of neighbouring key heads, which read the same keys'
//    neighbouring bytes at about the same time: a head's slice of a row is only 128 bytes in
//    8 bits (64 requests of 8 key heads: 262 us without teams, 253 in teams of 2, 4 or 8).
//    A (sequence, team's heads, row tile) unit counts ceil(L / 128) tiles and kUnitCost for
//    its start and end; the line of all units is cut into equal parts, one per team (one CTA
//    per SM), whatever the lengths.  A unit that lies in one part is finished there; others
//    leave fp32 partial states, two at most per CTA, that paged_merge_kernel joins in order.
//    No atomics: results do not depend on timing.
//  * Warp roles: 0 MMA issuer, 1 page lookup, then K loaders, V loaders, and four warps for
//    softmax and epilogue.  The lookup warp turns tiles into rows of the cache, up to eight tiles
//    ahead, in a ring that the loaders copy from, and fetches the rows' scale bytes: as the
//    aligned words that hold them (asynchronous copies have no smaller size), cut out by
//    the softmax.
//  * Every role is a small loop: one warp of each runs per scheduler, and with the loaders'
//    loops unrolled (2000 instructions each) two fifths of all stalls were for instructions
//    not yet fetched (64 requests, 8 key heads: 499 us; 272 with small loops over a ring of rows).
//  * What it measures (device time): 64 requests of 512 to 16384 keys, 32 query and 8 key
//    heads of 128, 8 bit: 225 us, 85% of the measured copy rate; bound by the softmax and MMA
//    chain of a tile, which takes about as long as its bytes.  Four tokens each: 318 us, bound
//    by the softmax of 16 rows a key, each weight cut into its pieces (two e4m3 pieces with one
//    scale took 284).  Over a bf16 cache 361 us, at the measured copy rate.  One sequence of
//    8192 keys, 32 heads, 8 bit: 21.5 us for 10 us of bytes, the rest the start (four
//    dependent loads, lengths, page, keys, and the first scores: 5.5 us), the epilogue and the
//    join (1 and 3 us).
//  * Few waits: the issue order Q K^T of step s + 1, then P V of step s, makes the scores'
//    barrier of a step imply that the products of two steps before have read their
//    weights, and the weights' barrier that the scores have been read; the barrier that
//    frees a tile's slot tells that its P V is in O.
#include "paged_common.cuh"

namespace fa {

using namespace paged;

namespace {

// Loader warps, half of them for K.  One warp each takes about 1050 cycles for a tile of 8
// bit keys, as long as its bytes do: two are never ahead (eight: 234 us for 64 requests, four
// 228).  With 32 rows the 8 bit softmax takes longer and needs the registers: 32 tokens, 16 x
// 4000 keys, 32 heads of 128, with two and four 287 and 320 us, in bf16 177 and 174.
template <int N, bool kQ8>
constexpr int kLoaders = kQ8 && N == 32 ? 2 : 4;
template <int N, bool kQ8>
constexpr int kThreads = (2 + kLoaders<N, kQ8> + 4) * 32;
// Exponent offset and threshold of the running maximum, log2 units.  8 bit: weights
// up to 2^(14 + 1) use the range of e5m2 (57344) and of fp16 (65504).  bf16: as in the dense
// forward.
template <bool kQ8>
struct SoftmaxRange {
  static constexpr float kOffset = kQ8 ? 14.f : 0.f;
  static constexpr float kThreshold = kQ8 ? 1.f : 8.f;
};

template <int N, bool kQ8>
struct PagedLayout {
  // Tiles of one step of the MMA issuer and the softmax.  A step has fixed costs (a look at
  // three barriers, commits, a barrier of the softmax group, latencies in a row) of some
  // 700 cycles, about the time of an 8 bit tile's bytes: two tiles share them.
  static constexpr int kPer = kQ8 ? 2 : 1;
  static constexpr int kTileBytes = kTile * 128 * (kQ8 ? 1 : 2);  // a K or V tile
  // Slots of one tile each, K and V in turn: K's is free as soon as its scores are there.
  // (K and V in one slot, a wait less, left the loaders too little room: 287 against 259 us.)
  static constexpr int kSlotBytes = kTileBytes;
  static constexpr int kSlots = kQ8 ? (N == 16 ? 11 : 9) : 6;    // what fits
  static constexpr int kRowBlock = N * 128;      // one 128-byte column block of the N rows
  static constexpr int kOffQ = kSlots * kSlotBytes;  // two e4m3 pieces, or two 64-dim blocks
  static constexpr int kOffP = kOffQ + 2 * kRowBlock;  // [2 steps][kPer] of three e5m2 pieces, or of bf16
  static constexpr int kBlocksP = kQ8 ? 3 : 2;         // row blocks of the weights of one tile
  static constexpr int kOffBar = kOffP + 2 * kPer * kBlocksP * kRowBlock;
  // kv_full[S], kv_empty[S], q_full, s_full[2], p_full[2], rows_full[R], rows_empty[R], scaled[R]
  static constexpr int kRing = 8;  // tiles that the page lookup may be ahead
  static constexpr int kNumBars = 2 * kSlots + 5 + 3 * kRing;
  static constexpr int kOffMisc = kOffBar + ((kNumBars * 8 + 15) & ~15);
  static constexpr int kOffRows = kOffMisc + 64;
  // per row: factor, limit, threshold, reference, rescale, running max, output row; per warp and row: two sums
  static constexpr int kOffRing = (kOffRows + 15 * N * 4 + 15) & ~15;  // per tile: 128 cache rows
  static constexpr int kOffTile = kOffRing + kRing * kTile * 4;         // per tile: head (or pair), -1: no more tiles
  // per tile and key: the words of K's and V's scale bytes, two each when two heads may
  // lie in different words
  static constexpr int kOffScales = kOffTile + kRing * 4;
  static constexpr int kSmemBytes = kOffScales + (kQ8 ? kRing * kTile * 16 : 0) + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 232448, "shared memory of one SM");
  // columns of the products: rows, in 8 bits as many pieces of each
  static constexpr int kPiecesQ = kQ8 ? 2 : 1, kPiecesP = kQ8 ? 3 : 1;
  static constexpr int kCols = kPiecesQ * N, kColsO = kPiecesP * N;
  static constexpr int kColO = 2 * kPer * kCols;  // behind the scores of two steps
  static constexpr uint32_t kTmemCols = (N == 16 ? 64 : 128) * (kQ8 ? 4 : 1);
  static_assert(kColO + kColsO <= (int)kTmemCols, "scores of two steps and O");
};

// rows of one tile that belong to one key head
template <int N, int D>
__host__ __device__ constexpr int head_rows() {
  return D == 64 ? N / 2 : N;
}

template <int N, int D>
__device__ __forceinline__ int row_tiles(const PagedArgs& a, int nq) {
  return nq <= 0 ? 0 : (nq * a.G + head_rows<N, D>() - 1) / head_rows<N, D>();
}

// Tiles of one unit of a sequence (one, fully masked, when it has no key).
__device__ __forceinline__ int unit_tiles(int lk) { return max(1, (lk + kTile - 1) / kTile); }

// A unit's start and end (Q in, O out, the pipeline filled and drained) take about as long as
// some tiles; each unit counts as many more, at its beginning, so that a CTA with the end of
// one unit and the beginning of the next is not 2.5 us behind the others.  One sequence of
// 8192 keys, 32 heads, with 0, 2, 3, 4 and 6 in 8 bits: 24.5, 23.4, 23.2, 22.6 and 23.4 us;
// 16 sequences of 8 key heads of 64: 49.9, 40.1, 40.1, 38.9 and 39.4 us; with 0, 1, 2 and 3 in
// bf16 32.0, 31.1, 31.0 and 31.2 us.
template <bool kQ8>
constexpr int kUnitCost = kQ8 ? 4 : 2;

// This CTA's (its team's) stretch [pos, end) of the line of what units count, as pieces of
// units.
struct Work {
  long long pos, end, total;
  int b, off;  // sequence of pos, and pos's place in what its units count
  int teams;   // teams that have a stretch
};
struct Piece {
  int b, hg, rt, t0, t1, tiles;
  int after;  // of what the unit counts, behind the stretch
  SeqInfo s;
};
template <int N, bool kQ8, int D>
__device__ __forceinline__ bool next_piece(const PagedArgs& a, Work& w, Piece& p) {
  if (w.pos >= w.end) return false;
  for (; w.b < a.B; ++w.b) {
    p.s = seq_info(a, w.b);
    const int rts = row_tiles<N, D>(a, p.s.nq);
    p.tiles = unit_tiles(p.s.lk);
    const int each = p.tiles + kUnitCost<kQ8>, cost = rts * a.sets * each;
    if (w.off < cost) {
      const int u = w.off / each, at = w.off - u * each;
      const int n = (int)min((long long)(each - at), w.end - w.pos);
      p.t0 = max(0, at - kUnitCost<kQ8>);
      p.t1 = at + n - kUnitCost<kQ8>;
      p.after = each - at - n;
      w.pos += n;
      w.off += n;
      if (p.t1 <= p.t0) return false;  // only of what the unit counts more: the next CTA begins it
      p.b = w.b;
      const int set = u / rts;
      p.hg = set * a.team + (int)blockIdx.x % a.team;
      p.rt = u - set * rts;
      return true;
    }
    w.off -= cost;
  }
  return false;
}

// Run by one warp: the line's length and where this CTA's stretch begins.
template <int N, bool kQ8, int D>
__device__ __forceinline__ Work find_work(const PagedArgs& a) {
  const int lane = lane_id();
  Work w;
  auto cost_of = [&](int b) {
    if (b >= a.B) return 0;
    const SeqInfo s = seq_info(a, b);
    return row_tiles<N, D>(a, s.nq) * a.sets * (unit_tiles(s.lk) + kUnitCost<kQ8>);
  };
  long long total = 0;
  for (int b = lane; b < a.B; b += 32) {
    total += cost_of(b);
    if (blockIdx.x == 0 && a.cu_q != nullptr && seq_info(a, b).nq < 0) atomicExch(a.status, kStatusBadArg);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  w.total = total;
  w.teams = (int)min((long long)a.teams, total);
  const int team = blockIdx.x / a.team;
  w.b = 0;
  w.off = 0;
  w.pos = w.end = 0;
  if (team >= w.teams) return w;
  w.pos = total * team / w.teams;
  w.end = total * (team + 1) / w.teams;
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int mine = cost_of(b0 + lane);
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
      w.off = (int)(w.pos - (before + __shfl_sync(0xffffffffu, upto - mine, src)));
      break;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return w;
}

// Does `pred` hold in any of the 128 softmax threads?  (Also their barrier.)
__device__ __forceinline__ bool any_of_group(bool pred) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)pred)
      : "memory");
  return any != 0;
}

// x to the nearest e4m3 pair and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 of_e4m3x2(uint32_t q) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)q, __NV_E4M3)));
}

// Four weights as the bytes of their three e5m2 pieces.  An e5m2 number is the upper byte of an
// fp16 one, so the nearest (ties away from zero) is that of its bits + 0x80, up to 57344, and
// the remainder is an fp16 number, as is 8 times it.  A NaN may come out as anything: it is in
// the sum that divides.
__device__ __forceinline__ void split_weights(const float (&w)[4], uint32_t& p1, uint32_t& p2, uint32_t& p3) {
  const __half2 eight = __float2half2_rn(8.f);
  __half2 lo = __floats2half2_rn(w[0], w[1]), hi = __floats2half2_rn(w[2], w[3]);
  auto piece = [&](uint32_t& codes) {
    uint32_t a = *reinterpret_cast<const uint32_t*>(&lo) + 0x00800080u, b = *reinterpret_cast<const uint32_t*>(&hi) + 0x00800080u;
    codes = __byte_perm(a, b, 0x7531);
    a &= 0xFF00FF00u;
    b &= 0xFF00FF00u;
    lo = __hmul2(__hsub2(lo, *reinterpret_cast<const __half2*>(&a)), eight);
    hi = __hmul2(__hsub2(hi, *reinterpret_cast<const __half2*>(&b)), eight);
  };
  piece(p1);
  piece(p2);
  piece(p3);
}

// Lane i < N ends with the sum over the warp of everyone's v[i]; v is used up.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  static_assert(N == 4 || N == 8 || N == 16 || N == 32, "one value per lane at most");
  const uint32_t lane = lane_id();
#pragma unroll
  for (int off = 16; off >= N; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
#pragma unroll
  for (int off = N / 2; off > 0; off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const float give = up ? v[i] : v[i + off];
      const float keep = up ? v[i + off] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
  return v[0];
}

// The rows of a product that there are, for this thread's key or dim: kHeads heads' first kLive
// columns of kHeadRows each, kPieces pieces of them N columns apart, added up, each `step` of
// the one before it.
template <int N, int kHeads, int kHeadRows, int kLive, int kPieces>
__device__ __forceinline__ void ld_rows(uint32_t at, float step, float (&x)[kHeads * kLive]) {
  constexpr int kRows = kHeads * kLive;
  uint32_t v[kRows * kPieces];
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
#pragma unroll
    for (int i = 0; i < kPieces; ++i) tmem_ld_some<kLive>(at + h * kHeadRows + i * N, v, (i * kHeads + h) * kLive);
  tmem_ld_done(v);
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    x[n] = __uint_as_float(v[(kPieces - 1) * kRows + n]);
#pragma unroll
    for (int i = kPieces - 2; i >= 0; --i) x[n] = fmaf(x[n], step, __uint_as_float(v[i * kRows + n]));
  }
}

// kLive: rows of each key head that there can be, 4 or all of the tile's.  (Four query heads
// to a key head, or one, and a single token: most decoding.  With the other rows' scores
// left in place the softmax loop is a quarter of its instructions.)
template <int N, bool kQ8, int D, int kLive>
__global__ void __launch_bounds__(kThreads<N, kQ8>, 1)
    paged_kernel(const PagedArgs a) {
  using L = PagedLayout<N, kQ8>;
  using R = SoftmaxRange<kQ8>;
  constexpr int kHeadRows = head_rows<N, D>();
  constexpr int kHeads = D == 64 ? 2 : 1;   // key heads side by side
  constexpr int kRows = kHeads * kLive;     // rows that the softmax looks at
  // column (row of the tile) of the n-th of them
  auto col = [](int n) constexpr { return n / kLive * kHeadRows + n % kLive; };
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = bars + L::kSlots;
  uint64_t* q_full = bars + 2 * L::kSlots;
  uint64_t* s_full = q_full + 1;
  uint64_t* p_full = q_full + 3;
  uint64_t* rows_full = q_full + 5;
  uint64_t* rows_empty = rows_full + L::kRing;
  uint64_t* scaled = rows_empty + L::kRing;
  uint32_t* ring_rows = reinterpret_cast<uint32_t*>(smem + L::kOffRing);
  volatile int* ring_tile = reinterpret_cast<volatile int*>(smem + L::kOffTile);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  // a softmax wait gave up: set before the tile's first barrier or after its last, read between
  volatile int* group_dead = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 8);
  Work* work = reinterpret_cast<Work*>(smem + L::kOffMisc + 16);
  static_assert(sizeof(Work) <= 48, "the stretch fits its place");
  const uint32_t warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(kv_full + s, kLoaders<N, kQ8> / 2);  // the warps that share a tile
      mbar_init(kv_empty + s, 1);
    }
    mbar_init(q_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
    }
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(rows_full + i, 1);
      mbar_init(scaled + i, 32);  // the lookup warp's lanes, 8 bits only
      mbar_init(rows_empty + i, kLoaders<N, kQ8> + (kQ8 ? 4 : 0));  // the loaders, and the softmax warps for the scales' words
    }
    *abort_flag = 0;
    *group_dead = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  // up to here the kernel before may still run
  grid_dependency_wait();
  if (warp == 2) {
    const Work w = find_work<N, kQ8, D>(a);
    if (lane == 0) {
      *work = w;
      a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Work w = *work;
  auto give_up = [&]() {
    *abort_flag = 1;
    atomicCAS(a.status, 0, kStatusTimeout);
  };

  if (warp == 1) {
    // -------------------------------------------------------------------- page lookup
    const PageRing ring{ring_rows, ring_tile, smem_u32(smem + L::kOffScales), rows_full, scaled, rows_empty};
    const bool ok = look_up_pages<L::kRing, kQ8, D == 64>(a, ring, abort_flag, [&](int& b, int& hg, int& t0, int& t1, int& lk) {
      Piece p;
      if (!next_piece<N, kQ8, D>(a, w, p)) return false;
      b = p.b, hg = p.hg, t0 = p.t0, t1 = p.t1, lk = p.s.lk;
      return true;
    });
    if (!ok && lane == 0) give_up();
  } else if (warp >= 2 && warp < 2 + kLoaders<N, kQ8>) {
    // -------------------------------------------------------------------- K and V loaders
    constexpr int kParts = kLoaders<N, kQ8> / 2;  // warps that share a tile
    const bool is_v = warp >= 2 + kParts;
    const int part = (warp - 2) % kParts;
    const uint32_t row_bytes = (uint32_t)a.Hkv * D * (kQ8 ? 1 : 2);
    const int chunk = lane & 7, sub = lane >> 3;  // 16-byte chunk of a 128-byte row, key of four
    const uint32_t to0 = sub * 128 + ((chunk ^ sub) << 4), to1 = (sub + 4) * 128 + ((chunk ^ (sub + 4)) << 4);
    const uint32_t ring = smem_u32(ring_rows);
    bool ok = true;
    uint32_t c = 0;
    // A tile is handed over once its copies have landed and been made visible to the tensor
    // core: when the next tile's are on their way, or when there is no slot for the next.
    // (The fence costs the MMA issuer more than it costs here.  64 requests: handed over at
    // once 316 us, always two tiles late 252, one 241.)
    bool pending = false;
    auto hand_over = [&](uint32_t x) {
      fence_proxy_async_smem();
      mbar_arrive_warp(kv_full + (2 * x + is_v) % L::kSlots);
    };
    for (;; ++c) {
      const uint32_t at = c % L::kRing, g = 2 * c + is_v, slot = g % L::kSlots;
      ok = warp_wait(rows_full + at, (c / L::kRing) & 1, a.timeout_ns, abort_flag);
      if (!ok) break;
      const int hg = ring_tile[at];
      if (hg < 0) break;
      const uint32_t free_parity = ((g / L::kSlots) & 1) ^ 1;
      if (pending && !__all_sync(0xffffffffu, mbar_try_wait(kv_empty + slot, free_parity))) {
        cp_async_wait_all();
        hand_over(c - 1);
        pending = false;
      }
      ok = warp_wait(kv_empty + slot, free_parity, a.timeout_ns, abort_flag);
      if (!ok) break;
      // a pair of 64-dim heads whose second is past the last has no bytes for it
      const bool lone = D == 64 && 2 * hg + 1 >= a.Hkv;
      const uint8_t* src = (is_v ? a.v_pages : a.k_pages) + hg * (kQ8 ? 128 : 256) + chunk * 16;
      uint32_t dst = smem_u32(smem + slot * L::kSlotBytes) + part * (128 / kParts) * 128;
      uint32_t rows = ring + (at * kTile + part * (128 / kParts) + sub) * 4;
      const bool mine = !(kQ8 && lone && chunk >= 4);
#pragma unroll 1
      for (int i = 0; i < 4 / kParts; ++i, dst += 4096, rows += 128) {
        uint32_t rw[8];  // of keys 32 i + 4 j + sub
#pragma unroll
        for (int j = 0; j < 8; ++j) rw[j] = ld_shared_u32(rows + 16 * j);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool have = rw[j] != kNoRow && mine;
          const uint8_t* from = src + (uint64_t)(have ? rw[j] : 0u) * row_bytes;
          const uint32_t to = dst + (j / 2) * 1024 + (j % 2 ? to1 : to0);
          cp_async16_or_zero(to, from, have);
          if constexpr (!kQ8) cp_async16_or_zero(to + kTile * 128, lone ? from : from + 128, have && !lone);
        }
      }
      mbar_arrive_warp(rows_empty + at);
      cp_async_commit();
      if (pending) {
        cp_async_wait<1>();
        hand_over(c - 1);
      }
      pending = true;
    }
    cp_async_wait_all();  // (also before the CTA retires after a wait that gave up)
    if (ok && pending) hand_over(c - 1);
    if (!ok && lane == 0) give_up();
  } else if (warp == 0) {
    // -------------------------------------------------------------------- MMA issuer
    if (elect_one()) {
      constexpr uint32_t kIdescS = kQ8 ? idesc_e4m3_f32(128, 2 * N, false, false) : idesc_bf16_f32(128, N, false, false);
      constexpr uint32_t kIdescO = kQ8 ? idesc_e4m3_e5m2_f32(128, 3 * N, true, true) : idesc_bf16_f32(128, N, true, true);
      const uint32_t base = smem_u32(smem);
      const SDesc k_desc = sdesc_make(base, 16, 1024);                     // K-major keys
      const SDesc v_desc = sdesc_make(base, kQ8 ? 16 : 16384, 1024);       // dims along M: MN-major
      const SDesc q_desc = sdesc_make(base + L::kOffQ, 16, 1024);
      const SDesc p_desc = sdesc_make_mn_plain(base + L::kOffP, 128, kTile * 16);  // rows along N: MN-major
      constexpr uint32_t kSlot16 = L::kSlotBytes / 16, kBlock16 = L::kRowBlock / 16;
      const uint32_t tO = tmem + L::kColO;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !thread_wait(bar, parity, a.timeout_ns, abort_flag)) {
          give_up();
          ok = false;
        }
        return ok;
      };
      // one step of a product: 32 deep in 8 bits, 16 in bf16
      auto step = [&](uint32_t d, uint64_t x, uint64_t y, uint32_t idesc, bool accumulate) {
        if constexpr (kQ8)
          umma_ss_f8(d, x, y, idesc, accumulate ? 1u : 0u);
        else
          umma_ss(d, x, y, idesc, accumulate ? 1u : 0u);
      };
      uint32_t c = 0, st = 0, piece = 0;  // tiles, steps and pieces so far
      // P V of step x, tiles c0 ..; its commits free the tiles' slots, and tell the softmax that O is up to date
      auto pv = [&](uint32_t x, uint32_t c0, int n, bool accumulate) {
        if (!wait(p_full + (x & 1), (x >> 1) & 1)) return;
        tc_fence_after();
#pragma unroll
        for (int u = 0; u < L::kPer; ++u) {
          if (u >= n) break;
          const uint32_t g = 2 * (c0 + u) + 1, slot = g % L::kSlots;
          if (!wait(kv_full + slot, (g / L::kSlots) & 1)) return;
          tc_fence_after();
          const SDesc v = SDesc{v_desc.lo + slot * kSlot16, v_desc.hi};
          const SDesc pd = SDesc{p_desc.lo + ((x & 1) * L::kPer + u) * L::kBlocksP * kBlock16, p_desc.hi};
          // keys 32 i .. or 16 i ..
#pragma unroll
          for (int i = 0; i < (kQ8 ? 4 : 8); ++i)
            step(tO, sdesc_at(v, i * (kQ8 ? 256 : 128)), sdesc_at(pd, i * (kQ8 ? 32 : 16)), kIdescO,
                 accumulate || u > 0 || i > 0);
          umma_commit(kv_empty + slot);
        }
      };
      Piece p;
      while (ok && next_piece<N, kQ8, D>(a, w, p)) {
        if (!wait(q_full, piece++ & 1)) break;
        tc_fence_after();
        const int tiles = p.t1 - p.t0;
        int last = 0;  // tiles of the step before
        for (int t = 0; ok && t < tiles; t += L::kPer, ++st) {
          const int n = min(L::kPer, tiles - t);
#pragma unroll
          for (int u = 0; u < L::kPer; ++u) {
            if (u >= n) break;
            const uint32_t g = 2 * (c + u), slot = g % L::kSlots;
            if (!wait(kv_full + slot, (g / L::kSlots) & 1)) break;
            tc_fence_after();
            const SDesc k = SDesc{k_desc.lo + slot * kSlot16, k_desc.hi};
            // dims 32 i .. or 16 i .. of two 64-dim blocks
#pragma unroll
            for (int i = 0; i < (kQ8 ? 4 : 8); ++i)
              step(tmem + ((st & 1) * L::kPer + u) * L::kCols, sdesc_at(k, (i >> 2) * 1024 + (i & 3) * 2),
                   sdesc_at(q_desc, (i >> 2) * kBlock16 + (i & 3) * 2), kIdescS, i > 0);
            if (u + 1 < n) umma_commit(kv_empty + slot);
          }
          if (!ok) break;
          umma_commit(s_full + (st & 1));
          umma_commit(kv_empty + 2 * (c + n - 1) % L::kSlots);
          if (t > 0) pv(st - 1, c - last, last, t > L::kPer);
          c += n;
          last = n;
        }
        if (ok) pv(st - 1, c - last, last, tiles > L::kPer);
      }
    }
  } else {
    // -------------------------------------------------------------------- softmax and epilogue
    const uint32_t quarter = warp & 3;
    const int r = quarter * 32 + lane;         // key of the tile, then dim of O
    const int tid = threadIdx.x - 64 - 32 * kLoaders<N, kQ8>;  // 0 .. 127
    const uint32_t lanes = (quarter * 32) << 16;
    float* factor = reinterpret_cast<float*>(smem + L::kOffRows);  // of the scores: scale, log2 e, Q's scale
    int* limit = reinterpret_cast<int*>(factor + N);               // first key that the row does not see
    float* thresh = factor + 2 * N;  // running maximum + threshold
    float* ref = factor + 3 * N;     // what the weights' exponents are taken from
    float* alpha = factor + 4 * N;
    float* top = factor + 5 * N;     // running maximum
    int* out_row = reinterpret_cast<int*>(factor + 6 * N);  // token * Hq + head, -1: no row
    float* wred = factor + 7 * N;    // [4][N] maxima, then sums
    float* wred2 = wred + 4 * N;
    uint32_t c = 0, st = 0;  // tiles and steps so far
    // A wait that gives up does not leave at once: the group's barriers need all four
    // warps, so the warp goes on (waiting no more) to the next place where all leave
    // together.
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok && !warp_wait(bar, parity, a.timeout_ns, abort_flag)) {
        if (lane == 0) {
          give_up();
          *group_dead = 1;
        }
        __syncwarp();
        ok = false;
      }
    };
    Piece p;
    while (next_piece<N, kQ8, D>(a, w, p)) {
      const int tiles = p.t1 - p.t0;
      // ---- the piece's rows: kThreadsPerRow threads share a row of 128 dims
      {
        constexpr int kTpr = 128 / N, kPer = 128 / kTpr;  // threads per row, dims per thread
        const int n = tid / kTpr, d0 = (tid % kTpr) * kPer;
        const int half = D == 64 ? n / kHeadRows : 0;   // which of the pair's heads
        const int row = p.rt * kHeadRows + (D == 64 ? n % kHeadRows : n);
        const int token = row / a.G, hk = D == 64 ? 2 * p.hg + half : p.hg;
        const bool have = token < p.s.nq && hk < a.Hkv;
        const int head = hk * a.G + row % a.G;
        // dims d0 .. d0 + kPer - 1 of the 128: this row's head has its own D of them
        const bool mine = have && (D == 128 || d0 / 64 == half);
        const __nv_bfloat16* src = a.q + (long long)(p.s.qoff + token) * a.q_stride + (long long)head * D + (D == 64 ? d0 % 64 : d0);
        uint32_t qw[kPer / 2];
#pragma unroll
        for (int i = 0; i < kPer / 8; ++i) {
          const uint4 x = mine ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
          qw[4 * i] = x.x, qw[4 * i + 1] = x.y, qw[4 * i + 2] = x.z, qw[4 * i + 3] = x.w;
        }
        float f = a.scale_log2;
        const uint32_t row_at = smem_u32(smem + L::kOffQ) + n * 128;
        if constexpr (kQ8) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < kPer / 2; ++i) m = __vmaxu2(m, qw[i] & 0x7FFF7FFFu);
          m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
          for (int off = 1; off < kTpr; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
          // times 2^(7 - exponent): the largest element in [128, 256)
          const int e = m == 0 ? 0 : min(120, max(-112, (int)(m >> 7) - 127 - 7));
          const float up = __uint_as_float((uint32_t)(127 - e) << 23);
          f *= __uint_as_float((uint32_t)(127 + e) << 23);
          if (m >= 0x7F80u) f = __uint_as_float(0x7FC00000u);  // an infinity or NaN in the row: NaN scores
#pragma unroll
          for (int i = 0; i < kPer / 16; ++i) {
            uint32_t q1[4], q2[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t h1[2], h2[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t x = qw[8 * i + 2 * j + k];
                const float lo = __uint_as_float(x << 16) * up, hi = __uint_as_float(x & 0xFFFF0000u) * up;
                h1[k] = to_e4m3x2(lo, hi);
                const float2 back = of_e4m3x2(h1[k]);
                h2[k] = to_e4m3x2((lo - back.x) * 32.f, (hi - back.y) * 32.f);  // at most 8 times 32
              }
              q1[j] = h1[0] | (h1[1] << 16);
              q2[j] = h2[0] | (h2[1] << 16);
            }
            const uint32_t at = row_at + ((((d0 >> 4) + i) ^ (n & 7)) << 4);
            st_shared_v4(at, q1[0], q1[1], q1[2], q1[3]);
            st_shared_v4(at + L::kRowBlock, q2[0], q2[1], q2[2], q2[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kPer / 8; ++i) {
            const int chunk = (d0 >> 3) + i;  // of 16: two blocks of 64 dims
            st_shared_v4(row_at + (chunk >> 3) * L::kRowBlock + (((chunk & 7) ^ (n & 7)) << 4), qw[4 * i], qw[4 * i + 1],
                         qw[4 * i + 2], qw[4 * i + 3]);
          }
        }
        if (tid % kTpr == 0) {
          factor[n] = have ? f : 0.f;
          limit[n] = (have && a.causal) ? max(0, min(p.s.lk, p.s.lk0 + token + 1)) : p.s.lk;
          thresh[n] = -INFINITY;
          top[n] = -INFINITY;
          ref[n] = -R::kOffset;
          out_row[n] = have ? (p.s.qoff + token) * a.Hq + head : -1;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(q_full);
      named_bar_sync(1, 128);
      // keys that every row of the tile sees: [0, all_see)
      const int first_token = (p.rt * kHeadRows) / a.G;
      const int all_see = a.causal ? max(0, min(p.s.lk, p.s.lk0 + first_token + 1)) : p.s.lk;

      float l[kRows], lr[kQ8 ? 1 : kRows];
#pragma unroll
      for (int n = 0; n < kRows; ++n) {
        l[n] = 0.f;
        if constexpr (!kQ8) lr[n] = 0.f;
      }

      for (int t = 0; t < tiles; t += L::kPer, ++st) {
        const int n_tiles = min(L::kPer, tiles - t);
        const int key0 = (p.t0 + t) * kTile + r;  // this thread's key of the step's first tile
        wait(s_full + (st & 1), (st >> 1) & 1);
        tc_fence_after();
        float kf[L::kPer][2], ve[L::kPer][2], vinv[L::kPer][2];  // the keys' scales, two heads' when d = 64
        float y[L::kPer][kRows];
        bool over = !ok;
#pragma unroll
        for (int u = 0; u < L::kPer; ++u) {
#pragma unroll
          for (int h = 0; h < 2; ++h) kf[u][h] = vinv[u][h] = 1.f, ve[u][h] = 0.f;
          if (u >= n_tiles) break;
          if constexpr (kQ8) {
            const uint32_t at = (c + u) % L::kRing, rw = ring_rows[at * kTile + r];
            wait(scaled + at, ((c + u) / L::kRing) & 1);
            uint4 words;
            if constexpr (D == 64) {
              words = reinterpret_cast<const uint4*>(smem + L::kOffScales)[at * kTile + r];
            } else {
              const uint2 w2 = reinterpret_cast<const uint2*>(smem + L::kOffScales)[at * kTile + r];
              words = make_uint4(w2.x, 0, w2.y, 0);
            }
            mbar_arrive_warp(rows_empty + at);
            // byte of the head in its word, and the pair's second head's after it
            const uint32_t cut = ((rw * (uint32_t)a.Hkv + (D == 64 ? 2 : 1) * p.hg) & 3u) * 8;
            uint32_t kb = D == 64 ? __funnelshift_r(words.x, words.y, cut) : words.x >> cut;
            uint32_t vb = D == 64 ? __funnelshift_r(words.z, words.w, cut) : words.z >> cut;
            if (rw == kNoRow) kb = vb = 0x7F7Fu;  // 2^0
#pragma unroll
            for (int h = 0; h < (D == 64 ? 2 : 1); ++h) {
              kf[u][h] = __uint_as_float(((kb >> (8 * h)) & 0xFFu) << 23);
              const int e = (int)((vb >> (8 * h)) & 0xFFu) - 127;
              ve[u][h] = (float)e;
              vinv[u][h] = __uint_as_float((uint32_t)(127 - e) << 23);
            }
          }
          ld_rows<N, kHeads, kHeadRows, kLive, L::kPiecesQ>(tmem + lanes + ((st & 1) * L::kPer + u) * L::kCols, 0.03125f, y[u]);
          const int key = key0 + u * kTile;
          const bool masked = key - r + kTile > all_see;
#pragma unroll
          for (int n = 0; n < kRows; ++n) {
            float x = y[u][n] * factor[col(n)];
            if constexpr (kQ8) x = fmaf(x, kf[u][n / kLive], ve[u][n / kLive]);
            if (masked && key >= limit[col(n)]) x = -INFINITY;
            y[u][n] = x;
            over |= x > thresh[col(n)];
          }
        }
        if (any_of_group(over)) {
          // some key exceeds its row's running maximum: the step's maximum of every row
          float mine = -INFINITY;
#pragma unroll
          for (int n = 0; n < kRows; ++n) {
            float best = y[0][n];
#pragma unroll
            for (int u = 1; u < L::kPer; ++u)
              if (u < n_tiles) best = fmaxf(best, y[u][n]);
            const float m = redux_max(best);
            if (lane == (uint32_t)n) mine = m;
          }
          if (lane < (uint32_t)kRows) wred[quarter * N + lane] = mine;
          const bool dead = *group_dead != 0;
          named_bar_sync(1, 128);
          if (dead) {
            ok = false;
            break;
          }
          if (tid < kRows) {
            const float m = fmaxf(fmaxf(wred[tid], wred[N + tid]), fmaxf(wred[2 * N + tid], wred[3 * N + tid]));
            const int x = col(tid);
            const float old = top[x];
            float al = 1.f;
            if (m > thresh[x]) {
              al = old == -INFINITY ? 0.f : ex2(old - m);
              top[x] = m;
              thresh[x] = m + R::kThreshold;
              ref[x] = m - R::kOffset;
            }
            alpha[x] = al;
          }
          named_bar_sync(1, 128);
#pragma unroll
          for (int n = 0; n < kRows; ++n) {
            l[n] *= alpha[col(n)];
            if constexpr (!kQ8) lr[n] *= alpha[col(n)];
          }
          if (t > 0) {  // O holds earlier tiles: rescale it once the last product is in
            wait(kv_empty + (2 * c - 1) % L::kSlots, ((2 * c - 1) / L::kSlots) & 1);
            tc_fence_after();
            // columns past the rows there are get whatever alpha holds; they are never read
            uint32_t o[16];
#pragma unroll 1
            for (int n0 = 0; n0 < L::kColsO; n0 += 16) {
              tmem_ld16(tmem + lanes + L::kColO + n0, o);
              tmem_ld_wait16(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[n0 % N + i]);
              tmem_st16(tmem + lanes + L::kColO + n0, o);
            }
            tmem_st_wait();
          }
        }
        // weights, into the buffer that the product of two steps ago has read: 16 bytes of
        // rows at a time for a key; rows past the chunk's last are left out
        constexpr int kGroup = kQ8 ? 16 : 8;
#pragma unroll
        for (int u = 0; u < L::kPer; ++u) {
          if (u >= n_tiles) break;
          const uint32_t pbuf = smem_u32(smem + L::kOffP) + ((st & 1) * L::kPer + u) * L::kBlocksP * L::kRowBlock + r * 16;
          // a word of four e5m2 codes, or two words of two bf16 values, for four rows
          uint32_t p1[N / kGroup][4], p2[N / kGroup][4], p3[N / kGroup][4];
#pragma unroll
          for (int i = 0; i < N / kGroup; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) p1[i][j] = p2[i][j] = p3[i][j] = 0;
#pragma unroll
          for (int n = 0; n < kRows; n += 4) {
            const int h = n / kLive, x = col(n);
            float pw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              pw[j] = ex2(y[u][n + j] - ref[x + j]);
              l[n + j] = fmaf(pw[j], vinv[u][h], l[n + j]);
            }
            if constexpr (kQ8) {
              const int i = x / 16, j = x % 16 / 4;
              split_weights(pw, p1[i][j], p2[i][j], p3[i][j]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                const uint32_t k2 = pack_bf16x2(pw[j], pw[j + 1]);
                p1[x / 8][(x % 8 + j) / 2] = k2;
                lr[n + j] += __uint_as_float(k2 << 16);
                lr[n + j + 1] += __uint_as_float(k2 & 0xFFFF0000u);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < N / kGroup; ++i) {
            const uint32_t at = pbuf + i * kTile * 16;
            st_shared_v4(at, p1[i][0], p1[i][1], p1[i][2], p1[i][3]);
            if constexpr (kQ8) {
              st_shared_v4(at + L::kRowBlock, p2[i][0], p2[i][1], p2[i][2], p2[i][3]);
              st_shared_v4(at + 2 * L::kRowBlock, p3[i][0], p3[i][1], p3[i][2], p3[i][3]);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive_warp(p_full + (st & 1));
        c += n_tiles;
      }
      // ---- epilogue: all products of the piece are in (a group that broke off has ok =
      // false in every warp and leaves here)
      if (ok) wait(kv_empty + (2 * c - 1) % L::kSlots, ((2 * c - 1) / L::kSlots) & 1);
      if (any_of_group(!ok)) break;
      tc_fence_after();
      {
        float v[kRows];
#pragma unroll
        for (int n = 0; n < kRows; ++n) v[n] = l[n];
        const float s1 = warp_sums<kRows>(v);
        float s2 = s1;
        if constexpr (!kQ8) {
#pragma unroll
          for (int n = 0; n < kRows; ++n) v[n] = lr[n];
          s2 = warp_sums<kRows>(v);
        }
        if (lane < (uint32_t)kRows) {
          wred[quarter * N + lane] = s1;
          wred2[quarter * N + lane] = s2;
        }
      }
      named_bar_sync(1, 128);
      auto sum_of = [&](const float* x, int n) { return (x[n] + x[N + n]) + (x[2 * N + n] + x[3 * N + n]); };
      float o[kRows];
      ld_rows<N, kHeads, kHeadRows, kLive, L::kPiecesP>(tmem + lanes + L::kColO, 0.125f, o);
      const bool whole = p.t0 == 0 && p.t1 == p.tiles;
      if (whole) {
#pragma unroll
        for (int n = 0; n < kRows; ++n) {
          const float sum = sum_of(wred2, n);
          const float inv = sum > 0.f ? 1.f / sum : sum;
          const float x = sum == 0.f ? 0.f : o[n] * inv;  // every key hidden: O = 0, whatever V holds
          const int row = out_row[col(n)];
          const bool mine = D == 128 || n / kLive == r / 64;  // a pair's head has its half of O^T
          if (row >= 0 && mine) a.o[(size_t)row * D + (D == 64 ? (r & 63) : r)] = __float2bfloat16(x);
        }
        if (tid < kRows && out_row[col(tid)] >= 0) {
          const float sum = sum_of(wred, tid);
          const int row = out_row[col(tid)], token = row / a.Hq, head = row - token * a.Hq;
          a.lse[token * a.lse_row + head * a.lse_head] =
              sum == 0.f ? -INFINITY : (ref[col(tid)] + __log2f(sum)) * 0.69314718055994530942f;
        }
      } else {
        // slot 0: a piece that goes on with a unit begun before; slot 1: a unit begun here
        const size_t slot = 2 * (size_t)blockIdx.x + (p.t0 == 0 ? 1 : 0);
#pragma unroll
        for (int n = 0; n < kRows; ++n) a.part_o[(slot * N + col(n)) * 128 + r] = o[n];
        if (tid < kRows) {
          a.part_m[slot * N + col(tid)] = ref[col(tid)];
          a.part_l[slot * N + col(tid)] = sum_of(wred, tid);
          a.part_lr[slot * N + col(tid)] = sum_of(wred2, tid);
        }
        if (p.t0 == 0 && tid < N) a.part_rows[(size_t)blockIdx.x * N + tid] = out_row[tid];
        if (p.t0 == 0 && tid == 0) {
          // parts up to the team that has the unit's end
          const long long last = w.pos + p.after - 1;
          a.meta[blockIdx.x] =
              make_int4((int)(((last + 1) * w.teams - 1) / w.total) - (int)blockIdx.x / a.team + 1, 0, 0, 0);
        }
      }
      named_bar_sync(1, 128);  // the rows' places are written again for the next piece
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) grid_dependents_launch();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Joins the partial states of the unit that begins in attention CTA blockIdx.x (none:
// nothing to do), a warp per row: with M the largest reference, every part's sums and
// O count 2^(m - M).  Part 0 is that CTA's slot 1, part i the slot 0 of the same member of
// the i-th team after its.  Latency is all it costs (a few parts, in L2): what does not
// depend on one another is loaded together.
template <int N, int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedArgs a) {
  grid_dependency_wait();  // launched while the attention kernel still runs
  grid_dependents_launch();
  const int cta = blockIdx.x, n = blockIdx.y * 4 + warp_id(), lane = lane_id();
  const int parts = a.meta[cta].x, row = a.part_rows[(size_t)cta * N + n];
  if (parts == 0 || row < 0) return;
  auto at = [&](int i) { return (2 * (size_t)(cta + i * a.team) + (i == 0 ? 1 : 0)) * N + n; };
  constexpr int kPer = D / 32;
  const int d0 = lane * kPer + (D == 64 && n >= N / 2 ? 64 : 0);
  float M = -INFINITY, acc[kPer], l = 0.f, lr = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  constexpr int kBatch = 16;
  for (int i0 = 0; i0 < parts; i0 += kBatch) {
    // lane i: the sums of part i0 + i
    const bool have = lane < kBatch && i0 + lane < parts;
    const size_t own = at(have ? i0 + lane : 0);
    const float pl = have ? a.part_l[own] : 0.f, pm = have ? a.part_m[own] : -INFINITY, plr = have ? a.part_lr[own] : 0.f;
    // and everyone its dims of all of them
    float x[kBatch][kPer];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i0 + i >= parts) break;
      const float* src = a.part_o + at(i0 + i) * 128 + d0;
      if constexpr (kPer == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        x[i][0] = v.x, x[i][1] = v.y;
      }
    }
    const float top = fmaxf(M, redux_max(pl == 0.f ? -INFINITY : pm));
    const float keep = M == -INFINITY ? 0.f : ex2(M - top);
    const float wt = pl == 0.f ? 0.f : ex2(pm - top);
    M = top;
    l = l * keep + wt * pl;
    lr = lr * keep + wt * plr;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= keep;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i0 + i >= parts) break;
      const float w = __shfl_sync(0xffffffffu, wt, i);
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, x[i][e], acc[e]);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, off);
    lr += __shfl_xor_sync(0xffffffffu, lr, off);
  }
  const float inv = lr > 0.f ? 1.f / lr : (lr == 0.f ? 0.f : lr);
  __nv_bfloat16* out = a.o + (size_t)row * D + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) {
    const int token = row / a.Hq, head = row - token * a.Hq;
    a.lse[token * a.lse_row + head * a.lse_head] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.69314718055994530942f;
  }
}

// Key heads (or pairs) whose CTAs form a team: a divisor of them, up to kMaxTeam, that leaves
// next to no CTA without a team.
constexpr int kMaxTeam = 4;
int team_size(int groups, int ctas) {
  int best = 1;
  for (int t = 2; t <= std::min({groups, ctas, kMaxTeam}); ++t)
    if (groups % t == 0 && ctas / t * t >= ctas / best * best * 31 / 32) best = t;
  return best;
}

template <int N, bool kQ8, int D, int kLive>
fa_status launch_paged_impl(const PagedLaunch& L0, cudaStream_t stream) {
  using L = PagedLayout<N, kQ8>;
  static PerDeviceOnce attr_once;
  if (!attr_once.run([] {
        return cudaFuncSetAttribute(paged_kernel<N, kQ8, D, kLive>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    L::kSmemBytes) == cudaSuccess;
      }))
    return FA_ERR_CUDA;
  const int ctas = num_sms();
  PagedArgs a = paged_args(L0);
  const PagedCarve c = paged_carve(ctas, N, 128);
  const int groups = D == 64 ? (L0.Hkv + 1) / 2 : L0.Hkv;
  a.team = team_size(groups, ctas);
  a.teams = ctas / a.team;
  a.sets = groups / a.team;
  a.min_rows = 0;
  a.max_rows = L0.few_rows;
  c.place(a, L0.workspace);
  prof_before(stream, kKPaged);
  cudaError_t err =
      launch_dependent(paged_kernel<N, kQ8, D, kLive>, dim3(a.teams * a.team), kThreads<N, kQ8>, L::kSmemBytes, stream, a);
  prof_after(stream, kKPaged);
  if (err != cudaSuccess) return FA_ERR_CUDA;
  if (L0.max_k <= kTile) return FA_OK;  // units of one tile are never split
  prof_before(stream, kKPagedMerge);
  err = launch_dependent(paged_merge_kernel<N, D>, dim3(a.teams * a.team, N / 4), 128, 0, stream, a);
  prof_after(stream, kKPagedMerge);
  return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <bool kQ8, int D>
fa_status launch_paged_type(const PagedLaunch& L, cudaStream_t stream) {
  // rows of one key head's longest chunk that this kernel takes
  const long long rows = std::min((long long)L.max_q * (L.Hq / L.Hkv), (long long)L.few_rows);
  if (rows <= 4) return launch_paged_impl<16, kQ8, D, 4>(L, stream);
  if (rows <= head_rows<16, D>()) return launch_paged_impl<16, kQ8, D, head_rows<16, D>()>(L, stream);
  return launch_paged_impl<32, kQ8, D, head_rows<32, D>()>(L, stream);
}

}  // namespace

size_t paged_few_workspace() { return paged_carve(num_sms(), 32, 128).bytes; }

fa_status launch_paged_few(const PagedLaunch& L, cudaStream_t stream) {
  if (L.d == 64) return L.k_scales ? launch_paged_type<true, 64>(L, stream) : launch_paged_type<false, 64>(L, stream);
  return L.k_scales ? launch_paged_type<true, 128>(L, stream) : launch_paged_type<false, 128>(L, stream);
}

}  // namespace fa
