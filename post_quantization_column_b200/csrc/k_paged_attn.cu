// k_paged_attn.cu — attention of one new token per sequence over a paged key-value cache.
//
//   o_h = (sum_t p_t v_t) / (sum_t p_t),  p_t = 2^(s_t - m),  s_t = scale log2(e) q_h . k_t
//
// over the sequence's first `length` cached tokens, with the running maximum m of the scores
// met so far (the sums are rescaled when it grows), so the cache is read once for up to 8 query heads
// of a key-value head (16 where heads have 64 or 128 dims), which share its bytes. More query
// heads than that make another pass over them.
//
// What bounds it: the cache's bytes (each of 2 D values per token and key-value head is used in
// Hq / Hkv multiply-adds), so the kernel is a stream.
//
// Work. The unit is 64 tokens of one (sequence, key-value head), more where rows are shorter than 256
// bytes: 32 KB of the cache, or 64 KB with 16-bit heads of 256. All units of the batch, sequence-major,
// are dealt to a grid of as many CTAs as fit the SMs, in equal contiguous runs; a CTA finds its run from the lengths on the device. A (sequence, head) that lies within one run is
// finished there; one that crosses runs leaves a partial (o, m, l) per run, and a second
// kernel adds them in run order (fixed order: equal inputs give equal bits). That join costs
// 3 to 5 us, so where the longest sequence has at most kWhole units runs begin and end with
// segments instead (55 sequences of 128 tokens, 8 heads: 8.7 us against 12.4 cut and joined).
//
// Tile. A warp takes a quarter of a unit (8 KB: 16 tokens at D = 128 in 16 bits) with its own running
// maximum; the four warps meet once per (sequence, head). Tokens are the rows of both products,
// so a group of up to 8 heads fills the 8 columns of an m16n8k16 MMA and none of the 16 rows is
// padding:
//   S^T (16 tokens x 8 heads) = K Q^T,   O^T (16 dims x 8 heads) += V^T P^T.
// The sum over dims in q . k may run in any order and the rows of O^T may be any dims, so
// each lane is given dims that lie together in memory: 32-byte pieces of the cache rows are
// its MMA fragments as they are (keys) or after a byte shuffle of two tokens' words (values).
// The cache therefore goes from memory to the fragments' registers without shared memory: a
// warp loads the keys of its next tile when it has used these keys, the next values when it
// has used these values, and the twelve warps of an SM keep some 90 KB on the way. (A ring of
// cp.async stages took twice the time: eight warps' chains of shared-memory reads, shuffles
// and products were longer than the loads; bulk copies of 128-byte rows stop at 3.9 TB/s.)
// The MMAs are mma.sync: tcgen05 wants 64 rows or more of a tile in shared memory, and at one
// token per sequence the tensor pipe is 15 % busy here.
//
// Measured (B200, device time in a captured graph; the copy rate is 6.55 TB/s): 16 x 4096 tokens
// of 32 fp16 heads 164 us, 6.6 TB/s; 67 ragged sequences up to 8192, 8 bf16 heads shared by 64,
// 189 us, 6.4 TB/s; one sequence of 131072 tokens 89 us, 6.1 TB/s; 96 ragged sequences up to
// 4099 on an e4m3 cache 96 us, 4.6 TB/s (bound by the latency of a tile's chain: 128 conversions and 32
// byte shuffles of its 647 instructions unpack e4m3; 6.7 TB/s at the margin of longer sequences); one of
// 33 tokens 4.7 us.
#include "decode_kernels.h"

#include <algorithm>
#include <cmath>

namespace awq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 3 * 148;  // three CTAs on each of a B200's SMs
constexpr int kWhole = 4;           // units of the longest segment that is not cut
// Over short rows (kShort), the four warps of a CTA can take four heads of the same tokens instead of
// four parts of one head's tokens (Geometry::side). That pays
// - in batches where no sequence has more than one unit, with kMany units a CTA or more: a
//   segment's end, where the warps meet, then comes once for four heads (243 ragged sequences up
//   to 86, 32 e4m3 heads: 49 against 68 us);
// - in long runs where the heads lie side by side in memory, with kLong units a CTA or
//   more: what is read at one time lies together (e4m3, D = 128, 8 heads: 55 x 8192 tokens 161
//   against 165 us, 55 x 4096 91 against 88; 32 heads, 32 ragged sequences up to 8192: 195 against
//   210 us). Units are a quarter as deep there and leave four heads' partial sums at a run's ends.
constexpr int kMany = 2, kLong = 40;

template <int D, int TYPE, int NB>
struct Tile {
  static constexpr int ES = type_bytes(TYPE);
  static constexpr int kKBytes = D * ES / 4 < 32 ? D * ES / 4 : 32;  // bytes of a lane's piece of a key row (4 lanes a row)
  static constexpr int kKChunks = D * ES / 4 / kKBytes;              // pieces per key row and lane
  static constexpr int kVBytes = D * ES / 8 < 32 ? D * ES / 8 : 32;  // the same of a value row (8 lanes a row)
  static constexpr int kVChunks = D * ES / 8 / kVBytes;
  static constexpr int kSteps = D / 16;                              // k16 steps of q . k; also tiles of 16 dims of O^T
  static constexpr int kBlocks = 256 / (D * ES) > 1 ? 256 / (D * ES) : 1;  // blocks of 16 tokens of a warp's tile
  static constexpr int kTok = 16 * kBlocks;
  static constexpr bool kShort = D * ES <= 128;                      // rows of which a CTA may take several heads'
  static constexpr int kSub = kShort ? kWarps : 1;                   // places of a run's partial sums
  static constexpr int kHeads = NB * 8;                              // query heads of a work segment
  static constexpr int kPitch = D + 2;                               // floats between heads in the join buffer
  static constexpr int kCtas = D * NB > 128 || (D == 64 && NB == 2) ? 2 : 3;                // per SM, by registers
};

template <int TYPE>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if constexpr (TYPE == kTypeBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit values held in MMA fragment order.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The four e4m3 values of a word as two fp16 pairs, exactly.
__device__ __forceinline__ void e4m3_pairs(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// A piece of a cache row, read once.
template <int BYTES>
struct Piece {
  uint32_t w[BYTES / 4];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (BYTES == 32)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p));
    else if constexpr (BYTES == 16)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
    else
      asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) w[i] = 0u;
  }
};

// `from` + 32 `place`.
__device__ __forceinline__ const uint8_t* at_place(const uint8_t* from, uint32_t place) {
  uint64_t p;
  asm("mad.wide.u32 %0, %1, 32, %2;" : "=l"(p) : "r"(place), "l"(from));
  return reinterpret_cast<const uint8_t*>(p);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A sequence's tokens as the kernel takes them: never more than its table row can name.
__device__ __forceinline__ int clamped_length(const int32_t* lengths, int64_t b, int cap) {
  return min(max(lengths[b], 0), cap);
}

// The run of CTA c when T units are dealt to C CTAs, and the CTA whose run holds unit l.
__host__ __device__ __forceinline__ int64_t run_start(int64_t c, int64_t T, int64_t C) { return c * T / C; }
__device__ __forceinline__ int64_t unit_owner(int64_t l, int64_t T, int64_t C) { return ((l + 1) * C - 1) / T; }

constexpr uint32_t kNoRow = 0xFFFFFFFFu;        // a row without a place (the last 32 bytes below 128 GB)
constexpr float kNoMax = -3.402823466e38f;  // the maximum before any score: finite, so that m - m is 0

// A place in the sequence-major list of units: sequence, group of key-value heads, block of their
// query heads, unit.
struct Cursor {
  int b, kg, hg, blk, len;
};

struct Space {       // the work space of a launch
  float* o;          // [2 C][kSub][heads][D] partial sums of run c: slot 2 c of the segment that begins in it and
                     // goes on, slot 2 c + 1 of the one that began before it
  float2* ml;        // [2 C][kSub][heads] (m, l)
  int4* joins;       // what the second kernel joins: pieces (0: nothing), the first piece's place, sequence, head
                     // block; one per segment if there are no more segments than CTAs, else kSub per CTA
};

struct Geometry {
  int cap;           // tokens a table row can name
  int heads_per;     // Hq / Hkv
  int hgroups;       // blocks of query heads per key-value head
  int side;          // key-value heads that may go side by side in a CTA: 1, 2 or 4, of kWarps / side warps each
  int adjacent;      // the heads of a token lie side by side in memory
  int64_t ctas;
  int by_segment;    // the joins are listed by segment
  int64_t listed;
  uint32_t page32, slot32, head32;  // the cache's strides in units of 32 bytes
  uint32_t page_mul;  // p / page_size = (p * page_mul) >> page_shift for 0 <= p < 2^31
  int page_shift;
};

// WHOLE: every block of 16 tokens lies in one page (the page size is a multiple of 16).
template <int D, int TYPE, int NB, bool WHOLE>
__global__ void __launch_bounds__(kThreads, Tile<D, TYPE, NB>::kCtas)
    paged_attn_kernel(PagedAttnArgs a, Geometry geo, Space sp) {
  using T_ = Tile<D, TYPE, NB>;
  constexpr int ES = T_::ES, KB = T_::kKBytes, KC = T_::kKChunks, VB = T_::kVBytes, VC = T_::kVChunks, S = T_::kSteps, TB = T_::kBlocks, SUB = T_::kSub;
  constexpr int kTok = T_::kTok;
  constexpr int MMA = TYPE == kTypeBf16 ? kTypeBf16 : kTypeF16;
  // Over a 16-bit cache the weights enter the product as two 16-bit values, the rounded weight and the rest,
  // for as many bits as fp32 sums keep: with the rounded weight alone the error against 64 bits was 0.0021 of
  // the output for bf16 and 0.00027 for fp16, with both it is that of the output's own rounding (0.0017 and
  // 0.00021). The second product costs 0.2 to 0.4 us of 160 to 190 over long sequences, 3 % of short
  // ones and 4 % of groups of 16 heads. Over an e4m3 cache, whose values hold 4 bits, it would cost
  // 18 % (96 ragged sequences: 113 against 95 us) and the weights are fp16 alone.
  constexpr bool kRest = ES == 2;
  // The maximum in use may lag behind the scores by 2^kLag before the sums are rescaled: weights
  // are p 2^kBias, 2^(kBias + kLag) at most, and in fp16 stay representable down to p = 2^-31 of
  // the maximum in use. Both factors cancel in o / l.
  constexpr float kLag = 8.0f, kBias = MMA == kTypeF16 ? 7.0f : 0.0f;
  __shared__ __align__(16) float join_buf[kWarps * 8 * T_::kPitch];
  __shared__ float sM[kWarps][T_::kHeads], sL[kWarps][T_::kHeads];
  __shared__ int sBad[kWarps];
  __shared__ int64_t sScan[kWarps + 1];
  __shared__ int sSnap[2];  // units from the run's even ends to those of segments
  __shared__ Cursor sStart;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t = lane & 3;
  const PagedCache& c = a.c;
  wait_for_previous();
  start_next();  // the join is set up meanwhile

  // ---- the run: exclusive sums of the sequences' units, then the places of its two ends
  const int64_t per = ceil_div(a.B, kThreads), b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  if (tid < 2) sSnap[tid] = 0;
  int64_t mine, before, total;
  int longest;
  auto count_units = [&](int unit) {
    mine = 0;
    longest = 0;
    for (int64_t b = b0; b < b1; ++b) {
      const int nblk = (clamped_length(a.lengths, b, geo.cap) + unit - 1) / unit;
      mine += nblk;
      longest = max(longest, nblk);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += up;
    }
    longest = __reduce_max_sync(~0u, longest);
    if (lane == 31) {
      sScan[warp] = incl;
      sBad[warp] = longest;
    }
    __syncthreads();
    before = incl - mine;
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sScan[w];
      total += sScan[w];
      longest = max(longest, sBad[w]);
    }
  };
  int side = 1;
  count_units(kTok * kWarps);
  const bool snap = longest <= kWhole;
  const int64_t all = total * c.heads * geo.hgroups;
  if (T_::kShort && geo.side > 1 &&
      (longest <= 1 ? all >= kMany * geo.ctas : geo.adjacent && all >= kLong * geo.ctas)) {
    side = geo.side;
    __syncthreads();  // the sums have been read
    count_units(kTok * kWarps / side);
  }
  const int unit = kTok * kWarps / side;
  const int HH = c.heads / side * geo.hgroups;
  const int deep = kWarps / side, head_of = warp / deep, tok_of = warp % deep * kTok;  // the warp's head and tokens of a unit
  // No run is empty: with fewer units than CTAs the later CTAs have none. Where segments are short a
  // run begins and ends with one instead (and may be empty): a join takes longer than kWhole units.
  const int64_t units = total * HH, C = min(geo.ctas, units);
  int64_t ends_at[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    ends_at[e] = blockIdx.x < C ? run_start(blockIdx.x + e, units, C) : 0;
    const int64_t u = ends_at[e];
    if (before * HH <= u && u < (before + mine) * HH) {
      int64_t at = before * HH;
      for (int64_t b = b0; b < b1; ++b) {
        const int len = clamped_length(a.lengths, b, geo.cap), nblk = (len + unit - 1) / unit;
        if (u < at + static_cast<int64_t>(nblk) * HH) {
          const int64_t rel = u - at;
          int hh = static_cast<int>(rel / nblk), blk = static_cast<int>(rel % nblk);
          if (snap && blk > 0) {
            sSnap[e] = nblk - blk;
            blk = nblk - 1;  // the unit before the run: it goes on from there
          }
          if (e == 0) sStart = {static_cast<int>(b), hh / geo.hgroups, hh % geo.hgroups, blk, len};
          break;
        }
        at += static_cast<int64_t>(nblk) * HH;
      }
    }
  }
  // sequences without tokens have no units: their rows of zeros are dealt out too
  for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x)
    if (a.lengths[b] <= 0) {
      if (geo.by_segment)
        for (int i = tid; i < c.heads * geo.hgroups; i += kThreads) sp.joins[b * c.heads * geo.hgroups + i] = make_int4(0, 0, 0, 0);
      for (int64_t i = tid; i < static_cast<int64_t>(a.Hq) * D / 2; i += kThreads)
        static_cast<uint32_t*>(a.out)[b * a.Hq * D / 2 + i] = 0u;
    }
  __syncthreads();
  const int64_t u0 = ends_at[0] + sSnap[0];
  const int n = static_cast<int>(ends_at[1] + sSnap[1] - u0);
  if (n <= 0) {
    if (tid < SUB && !geo.by_segment) sp.joins[blockIdx.x * SUB + tid] = make_int4(0, 0, 0, 0);
    return;
  }

  auto advance = [&](Cursor& k) {
    if (++k.blk * unit < k.len) return;
    k.blk = 0;
    if (++k.hg < geo.hgroups) return;
    k.hg = 0;
    if (++k.kg < c.heads / side) return;
    k.kg = 0;
    do {
      ++k.b;
      k.len = k.b < a.B ? clamped_length(a.lengths, k.b, geo.cap) : 1;
    } while (k.len == 0);
  };

  // ---- the loading side. look_up() asks the block table for a tile's pages one tile before
  // place() turns them into places of the cache, in units of 32 bytes: per block of 16 tokens
  // that of its first row if WHOLE, of row lane % 16 otherwise.
  Cursor first = sStart;
  if (sSnap[0] > 0) advance(first);
  Cursor ic = first;
  int looked = 0;
  int32_t page[TB];            // asked for
  uint32_t within[TB];         // places from the page's to the row's
  uint32_t row[TB];            // placed
  int ask_rows = 0, rows = 0;  // rows left of the sequence from the tile's first on
  bool full = false;           // every block of the placed tile has its 16 rows
  bool bad_tile = false;       // the placed tile needs a page outside the cache
  const int own = WHOLE ? 0 : lane & 15;
  auto look_up = [&]() {
    if (looked >= n) {
      ask_rows = 0;
    } else {
      if (looked > 0) advance(ic);
      ask_rows = ic.len - (ic.blk * unit + tok_of);
    }
    ++looked;
    const int tok0 = ic.blk * unit + tok_of + own;
    const int32_t* table = c.table + ic.b * c.table_stride;
#pragma unroll
    for (int k = 0; k < TB; ++k) {
      const int tok = tok0 + 16 * k;
      const uint32_t pi = static_cast<uint32_t>(static_cast<uint64_t>(tok) * geo.page_mul >> geo.page_shift);
      within[k] = (tok - pi * c.page_size) * geo.slot32 + (ic.kg * side + head_of) * geo.head32;
      page[k] = -1;
      if (16 * k + own < ask_rows) page[k] = table[pi];
    }
  };
  auto place = [&]() {
    rows = ask_rows;
    bool inside = true;
#pragma unroll
    for (int k = 0; k < TB; ++k) {
      const bool in = static_cast<uint32_t>(page[k]) < static_cast<uint32_t>(c.num_pages);
      row[k] = in ? page[k] * geo.page32 + within[k] : kNoRow;
      inside = inside && in;
    }
    full = WHOLE && inside && rows >= kTok;
    bad_tile = false;
    if (!inside)
#pragma unroll
      for (int k = 0; k < TB; ++k) bad_tile = bad_tile || (row[k] == kNoRow && 16 * k + own < rows);
  };
  Piece<KB> kr[TB][2][KC];
  Piece<VB> vr[TB][4][VC];
  // The lane's rows of a block: tokens g, g + 8 of the keys, 2t, 2t + 1, 2t + 8, 2t + 9 of the values.
  uint32_t k_at[2], v_at[4];
#pragma unroll
  for (int r = 0; r < 2; ++r) k_at[r] = (g + 8 * r) * geo.slot32;
#pragma unroll
  for (int r = 0; r < 4; ++r) v_at[r] = (2 * t + (r & 1) + 8 * (r >> 1)) * geo.slot32;
  const uint8_t* k_from = static_cast<const uint8_t*>(c.k) + KB * t;
  const uint8_t* v_from = static_cast<const uint8_t*>(c.v) + VB * g;
  auto load_keys = [&]() {
    if (full) {
#pragma unroll
      for (int k = 0; k < TB; ++k)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* src = at_place(k_from, row[k] + k_at[r]);
#pragma unroll
          for (int j = 0; j < KC; ++j) kr[k][r][j].load(src + 4 * KB * j);
        }
      return;
    }
#pragma unroll
    for (int k = 0; k < TB; ++k)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = g + 8 * r;
        const uint32_t off = WHOLE ? row[k] + k_at[r] : __shfl_sync(~0u, row[k], tok);
        const bool live = (WHOLE ? row[k] : off) != kNoRow && 16 * k + tok < rows;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          kr[k][r][j].zero();
          if (live) kr[k][r][j].load(at_place(k_from, off) + 4 * KB * j);
        }
      }
  };
  auto load_values = [&]() {
    if (full) {
#pragma unroll
      for (int k = 0; k < TB; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* src = at_place(v_from, row[k] + v_at[r]);
#pragma unroll
          for (int j = 0; j < VC; ++j) vr[k][r][j].load(src + 8 * VB * j);
        }
      return;
    }
#pragma unroll
    for (int k = 0; k < TB; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tok = 2 * t + (r & 1) + 8 * (r >> 1);
        const uint32_t off = WHOLE ? row[k] + v_at[r] : __shfl_sync(~0u, row[k], tok);
        const bool live = (WHOLE ? row[k] : off) != kNoRow && 16 * k + tok < rows;
#pragma unroll
        for (int j = 0; j < VC; ++j) {
          vr[k][r][j].zero();
          if (live) vr[k][r][j].load(at_place(v_from, off) + 8 * VB * j);
        }
      }
  };
  look_up();
  place();
  load_keys();
  load_values();
  bool bad_now = bad_tile;
  look_up();

  // ---- the computing side
  Cursor cc = first;
  uint32_t qf[NB][S][2];          // Q^T fragments: heads g of each block, this lane's dims
  float acc[NB][S][4];            // O^T: per 16-dim tile, (dim, dim + 1) x (heads 2t, 2t + 1)
  float ls[NB][2];                // l of heads 2t, 2t + 1
  float m[NB][2], sc[NB][2];      // the maximum in use, lowered by kBias; the factor of the products, base 2
  bool bad = false;
  auto load_queries = [&](const Cursor& at) {
    const int kvh = at.kg * side + head_of, hb = at.hg * T_::kHeads;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int h = hb + nb * 8 + g;
      const bool live = h < geo.heads_per;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + at.b * a.q_sb +
                          static_cast<int64_t>(kvh * geo.heads_per + (live ? h : 0)) * a.q_sh;
#pragma unroll
      for (int st = 0; st < S; ++st) {
        // dims of step st: 4 elements of the lane's piece st / PER
        constexpr int PER = KB / (4 * ES);  // steps that a piece serves
        const int d = (st / PER) * (4 * KB / ES) + (KB / ES) * t + 4 * (st % PER);
        qf[nb][st][0] = qf[nb][st][1] = 0u;
        if (live) asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(qf[nb][st][0]), "=r"(qf[nb][st][1]) : "l"(q + d));
      }
    }
  };
  auto begin_segment = [&]() {
    bad = a.lengths[cc.b] > geo.cap;
    const float k_scale = TYPE == kTypeE4m3 ? c.k_scale[cc.kg * side + head_of] : 1.0f;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;  // the factor of the scores is not negative
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int st = 0; st < S; ++st) {
        qf[nb][st][0] ^= flip;
        qf[nb][st][1] ^= flip;
      }
      float up = 1.0f;
      if (TYPE == kTypeE4m3 && a.q_type == kTypeBf16) {
        // the products run in fp16: bf16 queries are brought to [1, 2) by a power of two
        float peak = 0.0f;
#pragma unroll
        for (int st = 0; st < S; ++st)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 f = unpack16(qf[nb][st][x], kTypeBf16);
            peak = fmaxf(peak, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        peak = fmaxf(peak, __shfl_xor_sync(~0u, peak, 1));
        peak = fmaxf(peak, __shfl_xor_sync(~0u, peak, 2));
        const uint32_t e = __float_as_uint(peak) & 0x7F800000u;
        float down = 1.0f;
        if (e > 0x01000000u && e < 0x7E000000u) {
          up = __uint_as_float(e);
          down = __uint_as_float(0x7F000000u - e);
        }
#pragma unroll
        for (int st = 0; st < S; ++st)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 f = unpack16(qf[nb][st][x], kTypeBf16);
            qf[nb][st][x] = pack16(f.x * down, f.y * down, kTypeF16);
          }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sc[nb][x] = fabsf(a.scale * 1.4426950408889634f) * k_scale * __shfl_sync(~0u, up, (2 * t + x) * 4);
        m[nb][x] = kNoMax;
      }
#pragma unroll
      for (int st = 0; st < S; ++st) acc[nb][st][0] = acc[nb][st][1] = acc[nb][st][2] = acc[nb][st][3] = 0.0f;
      ls[nb][0] = ls[nb][1] = 0.0f;
    }
  };
  load_queries(cc);
  begin_segment();
  for (int i = 0; i < n; ++i) {
    const bool ends = (cc.blk + 1) * unit >= cc.len, last = i + 1 == n;
    bad = bad || bad_now;
    const int tok0 = cc.blk * unit + tok_of;
    // one block and one group of heads: two chains of products, for their latency
    constexpr int CHAINS = TB * NB == 1 ? 2 : 1;
    float s[TB][NB][4];
    {
      float s2[CHAINS][TB][NB][4];
#pragma unroll
      for (int k = 0; k < TB; ++k) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < CHAINS; ++h) s2[h][k][nb][0] = s2[h][k][nb][1] = s2[h][k][nb][2] = s2[h][k][nb][3] = 0.0f;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          const auto& wl = kr[k][0][j].w;  // row g
          const auto& wh = kr[k][1][j].w;  // row g + 8
          constexpr int PER = KB / (4 * ES);
          if constexpr (ES == 2) {
#pragma unroll
            for (int st = 0; st < PER; ++st)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma_16816<MMA>(s2[st % CHAINS][k][nb], wl[2 * st], wh[2 * st], wl[2 * st + 1], wh[2 * st + 1], qf[nb][PER * j + st][0],
                               qf[nb][PER * j + st][1]);
          } else {
#pragma unroll
            for (int st = 0; st < PER; ++st) {
              uint32_t a0, a1, a2, a3;
              e4m3_pairs(wl[st], a0, a2);
              e4m3_pairs(wh[st], a1, a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma_16816<MMA>(s2[st % CHAINS][k][nb], a0, a1, a2, a3, qf[nb][PER * j + st][0], qf[nb][PER * j + st][1]);
            }
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[k][nb][x] = CHAINS == 2 ? s2[0][k][nb][x] + s2[CHAINS - 1][k][nb][x] : s2[0][k][nb][x];
      }
    }
    Cursor next = cc;
    if (!last) advance(next);
    if (ends && !last) load_queries(next);  // these have been used
    place();
    load_keys();
    {
      // products of rows g (values 0, 1) and g + 8 (2, 3) of each block with heads 2t and 2t + 1
      const bool ragged = tok0 + kTok > cc.len;  // the sequence ends within the tile
      if (ragged) {
#pragma unroll
        for (int k = 0; k < TB; ++k)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (tok0 + 16 * k + g + 8 * (x >> 1) >= cc.len) s[k][nb][x] = -INFINITY;
      }
      float top[NB][2];
      bool grow = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[nb][x] = fmaxf(s[0][nb][x], s[0][nb][2 + x]);
#pragma unroll
          for (int k = 1; k < TB; ++k) top[nb][x] = fmaxf(top[nb][x], fmaxf(s[k][nb][x], s[k][nb][2 + x]));
          grow = grow || top[nb][x] * sc[nb][x] - m[nb][x] > kLag + kBias;
        }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top[nb][x] = fmaxf(top[nb][x], __shfl_xor_sync(~0u, top[nb][x], o));
            const float up = fmaxf(m[nb][x], top[nb][x] * sc[nb][x] - kBias);
            const float f = exp2f(m[nb][x] - up);
            m[nb][x] = up;
            ls[nb][x] *= f;
#pragma unroll
            for (int st = 0; st < S; ++st) {
              acc[nb][st][x] *= f;
              acc[nb][st][2 + x] *= f;
            }
          }
        }
      }
      // l sums the weights as they enter the product, so that they still add up to one
#pragma unroll
      for (int k = 0; k < TB; ++k) {
        uint32_t pf[NB][2], rest[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = exp2_approx(s[k][nb][2 * r] * sc[nb][0] - m[nb][0]), p1 = exp2_approx(s[k][nb][2 * r + 1] * sc[nb][1] - m[nb][1]);
            const bool none = ragged && tok0 + 16 * k + g + 8 * r >= cc.len;
            const uint32_t w = none ? 0u : pack16(p0, p1, MMA);
            pf[nb][r] = transposed(w);
            if constexpr (kRest) {
              const float2 f = unpack16(w, MMA);
              rest[nb][r] = transposed(none ? 0u : pack16(p0 - f.x, p1 - f.y, MMA));
            }
          }
          constexpr uint32_t kOnes = MMA == kTypeBf16 ? 0x3F803F80u : 0x3C003C00u;
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // a row of ones times P^T
          mma_16816<MMA>(sum, kOnes, kOnes, kOnes, kOnes, pf[nb][0], pf[nb][1]);
          if constexpr (kRest) mma_16816<MMA>(sum, kOnes, kOnes, kOnes, kOnes, rest[nb][0], rest[nb][1]);
          ls[nb][0] += sum[0];
          ls[nb][1] += sum[1];
        }
#pragma unroll
        for (int j = 0; j < VC; ++j) {
#pragma unroll
          for (int w = 0; w < VB / 4; ++w) {  // the words of tokens 2t, 2t + 1, 2t + 8, 2t + 9
            const uint32_t w0 = vr[k][0][j].w[w], w1 = vr[k][1][j].w[w], w2 = vr[k][2][j].w[w], w3 = vr[k][3][j].w[w];
            if constexpr (ES == 2) {  // word w: dims 2w, 2w + 1 of the piece
              const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
              const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma_16816<MMA>(acc[nb][j * (VB / 4) + w], a0, a1, a2, a3, pf[nb][0], pf[nb][1]);
                if constexpr (kRest) mma_16816<MMA>(acc[nb][j * (VB / 4) + w], a0, a1, a2, a3, rest[nb][0], rest[nb][1]);
              }
            } else {  // word w: dims 4w .. 4w + 3
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t a0, a1, a2, a3;
                e4m3_pairs(__byte_perm(w0, w1, e ? 0x7362 : 0x5140), a0, a1);
                e4m3_pairs(__byte_perm(w2, w3, e ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                  mma_16816<MMA>(acc[nb][(j * (VB / 4) + w) * 2 + e], a0, a1, a2, a3, pf[nb][0], pf[nb][1]);
                  if constexpr (kRest) mma_16816<MMA>(acc[nb][(j * (VB / 4) + w) * 2 + e], a0, a1, a2, a3, rest[nb][0], rest[nb][1]);
                }
              }
            }
          }
        }
      }
    }
    load_values();
    bad_now = bad_tile;
    look_up();

    if (ends || last) {
      // ---- the four warps meet: factors to the common maximum, then one sum per head and dim
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (g == 0) {
            sM[warp][nb * 8 + 2 * t + x] = m[nb][x];
            sL[warp][nb * 8 + 2 * t + x] = ls[nb][x];
          }
      bad = __any_sync(~0u, bad);
      if (lane == 0) sBad[warp] = bad;
      __syncthreads();
      const bool any_bad = sBad[0] | sBad[1] | sBad[2] | sBad[3];
      const int64_t seg0 = u0 + i - cc.blk;  // the segment's first unit
      const bool whole = ends && seg0 >= u0;
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (seg0 < u0 ? 1 : 0);
      const int hb = cc.hg * T_::kHeads;
      const int live = min(T_::kHeads, geo.heads_per - hb);
      if (any_bad && tid == 0 && a.status) *a.status = 1;
      const bool begins = seg0 >= u0;
      if (tid < kWarps && (geo.by_segment ? begins && tid < side : last && tid < SUB)) {
        const int hh = (cc.kg * side + tid) * geo.hgroups + cc.hg;
        int pieces = 0;
        if (begins && !ends && tid < side)
          pieces = static_cast<int>(unit_owner(seg0 + (cc.len + unit - 1) / unit - 1, units, C) - blockIdx.x) + 1;
        const int64_t at = geo.by_segment ? static_cast<int64_t>(cc.b) * c.heads * geo.hgroups + hh : blockIdx.x * SUB + tid;
        sp.joins[at] = make_int4(pieces, 2 * SUB * blockIdx.x + tid, cc.b, hh);
      }
      auto top_of = [&](int hs, int h) {  // the maximum of head h of the hs-th key-value head
        float top = sM[hs * deep][h];
        for (int w = hs * deep + 1; w < (hs + 1) * deep; ++w) top = fmaxf(top, sM[w][h]);
        return top;
      };
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (nb) __syncthreads();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int h = nb * 8 + 2 * t + x;
          if (h < live) {
            const float f = exp2f(m[nb][x] - top_of(head_of, h));
            float* dst = join_buf + (warp * 8 + 2 * t + x) * T_::kPitch;
#pragma unroll
            for (int st = 0; st < S; ++st) {
              constexpr int TPP = VB / ES / 2;  // 16-dim tiles a piece serves: its element pairs
              const int d = (st / TPP) * (8 * VB / ES) + (VB / ES) * g + 2 * (st % TPP);
              *reinterpret_cast<float2*>(dst + d) = make_float2(acc[nb][st][x] * f, acc[nb][st][2 + x] * f);
            }
          }
        }
        __syncthreads();
        for (int e = tid; e < side * 8 * (D / 4); e += kThreads) {
          const int hs = e / (8 * (D / 4)), h8 = e / (D / 4) % 8, d = (e % (D / 4)) * 4, h = nb * 8 + h8;
          if (h >= live) continue;
          const float top = top_of(hs, h);
          float L = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int w = hs * deep; w < (hs + 1) * deep; ++w) {
            L += sL[w][h] * exp2f(sM[w][h] - top);
            const float2 x0 = *reinterpret_cast<const float2*>(join_buf + (w * 8 + h8) * T_::kPitch + d);
            const float2 x1 = *reinterpret_cast<const float2*>(join_buf + (w * 8 + h8) * T_::kPitch + d + 2);
            o[0] += x0.x;
            o[1] += x0.y;
            o[2] += x1.x;
            o[3] += x1.y;
          }
          if (any_bad) L = NAN;
          const int kvh = cc.kg * side + hs;
          if (whole) {
            const float r = (TYPE == kTypeE4m3 ? c.v_scale[kvh] : 1.0f) / L;
            const int64_t to = (static_cast<int64_t>(cc.b) * a.Hq + kvh * geo.heads_per + hb + h) * D + d;
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) =
                make_uint2(pack16(o[0] * r, o[1] * r, a.q_type), pack16(o[2] * r, o[3] * r, a.q_type));
          } else {
            const int64_t to = (part * SUB + hs) * T_::kHeads + h;
            *reinterpret_cast<float4*>(sp.o + to * D + d) = make_float4(o[0], o[1], o[2], o[3]);
            if (d == 0) sp.ml[to] = make_float2(top, L);
          }
        }
      }
      __syncthreads();
    }
    cc = next;
    if (ends && !last) begin_segment();
  }
}

// The segments that cross runs: o = (sum over the runs, in order, of o_c 2^(m_c - m)) / l. D / 4
// threads take a head's dims, four each, and `teams` teams of as many share its pieces out.
constexpr int kJoinThreads = 256;
template <int D, int HEADS, int SUB>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_join_kernel(PagedAttnArgs a, Geometry geo, Space sp, int teams) {
  constexpr int kTeam = D / 4, kAhead = 8;
  __shared__ float4 sO[kJoinThreads];
  __shared__ float2 sML[kJoinThreads / kTeam];
  const int tid = threadIdx.x, team = tid / kTeam, d = tid % kTeam * 4;
  const int per = kJoinThreads / kTeam / teams;          // heads of a CTA
  const int64_t head = static_cast<int64_t>(blockIdx.x) * per + team / teams, listed = head / HEADS;
  const int r = static_cast<int>(head % HEADS);
  wait_for_previous();
  start_next();
  const int4 job = listed < geo.listed ? sp.joins[listed] : make_int4(0, 0, 0, 0);
  const int pieces = job.x;                              // none: finished by its run
  const int kvh = job.w / geo.hgroups, h = (job.w % geo.hgroups) * HEADS + r;
  const bool live = pieces > 0 && h < geo.heads_per;
  float top = kNoMax, L = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](float m, float l, float4 v) {
    const float up = fmaxf(top, m), f = exp2f(top - up), fm = exp2f(m - up);
    top = up;
    L = L * f + l * fm;
    o.x = o.x * f + v.x * fm;
    o.y = o.y * f + v.y * fm;
    o.z = o.z * f + v.z * fm;
    o.w = o.w * f + v.w * fm;
  };
  if (live)
    for (int p0 = team % teams; p0 < pieces; p0 += kAhead * teams) {
      float2 ml[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int p = min(p0 + k * teams, pieces - 1);
        const int64_t at = (job.y + (2 * p + (p > 0 ? 1 : 0)) * SUB) * static_cast<int64_t>(HEADS) + r;  // it goes on in the next runs
        ml[k] = sp.ml[at];
        v[k] = *reinterpret_cast<const float4*>(sp.o + at * D + d);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (p0 + k * teams < pieces) add(ml[k].x, ml[k].y, v[k]);
    }
  if (teams > 1) {
    sO[tid] = o;
    if (d == 0) sML[team] = make_float2(top, L);
    __syncthreads();
    if (team % teams) return;
    for (int k = 1; k < teams; ++k) add(sML[team + k].x, sML[team + k].y, sO[tid + k * kTeam]);
  }
  if (!live) return;
  const float x = (a.c.type == kTypeE4m3 ? a.c.v_scale[kvh] : 1.0f) / L;
  const int64_t to = (static_cast<int64_t>(job.z) * a.Hq + kvh * geo.heads_per + h) * D + d;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) =
      make_uint2(pack16(o.x * x, o.y * x, a.q_type), pack16(o.z * x, o.w * x, a.q_type));
}

// Blocks of 8 query heads that share a pass over the cache: two where a group has more than 8 and
// the registers hold both (64 ragged sequences up to 8192, 4 bf16 heads of 128: 117 us for 64 query heads, 100
// for 32, whose pass of one block runs three CTAs an SM; the floor is 92). Larger groups read the
// cache again, from DRAM in long sequences, since a segment's passes follow one another: 211 us for
// 128 query heads there, and 190 for 64 on 4 heads of 256 (32 sequences) where 16 on 4 take 106.
int head_blocks(int Hq, int Hkv, int D) { return Hq / Hkv > 8 && D <= 128 ? 2 : 1; }

template <int D, int TYPE, int NB>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t s, int* launches) {
  using T_ = Tile<D, TYPE, NB>;
  Geometry geo;
  geo.cap = static_cast<int>(std::min<int64_t>(a.c.max_pages * a.c.page_size, INT32_MAX - 1024));
  geo.heads_per = a.Hq / a.c.heads;
  geo.hgroups = static_cast<int>(ceil_div(geo.heads_per, T_::kHeads));
  geo.side = a.c.heads % 4 == 0 ? 4 : (a.c.heads % 2 == 0 ? 2 : 1);
  geo.adjacent = a.c.head_stride < a.c.slot_stride;
  const int unit = T_::kTok * kWarps;  // tokens of a unit of one head
  const int64_t segments = a.B * a.c.heads * geo.hgroups;
  geo.ctas = std::min<int64_t>(std::min(kMaxCtas, T_::kCtas * num_sms), segments * ceil_div(geo.cap, unit));
  geo.by_segment = segments <= geo.ctas;
  geo.listed = geo.by_segment ? segments : geo.ctas * T_::kSub;
  Space sp;
  sp.o = static_cast<float*>(a.workspace);
  sp.ml = reinterpret_cast<float2*>(sp.o + 2 * kMaxCtas * T_::kSub * T_::kHeads * D);
  sp.joins = reinterpret_cast<int4*>(sp.ml + 2 * kMaxCtas * T_::kSub * T_::kHeads);
  const int es = type_bytes(TYPE);
  geo.page32 = static_cast<uint32_t>(a.c.page_stride * es / 32);
  geo.slot32 = static_cast<uint32_t>(a.c.slot_stride * es / 32);
  geo.head32 = static_cast<uint32_t>(a.c.head_stride * es / 32);
  // ceil(2^(31 + s) / page_size) with the least s of 2^s >= page_size is below 2^32 and exact
  geo.page_shift = 31;
  while ((int64_t(1) << (geo.page_shift - 31)) < a.c.page_size) ++geo.page_shift;
  geo.page_mul = static_cast<uint32_t>(((uint64_t(1) << geo.page_shift) + a.c.page_size - 1) / a.c.page_size);
  const bool whole = a.c.page_size % 16 == 0;
  auto kernel = whole ? paged_attn_kernel<D, TYPE, NB, true> : paged_attn_kernel<D, TYPE, NB, false>;
  cudaError_t e = launch_early(kernel, dim3(static_cast<unsigned>(geo.ctas)), kThreads, 0, s, launches, a, geo, sp);
  if (e != cudaSuccess) return e;
  if (geo.cap <= kWhole * unit) return cudaSuccess;  // no segment crosses runs
  // few segments have many pieces each: eight teams share a head's pieces out
  const int64_t heads = geo.listed * T_::kHeads;
  const int teams = heads <= kMaxCtas ? std::min(8, kJoinThreads / (D / 4)) : 1;
  const dim3 grid(static_cast<unsigned>(ceil_div(heads * teams, kJoinThreads / (D / 4))));
  return launch_early(paged_attn_join_kernel<D, T_::kHeads, T_::kSub>, grid, kJoinThreads, 0, s, launches, a, geo, sp, teams);
}

template <int D>
cudaError_t launch_d(const PagedAttnArgs& a, int num_sms, cudaStream_t s, int* launches) {
  if constexpr (D <= 128) {
    if (head_blocks(a.Hq, a.c.heads, D) == 2) switch (a.c.type) {
        case kTypeBf16: return launch<D, kTypeBf16, 2>(a, num_sms, s, launches);
        case kTypeF16: return launch<D, kTypeF16, 2>(a, num_sms, s, launches);
        default: return launch<D, kTypeE4m3, 2>(a, num_sms, s, launches);
      }
  }
  switch (a.c.type) {
    case kTypeBf16: return launch<D, kTypeBf16, 1>(a, num_sms, s, launches);
    case kTypeF16: return launch<D, kTypeF16, 1>(a, num_sms, s, launches);
    default: return launch<D, kTypeE4m3, 1>(a, num_sms, s, launches);
  }
}

}  // namespace

int64_t paged_attn_workspace(int Hq, int Hkv, int D, int type) {
  const int64_t places = kMaxCtas * (D * type_bytes(type) <= 128 ? kWarps : 1), heads = head_blocks(Hq, Hkv, D) * 8;
  return places * (2 * heads * (D * 4 + 8) + 16);  // Space: partial sums, their (m, l), joins
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int num_sms, cudaStream_t s, int* launches) {
  switch (a.c.head_dim) {
    case 64: return launch_d<64>(a, num_sms, s, launches);
    case 128: return launch_d<128>(a, num_sms, s, launches);
    default: return launch_d<256>(a, num_sms, s, launches);
  }
}

}  // namespace awq
