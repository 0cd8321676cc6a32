// k_paged_attn.cu — attention of one new token per sequence over a paged key-value cache.
//
//   o_h = (sum_t p_t v_t) / (sum_t p_t),  p_t = 2^(s_t - m),  s_t = scale log2(e) q_h . k_t
//
// over the sequence's first `length` cached tokens, with the running maximum m of the scores
// met so far (the sums are rescaled when it grows), so the cache is read once. Every group
// of Hq / Hkv query heads shares its key-value head's bytes: they are read once for the group.
//
// What bounds it: the cache's bytes (2 D bytes of keys and as much of values per token and
// key-value head, against 4 D multiply-adds per query head), so the kernel is a stream.
//
// Work. The unit is 64 tokens of one (sequence, key-value head): all units of the batch,
// sequence-major, are dealt to a grid of as many CTAs as fit the SMs, in equal contiguous
// runs, whatever the lengths are. A CTA finds its run from the lengths on the device. A
// (sequence, head) that lies within one run is finished there; one that crosses runs leaves
// a partial (o, m, l) per run, and a second kernel adds them in run order (fixed order:
// equal inputs give equal bits).
//
// Tile. A warp takes 16 tokens (more where rows are short: 8 KB of cache) of a unit with its
// own running maximum; the four warps meet once per (sequence, head). Tokens are the rows of
// both products, so a group of up to 8 heads fills the 8 columns of an m16n8k16 MMA and none
// of the 16 rows is padding:
//   S^T (16 tokens x 8 heads) = K Q^T,   O^T (16 dims x 8 heads) += V^T P^T.
// The sum over dims in q . k may run in any order and the rows of O^T may be any dims, so
// each lane is given dims that lie together in memory: 16-byte pieces of the cache rows are
// its MMA fragments as they are (keys) or after a byte shuffle of two tokens' words (values).
// The cache therefore goes from memory to the fragments' registers without shared memory: a
// warp loads the keys of its next tile when it has used these keys, the next values when it
// has used these values, and the twelve warps of an SM keep some 90 KB on the way.
#include "decode_kernels.h"

#include <algorithm>
#include <cmath>

namespace awq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <int D, int TYPE, int NB>
struct Tile {
  static constexpr int ES = type_bytes(TYPE);
  static constexpr int kKChunks = D * ES / 64;                       // 16-byte pieces per key row and lane
  static constexpr int kVBytes = D * ES / 8 < 16 ? D * ES / 8 : 16;  // bytes of a piece of a value row
  static constexpr int kVChunks = D * ES / 8 / kVBytes;              // pieces per value row and lane
  static constexpr int kSteps = D / 16;                              // k16 steps of q . k; also tiles of 16 dims of O^T
  static constexpr int kBlocks = 256 / (D * ES) > 1 ? 256 / (D * ES) : 1;  // blocks of 16 tokens of a warp's tile
  static constexpr int kUnit = kWarps * 16 * kBlocks;                // tokens of a unit
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
    if constexpr (BYTES == 16)
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
    else
      asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) w[i] = 0u;
  }
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A sequence's tokens as the kernel takes them: never more than its table row can name.
__device__ __forceinline__ int clamped_length(const int32_t* lengths, int64_t b, int cap) {
  return min(max(__ldg(lengths + b), 0), cap);
}

// The run of CTA c when T units are dealt to C CTAs, and the CTA whose run holds unit l.
__host__ __device__ __forceinline__ int64_t run_start(int64_t c, int64_t T, int64_t C) { return c * T / C; }
__device__ __forceinline__ int64_t unit_owner(int64_t l, int64_t T, int64_t C) { return ((l + 1) * C - 1) / T; }

constexpr uint32_t kNoRow = 0xFFFFFFFFu;        // a row without a place (a place of the last 16 bytes below 64 GB)
constexpr float kNoMax = -3.402823466e38f;  // the maximum before any score: finite, so that m - m is 0

// A place in the sequence-major list of units: sequence, (key-value head, head block), unit.
struct Cursor {
  int b, kvh, hg, blk, len;
};

struct Space {       // the work space of a launch
  float* o;          // [2 C][heads][D] partial sums of run c: slot 2 c of the segment that begins in it and
                     // goes on, slot 2 c + 1 of the one that began before it
  float2* ml;        // [2 C][heads] (m, l)
  int64_t* prefix;   // [B + 1] units per (key-value head, head block) before each sequence
};

struct Geometry {
  int cap;           // tokens a table row can name
  int heads_per;     // Hq / Hkv
  int hgroups;       // head blocks per key-value head
  int64_t ctas;
  uint32_t page16, slot16, head16;  // the cache's strides in units of 16 bytes
  uint32_t page_mul;  // p / page_size = (p * page_mul) >> page_shift for 0 <= p < 2^31
  int page_shift;
  int block_pages;    // every block of 16 tokens lies in one page
};

template <int D, int TYPE, int NB>
__global__ void __launch_bounds__(kThreads, Tile<D, TYPE, NB>::kCtas)
    paged_attn_kernel(PagedAttnArgs a, Geometry geo, Space sp) {
  using T_ = Tile<D, TYPE, NB>;
  constexpr int ES = T_::ES, KC = T_::kKChunks, VB = T_::kVBytes, VC = T_::kVChunks, S = T_::kSteps, TB = T_::kBlocks;
  constexpr int kUnit = T_::kUnit, kTok = 16 * TB;
  constexpr int MMA = TYPE == kTypeBf16 ? kTypeBf16 : kTypeF16;
  // The maximum in use may lag behind the scores by 2^kLag before the sums are rescaled: weights
  // are p 2^kBias, 2^(kBias + kLag) at most, and in fp16 stay representable down to p = 2^-31 of
  // the maximum in use. Both factors cancel in o / l.
  constexpr float kLag = 8.0f, kBias = MMA == kTypeF16 ? 7.0f : 0.0f;
  __shared__ __align__(16) float join_buf[kWarps * 8 * T_::kPitch];
  __shared__ float sM[kWarps][T_::kHeads], sL[kWarps][T_::kHeads];
  __shared__ int sBad[kWarps];
  __shared__ int64_t sScan[kWarps + 1];
  __shared__ Cursor sStart;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t = lane & 3;
  const PagedCache& c = a.c;
  const int HH = c.heads * geo.hgroups;

  // ---- the run: exclusive sums of the sequences' units, then the sequence of its first unit
  const int64_t per = ceil_div(a.B, kThreads), b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t mine = 0;
  for (int64_t b = b0; b < b1; ++b) mine += (clamped_length(a.lengths, b, geo.cap) + kUnit - 1) / kUnit;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) sScan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sScan[w];
    total += sScan[w];
  }
  if (blockIdx.x == 0) {
    int64_t at = before;
    for (int64_t b = b0; b < b1; ++b) {
      sp.prefix[b] = at;
      at += (clamped_length(a.lengths, b, geo.cap) + kUnit - 1) / kUnit;
    }
    if (tid == 0) sp.prefix[a.B] = total;
  }
  // no run is empty: with fewer units than CTAs the later CTAs have none
  const int64_t units = total * HH, C = min(geo.ctas, units);
  const int64_t u0 = blockIdx.x < C ? run_start(blockIdx.x, units, C) : 0;
  const int n = blockIdx.x < C ? static_cast<int>(run_start(blockIdx.x + 1, units, C) - u0) : 0;
  if (n > 0 && before * HH <= u0 && u0 < (before + mine) * HH) {
    int64_t at = before * HH;
    for (int64_t b = b0; b < b1; ++b) {
      const int len = clamped_length(a.lengths, b, geo.cap), nblk = (len + kUnit - 1) / kUnit;
      if (u0 < at + static_cast<int64_t>(nblk) * HH) {
        const int64_t rel = u0 - at;
        const int hh = static_cast<int>(rel / nblk);
        sStart = {static_cast<int>(b), hh / geo.hgroups, hh % geo.hgroups, static_cast<int>(rel % nblk), len};
        break;
      }
      at += static_cast<int64_t>(nblk) * HH;
    }
  }
  // sequences without tokens have no units: their rows of zeros are dealt out too
  for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x)
    if (__ldg(a.lengths + b) <= 0)
      for (int64_t i = tid; i < static_cast<int64_t>(a.Hq) * D / 2; i += kThreads)
        static_cast<uint32_t*>(a.out)[b * a.Hq * D / 2 + i] = 0u;
  __syncthreads();
  if (n == 0) return;

  auto advance = [&](Cursor& k) {
    if (++k.blk * kUnit < k.len) return;
    k.blk = 0;
    if (++k.hg < geo.hgroups) return;
    k.hg = 0;
    if (++k.kvh < c.heads) return;
    k.kvh = 0;
    do {
      ++k.b;
      k.len = k.b < a.B ? clamped_length(a.lengths, k.b, geo.cap) : 1;
    } while (k.len == 0);
  };

  // ---- the loading side. look_up() asks the block table for a tile's pages one tile before
  // place() turns them into places of the cache, in units of 16 bytes: per block of 16 tokens
  // that of its first row where blocks lie in one page, of row lane % 16 otherwise.
  Cursor ic = sStart;
  int looked = 0;
  int32_t page[TB];        // asked for
  uint32_t row[TB];        // placed
  int ask_rows = 0, rows = 0;  // rows left of the sequence from the tile's first on
  int ask_tok = 0;
  uint32_t ask_head = 0;
  bool full = false;       // every block of the placed tile has its 16 rows, in one page
  bool bad_tile = false;   // the placed tile needs a page outside the cache
  auto page_of = [&](int tok) { return static_cast<int>(static_cast<uint64_t>(tok) * geo.page_mul >> geo.page_shift); };
  auto look_up = [&]() {
    if (looked >= n) {
      ask_rows = 0;
    } else {
      if (looked > 0) advance(ic);
      ask_rows = ic.len - (ic.blk * kUnit + warp * kTok);
    }
    ++looked;
    ask_tok = ic.blk * kUnit + warp * kTok + (geo.block_pages ? 0 : lane & 15);
    ask_head = ic.kvh * geo.head16;
    const int32_t* table = c.table + ic.b * c.table_stride;
#pragma unroll
    for (int k = 0; k < TB; ++k) {
      page[k] = -1;
      if (16 * k + (geo.block_pages ? 0 : lane & 15) < ask_rows) page[k] = __ldg(table + page_of(ask_tok + 16 * k));
    }
  };
  auto place = [&]() {
    rows = ask_rows;
    full = geo.block_pages && rows >= kTok;
    bad_tile = false;
#pragma unroll
    for (int k = 0; k < TB; ++k) {
      const int tok = ask_tok + 16 * k;
      const bool inside = static_cast<uint32_t>(page[k]) < static_cast<uint32_t>(c.num_pages);
      row[k] = inside ? static_cast<uint32_t>(page[k]) * geo.page16 +
                            static_cast<uint32_t>(tok - page_of(tok) * c.page_size) * geo.slot16 + ask_head
                      : kNoRow;
      full = full && inside;
      bad_tile = bad_tile || (!inside && 16 * k + (geo.block_pages ? 0 : lane & 15) < rows);
    }
  };
  Piece<16> kr[TB][2][KC];
  Piece<VB> vr[TB][4][VC];
  // Loads the lane's rows of a tile: its row r of a block is token at(r), its bytes from `from` on.
  auto load_tile = [&](const uint8_t* from, auto at, auto& piece) {
    constexpr int ROWS = sizeof(piece[0]) / sizeof(piece[0][0]);
    constexpr int PIECES = sizeof(piece[0][0]) / sizeof(piece[0][0][0]);
    constexpr int STEP = ROWS == 2 ? 64 : 8 * static_cast<int>(sizeof(piece[0][0][0]));
    if (full) {
#pragma unroll
      for (int k = 0; k < TB; ++k)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const uint8_t* src = from + static_cast<uint64_t>(row[k] + at(r) * geo.slot16) * 16u;
#pragma unroll
          for (int j = 0; j < PIECES; ++j) piece[k][r][j].load(src + STEP * j);
        }
      return;
    }
#pragma unroll
    for (int k = 0; k < TB; ++k)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        uint32_t off = __shfl_sync(~0u, row[k], at(r));
        if (geo.block_pages)
          off = row[k] != kNoRow && 16 * k + static_cast<int>(at(r)) < rows ? row[k] + at(r) * geo.slot16 : kNoRow;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
          piece[k][r][j].zero();
          if (off != kNoRow) piece[k][r][j].load(from + static_cast<uint64_t>(off) * 16u + STEP * j);
        }
      }
  };
  const uint8_t* k_from = static_cast<const uint8_t*>(c.k) + 16 * t;
  const uint8_t* v_from = static_cast<const uint8_t*>(c.v) + VB * g;
  auto load_keys = [&]() { load_tile(k_from, [&](uint32_t r) { return g + 8 * r; }, kr); };
  auto load_values = [&]() { load_tile(v_from, [&](uint32_t r) { return 2 * t + (r & 1) + 8 * (r >> 1); }, vr); };
  look_up();
  place();
  load_keys();
  load_values();
  bool bad_now = bad_tile;
  look_up();

  // ---- the computing side
  Cursor cc = sStart;
  uint32_t qf[NB][S][2];          // Q^T fragments: heads g of each block, this lane's dims
  float acc[NB][S][4];            // O^T: per 16-dim tile, (dim, dim + 1) x (heads 2t, 2t + 1)
  float ls[NB][2];                // l of heads 2t, 2t + 1
  float m[NB][2], sc[NB][2];      // the maximum in use, lowered by kBias; the factor of the products, base 2
  bool bad = false, fresh = true;
  for (int i = 0; i < n; ++i) {
    if (fresh) {  // a segment of the run begins
      fresh = false;
      bad = __ldg(a.lengths + cc.b) > geo.cap;
      const int kvh = cc.kvh, hb = cc.hg * T_::kHeads;
      const float k_scale = TYPE == kTypeE4m3 ? __ldg(c.k_scale + kvh) : 1.0f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int h = hb + nb * 8 + g;
        const bool live = h < geo.heads_per;
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;  // the factor of the scores is not negative
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + cc.b * a.q_sb +
                            static_cast<int64_t>(kvh * geo.heads_per + (live ? h : 0)) * a.q_sh;
#pragma unroll
        for (int st = 0; st < S; ++st) {
          // dims of step st: 4 elements of the lane's piece st / PER
          constexpr int PER = 4 / ES;  // steps a 16-byte piece serves: 2 (16 bits) or 4 (8 bits)
          const int d = (st / PER) * (64 / ES) + (16 / ES) * t + 4 * (st % PER);
          const uint2 w = live ? __ldg(reinterpret_cast<const uint2*>(q + d)) : make_uint2(0u, 0u);
          qf[nb][st][0] = w.x ^ flip;
          qf[nb][st][1] = w.y ^ flip;
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
    }
    bad = bad || bad_now;
    const int tok0 = cc.blk * kUnit + warp * kTok;
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
          const uint32_t(&wl)[4] = kr[k][0][j].w;  // row g
          const uint32_t(&wh)[4] = kr[k][1][j].w;  // row g + 8
          if constexpr (ES == 2) {
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma_16816<MMA>(s2[st % CHAINS][k][nb], wl[2 * st], wh[2 * st], wl[2 * st + 1], wh[2 * st + 1], qf[nb][2 * j + st][0],
                               qf[nb][2 * j + st][1]);
          } else {
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              uint32_t a0, a1, a2, a3;
              e4m3_pairs(wl[st], a0, a2);
              e4m3_pairs(wh[st], a1, a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma_16816<MMA>(s2[st % CHAINS][k][nb], a0, a1, a2, a3, qf[nb][4 * j + st][0], qf[nb][4 * j + st][1]);
            }
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[k][nb][x] = CHAINS == 2 ? s2[0][k][nb][x] + s2[CHAINS - 1][k][nb][x] : s2[0][k][nb][x];
      }
    }
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
      // the weights enter the product in 16 bits; l sums those same rounded weights, so that
      // they still add up to one
#pragma unroll
      for (int k = 0; k < TB; ++k) {
        uint32_t pf[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t w = pack16(exp2_approx(s[k][nb][2 * r] * sc[nb][0] - m[nb][0]),
                                exp2_approx(s[k][nb][2 * r + 1] * sc[nb][1] - m[nb][1]), MMA);
            if (ragged && tok0 + 16 * k + g + 8 * r >= cc.len) w = 0u;
            pf[nb][r] = transposed(w);
          }
          constexpr uint32_t kOnes = MMA == kTypeBf16 ? 0x3F803F80u : 0x3C003C00u;
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // a row of ones times P^T
          mma_16816<MMA>(sum, kOnes, kOnes, kOnes, kOnes, pf[nb][0], pf[nb][1]);
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
              for (int nb = 0; nb < NB; ++nb)
                mma_16816<MMA>(acc[nb][j * (VB / 4) + w], a0, a1, a2, a3, pf[nb][0], pf[nb][1]);
            } else {  // word w: dims 4w .. 4w + 3
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t a0, a1, a2, a3;
                e4m3_pairs(__byte_perm(w0, w1, e ? 0x7362 : 0x5140), a0, a1);
                e4m3_pairs(__byte_perm(w2, w3, e ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma_16816<MMA>(acc[nb][(j * (VB / 4) + w) * 2 + e], a0, a1, a2, a3, pf[nb][0], pf[nb][1]);
              }
            }
          }
        }
      }
    }
    load_values();
    bad_now = bad_tile;
    look_up();

    const bool ends = (cc.blk + 1) * kUnit >= cc.len, last = i + 1 == n;
    if (ends || last) {
      // ---- the four warps meet: factors to the common maximum, then one sum per head and dim
      if (last) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
      const int kvh = cc.kvh, hb = cc.hg * T_::kHeads;
      const int live = min(T_::kHeads, geo.heads_per - hb);
      const float v_scale = TYPE == kTypeE4m3 ? __ldg(c.v_scale + kvh) : 1.0f;
      if (any_bad && tid == 0 && a.status) *a.status = 1;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (nb) __syncthreads();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int h = nb * 8 + 2 * t + x;
          if (h < live) {
            const float top = fmaxf(fmaxf(sM[0][h], sM[1][h]), fmaxf(sM[2][h], sM[3][h]));
            const float f = exp2f(m[nb][x] - top);
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
        for (int e = tid; e < min(8, live - nb * 8) * (D / 4); e += kThreads) {
          const int h8 = e / (D / 4), d = (e % (D / 4)) * 4, h = nb * 8 + h8;
          const float top = fmaxf(fmaxf(sM[0][h], sM[1][h]), fmaxf(sM[2][h], sM[3][h]));
          float L = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            L += sL[w][h] * exp2f(sM[w][h] - top);
            const float2 x0 = *reinterpret_cast<const float2*>(join_buf + (w * 8 + h8) * T_::kPitch + d);
            const float2 x1 = *reinterpret_cast<const float2*>(join_buf + (w * 8 + h8) * T_::kPitch + d + 2);
            o[0] += x0.x;
            o[1] += x0.y;
            o[2] += x1.x;
            o[3] += x1.y;
          }
          if (any_bad) L = NAN;
          if (whole) {
            const float r = v_scale / L;
            const int64_t to = (static_cast<int64_t>(cc.b) * a.Hq + kvh * geo.heads_per + hb + h) * D + d;
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) =
                make_uint2(pack16(o[0] * r, o[1] * r, a.q_type), pack16(o[2] * r, o[3] * r, a.q_type));
          } else {
            *reinterpret_cast<float4*>(sp.o + (part * T_::kHeads + h) * D + d) = make_float4(o[0], o[1], o[2], o[3]);
            if (d == 0) sp.ml[part * T_::kHeads + h] = make_float2(top, L);
          }
        }
      }
      __syncthreads();
      fresh = true;
    }
    if (!last) advance(cc);
  }
}

// The segments that cross runs: o = (sum over the runs, in order, of o_c 2^(m_c - m)) / l.
// One CTA per (segment, head): kGroups groups of D / 4 threads take every kGroups-th run.
constexpr int kJoinThreads = 256;
template <int D, int HEADS>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_join_kernel(PagedAttnArgs a, Geometry geo, Space sp) {
  constexpr int kGroups = kJoinThreads / (D / 4);
  __shared__ float4 sO[kGroups][D / 4];
  __shared__ float sW[kJoinThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int HH = a.c.heads * geo.hgroups;
  const int64_t b = blockIdx.x / HH;
  const int hh = static_cast<int>(blockIdx.x % HH), h = blockIdx.y;
  const int kvh = hh / geo.hgroups, hb = (hh % geo.hgroups) * HEADS;
  if (hb + h >= geo.heads_per) return;
  const int64_t before = sp.prefix[b], nblk = sp.prefix[b + 1] - before, units = sp.prefix[a.B] * HH;
  const int64_t C = min(geo.ctas, units);
  if (nblk == 0) return;
  const int64_t s0 = before * HH + hh * nblk, s1 = s0 + nblk;
  const int64_t c0 = unit_owner(s0, units, C), c1 = unit_owner(s1 - 1, units, C);
  if (c0 == c1) return;  // finished by its run
  const int pieces = static_cast<int>(c1 - c0 + 1);
  const int tid = threadIdx.x;
  auto at = [&](int p) {  // the segment begins in run c0 and goes on in the later ones
    return (2 * (c0 + p) + (p > 0 ? 1 : 0)) * HEADS + h;
  };
  float top = kNoMax;
  for (int p = tid; p < pieces; p += kJoinThreads) top = fmaxf(top, sp.ml[at(p)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (tid % 32 == 0) sW[tid / 32] = top;
  __syncthreads();
  for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, sW[w]);
  const int grp = tid / (D / 4), d4 = tid % (D / 4);
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float L = 0.0f;
#pragma unroll 4
  for (int p = grp; p < pieces; p += kGroups) {
    const float2 ml = sp.ml[at(p)];
    const float4 v = *reinterpret_cast<const float4*>(sp.o + static_cast<int64_t>(at(p)) * D + 4 * d4);
    const float f = exp2f(ml.x - top);
    L += ml.y * f;
    o.x += v.x * f;
    o.y += v.y * f;
    o.z += v.z * f;
    o.w += v.w * f;
  }
  sO[grp][d4] = o;
  __shared__ float sL[kGroups];
  if (d4 == 0) sL[grp] = L;
  __syncthreads();
  if (grp == 0) {
    for (int k = 1; k < kGroups; ++k) {
      const float4 v = sO[k][d4];
      o.x += v.x;
      o.y += v.y;
      o.z += v.z;
      o.w += v.w;
      L += sL[k];
    }
    const float r = (a.c.type == kTypeE4m3 ? __ldg(a.c.v_scale + kvh) : 1.0f) / L;
    const int64_t to = (b * a.Hq + kvh * geo.heads_per + hb + h) * D + 4 * d4;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) =
        make_uint2(pack16(o.x * r, o.y * r, a.q_type), pack16(o.z * r, o.w * r, a.q_type));
  }
}

constexpr int kMaxCtas = 3 * 148;  // three CTAs on each of a B200's SMs

int head_blocks(int Hq, int Hkv, int D) { return Hq / Hkv > 8 && D <= 128 ? 2 : 1; }

template <int D, int TYPE, int NB>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t s, int* launches) {
  using T_ = Tile<D, TYPE, NB>;
  Geometry geo;
  geo.cap = static_cast<int>(std::min<int64_t>(a.c.max_pages * a.c.page_size, INT32_MAX - 1024));
  geo.heads_per = a.Hq / a.c.heads;
  geo.hgroups = static_cast<int>(ceil_div(geo.heads_per, T_::kHeads));
  const int64_t segments = a.B * a.c.heads * geo.hgroups;
  geo.ctas = std::min<int64_t>(std::min(kMaxCtas, T_::kCtas * num_sms), segments * ceil_div(geo.cap, T_::kUnit));
  Space sp;
  sp.o = static_cast<float*>(a.workspace);
  sp.ml = reinterpret_cast<float2*>(sp.o + 2 * kMaxCtas * T_::kHeads * D);
  sp.prefix = reinterpret_cast<int64_t*>(sp.ml + 2 * kMaxCtas * T_::kHeads);
  geo.block_pages = a.c.page_size % 16 == 0;
  const int es = type_bytes(TYPE);
  geo.page16 = static_cast<uint32_t>(a.c.page_stride * es / 16);
  geo.slot16 = static_cast<uint32_t>(a.c.slot_stride * es / 16);
  geo.head16 = static_cast<uint32_t>(a.c.head_stride * es / 16);
  // ceil(2^(31 + s) / page_size) with the least s of 2^s >= page_size is below 2^32 and exact
  geo.page_shift = 31;
  while ((int64_t(1) << (geo.page_shift - 31)) < a.c.page_size) ++geo.page_shift;
  geo.page_mul = static_cast<uint32_t>(((uint64_t(1) << geo.page_shift) + a.c.page_size - 1) / a.c.page_size);
  paged_attn_kernel<D, TYPE, NB><<<static_cast<unsigned>(geo.ctas), kThreads, 0, s>>>(a, geo, sp);
  *launches += 1;
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (geo.cap <= T_::kUnit) return cudaSuccess;  // a segment is one unit: none crosses runs
  // The join may be set up while the runs still work; it waits for them before it reads.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(segments), static_cast<unsigned>(std::min(T_::kHeads, geo.heads_per)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<D, T_::kHeads>, a, geo, sp);
  *launches += 1;
  return e;
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

int64_t paged_attn_workspace(int64_t B, int Hq, int Hkv, int D) {
  const int64_t heads = head_blocks(Hq, Hkv, D) * 8;
  return 2 * kMaxCtas * heads * (D * 4 + 8) + (B + 1) * 8;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int num_sms, cudaStream_t s, int* launches) {
  switch (a.c.head_dim) {
    case 64: return launch_d<64>(a, num_sms, s, launches);
    case 128: return launch_d<128>(a, num_sms, s, launches);
    default: return launch_d<256>(a, num_sms, s, launches);
  }
}

}  // namespace awq
