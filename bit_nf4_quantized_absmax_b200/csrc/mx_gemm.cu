// Products of MX operands: Y[m, n] = sum_k x[m, k] w[n, k] with x in e4m3 or e2m1
// and w in e2m1, each with a power-of-two scale per 32 elements along k. The
// tensor cores apply the scales (tcgen05.mma kind::mxf8f6f4.block_scale), so no
// operand is decoded in software and the sums stay in fp32.
//
// The product is computed transposed: a tile is 128 weight rows (the MMA's M, one
// TMEM lane each) by TN tokens (its N, one TMEM column each), so the same kernel
// serves one token, where the weights' bytes are all that counts, and hundreds.
//
// Operand stages hold 128 elements of k. e4m3 rows are copied as they are; e2m1
// rows are widened by TMA to the 8-bit containers that this MMA kind reads (16
// codes become 8 bytes of codes and 8 of padding; a copy counts the codes' bytes),
// so both take 128 bytes a row and one swizzle. Scale words (4 bytes: the row's 4
// blocks of the stage) are read ahead into registers and stored where tcgen05.cp
// wants them: row r of 128 at byte (r % 32) * 16 + (r / 32) * 4. The MMA of block j
// reads byte j of each word.
//
// Two kernels: k_mx_gemm, one tile a CTA or a cluster, for few tokens and for as many
// tiles as there are SMs; k_mx_gemm_pair, persistent CTA pairs (for groups of up to 128
// rows: single CTAs), beyond. Measured on
// the device (x already MX, weights in rotation over three sets):
//   one token       4096x4096  5.9 us   11008x4096  7.3 us (24 MB: 3.3 TB/s)
//   512 tokens      4096x4096 11.8 us   11008x4096 25.9 us
//   4096 tokens     4096x4096 55 us (2500 TFLOP/s)   11008x4096 138 us (2680)
// The first line is latency (launch, first copies, a reduction over the cluster), the
// last the MMAs at the clock that 1000 W allow (1300 to 1400 MHz of 1965).
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace qlora {
namespace {

constexpr int kMxBK = 128;     // elements of k a stage
constexpr int kMxRows = 128;   // weight rows a tile
constexpr int kMxThreads = 128;  // and four warps more where the kernel quantizes x

// Scale words are handled four k-blocks at a time, in a ring of two such blocks: a
// warp's stores, fence and arrival take some 300 clocks, as long as a k-block's
// copies and MMAs, so once per k-block they bounded the small products.
constexpr int kSfDepth = 4;           // k-blocks a block of scales
constexpr int kSfSlots = 2;
constexpr int kSfOne = 1024;          // bytes a k-block: words of 128 weight rows, of 128 tokens

template <int TN, bool DEEP>
struct MxCfg {
  static constexpr int W_BYTES = kMxRows * kMxBK;
  static constexpr int X_BYTES = TN * kMxBK;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int SF_BYTES = kSfSlots * kSfDepth * kSfOne;
  // The ring's round trip (a k-block's MMAs done, slot free, copy issued, data there) takes 1500 to 2000 clocks. With
  // two CTAs on an SM one streams while the other waits; DEEP is for grids that leave a CTA alone on its SM.
  static constexpr int ROOM = (DEEP ? 220 : 110) * 1024 - 1536 - SF_BYTES;
  static constexpr int STAGES = ROOM / STAGE_BYTES < kSfSlots * kSfDepth ? ROOM / STAGE_BYTES : kSfSlots * kSfDepth;
  static constexpr int SF_COL = TN < 32 ? 32 : TN;  // first TMEM column of the scales, 8 a k-block
  static constexpr int TMEM_NEED = SF_COL + 8 * kSfSlots * kSfDepth;
  static constexpr int TMEM_COLS = TMEM_NEED <= 128 ? 128 : 256;
  static constexpr int SMEM = STAGES * STAGE_BYTES + SF_BYTES + 1024 /*align*/ + 256 /*barriers*/;
  static_assert(STAGES * STAGE_BYTES >= TN * kMxRows * 4, "the partial tile reuses the stages");
  static_assert(STAGES <= kSfSlots * kSfDepth, "a free stage has to mean free scales");
};

// Instruction descriptor of kind::mxf8f6f4.block_scale (fp32 accumulator, ue8m0
// scales, both operands K-major): A format at bit 7, B format at bit 10 (0 e4m3,
// 5 e2m1), N / 8 at bit 17, ue8m0 at bit 23, M / 16 at bit 24; the scale byte of
// B at bits 4-5 and of A at bits 29-30 are added per MMA.
constexpr uint32_t kFmtE4M3 = 0, kFmtE2M1 = 5;
inline uint32_t mx_instr_desc(uint32_t a_fmt, uint32_t b_fmt, int M, int N) {
  return (a_fmt << 7) | (b_fmt << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_mx(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc));
}

// 512 bytes of scale words (32 rows of 16 bytes) to 4 TMEM columns, repeated in
// the four groups of 32 lanes.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc));
}

// Shared-memory descriptor without swizzle: 8-row groups of 16-byte rows, 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One lane of a converged warp (always the same one). Code that it guards may use
// uniform registers, which the operands of tcgen05 instructions have to be in: with
// `if (lane == 0)` around the MMA loop each MMA took 70 clocks to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// The scale words of GROUPS x 128 rows from r0 on, for the k-blocks of a tile, kept
// AHEAD stages ahead in a warp's registers: lane l holds rows l, l + 32, l + 64 and
// l + 96 of each 128, the 16 bytes that tcgen05.cp wants together. Rows past `count` or
// at or past `rows` read as 0. (cp.async instead of registers: the proxy fence after it
// waited for all that were in flight, 20% of a large product.)
template <int GROUPS, int AHEAD>
struct ScaleWords {
  uint32_t w[AHEAD][GROUPS * 4];
  const uint32_t* src;
  int64_t rows;
  uint32_t in;  // bit q: row l + 32 q exists
  __device__ __forceinline__ void start(const uint8_t* scales, int64_t rows_, int64_t r0, int count, int kb0, int kb1) {
    const int lane = threadIdx.x & 31;
    rows = rows_;
    src = reinterpret_cast<const uint32_t*>(scales) + r0 + lane;
    in = 0;
#pragma unroll
    for (int q = 0; q < GROUPS * 4; ++q)
      if (q * 32 + lane < count && r0 + q * 32 + lane < rows) in |= 1u << q;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(i, kb0 + i, kb1);
  }
  __device__ __forceinline__ void load(int i, int kb, int kb1) {
    const uint32_t* line = src + static_cast<int64_t>(kb) * rows;
#pragma unroll
    for (int q = 0; q < GROUPS * 4; ++q) w[i][q] = (kb < kb1 && (in >> q & 1u)) ? __ldg(line + q * 32) : 0u;
  }
  __device__ __forceinline__ void store(int i, uint8_t* dst) const {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
      *reinterpret_cast<uint4*>(dst + g * 512 + (threadIdx.x & 31) * 16) =
          make_uint4(w[i][4 * g], w[i][4 * g + 1], w[i][4 * g + 2], w[i][4 * g + 3]);
  }
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// 16 TMEM lanes by 64 columns of fp32 to 4 x four 8 x 8 bf16 matrix fragments, per 16
// columns {lanes 0-7, columns 0-7}, {8-15, 0-7}, {0-7, 8-15}, {8-15, 8-15}. One load
// for all: with a wait after every 16 columns a tile's accumulator was held for 1900
// clocks instead of some 500.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&o)[4][4]) {
  float v[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[c][i] = pack_bf16x2(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
}

// Where 8 weight rows (n8 of 4) of token `tok` of 16 stand in a warp's 1 KB: 64-byte
// rows whose 16-byte pieces are permuted so that 8 consecutive tokens of one piece
// fall into different banks.
__device__ __forceinline__ uint32_t staged_at(int tok, int n8) {
  return static_cast<uint32_t>(tok * 64 + ((n8 ^ ((tok >> 1) & 3)) << 4));
}

// 32 weight rows (lo: 0-15, hi: 16-31) by 16 tokens, transposed on the way into
// shared memory: a token's weight rows, which are adjacent in Y, become adjacent.
__device__ __forceinline__ void stage_transposed(uint8_t* stg, const uint32_t (&lo)[4], const uint32_t (&hi)[4]) {
  const int lane = threadIdx.x & 31;
  const int m = lane >> 3, r = lane & 7;  // this lane gives the address of row (token) r of matrix m
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t at = smem_u32(stg) + staged_at((m >> 1) * 8 + r, h * 2 + (m & 1));
    const uint32_t(&o)[4] = h ? hi : lo;
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[0]),
                 "r"(o[1]), "r"(o[2]), "r"(o[3])
                 : "memory");
  }
}

// `tokens` of 16 staged tokens to Y (dst: the first token's first weight row, ld
// elements a token), `rows` of 32 weight rows each.
__device__ __forceinline__ void store_tokens(const uint8_t* stg, __nv_bfloat16* dst, int64_t ld, int tokens, int rows) {
  const int lane = threadIdx.x & 31;
  if (rows == 32 && ld % 8 == 0) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int tok = p * 8 + (lane >> 2), n8 = lane & 3;
      if (tok < tokens)
        *reinterpret_cast<uint4*>(dst + tok * ld + n8 * 8) = *reinterpret_cast<const uint4*>(stg + staged_at(tok, n8));
    }
  } else if (rows == 32 && ld % 4 == 0) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int tok = p * 4 + (lane >> 3), n4 = lane & 7;
      if (tok < tokens)
        *reinterpret_cast<uint2*>(dst + tok * ld + n4 * 4) =
            *reinterpret_cast<const uint2*>(stg + staged_at(tok, n4 >> 1) + (n4 & 1) * 8);
    }
  } else if (lane < rows) {
#pragma unroll
    for (int tok = 0; tok < 16; ++tok)
      if (tok < tokens)
        dst[tok * ld + lane] = *reinterpret_cast<const __nv_bfloat16*>(stg + staged_at(tok, lane >> 3) + (lane & 7) * 2);
  }
}

// Token tiles of the grouped rows, found by a whole warp. A group of m rows has
// ceil(m / tn) tiles of equal size, rounded up to a multiple of `unit`. Offsets are read
// as they are but clamped to [0, M] and to their running maximum, so that no offsets lead
// outside of x and Y. Tiles are asked for in ascending order: 32 groups at a time are
// scanned and kept in the lanes, so that a warp that goes from tile to tile reads and
// scans each group once (anew for every tile it took 2000 clocks with 64 groups, a fifth
// of a tile of 16 k-blocks).
struct TokenTile {
  int group;
  int64_t row0, end;
  bool found;
};
struct GroupScan {
  const int32_t* offsets;
  int groups, M, tn, unit;
  int e0 = -32;           // first group of the lanes' 32
  int base = 0, next = 0;  // tiles before them, and before the next 32
  int carry = 0;          // running maximum of the offsets so far
  // the lane's group: first row, row behind its last, tiles, rows of a tile; tiles up to and with it
  int b = 0, t = 0, tiles = 0, step = 0, upto = 0;
  __device__ __forceinline__ GroupScan(const int32_t* offsets_, int groups_, int64_t M_, int tn_, int unit_)
      : offsets(offsets_), groups(groups_), M(static_cast<int>(M_)), tn(tn_), unit(unit_) {}
  __device__ __forceinline__ void advance() {
    const int lane = threadIdx.x & 31;
    e0 += 32;
    base = next;
    const int e = e0 + lane;
    const bool in = e < groups;
    b = max(in ? offsets[e] : 0, carry);
    t = in ? offsets[e + 1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) b = max(b, v);
    }
    t = min(max(t, b), M);
    b = min(b, M);
    const int rows = in ? t - b : 0;
    tiles = rows / tn + (rows % tn != 0);
    step = tiles ? (rows / tiles + (rows % tiles != 0) + unit - 1) / unit * unit : 0;
    upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    upto += base;
    next = __shfl_sync(0xffffffffu, upto, 31);
    carry = __shfl_sync(0xffffffffu, t, 31);
  }
  __device__ __forceinline__ TokenTile find(int want) {
    while (want >= next && e0 + 32 < groups) advance();
    TokenTile r{0, 0, 0, false};
    if (want >= next) return r;
    const int src = __ffs(__ballot_sync(0xffffffffu, want < upto)) - 1;
    const int index = want - __shfl_sync(0xffffffffu, upto - tiles, src);
    const int size = __shfl_sync(0xffffffffu, step, src);
    r.group = e0 + src;
    r.row0 = static_cast<int64_t>(__shfl_sync(0xffffffffu, b, src)) + static_cast<int64_t>(index) * size;
    r.end = min(static_cast<int64_t>(__shfl_sync(0xffffffffu, t, src)), r.row0 + size);
    r.found = true;
    return r;
  }
};

struct MxArgs {
  const uint4* x_bf16;     // QUANT: activations still to be quantized, [M, K]
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  const int32_t* offsets;  // null: one group of all M rows
  int groups;
  int64_t M, N, w_rows;
  int n_tiles, nkb, K;
  int stages, stage_bytes;  // pairs: the operands' ring
  int tile_rows;            // pairs: weight rows a tile
  int tn, step, tok_tiles;  // pairs: most tokens a tile; without groups, tokens of all tiles but the last and their count
  uint32_t idesc;
  bool x_fp4;  // the widening copies of e2m1 count the bytes of codes, not of containers
  __nv_bfloat16* Y;
};

// The tokens' side of the stages, from bf16 (warps 4..7 of the QUANT kernel): warp q
// writes every fourth k-block, lane l the 64 elements (two MX blocks) of half l % 2 of
// token l / 2, one k-block of its own ahead in registers. The scale words go to the
// k-block's place in the scales' ring, which is free when the stage is (the ring of
// scales holds more k-blocks than the ring of stages).
template <int TN, bool DEEP, int FMT>
__device__ __forceinline__ void quantize_stages(const MxArgs& a, int64_t row0, int tokens, int kb0, int kb1,
                                                uint8_t* smem, uint8_t* sf, uint64_t* full, uint64_t* empty,
                                                volatile int* abort_flag, int32_t* err) {
  using C = MxCfg<TN, DEEP>;
  static_assert(TN == 16, "a lane holds half a token's k-block");
  // A warp that goes from k-block n - 4 to n has seen n - 4 - STAGES consumed; the parity of n's barrier tells n -
  // STAGES from n - 2 STAGES only if the latter is among those.
  static_assert(C::STAGES >= 4, "the parity of a stage's barrier would be ambiguous");
  const int lane = threadIdx.x & 31;
  const int row = lane >> 1, h = lane & 1;
  const bool mine = row < tokens;
  const uint4* src = a.x_bf16 + ((row0 + (mine ? row : 0)) * a.K + h * 64) / 8;
  uint4 q[8];
  auto load = [&](int kb) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = make_uint4(0u, 0u, 0u, 0u);
      if (mine && kb < kb1 && kb * kMxBK + h * 64 + (i >> 2) * 32 < a.K) q[i] = __ldg(src + kb * (kMxBK / 8) + i);
    }
  };
  const int first = kb0 + (threadIdx.x >> 5) - kMxThreads / 32;
  load(first);
  for (int kb = first; kb < kb1; kb += 4) {
    const int n = kb - kb0, stage = n % C::STAGES;
    const uint32_t phase = (n / C::STAGES) & 1;
    uint32_t o[2][8];
    uint32_t bytes = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[4 * i] = q[4 * b + i].x;
        v[4 * i + 1] = q[4 * b + i].y;
        v[4 * i + 2] = q[4 * b + i].z;
        v[4 * i + 3] = q[4 * b + i].w;
      }
      bytes |= mx_quantize_block<FMT>(v, o[b]) << (8 * b);
    }
    load(kb + 4);
    if (!__all_sync(0xffffffffu, wait_or_abort(&empty[stage], phase ^ 1u, abort_flag, err, DEV_TIMEOUT_SMEM_EMPTY)))
      return;
    if (mine) {
      uint8_t* line = smem + stage * C::STAGE_BYTES + C::W_BYTES + row * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // 16 elements: a 16-byte piece of the row, at its place in the 128-byte swizzle
        uint8_t* dst = line + (((h * 4 + c) ^ (row & 7)) << 4);
        const uint32_t(&p)[8] = o[c >> 1];
        if (FMT == kMxE4M3)
          *reinterpret_cast<uint4*>(dst) =
              make_uint4(p[4 * (c & 1)], p[4 * (c & 1) + 1], p[4 * (c & 1) + 2], p[4 * (c & 1) + 3]);
        else  // 8 bytes of codes, 8 unused
          *reinterpret_cast<uint2*>(dst) = make_uint2(p[2 * (c & 1)], p[2 * (c & 1) + 1]);
      }
      *reinterpret_cast<uint16_t*>(sf + (n % (kSfSlots * kSfDepth)) * kSfOne + 512 + row * 16 + h * 2) =
          static_cast<uint16_t>(bytes);
    }
    fence_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[stage]);
  }
}

// One tile a cluster of S CTAs, CTA r of the cluster taking k-blocks [r nkb / S,
// (r + 1) nkb / S). Warp 0 issues the TMA copies, warp 1 the MMAs, warps 2 and 3
// the scale words of the weights and the tokens; all four then drain the
// accumulator. With S > 1 each CTA leaves its fp32 partial in shared memory and
// adds up its share of the tokens over the cluster, in the order of the CTAs.
//
// QUANT (TN = 16): x is bf16, and four more warps write the tokens' side of the stages
// themselves, so that a decode step is one launch and its activations are never
// stored. A few tokens are quantized again by every CTA, which costs less (one token
// 0.8 us, 16 tokens 2 us) than a launch and a round trip through memory.
template <int TN, bool QUANT, bool DEEP>
__global__ void __launch_bounds__(QUANT ? kMxThreads + 128 : kMxThreads)
k_mx_gemm(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const MxArgs a,
          int32_t* err) {
  using C = MxCfg<TN, DEEP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf = smem + C::STAGES * C::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf + C::SF_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* sf_full = empty + C::STAGES;
  uint64_t* sf_empty = sf_full + kSfSlots;
  uint64_t* accf = sf_empty + kSfSlots;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(accf + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t S;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(S));
  const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], QUANT ? 2 : 1);  // the TMA warp, the warp that quantizes the stage
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sf_full[s], QUANT ? 1 : 2);  // the scale warps
      mbar_init(&sf_empty[s], 1);
    }
    mbar_init(accf, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_w);
    if (!QUANT) prefetch_tmap(&tm_x);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  pdl_enter();

  const int tile = blockIdx.x / S;
  const int tok = tile / a.n_tiles;
  const int64_t n0 = static_cast<int64_t>(tile - tok * a.n_tiles) * kMxRows;
  TokenTile tt{0, static_cast<int64_t>(tok) * TN, a.M, true};
  if (a.offsets) tt = GroupScan(a.offsets, a.groups, a.M, TN, TN).find(tok);
  const int64_t w0 = tt.group * a.N + n0;  // first weight row in w's storage
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.nkb) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(a.nkb) * (rank + 1) / S);

  if (tt.found) {  // the same in every thread of the cluster
    int issued = 0;  // copies, in the thread that issues them
    if (warp == 0) {
      const uint32_t bytes = C::W_BYTES / 2 + (QUANT ? 0 : a.x_fp4 ? C::X_BYTES / 2 : C::X_BYTES);
      const int32_t wrow = static_cast<int32_t>(w0), xrow = static_cast<int32_t>(tt.row0);
      if (elect_one()) {
        bool ok = true;
        for (int round = 0, kb = kb0; kb < kb1 && ok; ++round) {
#pragma unroll
          for (int st = 0; st < C::STAGES; ++st, ++kb) {
            if (kb < kb1 && ok) {
              if (round > 0)
                ok = wait_or_abort(&empty[st], (round - 1) & 1, abort_flag, err, DEV_TIMEOUT_SMEM_EMPTY);
              if (ok) {
                uint8_t* sw = smem + st * C::STAGE_BYTES;
                mbar_arrive_expect_tx(&full[st], bytes);
                tma_load_2d(sw, &tm_w, &full[st], kb * kMxBK, wrow);
                if (!QUANT) tma_load_2d(sw + C::W_BYTES, &tm_x, &full[st], kb * kMxBK, xrow);
                ++issued;
              }
            }
          }
        }
      }
    } else if (warp == 1) {
      const uint32_t s0 = smem_u32(smem);
      const uint64_t dw0 = smem_desc(s0, 16, 1024), dx0 = smem_desc(s0 + C::W_BYTES, 16, 1024);
      const uint64_t df0 = smem_desc_scales(smem_u32(sf));
      int stage = 0, slot = 0;
      uint32_t phase = 0, sf_phase = 0;
      bool ok = true;
      for (int base = kb0; base < kb1; base += kSfDepth) {
        ok = __all_sync(0xffffffffu, wait_or_abort(&sf_full[slot], sf_phase, abort_flag, err, DEV_TIMEOUT_TMA_FULL));
        if (!ok) break;
        int st[kSfDepth];
        uint32_t ph[kSfDepth];
#pragma unroll
        for (int i = 0; i < kSfDepth; ++i) {
          st[i] = stage;
          ph[i] = phase;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (elect_one()) {
          bool good = true;
#pragma unroll
          for (int i = 0; i < kSfDepth; ++i) {
            if (base + i < kb1 && good) {
              good = wait_or_abort(&full[st[i]], ph[i], abort_flag, err, DEV_TIMEOUT_TMA_FULL);
              if (good) {
                tc_fence_after();
                const uint64_t at = static_cast<uint32_t>(st[i] * C::STAGE_BYTES) >> 4;  // 16-byte units, as descriptors
                const uint64_t df = df0 + ((slot * kSfDepth + i) * (kSfOne >> 4));
                // TMEM columns of the k-block's own place: the MMAs that read them last have completed, or the scales
                // would not have been refilled
                const uint32_t tsf = tmem_base + C::SF_COL + 8 * (slot * kSfDepth + i);
                tmem_copy_scales(tsf, df);
                tmem_copy_scales(tsf + 4, df + (512 >> 4));
#pragma unroll
                for (uint32_t j = 0; j < kMxBK / 32; ++j)
                  mma_mx(tmem_base, dw0 + at + j * 2, dx0 + at + j * 2, a.idesc | (j << 4) | (j << 29), tsf, tsf + 4,
                         (base + i > kb0 || j > 0) ? 1u : 0u);
                mma_commit(&empty[st[i]]);
              }
            }
          }
          if (good) mma_commit(&sf_empty[slot]);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, *abort_flag == 0);
        if (!ok) break;
        if (++slot == kSfSlots) {
          slot = 0;
          sf_phase ^= 1u;
        }
      }
      if (ok && elect_one()) mma_commit(accf);
    } else if (QUANT && warp >= 4) {
      if constexpr (QUANT) {
        const int tokens = static_cast<int>(min(static_cast<int64_t>(TN), tt.end - tt.row0));
        if (a.x_fp4)
          quantize_stages<TN, DEEP, kMxE2M1>(a, tt.row0, tokens, kb0, kb1, smem, sf, full, empty, abort_flag, err);
        else
          quantize_stages<TN, DEEP, kMxE4M3>(a, tt.row0, tokens, kb0, kb1, smem, sf, full, empty, abort_flag, err);
      }
    } else if (!QUANT || warp == 2) {
      // scale words of 128 weight rows (warp 2) or TN tokens (warp 3)
      const bool wside = warp == 2;
      ScaleWords<1, kSfDepth> sc;
      if (wside)
        sc.start(a.w_scales, a.w_rows, w0, kMxRows, kb0, kb1);
      else
        sc.start(a.x_scales, a.M, tt.row0, TN, kb0, kb1);
      uint8_t* dst = sf + (wside ? 0 : 512);
      int slot = 0;
      uint32_t phase = 0;
      for (int base = kb0; base < kb1; base += kSfDepth) {
        if (!__all_sync(0xffffffffu,
                        wait_or_abort(&sf_empty[slot], phase ^ 1u, abort_flag, err, DEV_TIMEOUT_SMEM_EMPTY)))
          break;
#pragma unroll
        for (int i = 0; i < kSfDepth; ++i) sc.store(i, dst + (slot * kSfDepth + i) * kSfOne);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[slot]);
#pragma unroll
        for (int i = 0; i < kSfDepth; ++i) sc.load(i, base + kSfDepth + i, kb1);
        if (++slot == kSfSlots) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();

    const bool ok = wait_or_abort(accf, 0, abort_flag, err, DEV_TIMEOUT_ACCUM);
    if (!ok)  // whichever role gave up: the copies already issued land before the CTA leaves
      for (int i = max(0, issued - C::STAGES); i < issued; ++i)
        mbar_wait_bounded(&full[i % C::STAGES], (i / C::STAGES) & 1, err, DEV_TIMEOUT_TMA_FULL);
    tc_fence_after();
    const int tokens = static_cast<int>(min(static_cast<int64_t>(TN), tt.end - tt.row0));
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool drain = warp < 4 && __all_sync(0xffffffffu, ok);
    if (S == 1) {
      const int64_t n = n0 + warp * 32;
      if (drain && n < a.N) {
        uint8_t* stg = smem + warp * 1024;  // the stages are free
        const int rows = static_cast<int>(min(static_cast<int64_t>(32), a.N - n));
#pragma unroll 1
        for (int c = 0; c < tokens; c += 64) {
          uint32_t lo[4][4], hi[4][4];
          tmem_ld_16x64(tacc + c, lo);
          tmem_ld_16x64(tacc + (16u << 16) + c, hi);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = c + k * 16;
            if (at < tokens) {
              stage_transposed(stg, lo[k], hi[k]);
              __syncwarp();
              store_tokens(stg, a.Y + (tt.row0 + at) * a.N + n, a.N, min(16, tokens - at), rows);
              __syncwarp();
            }
          }
        }
      }
    } else {
      float* part = reinterpret_cast<float*>(smem);  // [token][weight row]
      if (drain) {
#pragma unroll 1
        for (int c = 0; c < tokens; c += 32) {
          float v[32];
          tmem_ld32(tacc + c, v);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < tokens) part[(c + j) * kMxRows + threadIdx.x] = v[j];
        }
      }
      cluster_sync_all();
      if (warp < 4 && !*abort_flag) {
        // This CTA's share of the tokens, a warp every fourth of them and four at a time: the loads from the other
        // CTAs' shared memory are what this costs, so as many as possible are in flight.
        const int t0 = tokens * static_cast<int>(rank) / static_cast<int>(S);
        const int t1 = tokens * static_cast<int>(rank + 1) / static_cast<int>(S);
        const int64_t n = n0 + lane * 4;
        const uint32_t mine = smem_u32(part) + lane * 16;
        for (int j0 = t0 + warp; j0 < t1; j0 += 16) {
          float4 sum[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) sum[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
          for (uint32_t r = 0; r < S; ++r) {
            const uint32_t peer = map_to_cta(mine, r);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int j = j0 + 4 * u;
              if (j < t1) {
                const float4 v = ld_cluster_f32x4(peer + j * (kMxRows * 4));
                sum[u].x += v.x;
                sum[u].y += v.y;
                sum[u].z += v.z;
                sum[u].w += v.w;
              }
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int j = j0 + 4 * u;
            if (j < t1) {
              __nv_bfloat16* dst = a.Y + (tt.row0 + j) * a.N + n;
              const uint32_t p0 = pack_bf16x2(sum[u].x, sum[u].y), p1 = pack_bf16x2(sum[u].z, sum[u].w);
              if (a.N % 4 == 0) {
                if (n < a.N) *reinterpret_cast<uint2*>(dst) = make_uint2(p0, p1);
              } else {
                unsigned short* d = reinterpret_cast<unsigned short*>(dst);
                if (n < a.N) d[0] = static_cast<unsigned short>(p0);
                if (n + 1 < a.N) d[1] = static_cast<unsigned short>(p0 >> 16);
                if (n + 2 < a.N) d[2] = static_cast<unsigned short>(p1);
                if (n + 3 < a.N) d[3] = static_cast<unsigned short>(p1 >> 16);
              }
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync_all();  // no CTA leaves while another may still read its partial
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(C::TMEM_COLS)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------
// Many tokens: persistent CTA pairs, 256 weight rows by up to 256 tokens a tile
// (cta_group::2: each CTA stages 128 weight rows and half of the tokens, and keeps
// 128 rows of the accumulator). A k-block of the full tile is 24 KB of loads a CTA
// for 512 clocks of MMA at the 8-bit rate, where a 1-CTA tile of 128 x 128 needs as
// much for 256 (4096 tokens, 11008x4096: 234 us with those). The rows of a group are
// cut into tiles of equal width, a multiple of 32, so no MMA is wider than its rows
// need (8192 rows over 16 experts: 163 us with a remainder tile a group, 135 so).
// What bounds it at full width is the MMA pipe: 2048 clocks for four k-blocks, at the
// 8-bit rate, whatever the format of the tokens (kind::mxf4 would multiply e2m1 by e2m1 at
// twice the rate; it is not used). 384 threads leave 168 registers a thread, which all roles
// share: k_mx_gemm_pair<2> spills 72 bytes there.
//
// The accumulator takes 256 TMEM columns and the scales 192 more, so there is one
// accumulator; the epilogue's eight warps move it to registers (rounded to bf16, 64
// registers a thread) and release it before they store, which keeps the pause of
// the MMAs to the TMEM reads.
//
// The scales have a ring of their own, of blocks of eight k-blocks: two warps of each
// CTA store them (fence, arrive) once per block and a block ahead. The odd CTA's words
// reach the leader's barrier by a release at cluster scope, from a warp that has no
// loads in flight to wait for: it takes 1000 to 1600 clocks, which bounded the product
// while there was one in one k-block (1250 clocks a k-block) or in four (410).
//
// CG = 1 is the same kernel for single CTAs (128 weight rows by up to 128 tokens), for
// groups of few rows, where the weights' copies are what counts and have to go on from
// tile to tile without a pause: two accumulators, and nothing remote (8 groups of 125
// rows, 4100x4128 each: 45.5 us in pairs, 40.4 so).
constexpr int kPairMaxStages = 10;
constexpr int kPairRing = 6 * (kMxRows + 128) * kMxBK;  // bytes of the operands' ring: 6 stages of the widest tile
constexpr int kPairThreads = 384;  // warps: TMA, MMA (odd CTA: relay), scales of w, scales of x, eight for the epilogue
constexpr int kPairW = kMxRows * kMxBK;
constexpr int kPairBatch = 4;      // k-blocks that one elected region issues
constexpr int kPairSfDepth = 8;    // k-blocks a block of scales
constexpr int kPairSfSlots = 2;
constexpr int kPairOut = 1024;          // bytes an epilogue warp stages: 16 tokens of 32 weight rows
constexpr uint32_t kPairSfCol = 256;    // first TMEM column of the scales
template <int CG>
struct PairCfg {
  static constexpr int ROWS = 128 * CG;            // weight rows of a tile
  static constexpr int SF_ONE = 512 + 512 * CG;    // bytes a k-block: words of 128 weight rows, of 128 CG tokens
  static constexpr int SF_SLOT = kPairSfDepth * SF_ONE;
  static constexpr int SF_COLS = 4 + 4 * CG;       // TMEM columns a k-block
  static constexpr int ACCS = CG == 1 ? 2 : 1;     // accumulators of 128 CG columns
  static constexpr int EPI_COLS = 64 * CG;         // tokens of an epilogue warp
  static constexpr int SMEM = kPairRing + kPairSfSlots * SF_SLOT + 8 * kPairOut + 1024 + 256;
  static_assert(kPairSfCol + kPairSfSlots * kPairSfDepth * SF_COLS <= 512, "TMEM columns");
};

__device__ __forceinline__ void mma_mx_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc));
}

// Each CTA's own 512 bytes at `desc` to its own TMEM.
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc));
}

// An arrival that publishes no memory: the TMEM reads before it are ordered by the
// tcgen05 fences on both sides. (A release would wait for the warp's stores of the
// tile before: 1600 clocks with the accumulator held.)
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar_cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster_addr) : "memory");
}

// The same tokens in boxes of 128, 64, 32 and 16 rows.
struct MxBoxes {
  CUtensorMap m[4];
};

struct MxPairTile {
  int64_t row0;   // first token
  int64_t w0;     // first weight row of the pair, in w's storage
  int64_t n0;     // the same in Y's columns
  int rows;       // tokens
  int width;      // tokens rounded up to 32: the MMA's N
  bool found;
};
// The tiles of a CTA (pair) in turn, for one warp: tiles pair, pair + npairs, .. of
// token tile tok's n_tiles, then the next one's.
struct PairTiles {
  const MxArgs& a;
  GroupScan scan;
  int tok, part, dtok, dpart;
  __device__ __forceinline__ PairTiles(const MxArgs& a_, int pair, int npairs)
      : a(a_), scan(a_.offsets, a_.groups, a_.M, a_.tn, 32) {
    dtok = npairs / a.n_tiles;
    dpart = npairs - dtok * a.n_tiles;
    tok = pair / a.n_tiles;
    part = pair - tok * a.n_tiles;
  }
  __device__ __forceinline__ MxPairTile next() {
    const int64_t row0 = static_cast<int64_t>(tok) * a.step;
    TokenTile tt{0, row0, min(a.M, row0 + a.step), tok < a.tok_tiles};
    if (a.offsets) tt = scan.find(tok);
    MxPairTile t;
    t.found = tt.found;
    t.row0 = tt.row0;
    t.n0 = static_cast<int64_t>(part) * a.tile_rows;
    t.w0 = tt.group * a.N + t.n0;
    t.rows = static_cast<int>(tt.end - tt.row0);
    t.width = (t.rows + 31) / 32 * 32;
    tok += dtok;
    part += dpart;
    if (part >= a.n_tiles) {
      part -= a.n_tiles;
      ++tok;
    }
    return t;
  }
};

// The scales' side (one warp): this CTA's weight rows (WSIDE) or the tile's tokens.
template <int CG, bool WSIDE>
__device__ __forceinline__ void pair_scales(const MxArgs& a, const uint8_t* scales, int64_t rows, int pair, int npairs,
                                            uint32_t rank, uint8_t* dst, uint64_t* sf_full, uint64_t* sf_empty,
                                            volatile int* abort_flag, int32_t* err) {
  using C = PairCfg<CG>;
  int slot = 0;
  uint32_t phase = 0;
  PairTiles tiles(a, pair, npairs);
  while (true) {
    const MxPairTile t = tiles.next();
    if (!t.found) return;
    ScaleWords<WSIDE ? 1 : CG, kPairSfDepth> sc;
    sc.start(scales, rows, WSIDE ? t.w0 + rank * 128 : t.row0, WSIDE ? kMxRows : t.width, 0, a.nkb);
    for (int base = 0; base < a.nkb; base += kPairSfDepth) {
      if (!__all_sync(0xffffffffu, wait_or_abort(&sf_empty[slot], phase ^ 1u, abort_flag, err, DEV_TIMEOUT_SMEM_EMPTY)))
        return;
#pragma unroll
      for (int i = 0; i < kPairSfDepth; ++i) sc.store(i, dst + slot * C::SF_SLOT + i * C::SF_ONE);
      fence_async_shared();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sf_full[slot]);
#pragma unroll
      for (int i = 0; i < kPairSfDepth; ++i) sc.load(i, base + kPairSfDepth + i, a.nkb);
      if (++slot == kPairSfSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
}

// The odd CTA's scale words are stored by its own warps, but the leader issues the
// tcgen05.cp that reads them: their arrival is passed on to the leader's barrier
// with a release at cluster scope.
__device__ __forceinline__ void pair_relay(const MxArgs& a, int pair, int npairs, uint64_t* sf_full,
                                           volatile int* abort_flag, int32_t* err) {
  int slot = 0;
  uint32_t phase = 0;
  PairTiles tiles(a, pair, npairs);
  while (tiles.next().found) {
    for (int base = 0; base < a.nkb; base += kPairSfDepth) {
      if (!__all_sync(0xffffffffu, wait_or_abort(&sf_full[slot], phase, abort_flag, err, DEV_TIMEOUT_TMA_FULL))) return;
      if ((threadIdx.x & 31) == 0) mbar_arrive_cluster(map_to_cta(smem_u32(&sf_full[slot]), 0));
      __syncwarp();
      if (++slot == kPairSfSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
}

template <int CG>
__global__ void __launch_bounds__(kPairThreads, 1)
k_mx_gemm_pair(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ MxBoxes tm_x, const MxArgs a,
               int32_t* err) {
  using C = PairCfg<CG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf = smem + kPairRing;
  uint8_t* out = sf + kPairSfSlots * C::SF_SLOT;
  uint64_t* full = reinterpret_cast<uint64_t*>(out + 8 * kPairOut);
  uint64_t* empty = full + kPairMaxStages;
  uint64_t* sf_full = empty + kPairMaxStages;
  uint64_t* sf_empty = sf_full + kPairSfSlots;
  uint64_t* accf = sf_empty + kPairSfSlots;
  uint64_t* acce = accf + C::ACCS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acce + C::ACCS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const int pair = blockIdx.x / CG;
  const int npairs = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kPairSfSlots; ++s) {
      mbar_init(&sf_full[s], CG == 2 && rank == 0 ? 3 : 2);  // the CTA's scale warps; the leader's also the odd CTA's relay
      mbar_init(&sf_empty[s], 1);
    }
    for (int s = 0; s < C::ACCS; ++s) {
      mbar_init(&accf[s], 1);
      mbar_init(&acce[s], 8 * CG);  // the epilogue warps
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_w);
    for (int b = 0; b < 4; ++b) prefetch_tmap(&tm_x.m[b]);
  }
  if (warp == 1) {
    if (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // the peer's barriers are initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  pdl_enter();

  if (warp == 0) {
    // ---------------- TMA (both CTAs; the bytes count on the leader's barrier) ----------------
    const uint32_t fbar0 = CG == 2 ? map_to_cta(smem_u32(full), 0) : 0u;
    const bool leader = elect_one();
    PairTiles tiles(a, pair, npairs);
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    while (ok) {
      const MxPairTile t = tiles.next();
      if (!t.found) break;
      const int half = t.width / CG;  // tokens that this CTA stages
      const int32_t wrow = static_cast<int32_t>(t.w0 + rank * 128);
      const int32_t xrow = static_cast<int32_t>(t.row0 + rank * half);
      const uint32_t bytes = CG * (kPairW / 2 + half * (a.x_fp4 ? kMxBK / 2 : kMxBK));
      // The warp stays converged and only the copies are the elected lane's: within `if (elect_one())` around the loop the
      // copies' operands left the uniform registers (tiles of 64 tokens: 8% slower).
      for (int kb = 0; kb < a.nkb && ok; ++kb) {
        // (the vote also keeps every lane within a phase of the barrier that it waits on)
        ok = __all_sync(0xffffffffu,
                        wait_or_abort(&empty[stage], phase ^ 1u, abort_flag, err, DEV_TIMEOUT_SMEM_EMPTY));
        if (!ok) break;
        uint8_t* sw = smem + stage * a.stage_bytes;
        const uint32_t fbar = fbar0 + stage * 8;
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], bytes);
          if (CG == 2)
            tma_load_2d_pair(sw, &tm_w, fbar, kb * kMxBK, wrow);
          else
            tma_load_2d(sw, &tm_w, &full[stage], kb * kMxBK, wrow);
          int at = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) {  // half = a sum of boxes of 128, 64, 32 and 16 rows
            if (half & (128 >> b)) {
              if (CG == 2)
                tma_load_2d_pair(sw + kPairW + at * kMxBK, &tm_x.m[b], fbar, kb * kMxBK, xrow + at);
              else
                tma_load_2d(sw + kPairW + at * kMxBK, &tm_x.m[b], &full[stage], kb * kMxBK, xrow + at);
              at += 128 >> b;
            }
          }
        }
        ++issued;
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // The copies issued last, of both CTAs, land before the pair leaves, also where another role gives up after this one.
    if (leader && rank == 0)
      for (int64_t i = max(static_cast<int64_t>(0), issued - a.stages); i < issued; ++i)
        mbar_wait_bounded(&full[i % a.stages], (i / a.stages) & 1, err, DEV_TIMEOUT_TMA_FULL);
  } else if (warp == 1) {
    // ---------------- MMA (leader CTA), relay (odd CTA) ----------------
    if (CG == 2 && rank == 1) {
      pair_relay(a, pair, npairs, sf_full, abort_flag, err);
    } else {
      const uint32_t s0 = smem_u32(smem);
      const uint64_t dw0 = smem_desc(s0, 16, 1024), dx0 = smem_desc(s0 + kPairW, 16, 1024);
      const uint64_t df0 = smem_desc_scales(smem_u32(sf));
      PairTiles tiles(a, pair, npairs);
      int stage = 0, slot = 0, acc = 0;
      uint32_t phase = 0, sf_phase = 0, acc_phase = 0;
      bool ok = true;
      while (ok) {
        const MxPairTile t = tiles.next();
        if (!t.found) break;
        const uint32_t idesc = a.idesc | (static_cast<uint32_t>(t.width >> 3) << 17);
        const bool wide = t.width > 128;
        ok = __all_sync(0xffffffffu, wait_or_abort(&acce[acc], acc_phase ^ 1u, abort_flag, err, DEV_TIMEOUT_TMEM_EMPTY));
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 128;
        for (int base = 0; base < a.nkb && ok; base += kPairSfDepth) {
          ok = __all_sync(0xffffffffu,
                          CG == 2 ? wait_or_abort_cluster(&sf_full[slot], sf_phase, abort_flag, err, DEV_TIMEOUT_TMA_FULL)
                                  : wait_or_abort(&sf_full[slot], sf_phase, abort_flag, err, DEV_TIMEOUT_TMA_FULL));
          if (!ok) break;
          const int end = min(a.nkb, base + kPairSfDepth);
          for (int kb0 = base; kb0 < end && ok; kb0 += kPairBatch) {
            int st[kPairBatch];
            uint32_t ph[kPairBatch];
#pragma unroll
            for (int i = 0; i < kPairBatch; ++i) {
              st[i] = stage;
              ph[i] = phase;
              if (kb0 + i < end && ++stage == a.stages) {
                stage = 0;
                phase ^= 1u;
              }
            }
            if (elect_one()) {
              bool good = true;
#pragma unroll
              for (int i = 0; i < kPairBatch; ++i) {
                if (kb0 + i < end && good) {
                  good = wait_or_abort(&full[st[i]], ph[i], abort_flag, err, DEV_TIMEOUT_TMA_FULL);
                  if (good) {
                    tc_fence_after();
                    const uint64_t at = static_cast<uint32_t>(st[i] * a.stage_bytes) >> 4;
                    const uint32_t one = slot * kPairSfDepth + (kb0 - base) + i;  // this k-block's place among the scales
                    const uint64_t df = df0 + one * (C::SF_ONE >> 4);
                    // TMEM columns of its own: the MMAs that read them last have completed, or the slot would not have
                    // been refilled
                    const uint32_t tsf = tmem_base + kPairSfCol + C::SF_COLS * one;
                    if (CG == 2) {
                      tmem_copy_scales_pair(tsf, df);
                      tmem_copy_scales_pair(tsf + 4, df + (512 >> 4));
                      if (wide) tmem_copy_scales_pair(tsf + 8, df + (1024 >> 4));
                    } else {
                      tmem_copy_scales(tsf, df);
                      tmem_copy_scales(tsf + 4, df + (512 >> 4));
                    }
#pragma unroll
                    for (uint32_t j = 0; j < kMxBK / 32; ++j) {
                      const uint32_t id = idesc | (j << 4) | (j << 29), more = (kb0 + i > 0 || j > 0) ? 1u : 0u;
                      if (CG == 2)
                        mma_mx_pair(d_tmem, dw0 + at + j * 2, dx0 + at + j * 2, id, tsf, tsf + 4, more);
                      else
                        mma_mx(d_tmem, dw0 + at + j * 2, dx0 + at + j * 2, id, tsf, tsf + 4, more);
                    }
                    if (CG == 2)
                      mma_commit_pair(&empty[st[i]]);
                    else
                      mma_commit(&empty[st[i]]);
                  }
                }
              }
              if (good && kb0 + kPairBatch >= end) {
                if (CG == 2)
                  mma_commit_pair(&sf_empty[slot]);
                else
                  mma_commit(&sf_empty[slot]);
              }
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, *abort_flag == 0);
          }
          if (++slot == kPairSfSlots) {
            slot = 0;
            sf_phase ^= 1u;
          }
        }
        if (ok && elect_one()) {
          if (CG == 2)
            mma_commit_pair(&accf[acc]);
          else
            mma_commit(&accf[acc]);
        }
        __syncwarp();
        if (++acc == C::ACCS) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
  } else if (warp < 4) {
    // ---------------- scale words: this CTA's 128 weight rows (warp 2), all tokens of the tile (warp 3) ----------------
    if (warp == 2)
      pair_scales<CG, true>(a, a.w_scales, a.w_rows, pair, npairs, rank, sf, sf_full, sf_empty, abort_flag, err);
    else
      pair_scales<CG, false>(a, a.x_scales, a.M, pair, npairs, rank, sf + 512, sf_full, sf_empty, abort_flag, err);
  } else {
    // ---------------- epilogue: 32 weight rows by EPI_COLS tokens a warp ----------------
    const int quarter = warp & 3, col0 = ((warp - 4) >> 2) * C::EPI_COLS;
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
    uint8_t* stg = out + (warp - 4) * kPairOut;
    PairTiles tiles(a, pair, npairs);
    int acc = 0;
    uint32_t acc_phase = 0;
    while (true) {
      const MxPairTile t = tiles.next();
      if (!t.found) break;
      if (!__all_sync(0xffffffffu, wait_or_abort(&accf[acc], acc_phase, abort_flag, err, DEV_TIMEOUT_ACCUM))) break;
      tc_fence_after();
      // lo, hi: TMEM lanes 0-15 and 16-31, [64 columns][16 of them][fragment]
      uint32_t lo[CG][4][4], hi[CG][4][4];
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        if (col0 + c * 64 < t.width) {  // columns past the width are read but not stored
          tmem_ld_16x64(tacc + acc * 128 + c * 64, lo[c]);
          tmem_ld_16x64(tacc + acc * 128 + (16u << 16) + c * 64, hi[c]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster_relaxed(map_to_cta(smem_u32(&acce[acc]), 0));
        else
          mbar_arrive(&acce[acc]);
      }
      if (++acc == C::ACCS) {
        acc = 0;
        acc_phase ^= 1u;
      }
      const int64_t n = t.n0 + rank * 128 + quarter * 32;
      const int left = t.rows - col0;
      const int nleft = static_cast<int>(min(static_cast<int64_t>(32), a.N - n));
      __nv_bfloat16* dst = a.Y + (t.row0 + col0) * a.N + n;
#pragma unroll
      for (int c = 0; c < 4 * CG; ++c) {
        if (c * 16 < left && nleft > 0) {
          stage_transposed(stg, lo[c >> 2][c & 3], hi[c >> 2][c & 3]);
          __syncwarp();
          store_tokens(stg, dst + static_cast<int64_t>(c * 16) * a.N, a.N, min(16, left - c * 16), nleft);
          __syncwarp();
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
  }
}

// Tensor map of MX data [rows, kp]: a box is 128 elements by box_rows rows, 128
// swizzled bytes a row in shared memory for either format.
bool make_mx_map(CUtensorMap* m, const MxView& v, int box_rows) {
  PFN_encodeTiled enc = get_encoder();
  if (!enc) return false;
  const bool fp4 = v.fmt == kMxE2M1;
  const cuuint64_t kp = static_cast<cuuint64_t>((v.cols + 127) / 128 * 128);
  cuuint64_t dims[2] = {kp, static_cast<cuuint64_t>(v.rows)};
  cuuint64_t strides[1] = {fp4 ? kp / 2 : kp};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(kMxBK), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1u, 1u};
  return enc(m, fp4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, v.data, dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch in clusters of S CTAs, after the preceding kernel's trigger.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), int64_t ctas, int S, int threads, int smem, cudaStream_t stream,
                            Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(S);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

template <int TN, bool QUANT, bool DEEP>
cudaError_t launch_tiles(const CUtensorMap& tw, const CUtensorMap& tx, const MxArgs& a, int64_t tiles, int S,
                         int32_t* err, cudaStream_t stream) {
  using C = MxCfg<TN, DEEP>;
  const cudaError_t e = ensure_smem_limit<k_mx_gemm<TN, QUANT, DEEP>>(C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_clusters(k_mx_gemm<TN, QUANT, DEEP>, tiles * S, S, QUANT ? kMxThreads + 128 : kMxThreads, C::SMEM,
                         stream, tw, tx, a, err);
}

template <int TN, bool QUANT = false>
cudaError_t run_tiles(const MxView& x, const MxView& w, MxArgs a, int64_t tok_tiles, int num_sms, int32_t* err,
                      cudaStream_t stream) {
  CUtensorMap tw, tx;
  if (!make_mx_map(&tw, w, kMxRows)) return cudaErrorInvalidValue;
  if (QUANT)
    tx = tw;  // not used
  else if (!make_mx_map(&tx, x, TN))
    return cudaErrorInvalidValue;
  a.idesc = mx_instr_desc(kFmtE2M1, x.fmt == kMxE2M1 ? kFmtE2M1 : kFmtE4M3, kMxRows, TN);
  const int64_t tiles = tok_tiles * a.n_tiles;
  // CTAs a tile: one on each SM (one token, 4096x4096: 5.9 us with 4 a tile, 6.3 with 8, two to an SM), or where that
  // leaves SMs without one, two on each (11008x4096: 7.3 us with 3 a tile, 8.6 with 1; not with 128 tokens, whose partial
  // tiles cost more to add up: 13.9 and 12.1); each with at least 4 k-blocks.
  int64_t most = num_sms / tiles;
  if (most == 1 && TN <= 64) most = 2 * num_sms / tiles;
  if (most > 8) most = 8;
  if (most > a.nkb / 4) most = a.nkb / 4;
  const int S = most < 1 ? 1 : static_cast<int>(most);
  if (tiles * S <= num_sms) return launch_tiles<TN, QUANT, true>(tw, tx, a, tiles, S, err, stream);
  return launch_tiles<TN, QUANT, false>(tw, tx, a, tiles, S, err, stream);
}

// tn: most tokens a tile, a multiple of 32 up to 128 CG.
template <int CG>
cudaError_t run_pairs(const MxView& x, const MxView& w, MxArgs a, int tn, int64_t tok_tiles, int num_sms, int32_t* err,
                      cudaStream_t stream) {
  using C = PairCfg<CG>;
  CUtensorMap tw;
  MxBoxes tx;
  if (!make_mx_map(&tw, w, kMxRows)) return cudaErrorInvalidValue;
  for (int b = 0; b < 4; ++b)
    if (!make_mx_map(&tx.m[b], x, 128 >> b)) return cudaErrorInvalidValue;
  a.tn = tn;
  // A stage's round trip (MMAs done, slot free, copy issued, data there) takes some 2600 clocks, so narrow tiles, whose
  // MMAs are short, use the room that their operands leave for more stages.
  a.stage_bytes = kPairW + (tn / CG * kMxBK + 1023) / 1024 * 1024;
  a.stages = kPairRing / a.stage_bytes < kPairMaxStages ? kPairRing / a.stage_bytes : kPairMaxStages;
  a.tok_tiles = static_cast<int>(tok_tiles);
  a.step = static_cast<int>(((a.M + tok_tiles - 1) / tok_tiles + 31) / 32 * 32);
  a.tile_rows = C::ROWS;
  a.n_tiles = static_cast<int>((a.N + C::ROWS - 1) / C::ROWS);
  a.idesc = mx_instr_desc(kFmtE2M1, x.fmt == kMxE2M1 ? kFmtE2M1 : kFmtE4M3, C::ROWS, 0);  // N is the tile's
  const int64_t units = tok_tiles * a.n_tiles;
  const int pairs = static_cast<int>(units < num_sms / CG ? units : num_sms / CG);
  const cudaError_t e = ensure_smem_limit<k_mx_gemm_pair<CG>>(C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_clusters(k_mx_gemm_pair<CG>, CG * pairs, CG, kPairThreads, C::SMEM, stream, tw, tx, a, err);
}

}  // namespace

bool mx_gemm_fits(int64_t M, int64_t N, int64_t groups) {
  const int64_t used = groups < M ? groups : M;
  const int64_t n_tiles = (N + kMxRows - 1) / kMxRows;
  // the smallest token tile gives the most tiles; clusters of several CTAs only come with few
  return ((M + used * 15) / 16) <= 0x3FFFFFFFLL / n_tiles;
}

// Rows of a group that has any: all of them, or their mean over as many groups as can have some.
static int64_t rows_per_group(int64_t M, int64_t groups) {
  const int64_t used = groups < M ? groups : M;
  return used > 0 ? (M + used - 1) / used : 0;
}

// Every choice goes by the average group, since the offsets are on the device: with 512 rows of 64 experts, 2048x2048, all
// at one expert the call takes 29 us in 32 tiles of 16 tokens, where that expert's product alone would take 12 (and 43 with
// 8 rows at each).
//
// Most rows of a group, on average, for tiles of 16 tokens: groups are uneven, and a group that needs two tiles reads its
// weights twice (64 experts, 2048x2048, 500 rows: 42.5 us in tiles of 16, 41.2 of 32; 1000 rows: 58.8 and 44.7; 16
// experts, 4096x4096, 200 rows: 43.8 and 34.5).
static int64_t rows_of_16(int64_t groups) { return groups == 1 ? 16 : 8; }

bool mx_gemm_quantizes(int64_t M, int64_t groups) { return rows_per_group(M, groups) <= rows_of_16(groups); }

cudaError_t launch_mx_gemm(const MxView& x, const void* x_bf16, const MxView& w, const int32_t* offsets, int groups,
                           int64_t N, void* Y, int num_sms, int32_t* err, cudaStream_t stream) {
  MxArgs a{};
  a.x_bf16 = static_cast<const uint4*>(x_bf16);
  a.x_scales = x.scales;
  a.w_scales = w.scales;
  a.offsets = offsets;
  a.groups = groups;
  a.M = x.rows;
  a.N = N;
  a.w_rows = w.rows;
  a.n_tiles = static_cast<int>((N + kMxRows - 1) / kMxRows);
  a.K = static_cast<int>(x.cols);
  a.nkb = static_cast<int>((x.cols + kMxBK - 1) / kMxBK);
  a.x_fp4 = x.fmt == kMxE2M1;
  a.Y = static_cast<__nv_bfloat16*>(Y);
  const int64_t per = rows_per_group(a.M, groups);
  // most token tiles that any division of the rows into the groups can need
  const int64_t used = groups < a.M ? groups : a.M;
  auto bound = [&](int tn) { return (a.M + used * (tn - 1)) / tn; };
  if (per <= rows_of_16(groups))
    return x_bf16 ? run_tiles<16, true>(x, w, a, bound(16), num_sms, err, stream)
                  : run_tiles<16>(x, w, a, bound(16), num_sms, err, stream);
  // Groups of up to 128 rows whose tiles make several rounds of SMs: one CTA per SM that goes from tile to tile, copying
  // the next one's weights while it finishes. Averages of 16 to 64 rows want many rounds for it (256 groups of 16,
  // 2048x512: 124 -> 87 us; 128 of 23, 768x2048: 43.8 -> 40.6; 64 of 47, 2048x2048: 55.6 -> 47.9; but 128 of 12,
  // 768x2048: 35.7 and 38.5; 8 of 64, 4096x4096, in two rounds: 18.7 and 21.6), larger ones do not (8 of 125, 4096x4096:
  // 26.6 -> 23.5 us, in pairs before; 8 of 187: 28.9 and 37.5).
  if (offsets && per >= 16 && per <= 128 && bound(128) * a.n_tiles > num_sms &&
      (per > 64 || static_cast<int64_t>(groups) * a.n_tiles > 5 * static_cast<int64_t>(num_sms)))
    return run_pairs<1>(x, w, a, 128, bound(128), num_sms, err, stream);
  if (per <= 2 * rows_of_16(groups)) return run_tiles<32>(x, w, a, bound(32), num_sms, err, stream);
  // The narrowest tile that still gives every tile an SM (200 tokens, 4096x4096: 9.6 us in tiles of 64, 10.7 of 128; 333:
  // 13.0 and 11.7), then pairs, whose tiles read less (1024 tokens, 4096x4096: 19.0 us, 18.6 in 256 tiles of 128 tokens;
  // 512, 11008x4096: 27.0 and 33.1).
  if (per <= 64 || bound(64) * a.n_tiles <= num_sms) return run_tiles<64>(x, w, a, bound(64), num_sms, err, stream);
  if (bound(128) * a.n_tiles <= num_sms) return run_tiles<128>(x, w, a, bound(128), num_sms, err, stream);
  // Tokens a tile: a k-block takes 2 clocks a token, but not under 440 (the copies' round trip); the last round of tiles
  // is as long as the others. Groups come in all sizes, and their tiles shrink to fit: the widest.
  int tn = 256;
  if (!offsets) {
    int64_t best = INT64_MAX;
    for (int t = 256; t >= 128; t -= 32) {
      const int64_t tok = bound(t);
      const int64_t width = ((a.M + tok - 1) / tok + 31) / 32 * 32;
      const int64_t rounds = (tok * ((N + 255) / 256) + num_sms / 2 - 1) / (num_sms / 2);
      const int64_t cost = rounds * (2 * width > 440 ? 2 * width : 440);
      if (cost < best) {
        best = cost;
        tn = t;
      }
    }
  }
  return run_pairs<2>(x, w, a, tn, bound(tn), num_sms, err, stream);
}

}  // namespace qlora
