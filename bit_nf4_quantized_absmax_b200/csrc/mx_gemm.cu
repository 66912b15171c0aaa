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
// codes become 8 bytes of codes and 8 of padding), so both take 128 bytes a row
// and one swizzle. Scale words (4 bytes: the row's 4 blocks of the stage) are
// fetched by cp.async, one 128-byte run per 32 rows, to the place that
// tcgen05.cp wants them: row r of 128 at byte (r % 32) * 16 + (r / 32) * 4. The
// MMA of block j reads byte j of each word.
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
constexpr int kMxThreads = 128;   // and four warps more where the kernel quantizes x

template <int TN>
struct MxCfg {
  static constexpr int W_BYTES = kMxRows * kMxBK;
  static constexpr int X_BYTES = TN * kMxBK;
  static constexpr int SF_BYTES = 1024;  // 512 bytes of scale words of the weights, 512 of the tokens
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES + SF_BYTES;
  // two CTAs on an SM: while one fills or drains, the other streams
  static constexpr int STAGES = (110 * 1024 - 1536) / STAGE_BYTES;
  static constexpr int SF_COL = TN < 32 ? 32 : TN;  // first TMEM column of the scales
  static constexpr int TMEM_NEED = SF_COL + 8 * STAGES;
  static constexpr int TMEM_COLS = TMEM_NEED <= 64 ? 64 : (TMEM_NEED <= 128 ? 128 : 256);
  static constexpr int SMEM = STAGES * STAGE_BYTES + 1024 /*align*/ + 256 /*barriers*/;
  static_assert(STAGES * STAGE_BYTES >= TN * kMxRows * 4, "the partial tile reuses the stages");
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

// 4 bytes global -> shared without registers; zero when !ok (nothing is read).
__device__ __forceinline__ void cp_async_word(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Token tile `want` of the grouped rows, by a whole warp: group e, its first row
// of the tile and the group's end. Offsets are read as they are but clamped to
// [0, M] and to their running maximum, so that no offsets lead outside of x and Y.
struct TokenTile {
  int group;
  int64_t row0, end;
  bool found;
};
__device__ __forceinline__ TokenTile find_token_tile(const int32_t* __restrict__ offsets, int groups, int64_t M,
                                                     int tn, int want) {
  const int lane = threadIdx.x & 31;
  int64_t carry = 0;  // running maximum of the offsets so far
  int base = 0;       // tiles before this chunk
  for (int e0 = 0; e0 < groups; e0 += 32) {
    const int e = e0 + lane;
    const bool in = e < groups;
    int64_t b = in ? offsets[e] : 0, t = in ? offsets[e + 1] : 0;
    b = max(b, carry);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) b = max(b, v);
    }
    t = max(t, b);
    b = min(b, M);
    t = min(t, M);
    const int tiles = in ? static_cast<int>((t - b + tn - 1) / tn) : 0;
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const bool mine = in && want >= base + sum - tiles && want < base + sum;
    const uint32_t hit = __ballot_sync(0xffffffffu, mine);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int first = __shfl_sync(0xffffffffu, base + sum - tiles, src);
      TokenTile r;
      r.group = e0 + src;
      r.row0 = __shfl_sync(0xffffffffu, b, src) + static_cast<int64_t>(want - first) * tn;
      r.end = __shfl_sync(0xffffffffu, t, src);
      r.found = true;
      return r;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
    carry = __shfl_sync(0xffffffffu, t, 31);
    if (!__shfl_sync(0xffffffffu, in ? 1 : 0, 31)) break;
  }
  return TokenTile{0, 0, 0, false};
}

struct MxArgs {
  const uint4* x_bf16;     // QUANT: activations still to be quantized, [M, K]
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  const int32_t* offsets;  // null: one group of all M rows
  int groups;
  int64_t M, N, w_rows;
  int n_tiles, nkb, K;
  uint32_t idesc;
  bool x_fp4;  // the widening copies of e2m1 count the bytes of codes, not of containers
  __nv_bfloat16* Y;
};

// The tokens' side of the stages, from bf16 (warps 4..7 of the QUANT kernel).
template <int TN, int FMT>
__device__ __forceinline__ void quantize_stages(const MxArgs& a, int64_t row0, int tokens, int kb0, int kb1,
                                                uint8_t* smem, uint64_t* full, uint64_t* empty,
                                                volatile int* abort_flag, int32_t* err) {
  using C = MxCfg<TN>;
  static_assert(TN * 8 == 128, "a thread holds 16 elements of a stage");
  constexpr int AHEAD = 4;
  const int t = threadIdx.x - kMxThreads;
  const int row = t >> 3, h = t & 7;  // token, and which 16 of the stage's 128 elements
  const bool mine = row < tokens;
  const uint4* src = a.x_bf16 + ((row0 + (mine ? row : 0)) * a.K + h * 16) / 8;
  uint4 q[AHEAD][2];
  auto load = [&](int kb, uint4 (&d)[2]) {
    d[0] = d[1] = make_uint4(0u, 0u, 0u, 0u);
    if (mine && kb < kb1 && kb * kMxBK + h * 16 < a.K) {
      d[0] = __ldg(src + kb * (kMxBK / 8));
      d[1] = __ldg(src + kb * (kMxBK / 8) + 1);
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load(kb0 + i, q[i]);
  int stage = 0;
  uint32_t phase = 0;
  for (int base = kb0; base < kb1; base += AHEAD) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int kb = base + i;
      if (kb >= kb1) return;
      const uint32_t v[8] = {q[i][0].x, q[i][0].y, q[i][0].z, q[i][0].w, q[i][1].x, q[i][1].y, q[i][1].z, q[i][1].w};
      load(kb + AHEAD, q[i]);
      uint32_t m = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = __vmaxu2(m, v[j] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));  // the block's other half
      const uint32_t byte = mx_scale_byte<FMT>(m >> 7);
      const float inv = mx_inverse_scale(byte);
      float f[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const f32x2 p = mul_f32x2({bf16lo_to_f32(v[j]), bf16hi_to_f32(v[j])}, {inv, inv});
        f[2 * j] = p.x;
        f[2 * j + 1] = p.y;
      }
      const bool bad = byte == 255u;
      if (!__all_sync(0xffffffffu, wait_or_abort(&empty[stage], phase ^ 1u, abort_flag, err, DEV_TIMEOUT_SMEM_EMPTY)))
        return;
      uint8_t* sx = smem + stage * C::STAGE_BYTES + C::W_BYTES;
      if (mine) {
        uint8_t* dst = sx + row * 128 + ((h ^ (row & 7)) << 4);  // 128-byte swizzle
        if (FMT == kMxE4M3) {
          uint4 o;
          o.x = cvt_e4m3x2(f[0], f[1]) | (cvt_e4m3x2(f[2], f[3]) << 16);
          o.y = cvt_e4m3x2(f[4], f[5]) | (cvt_e4m3x2(f[6], f[7]) << 16);
          o.z = cvt_e4m3x2(f[8], f[9]) | (cvt_e4m3x2(f[10], f[11]) << 16);
          o.w = cvt_e4m3x2(f[12], f[13]) | (cvt_e4m3x2(f[14], f[15]) << 16);
          *reinterpret_cast<uint4*>(dst) = bad ? make_uint4(0u, 0u, 0u, 0u) : o;
        } else {
          const float lo[8] = {f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
          const float hi[8] = {f[8], f[9], f[10], f[11], f[12], f[13], f[14], f[15]};
          *reinterpret_cast<uint2*>(dst) = bad ? make_uint2(0u, 0u) : make_uint2(cvt_e2m1x8(lo), cvt_e2m1x8(hi));
        }
        if ((h & 1) == 0) sx[C::X_BYTES + 512 + row * 16 + (h >> 1)] = static_cast<uint8_t>(byte);
      }
      fence_async_shared();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&full[stage]);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

// One tile a cluster of S CTAs, CTA r of the cluster taking k-blocks [r nkb / S,
// (r + 1) nkb / S). Warp 0 issues the TMA copies, warp 1 the MMAs, warps 2 and 3
// the scale words of the weights and the tokens; all four then drain the
// accumulator. With S > 1 each CTA leaves its fp32 partial in shared memory and
// adds up its share of the tokens over the cluster, in the order of the CTAs.
//
// QUANT (TN = 16): x is bf16, and four more warps write the tokens' side of a stage
// themselves: thread t holds 16 elements, half an MX block, of token t / 8, four
// stages ahead in registers, so that a decode step is one launch and its
// activations are never stored. A few tokens are quantized again by every CTA,
// which costs less than a launch and a round trip through memory.
template <int TN, bool QUANT>
__global__ void __launch_bounds__(QUANT ? kMxThreads + 128 : kMxThreads)
k_mx_gemm(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const MxArgs a,
          int32_t* err) {
  using C = MxCfg<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* accf = empty + C::STAGES;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(accf + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t S;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(S));
  const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], QUANT ? 6 : 3);  // the TMA warp, the scale warp(s), the four quantizing warps
      mbar_init(&empty[s], 1);
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
  if (a.offsets) tt = find_token_tile(a.offsets, a.groups, a.M, TN, tok);
  const int64_t w0 = tt.group * a.N + n0;  // first weight row in w's storage
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.nkb) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(a.nkb) * (rank + 1) / S);

  if (tt.found) {  // the same in every thread of the cluster
    if (warp == 0) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0, outstanding = 0, out_parity = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_or_abort(&empty[stage], phase ^ 1u, abort_flag, err, DEV_TIMEOUT_SMEM_EMPTY)) {
            ok = false;
            break;
          }
          uint8_t* sw = smem + stage * C::STAGE_BYTES;
          mbar_arrive_expect_tx(&full[stage], C::W_BYTES / 2 + (QUANT ? 0 : a.x_fp4 ? C::X_BYTES / 2 : C::X_BYTES));
          tma_load_2d(sw, &tm_w, &full[stage], kb * kMxBK, static_cast<int32_t>(w0));
          if (!QUANT) tma_load_2d(sw + C::W_BYTES, &tm_x, &full[stage], kb * kMxBK, static_cast<int32_t>(tt.row0));
          outstanding |= 1u << stage;
          out_parity = (out_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok || *abort_flag) {  // let the copies already issued land before the CTA leaves
          for (int s = 0; s < C::STAGES; ++s)
            if (outstanding & (1u << s)) mbar_wait_bounded(&full[s], (out_parity >> s) & 1u, err, DEV_TIMEOUT_TMA_FULL);
        }
      }
    } else if (warp == 1) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_or_abort(&full[stage], phase, abort_flag, err, DEV_TIMEOUT_TMA_FULL)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sw = smem_u32(smem + stage * C::STAGE_BYTES);
          const uint32_t sx = sw + C::W_BYTES;
          const uint32_t sf = sx + C::X_BYTES;
          // the stage's own TMEM columns: the MMAs that read them last have
          // completed, or the stage would not have been refilled
          const uint32_t tsf = tmem_base + C::SF_COL + 8u * stage;
          tmem_copy_scales(tsf, smem_desc_scales(sf));
          tmem_copy_scales(tsf + 4, smem_desc_scales(sf + 512));
#pragma unroll
          for (uint32_t j = 0; j < kMxBK / 32; ++j)
            mma_mx(tmem_base, smem_desc(sw + j * 32, 16, 1024), smem_desc(sx + j * 32, 16, 1024),
                   a.idesc | (j << 4) | (j << 29), tsf, tsf + 4, (kb > kb0 || j > 0) ? 1u : 0u);
          mma_commit(&empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) mma_commit(accf);
      }
    } else if (QUANT && warp >= 4) {
      if constexpr (QUANT) {
        const int tokens = static_cast<int>(min(static_cast<int64_t>(TN), tt.end - tt.row0));
        if (a.x_fp4)
          quantize_stages<TN, kMxE2M1>(a, tt.row0, tokens, kb0, kb1, smem, full, empty, abort_flag, err);
        else
          quantize_stages<TN, kMxE4M3>(a, tt.row0, tokens, kb0, kb1, smem, full, empty, abort_flag, err);
      }
    } else if (!QUANT || warp == 2) {
      // scale words of 128 weight rows (warp 2) or TN tokens (warp 3)
      constexpr int LAG = 2;  // stages in flight behind the one being issued
      const bool wside = warp == 2;
      const uint8_t* src = wside ? a.w_scales : a.x_scales;
      const int64_t rows = wside ? a.w_rows : a.M;
      const int64_t r0 = wside ? w0 : tt.row0;
      const int per = wside ? 4 : (TN + 31) / 32;
      const uint32_t off = C::W_BYTES + C::X_BYTES + (wside ? 0 : 512);
      int stage = 0, done = 0;
      uint32_t phase = 0;
      bool ok = true;
      int issued = 0;
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        ok = wait_or_abort(&empty[stage], phase ^ 1u, abort_flag, err, DEV_TIMEOUT_SMEM_EMPTY);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t dst = smem_u32(smem + stage * C::STAGE_BYTES) + off + lane * 16;
        const uint8_t* line = src + static_cast<int64_t>(kb) * rows * 4;
        for (int q = 0; q < per; ++q) {
          const int64_t r = r0 + q * 32 + lane;
          const bool in = r < rows && q * 32 + lane < (wside ? kMxRows : TN);
          cp_async_word(dst + q * 4, line + (in ? r : 0) * 4, in);
        }
        cp_async_commit();
        ++issued;
        if (issued > LAG) {
          cp_async_wait<LAG>();
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[done]);
          if (++done == C::STAGES) done = 0;
        }
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      cp_async_wait<0>();
      fence_async_shared();
      __syncwarp();
      if (ok) {
        for (int left = min(issued, LAG); left > 0; --left) {
          if (lane == 0) mbar_arrive(&full[done]);
          if (++done == C::STAGES) done = 0;
        }
      }
    }
    __syncwarp();

    const bool ok = wait_or_abort(accf, 0, abort_flag, err, DEV_TIMEOUT_ACCUM);
    tc_fence_after();
    const int64_t n = n0 + threadIdx.x;  // lane of TMEM = weight row
    const int tokens = static_cast<int>(min(static_cast<int64_t>(TN), tt.end - tt.row0));
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float* part = reinterpret_cast<float*>(smem);
    if (warp < 4 && __all_sync(0xffffffffu, ok)) {
#pragma unroll 1
      for (int c = 0; c < TN; c += 32) {
        float v[32];
        tmem_ld32(tacc + c, v);
        if (S == 1) {
          __nv_bfloat16* dst = a.Y + (tt.row0 + c) * a.N + n;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < tokens && n < a.N) dst[static_cast<int64_t>(j) * a.N] = __float2bfloat16_rn(v[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < TN) part[(c + j) * kMxRows + threadIdx.x] = v[j];
        }
      }
    }
    if (S > 1) {
      cluster_sync_all();
      if (warp < 4 && !*abort_flag) {
        const uint32_t mine = smem_u32(part) + threadIdx.x * 4;
        for (int j = rank; j < tokens; j += S) {
          float sum = 0.0f;
          for (uint32_t r = 0; r < S; ++r) sum += ld_cluster_f32(map_to_cta(mine + j * kMxRows * 4, r));
          if (n < a.N) a.Y[(tt.row0 + j) * a.N + n] = __float2bfloat16_rn(sum);
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

template <int TN, bool QUANT = false>
cudaError_t run_tiles(const MxView& x, const MxView& w, MxArgs a, int64_t tok_tiles, int num_sms, int32_t* err,
                      cudaStream_t stream) {
  using C = MxCfg<TN>;
  CUtensorMap tw, tx;
  if (!make_mx_map(&tw, w, kMxRows)) return cudaErrorInvalidValue;
  if (QUANT)
    tx = tw;  // not used
  else if (!make_mx_map(&tx, x, TN))
    return cudaErrorInvalidValue;
  a.idesc = mx_instr_desc(kFmtE2M1, x.fmt == kMxE2M1 ? kFmtE2M1 : kFmtE4M3, kMxRows, TN);
  const int64_t tiles = tok_tiles * a.n_tiles;
  // CTAs a tile: as many as are on the card at once, with at least 4 stages of work each
  int S = static_cast<int>(2 * num_sms / tiles < 8 ? 2 * num_sms / tiles : 8);
  if (S > a.nkb / 4) S = a.nkb / 4;
  if (S < 1) S = 1;
  cudaError_t e = ensure_smem_limit<k_mx_gemm<TN, QUANT>>(C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * S));
  cfg.blockDim = dim3(QUANT ? kMxThreads + 128 : kMxThreads);
  cfg.dynamicSmemBytes = C::SMEM;
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
  return cudaLaunchKernelEx(&cfg, k_mx_gemm<TN, QUANT>, tw, tx, a, err);
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

bool mx_gemm_quantizes(int64_t M, int64_t groups) { return rows_per_group(M, groups) <= 16; }

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
  if (per <= 16) return x_bf16 ? run_tiles<16, true>(x, w, a, bound(16), num_sms, err, stream)
                               : run_tiles<16>(x, w, a, bound(16), num_sms, err, stream);
  if (per <= 32) return run_tiles<32>(x, w, a, bound(32), num_sms, err, stream);
  if (per <= 64) return run_tiles<64>(x, w, a, bound(64), num_sms, err, stream);
  return run_tiles<128>(x, w, a, bound(128), num_sms, err, stream);
}

}  // namespace qlora
