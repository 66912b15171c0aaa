// Conversion of bf16 matrices to MX storage and back, and the RMS norm whose
// output is MX. Conversion is bound by memory traffic (6.1 TB/s at 11008x4096), and so is
// nearly the norm with a residual at its largest (4096x4096: 5.2 TB/s); below that a norm
// is bound by the latency of a row and its sum.
//
// Storage of [rows, cols] (cols % 32 == 0; kp = cols rounded up to 128):
//   data   : [rows][kp] e4m3 bytes, or [rows][kp / 2] bytes of two e2m1 codes
//            (the lower index in the low nibble); columns >= cols are code 0.
//   scales : [kp / 128][rows][4] bytes, block kb of row r at
//            ((kb / 4) * rows + r) * 4 + kb % 4; blocks past cols hold 127.
// The four scale bytes that 128 elements of a row need are one 32-bit word, and
// the words of consecutive rows are adjacent, so a GEMM stage of 128 elements
// reads its scales in contiguous runs whatever row its tile starts at.
#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "nf4_lut.cuh"

namespace qlora {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kDeqUnits = 2;  // blocks a thread decodes at a time (11008x4096 e2m1: 22.0 us with one, 18.9 with two, 20.1 with four)

// Row and padded block of flat block index t (nkb blocks a row).
__device__ __forceinline__ void split_index(int64_t t, int nkb, int64_t total, int64_t& row, int& kb) {
  if (total <= 0xFFFFFFFFLL) {
    const uint32_t r = static_cast<uint32_t>(t) / static_cast<uint32_t>(nkb);
    row = r;
    kb = static_cast<int>(static_cast<uint32_t>(t) - r * static_cast<uint32_t>(nkb));
  } else {
    row = t / nkb;
    kb = static_cast<int>(t - row * nkb);
  }
}

// The scale bytes of lanes 4i..4i+3 as one word (valid in lane 4i).
__device__ __forceinline__ uint32_t gather_scale_word(uint32_t byte) {
  uint32_t w = byte;
  w |= __shfl_down_sync(0xffffffffu, byte, 1) << 8;
  w |= __shfl_down_sync(0xffffffffu, byte, 2) << 16;
  w |= __shfl_down_sync(0xffffffffu, byte, 3) << 24;
  return w;
}

// One thread quantizes one block of 32: 64 contiguous bytes in, 32 (e4m3) or 16
// (e2m1) out, no exchange between threads but the scale word's.
template <int FMT, bool V8>
__global__ void __launch_bounds__(kQuantThreads)
k_mx_quantize(const uint4* __restrict__ X, int64_t rows, int cols, uint8_t* __restrict__ data,
              uint32_t* __restrict__ scales) {
  pdl_enter();
  const int kp = (cols + 127) / 128 * 128;
  const int nkb = kp / 32, nvalid = cols / 32;
  const int64_t total = rows * nkb;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kQuantThreads;
  // total is a multiple of 4: the four lanes of a scale word are in range together
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kQuantThreads; t0 < total; t0 += stride) {
    const int64_t t = t0 + threadIdx.x;
    const bool in = t < total;
    int64_t row = 0;
    int kb = 0;
    if (in) split_index(t, nkb, total, row, kb);
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0u;
    const bool valid = in && kb < nvalid;
    if (valid) {
      const uint4* src = X + (row * cols + kb * 32) / 8;
      if (V8) {
        uint32_t a[8], b[8];
        ld_global_cs_v8(src, a);
        ld_global_cs_v8(src + 2, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = a[i];
          v[8 + i] = b[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 q = __ldcs(src + i);
          v[4 * i] = q.x;
          v[4 * i + 1] = q.y;
          v[4 * i + 2] = q.z;
          v[4 * i + 3] = q.w;
        }
      }
    }
    uint32_t o[8];
    uint32_t byte = mx_quantize_block<FMT>(v, o);
    if (!valid) byte = 127u;  // the padding; its codes are 0
    const uint32_t word = gather_scale_word(byte);
    if (in && (threadIdx.x & 3) == 0) scales[static_cast<int64_t>(kb >> 2) * rows + row] = word;
    if (!in) continue;
    if (FMT == kMxE4M3) {
      uint4* dst = reinterpret_cast<uint4*>(data + row * kp + kb * 32);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
      *reinterpret_cast<uint4*>(data + (row * kp + kb * 32) / 2) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// One thread decodes one block of 32 to 64 contiguous bytes of bf16. An element
// times its scale has at most 4 significant bits, so fp32 and bf16 hold it
// exactly except below bf16's smallest values (one rounding, nearest even) and from
// 2^128 on, which only imported storage reaches (infinite). The e2m1 codes go through the
// 16-entry table of the NF4 decoder.
template <int FMT, bool V8>
__global__ void __launch_bounds__(kQuantThreads)
k_mx_dequantize(const uint8_t* __restrict__ data, const uint8_t* __restrict__ scales, int64_t rows, int cols,
                uint4* __restrict__ out, const __grid_constant__ Nf4Codebook cb) {
  pdl_enter();
  const int kp = (cols + 127) / 128 * 128;
  const int nvalid = cols / 32;
  const int64_t total = rows * nvalid;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kQuantThreads;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x; t0 < total; t0 += stride * kDeqUnits) {
    // every load of the iteration before its first use
    uint4 q[kDeqUnits][2];
    uint32_t byte[kDeqUnits];
#pragma unroll
    for (int u = 0; u < kDeqUnits; ++u) {
      const int64_t t = t0 + u * stride;
      q[u][0] = q[u][1] = make_uint4(0u, 0u, 0u, 0u);
      byte[u] = 0;
      if (t < total) {
        int64_t row;
        int kb;
        split_index(t, nvalid, total, row, kb);
        byte[u] = scales[(static_cast<int64_t>(kb >> 2) * rows + row) * 4 + (kb & 3)];
        if (FMT == kMxE4M3) {
          const uint4* src = reinterpret_cast<const uint4*>(data + row * kp + kb * 32);
          q[u][0] = __ldcs(src);
          q[u][1] = __ldcs(src + 1);
        } else {
          q[u][0] = __ldcs(reinterpret_cast<const uint4*>(data + (row * kp + kb * 32) / 2));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kDeqUnits; ++u) {
      const int64_t t = t0 + u * stride;
      if (t >= total) continue;
      const float sc = mx_scale(byte[u]);
      uint32_t o[2][8];
      if (FMT == kMxE4M3) {
        const uint32_t w[8] = {q[u][0].x, q[u][0].y, q[u][0].z, q[u][0].w, q[u][1].x, q[u][1].y, q[u][1].z, q[u][1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const f32x2 a = mul_f32x2(e4m3x2_to_f32x2(w[i]), {sc, sc});
          const f32x2 b = mul_f32x2(e4m3x2_to_f32x2(w[i] >> 16), {sc, sc});
          o[i >> 2][2 * (i & 3)] = pack_bf16x2(a.x, a.y);
          o[i >> 2][2 * (i & 3) + 1] = pack_bf16x2(b.x, b.y);
        }
      } else {
        const Nf4Lut lut = make_nf4_lut(cb, sc);
        nf4_lookup8(lut, q[u][0].x, o[0]);
        nf4_lookup8(lut, q[u][0].y, o[0] + 4);
        nf4_lookup8(lut, q[u][0].z, o[1]);
        nf4_lookup8(lut, q[u][0].w, o[1] + 4);
      }
      uint4* dst = out + t * 4;
      if (V8) {
        st_global_cs_v8(dst, o[0]);
        st_global_cs_v8(dst + 2, o[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __stcs(dst + i, make_uint4(o[i >> 1][4 * (i & 1)], o[i >> 1][4 * (i & 1) + 1], o[i >> 1][4 * (i & 1) + 2],
                                     o[i >> 1][4 * (i & 1) + 3]));
      }
    }
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 1 / sqrt(v) as a head and a tail, to about 2^-43: the fp32 estimate and one Newton
// step in fp64 (an fp64 division and root in every thread took a third of the
// norm's time).
__device__ __forceinline__ void rsqrt_head_tail(double v, float& hi, float& lo) {
  double r;
  if (v > 1e-35 && v < 1e38) {
    const double e = static_cast<double>(rsqrtf(static_cast<float>(v)));
    r = e * (1.5 - 0.5 * v * e * e);
  } else {
    r = 1.0 / sqrt(v);
  }
  hi = static_cast<float>(r);
  lo = static_cast<float>(r - static_cast<double>(hi));
  if (!(fabsf(hi) < __int_as_float(0x7F800000))) lo = 0.0f;  // infinite or NaN
}

// a * b + c rounded toward zero
__device__ __forceinline__ f32x2 fma_rz_f32x2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rz.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// h = bf16(x + residual) (or x), rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd
// gamma, y to MX blocks: a CTA a row, the row read once and kept in registers
// (8 elements a chunk, CHUNKS chunks a thread), so x and the residual cross
// memory once in and the sum and the codes once out. A CTA takes every gridDim-th
// row, reads the next one before it reduces the present one, and keeps gamma.
//
// Squares, their sum, the mean and rstd are fp64: with the 16 + 16 squares of a thread
// added up in fp32, 2 or 3 of 16 million e4m3 codes were not those of the exact y (4096x4096
// with a residual 22.6 us either way; e2m1 without one 15.4 us then, 16.6 so). h * gamma is
// exact in fp32, and rstd enters as a head and a tail, so y carries one fp32 rounding. It is
// a rounding to odd (toward zero, then the last bit set), since a y that became a tie of the
// element type only by its rounding would be rounded a second time, to even (8 of 16 million
// e4m3 elements).
//
// Where rstd is itself a binary fraction p / 2^k, p odd, y is exact and may be a true tie,
// so the bit stays. Then t = sum(h^2) + eps cols, a binary fraction too, has t p^2 =
// cols 4^k, so p^2 divides the odd part of cols: p <= 31, since cols is a multiple of 32 up
// to 32768. Such an rstd is found by its five leading bits and rstd^2 t = cols, whose left
// side is exact up to its last rounding; h gamma rstd then has 21 bits at most.
//
// A zero becomes 2^-149, which is a zero again under every scale. Four neighbouring lanes
// hold a block; the sixteen lanes of 128 elements make a scale word.
template <int FMT, int CHUNKS, bool RES>
__global__ void __launch_bounds__(1024)
k_rmsnorm_mx(const uint4* __restrict__ X, const uint4* residual, const uint4* __restrict__ gamma, float eps,
             int64_t rows, int cols, uint4* residual_out, uint8_t* __restrict__ data, uint32_t* __restrict__ scales) {
  __shared__ double warp_sum[2][32];
  const int T = blockDim.x;
  const int kp = (cols + 127) / 128 * 128;
  const int nchunk = cols / 8, nchunk_p = kp / 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const double inv_cols = 1.0 / cols, eps_cols = static_cast<double>(eps) * cols;
  pdl_enter();
  uint4 xq[CHUNKS], rq[CHUNKS], gq[CHUNKS];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int i = c * T + threadIdx.x;
      xq[c] = rq[c] = make_uint4(0u, 0u, 0u, 0u);
      if (i < nchunk && row < rows) {
        xq[c] = __ldcs(X + row * nchunk + i);
        if (RES) rq[c] = __ldcs(residual + row * nchunk + i);
      }
    }
  };
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int i = c * T + threadIdx.x;
    gq[c] = i < nchunk ? __ldg(gamma + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  load(blockIdx.x);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, buf ^= 1) {
    uint32_t h[CHUNKS][4];
    double d = 0.0;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int i = c * T + threadIdx.x;
      h[c][0] = xq[c].x;
      h[c][1] = xq[c].y;
      h[c][2] = xq[c].z;
      h[c][3] = xq[c].w;
      if (RES) {
        const uint32_t rr[4] = {rq[c].x, rq[c].y, rq[c].z, rq[c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[c][j] = pack_bf16x2(bf16lo_to_f32(h[c][j]) + bf16lo_to_f32(rr[j]),
                                bf16hi_to_f32(h[c][j]) + bf16hi_to_f32(rr[j]));
        if (i < nchunk) residual_out[row * nchunk + i] = make_uint4(h[c][0], h[c][1], h[c][2], h[c][3]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double lo = bf16lo_to_f32(h[c][j]), hi = bf16hi_to_f32(h[c][j]);
        d = fma(lo, lo, d);
        d = fma(hi, hi, d);
      }
    }
    load(row + gridDim.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) warp_sum[buf][warp] = d;
    __syncthreads();  // one a row: the row after next is the first to write this half again
    d = lane < T / 32 ? warp_sum[buf][lane] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);  // the same order in every warp
    float r_hi, r_lo;
    const double t = d + eps_cols;
    rsqrt_head_tail(t * inv_cols, r_hi, r_lo);
    const bool fraction = (__float_as_uint(r_hi) & 0x7FFFFu) == 0u &&
                          static_cast<double>(r_hi) * static_cast<double>(r_hi) * t == static_cast<double>(cols);
    if (fraction) r_lo = 0.0f;
    const uint32_t odd = fraction ? 0u : 1u;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int i = c * T + threadIdx.x;
      const bool valid = i < nchunk;
      const uint32_t gg[4] = {gq[c].x, gq[c].y, gq[c].z, gq[c].w};
      f32x2 y[4];
      float big = 0.0f;  // of the magnitudes; NaN where one is
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 a = mul_f32x2({bf16lo_to_f32(h[c][j]), bf16hi_to_f32(h[c][j])},
                                  {bf16lo_to_f32(gg[j]), bf16hi_to_f32(gg[j])});
        y[j] = fma_rz_f32x2(a, {r_hi, r_hi}, mul_f32x2(a, {r_lo, r_lo}));
        y[j].x = __uint_as_float(__float_as_uint(y[j].x) | odd);
        y[j].y = __uint_as_float(__float_as_uint(y[j].y) | odd);
        big = max_nan(big, max_nan(fabsf(y[j].x), fabsf(y[j].y)));
      }
      uint32_t m = __float_as_uint(big);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t byte = valid ? mx_scale_byte<FMT>(m >> 23) : 127u;
      uint32_t word = byte;
      word |= __shfl_down_sync(0xffffffffu, byte, 4) << 8;
      word |= __shfl_down_sync(0xffffffffu, byte, 8) << 16;
      word |= __shfl_down_sync(0xffffffffu, byte, 12) << 24;
      if (i >= nchunk_p) continue;
      if ((lane & 15) == 0) scales[static_cast<int64_t>(i >> 4) * rows + row] = word;
      const float inv = mx_inverse_scale(byte);
      const bool zero = byte == 255u || !valid;
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = mul_f32x2(y[j], {inv, inv});
        v[2 * j] = y[j].x;
        v[2 * j + 1] = y[j].y;
      }
      if (FMT == kMxE4M3) {
        uint2 o = make_uint2(cvt_e4m3x2(v[0], v[1]) | (cvt_e4m3x2(v[2], v[3]) << 16),
                             cvt_e4m3x2(v[4], v[5]) | (cvt_e4m3x2(v[6], v[7]) << 16));
        if (zero) o = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(data + row * kp + static_cast<int64_t>(i) * 8) = o;
      } else {
        *reinterpret_cast<uint32_t*>(data + (row * kp + static_cast<int64_t>(i) * 8) / 2) = zero ? 0u : cvt_e2m1x8(v);
      }
    }
  }
}

int flat_grid(int64_t threads, int num_sms, int per_sm) {
  const int64_t want = (threads + kQuantThreads - 1) / kQuantThreads;
  const int64_t cap = static_cast<int64_t>(num_sms) * per_sm;
  return static_cast<int>(want < cap ? (want > 0 ? want : 1) : cap);
}

template <int FMT, bool RES>
cudaError_t run_rmsnorm(const void* X, const void* residual, const void* gamma, float eps, const MxView& q,
                        void* residual_out, int num_sms, cudaStream_t stream) {
  const int nchunk_p = static_cast<int>((q.cols + 127) / 128 * 16);
  // Two chunks a thread halve what a row's sum costs against its elements (4096x4096 with a residual: 24.8 us with one,
  // 22.8 with two, 33.3 with four, of which 224 bytes a thread are spilled at 64 registers), but narrow rows have too few
  // threads then (8192x256: 5.4 us with one, 6.5 with two). Four where two would need more than 512 threads, and must
  // where they would need more than 1024. (Between the two limits two are faster: 1024x12288 18.8 us and 25.5 with four,
  // 1024x16384 23.5 and 33.7.)
  const int chunks = nchunk_p <= 64 ? 1 : (nchunk_p <= 1024 ? 2 : 4);
  const int threads = ((nchunk_p + chunks - 1) / chunks + 31) / 32 * 32;
  // As many CTAs as are resident: 59 to 64 registers a thread leave room for 1024 threads an SM. (With twice as many CTAs,
  // half of them start when the others end, and each pays for gamma and its first row: 517x5152 e2m1 5.3 us, 4.8 so;
  // 512x32768 23.8 and 21.3.)
  const int64_t resident = static_cast<int64_t>(num_sms) * (1024 / threads < 16 ? 1024 / threads : 16);
  const int grid = static_cast<int>(q.rows < resident ? q.rows : resident);
  auto kern = chunks == 1 ? k_rmsnorm_mx<FMT, 1, RES> : (chunks == 2 ? k_rmsnorm_mx<FMT, 2, RES> : k_rmsnorm_mx<FMT, 4, RES>);
  return launch_pdl(kern, dim3(grid), dim3(threads), 0, stream, reinterpret_cast<const uint4*>(X),
                    reinterpret_cast<const uint4*>(residual), reinterpret_cast<const uint4*>(gamma), eps, q.rows,
                    static_cast<int>(q.cols), reinterpret_cast<uint4*>(residual_out), q.data,
                    reinterpret_cast<uint32_t*>(q.scales));
}

}  // namespace

cudaError_t launch_mx_quantize(const void* X, const MxView& q, int num_sms, cudaStream_t stream) {
  const bool v8 = (reinterpret_cast<uintptr_t>(X) & 31u) == 0;
  auto kern = q.fmt == kMxE4M3 ? (v8 ? k_mx_quantize<kMxE4M3, true> : k_mx_quantize<kMxE4M3, false>)
                               : (v8 ? k_mx_quantize<kMxE2M1, true> : k_mx_quantize<kMxE2M1, false>);
  const int64_t blocks = q.rows * ((q.cols + 127) / 128 * 4);
  return launch_pdl(kern, dim3(flat_grid(blocks, num_sms, 32)), dim3(kQuantThreads), 0, stream,
                    reinterpret_cast<const uint4*>(X), q.rows, static_cast<int>(q.cols), q.data,
                    reinterpret_cast<uint32_t*>(q.scales));
}

cudaError_t launch_mx_dequantize(const MxView& q, void* out, int num_sms, cudaStream_t stream) {
  // code order of e2m1: sign in bit 3
  const Nf4Codebook cb = {{0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f, -0.0f, -0.5f, -1.0f, -1.5f, -2.0f, -3.0f,
                           -4.0f, -6.0f}};
  const bool v8 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  auto kern = q.fmt == kMxE4M3 ? (v8 ? k_mx_dequantize<kMxE4M3, true> : k_mx_dequantize<kMxE4M3, false>)
                               : (v8 ? k_mx_dequantize<kMxE2M1, true> : k_mx_dequantize<kMxE2M1, false>);
  return launch_pdl(kern, dim3(flat_grid((q.rows * (q.cols / 32) + kDeqUnits - 1) / kDeqUnits, num_sms, 16)), dim3(kQuantThreads), 0, stream,
                    q.data, q.scales, q.rows, static_cast<int>(q.cols), reinterpret_cast<uint4*>(out), cb);
}

cudaError_t launch_rmsnorm_mx(const void* X, const void* residual, const void* gamma, float eps, const MxView& q,
                              void* residual_out, int num_sms, cudaStream_t stream) {
  if (q.fmt == kMxE4M3)
    return residual ? run_rmsnorm<kMxE4M3, true>(X, residual, gamma, eps, q, residual_out, num_sms, stream)
                    : run_rmsnorm<kMxE4M3, false>(X, residual, gamma, eps, q, residual_out, num_sms, stream);
  return residual ? run_rmsnorm<kMxE2M1, true>(X, residual, gamma, eps, q, residual_out, num_sms, stream)
                  : run_rmsnorm<kMxE2M1, false>(X, residual, gamma, eps, q, residual_out, num_sms, stream);
}

}  // namespace qlora
