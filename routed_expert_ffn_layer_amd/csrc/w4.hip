// w4.hip -- products with 4-bit weights for a few tokens: y = x . W^T (+ bias).
//
//   MXFP4: W[n][k] = E2M1(code) * 2^(scale[n][k/32] - 127)
//   INT4:  W[n][k] = s[n][k/G] * (q - z[n][k/G]),  q in 0..15
//
// Laid-out weights: tiles of 16 rows x 128 columns of 1 KB (row-tile major, then column
// step), so that a wave reads a tile as one contiguous KB and lane l's 16 bytes are the
// operands of four 32-column MFMAs.  MXFP4 keeps the layout of the expert slots.  An
// INT4 tile's fragment f = 16 g + row holds, in word m, the 8 codes of columns
// 32 m + 8 g .. + 7, so one MFMA covers 32 consecutive columns, one group or a part of
// one, and the group's scale is applied to its f32 sum: the operand stays the exact
// integer code, never a rounded product.  Inside a word, nibble order 0 2 4 6 1 3 5 7
// of columns 0 1 4 5 2 3 6 7 makes the bytes of (word & 0x0f0f0f0f) columns
// 0 1 2 3 and those of the shifted word columns 4 5 6 7.
// Scale and zero of a group are one 32-bit word (two f16), four consecutive groups of
// a row side by side: per row tile, blocks of 4 groups x 16 rows, 256 bytes each.
//
// INT4 codes become bf16 through E4M3: a byte 0 .. 15 is q * 2^-9 in that format (the
// subnormals and the first binade are one linear run), so the scaled convert by 2^9
// gives q exactly, two per instruction.
//   sum_k x W = sum over groups s * (sum_k x q - z sum_k x)
// and sum_k x over the same 32 columns is one more MFMA with an all-ones operand.
#include "kernels.hpp"
#include "stream_tile.hpp"

namespace moe {

constexpr int kW4Waves = 8;

size_t w4_code_bytes(int N, int K) { return (size_t)((N + 15) / 16) * ((K + 127) / 128) * 1024; }

static size_t w4_scale_bytes(int fmt, int N, int K, int group) {
  const size_t rt = (N + 15) / 16;
  if (fmt == kW4Mxfp4) return rt * (((K + 127) / 128 + 15) / 16) * 1024;
  const size_t groups = (K + group - 1) / group;
  return rt * ((groups + 3) / 4) * 256;
}

size_t w4_bytes(int fmt, int N, int K, int group) { return w4_code_bytes(N, K) + w4_scale_bytes(fmt, N, K, group); }

// ---------------------------------------------------------------------------
// Layout.  One thread per 16-byte code fragment, then per 16 bytes of scales.  Rows past
// N and columns past K become zero codes and zero scales.
// ---------------------------------------------------------------------------
// The 8 codes of 4 source bytes (element 2i in the low nibble of byte i) in the word order
// above: nibble 2j holds element j, nibble 2j + 1 element 4 + j (j < 4).
__device__ __forceinline__ uint32_t int4_word(uint32_t v) {
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) o |= ((v >> (4 * j)) & 15u) << (8 * j) | ((v >> (16 + 4 * j)) & 15u) << (8 * j + 4);
  return o;
}

template <int FMT>
__global__ __launch_bounds__(256) void w4_pack_codes(const uint8_t* __restrict__ codes, int N, int K, uint8_t* w) {
  const int nk = (K + 127) / 128;
  const int64_t total = (int64_t)((N + 15) / 16) * nk * 64;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int f = i & 63, r = f & 15, g = f >> 4;
  const int64_t ts = i >> 6;
  const int step = ts % nk;
  const int64_t row = ts / nk * 16 + r;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (row < N) {
    const uint8_t* src = codes + row * (K / 2);
    if constexpr (FMT == kW4Mxfp4) {
      if (step * 128 + 32 * g < K) v = ldg16(src + step * 64 + 16 * g);
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (step * 128 + 32 * m < K)
          v[m] = int4_word(*reinterpret_cast<const uint32_t*>(src + step * 64 + 16 * m + 4 * g));
    }
  }
  *reinterpret_cast<u32x4*>(w + i * 16) = v;
}

__global__ __launch_bounds__(256) void w4_pack_mx_scales(const uint8_t* __restrict__ scales, int N, int K, uint8_t* w) {
  const int nb = ((K + 127) / 128 + 15) / 16, groups = K / 32;
  const int64_t total = (int64_t)((N + 15) / 16) * nb * 64;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int f = i & 63, r = f & 15, g = f >> 4;
  const int blk = (i >> 6) % nb;
  const int64_t row = (i >> 6) / nb * 16 + r;
  for (int b = 0; b < 16; ++b) {
    const int grp = (blk * 16 + b) * 4 + g;
    w[i * 16 + b] = row < N && grp < groups ? scales[row * groups + grp] : 0;
  }
}

__global__ __launch_bounds__(256) void w4_pack_int4_scales(const uint16_t* __restrict__ scales,
                                                           const uint8_t* __restrict__ zeros, int N, int groups,
                                                           uint8_t* w) {
  const int nb = (groups + 3) / 4;
  const int64_t total = (int64_t)((N + 15) / 16) * nb * 64;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int q = i & 3, r = (i >> 2) & 15;
  const int grp = (i >> 6) % nb * 4 + q;
  const int64_t row = (i >> 6) / nb * 16 + r;
  uint32_t word = 0;
  if (row < N && grp < groups) {
    const int z = zeros ? zeros[row * groups + grp] : 8;
    word = scales[row * groups + grp] | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)z) << 16;
  }
  reinterpret_cast<uint32_t*>(w)[i] = word;
}

hipError_t launch_w4_pack(int fmt, const uint8_t* codes, const void* scales, const uint8_t* zeros, int N, int K,
                          int group, uint8_t* w, hipStream_t st) {
  const size_t cb = w4_code_bytes(N, K), sb = w4_scale_bytes(fmt, N, K, group);
  const dim3 gc((unsigned)((cb / 16 + 255) / 256)), block(256);
  if (fmt == kW4Mxfp4) {
    hipLaunchKernelGGL(w4_pack_codes<kW4Mxfp4>, gc, block, 0, st, codes, N, K, w);
    hipLaunchKernelGGL(w4_pack_mx_scales, dim3((unsigned)((sb / 16 + 255) / 256)), block, 0, st,
                       static_cast<const uint8_t*>(scales), N, K, w + cb);
  } else {
    hipLaunchKernelGGL(w4_pack_codes<kW4Int4>, gc, block, 0, st, codes, N, K, w);
    hipLaunchKernelGGL(w4_pack_int4_scales, dim3((unsigned)((sb / 4 + 255) / 256)), block, 0, st,
                       static_cast<const uint16_t*>(scales), zeros, N, (K + group - 1) / group, w + cb);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Product.  A block owns one row tile for up to 16 tokens; its waves split K and the
// block adds their parts in LDS in ascending order.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bf16x8 int4x8_to_bf16x8(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ float f16_lo(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)w); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16)); }

template <int FMT, int G, bool BF16OUT>
__global__ __launch_bounds__(64 * kW4Waves) void w4_linear_kernel(W4Args a) {
  __shared__ float red[kW4Waves][256];
  const int lane = threadIdx.x & 63, kp = uniform(threadIdx.x >> 6), g = lane >> 4, r = lane & 15;
  const int tile = blockIdx.x;
  const int t0 = blockIdx.y * 16, m = min(16, a.T - t0);
  const int nk = (a.K + 127) / 128, s0 = kp * nk / kW4Waves, s1 = (kp + 1) * nk / kW4Waves;
  const size_t rt = (a.N + 15) / 16;
  const uint8_t* scales = a.w + rt * nk * 1024;
  const __amdgpu_buffer_rsrc_t xbuf = make_rsrc(a.x + (size_t)t0 * a.x_ld, ((size_t)(m - 1) * a.x_ld + a.K) * 2);
  const int row_off = min(a_token(lane), m - 1) * (int)a.x_ld * 2;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if constexpr (FMT == kW4Mxfp4) {
    Mat w;
    w.nK = nk;
    w.nKs = (nk + 15) / 16;
    w.K = a.K;
    w.codes = make_rsrc(a.w + (size_t)tile * nk * 1024, (size_t)nk * 1024);
    w.scales = make_rsrc(scales + (size_t)tile * w.nKs * 1024, (size_t)w.nKs * 1024);
    stream_tile<W_MXFP4>(w, 0, s0, s1, xbuf, row_off, acc);
  } else {
    const int groups = (a.K + G - 1) / G, nb = (groups + 3) / 4;
    const __amdgpu_buffer_rsrc_t codes = make_rsrc(a.w + (size_t)tile * nk * 1024, (size_t)nk * 1024);
    const uint32_t* par = reinterpret_cast<const uint32_t*>(scales + (size_t)tile * nb * 256) + r * 4;
    const u32x4 one4 = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    constexpr int B = G / 32;  // MFMAs per group
    for (int s = s0; s < s1; ++s) {
      const u32x4 q = bld16(codes, lane * 16, s * 1024);
      f32x4 d = {0.f, 0.f, 0.f, 0.f}, xs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int o = frag_offset<W_INT4>(s, b, g, a.K);
        const u32x4 x = bld16(xbuf, o == kPastEnd ? kPastEnd : row_off + o, 0);
        d = mfma16(x, int4x8_to_bf16x8(q[b]), d);
        xs = mfma16(x, as_bf16x8(one4), xs);
        if (b % B == B - 1) {
          const int grp = min((s * 128 + b * 32) / G, groups - 1);
          const uint32_t p = par[grp / 4 * 64 + grp % 4];
          const float sc = f16_lo(p), z = f16_hi(p);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[v] = fmaf(sc, fmaf(-z, xs[v], d[v]), acc[v]);
          d = xs = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) red[kp][64 * v + lane] = acc[v];
  __syncthreads();
  const int o = threadIdx.x, t = o >> 4;
  if (o >= 256 || t >= m) return;
  const int64_t col = (int64_t)tile * 16 + (o & 15);
  if (col >= a.N) return;
  float y = 0.f;
#pragma unroll
  for (int q = 0; q < kW4Waves; ++q) y += red[q][o];
  if (a.bias) y += a.bias[col];
  const size_t at = (size_t)(t0 + t) * a.y_ld + col;
  if (BF16OUT)
    static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_rne(y);
  else
    static_cast<float*>(a.y)[at] = y;
}

template <int FMT, int G>
static void launch_t(const W4Args& a, bool bf16_out, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.T + 15) / 16)), block(64 * kW4Waves);
  if (bf16_out)
    hipLaunchKernelGGL((w4_linear_kernel<FMT, G, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((w4_linear_kernel<FMT, G, false>), grid, block, 0, st, a);
}

hipError_t launch_w4_linear(int fmt, const W4Args& a, bool bf16_out, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  if (fmt == kW4Mxfp4) launch_t<kW4Mxfp4, 32>(a, bf16_out, st);
  else if (a.group == 32) launch_t<kW4Int4, 32>(a, bf16_out, st);
  else if (a.group == 64) launch_t<kW4Int4, 64>(a, bf16_out, st);
  else launch_t<kW4Int4, 128>(a, bf16_out, st);
  return hipGetLastError();
}

}  // namespace moe
