// mx.cu - quantisation to microscaled 8- and 4-bit floating point and back (format: mx.cuh),
// and the RMS norm with the residual's addition whose output may be microscaled.
#include "kernels.h"
#include "mx.cuh"

namespace fh {

namespace {

// ------------------------------------------------------------------ quantise / dequantise
// One CTA per tile of 128 rows x 128 columns, i.e. per 512-byte scale tile. Sixteen lanes take a
// row's 128 columns, 8 values each; four lanes make a block, whose maximum crosses them by two
// shuffles. Bytes bound it: the values read once, the codes and scales written once.
constexpr int QT_THREADS = 256;

template <typename T, MxFormat F>
__global__ void __launch_bounds__(QT_THREADS) quantize_kernel(const T* __restrict__ x, long ldx, int M, int K,
                                                              uint8_t* __restrict__ data,
                                                              uint8_t* __restrict__ scales) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int PER = F == MX_FP8 ? 8 : 4;  // code bytes of 8 values
  const int ktiles = (K + 127) >> 7;
  const int kt = blockIdx.x % ktiles, rt = blockIdx.x / ktiles;
  const int lane16 = threadIdx.x & 15, hw = threadIdx.x >> 4;  // 16 half-warps
  const int col = kt * 128 + lane16 * 8;
  const long rowb = (long)K * PER / 8;
  __shared__ __align__(16) uint32_t words[128];  // the scale tile
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long r = (long)rt * 128 + hw + 16 * i;
    if (r < M && col < K) {
      load8(x + r * ldx + col, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rl = hw + 16 * i;
    const long r = (long)rt * 128 + rl;
    uint32_t m = mx_amax8(v[i]);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t byte = mx_scale_byte<F>(m);  // 0 for the zeros beyond the tensor
    uint32_t w = byte << (8 * (lane16 >> 2));
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    if (lane16 == 0) words[(rl & 31) * 4 + (rl >> 5)] = w;
    if (r < M && col < K) {
      const uint2 c = mx_encode8<F>(v[i], byte);
      uint8_t* dst = data + r * rowb + (long)col * PER / 8;
      if (F == MX_FP8)
        *reinterpret_cast<uint2*>(dst) = c;
      else
        *reinterpret_cast<uint32_t*>(dst) = c.x;
    }
  }
  __syncthreads();
  if (threadIdx.x < 32)
    reinterpret_cast<uint4*>(scales + (size_t)blockIdx.x * 512)[threadIdx.x] =
        reinterpret_cast<const uint4*>(words)[threadIdx.x];
}

template <typename T, MxFormat F>
__global__ void __launch_bounds__(QT_THREADS) dequantize_kernel(const uint8_t* __restrict__ data,
                                                                const uint8_t* __restrict__ scales, int M, int K,
                                                                T* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int PER = F == MX_FP8 ? 8 : 4;
  const int ktiles = (K + 127) >> 7;
  const int kt = blockIdx.x % ktiles, rt = blockIdx.x / ktiles;
  const int lane16 = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const int col = kt * 128 + lane16 * 8;
  const long rowb = (long)K * PER / 8;
  const uint8_t* sc = scales + (size_t)blockIdx.x * 512;
  uint2 c[8];
  uint32_t sb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rl = hw + 16 * i;
    const long r = (long)rt * 128 + rl;
    c[i] = make_uint2(0u, 0u);
    sb[i] = 0;
    if (r < M && col < K) {
      const uint8_t* src = data + r * rowb + (long)col * PER / 8;
      if (F == MX_FP8)
        c[i] = *reinterpret_cast<const uint2*>(src);
      else
        c[i].x = *reinterpret_cast<const uint32_t*>(src);
      sb[i] = sc[(rl & 31) * 16 + (rl >> 5) * 4 + (lane16 >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long r = (long)rt * 128 + hw + 16 * i;
    if (r < M && col < K) {
      const float s = mx_scale_value(sb[i]);
      float v[8];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float2 f;
        if (F == MX_FP8)
          f = mx_decode2_e4m3(((p < 2 ? c[i].x : c[i].y) >> (16 * (p & 1))) & 0xffffu, s);
        else
          f = mx_decode2_e2m1((c[i].x >> (8 * p)) & 0xffu, s);
        v[2 * p] = f.x;
        v[2 * p + 1] = f.y;
      }
      store8(out + r * K + col, v);
    }
  }
}

// ------------------------------------------------------------------ residual + RMS norm
// s = x + res, kept in x's type; y = s / sqrt(mean(s^2) + eps) * g + c on s as it is kept, with
// g = a (plain gain) or 1 + a, and a, c the stream's own vectors. W warps share a row, which
// stays in registers (NC chunks of 8 values per lane) between the sum of squares and the output:
// x and res are read once, the sum and y written once, so bytes bound it. Four lanes make a
// microscaled block. Rows past M up to the end of the last scale tile only zero their scales.
enum NormOut { NO_F32 = 0, NO_BF16 = 1, NO_FP8 = 2, NO_FP4 = 3 };

template <typename TX, typename TR, int OUT, int W, int NC>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W)
    add_rms_norm_kernel(const TX* x, const TR* res, TX* sum, const float* __restrict__ a,
                        const float* __restrict__ c, long bstride, int rows_per_batch, int M, int rows, int D,
                        float eps, void* __restrict__ out, uint8_t* __restrict__ scales) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int RPC = W == 1 ? 4 : 1;  // rows per CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long row = (long)blockIdx.x * RPC + (W == 1 ? warp : 0);
  const int t = W == 1 ? lane : threadIdx.x;  // thread within the row
  const int chunks = D >> 3;
  const long ktiles = (D + 127) >> 7;
  if (row >= rows) return;
  if (row >= M) {  // only for the microscaled outputs
    for (long kt = t; kt < ktiles; kt += 32 * W)
      *reinterpret_cast<uint32_t*>(scales + mx_scale_word(row, kt, ktiles)) = 0u;
    return;
  }
  float v[NC][8];
  {
    float r[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int ch = t + i * 32 * W;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = r[i][e] = 0.f;
      if (ch < chunks) {
        load8(x + row * D + ch * 8, v[i]);
        load8(res + row * D + ch * 8, r[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int ch = t + i * 32 * W;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = to_f(from_f<TX>(v[i][e] + r[i][e]));
      if (ch < chunks) store8(sum + row * D + ch * 8, v[i]);
    }
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(v[i][e], v[i][e], q);
  q = warp_sum(q);
  if constexpr (W > 1) {
    __shared__ float part[W];
    if (lane == 0) part[warp] = q;
    __syncthreads();
    q = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) q += part[w];
  }
  const float rstd = rsqrtf(q / (float)D + eps);
  const long mb = (row / rows_per_batch) * bstride;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int ch = t + i * 32 * W;
    const bool in = ch < chunks;
    float y[8];
    if (in) {
      float g[8], h[8];
      load8(a + mb + ch * 8, g);
      if (c) {
        load8(c + mb + ch * 8, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = v[i][e] * rstd * (1.f + g[e]) + h[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = v[i][e] * rstd * g[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = 0.f;
    }
    if constexpr (OUT == NO_F32) {
      if (in) store8(reinterpret_cast<float*>(out) + row * D + ch * 8, y);
    } else if constexpr (OUT == NO_BF16) {
      if (in) store8(reinterpret_cast<bf16*>(out) + row * D + ch * 8, y);
    } else {
      constexpr MxFormat F = OUT == NO_FP8 ? MX_FP8 : MX_FP4;
      uint32_t m = mx_amax8(y);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t byte = mx_scale_byte<F>(m);
      uint32_t w = byte << (8 * ((lane >> 2) & 3));
      w |= __shfl_xor_sync(0xffffffffu, w, 4);
      w |= __shfl_xor_sync(0xffffffffu, w, 8);
      if ((lane & 15) == 0 && in)
        *reinterpret_cast<uint32_t*>(scales + mx_scale_word(row, ch >> 4, ktiles)) = w;
      if (in) {
        const uint2 code = mx_encode8<F>(y, byte);
        if (F == MX_FP8)
          *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(out) + row * D + ch * 8) = code;
        else
          *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(out) + row * (D / 2) + ch * 4) = code.x;
      }
    }
  }
}

template <typename TX, typename TR, int OUT>
cudaError_t launch_norm(const void* x, const void* res, void* sum, const float* a, const float* c, long bstride,
                        int rows_per_batch, int M, int D, float eps, void* out, uint8_t* scales, cudaStream_t st) {
  const int rows = OUT >= NO_FP8 ? (M + 127) / 128 * 128 : M;
  const int chunks = D / 8;
#define FH_NORM(WV, NCV)                                                                                             \
  return launch_pdl(add_rms_norm_kernel<TX, TR, OUT, WV, NCV>, dim3(WV == 1 ? (rows + 3) / 4 : rows),                 \
                    dim3(WV == 1 ? 128 : 32 * WV), 0, st, (const TX*)x, (const TR*)res, (TX*)sum, a, c, bstride,      \
                    rows_per_batch, M, rows, D, eps, out, scales)
  if (chunks <= 32 * 2) FH_NORM(1, 2);
  if (chunks <= 32 * 4) FH_NORM(1, 4);
  if (chunks <= 32 * 6) FH_NORM(1, 6);
  if (chunks <= 32 * 8) FH_NORM(1, 8);
  if (chunks <= 128 * 4) FH_NORM(4, 4);
  if (chunks <= 256 * 4) FH_NORM(8, 4);
  if (chunks <= 256 * 8) FH_NORM(8, 8);
#undef FH_NORM
  return cudaErrorInvalidValue;
}

template <typename TX, typename TR>
cudaError_t norm_out(const void* x, const void* res, void* sum, const float* a, const float* c, long bstride,
                     int rows_per_batch, int M, int D, float eps, int out_kind, void* out, uint8_t* scales,
                     cudaStream_t st) {
  switch (out_kind) {
    case NO_F32:
      return launch_norm<TX, TR, NO_F32>(x, res, sum, a, c, bstride, rows_per_batch, M, D, eps, out, scales, st);
    case NO_BF16:
      return launch_norm<TX, TR, NO_BF16>(x, res, sum, a, c, bstride, rows_per_batch, M, D, eps, out, scales, st);
    case NO_FP8:
      return launch_norm<TX, TR, NO_FP8>(x, res, sum, a, c, bstride, rows_per_batch, M, D, eps, out, scales, st);
    default:
      return launch_norm<TX, TR, NO_FP4>(x, res, sum, a, c, bstride, rows_per_batch, M, D, eps, out, scales, st);
  }
}

}  // namespace

cudaError_t mx_quantize(const void* x, long ldx, int M, int K, bool x_bf16, int fmt, void* data, void* scales,
                        cudaStream_t st) {
  const long tiles = (long)((K + 127) / 128) * ((M + 127) / 128);
  if (tiles > 0x7fffffffL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)tiles);
  uint8_t *d = (uint8_t*)data, *s = (uint8_t*)scales;
  if (x_bf16)
    return fmt == MX_FP8
               ? launch_pdl(quantize_kernel<bf16, MX_FP8>, grid, dim3(QT_THREADS), 0, st, (const bf16*)x, ldx, M, K, d, s)
               : launch_pdl(quantize_kernel<bf16, MX_FP4>, grid, dim3(QT_THREADS), 0, st, (const bf16*)x, ldx, M, K, d, s);
  return fmt == MX_FP8
             ? launch_pdl(quantize_kernel<float, MX_FP8>, grid, dim3(QT_THREADS), 0, st, (const float*)x, ldx, M, K, d, s)
             : launch_pdl(quantize_kernel<float, MX_FP4>, grid, dim3(QT_THREADS), 0, st, (const float*)x, ldx, M, K, d, s);
}

cudaError_t mx_dequantize(const void* data, const void* scales, int M, int K, int fmt, void* out, bool out_bf16,
                          cudaStream_t st) {
  const long tiles = (long)((K + 127) / 128) * ((M + 127) / 128);
  if (tiles > 0x7fffffffL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)tiles);
  const uint8_t *d = (const uint8_t*)data, *s = (const uint8_t*)scales;
  if (out_bf16)
    return fmt == MX_FP8 ? launch_pdl(dequantize_kernel<bf16, MX_FP8>, grid, dim3(QT_THREADS), 0, st, d, s, M, K, (bf16*)out)
                         : launch_pdl(dequantize_kernel<bf16, MX_FP4>, grid, dim3(QT_THREADS), 0, st, d, s, M, K, (bf16*)out);
  return fmt == MX_FP8 ? launch_pdl(dequantize_kernel<float, MX_FP8>, grid, dim3(QT_THREADS), 0, st, d, s, M, K, (float*)out)
                       : launch_pdl(dequantize_kernel<float, MX_FP4>, grid, dim3(QT_THREADS), 0, st, d, s, M, K, (float*)out);
}

cudaError_t add_rms_norm(const void* x, bool x_bf16, const void* res, bool res_bf16, void* sum, const float* a,
                         const float* c, long bstride, int rows_per_batch, int M, int D, float eps, int out_kind,
                         void* out, void* scales, cudaStream_t st) {
  uint8_t* s = (uint8_t*)scales;
  if (x_bf16)
    return res_bf16 ? norm_out<bf16, bf16>(x, res, sum, a, c, bstride, rows_per_batch, M, D, eps, out_kind, out, s, st)
                    : norm_out<bf16, float>(x, res, sum, a, c, bstride, rows_per_batch, M, D, eps, out_kind, out, s, st);
  return res_bf16 ? norm_out<float, bf16>(x, res, sum, a, c, bstride, rows_per_batch, M, D, eps, out_kind, out, s, st)
                  : norm_out<float, float>(x, res, sum, a, c, bstride, rows_per_batch, M, D, eps, out_kind, out, s, st);
}

}  // namespace fh
