// mx.cu - quantisation to microscaled 8- and 4-bit floating point and back (format: mx.cuh),
// and the RMS norm with the residual's addition whose output may be microscaled.
#include "kernels.h"
#include "mx.cuh"

namespace fh {

namespace {

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// Eight consecutive values: fp32 in one access, which fills whole sectors, where `wide` says that they
// lie on 32 bytes
__device__ __forceinline__ void store8w(bf16* p, const float (&v)[8], bool) { store8(p, v); }
__device__ __forceinline__ void store8w(float* p, const float (&v)[8], bool wide) {
  if (wide)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  else
    store8(p, v);
}

// ------------------------------------------------------------------ quantise
// A warp takes units of 4 rows x 128 columns, 16 columns a lane: two lanes make a block, so its
// maximum crosses lanes once, and the four scale bytes of a row are one word. QU units are loaded
// before the first is worked on, and no warp waits for another. Bytes bound it: the values read
// once, the codes and scales written once (8640 x 8960 bf16 to mxfp8: 37.0 us, 6.3 TB/s; with 8 values
// a lane, four shuffles for them and a scale tile gathered by the CTA 60.5).
constexpr int QT_THREADS = 256;

// Sixteen consecutive values as they lie in memory: 4 * sizeof(T) words
template <typename T>
__device__ __forceinline__ void load16(const T* p, uint32_t (&w)[4 * sizeof(T)]) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
  }
}
template <typename T>
__device__ __forceinline__ void unpack16(const uint32_t (&w)[4 * sizeof(T)], float (&v)[16]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
  }
}

template <typename T, MxFormat F, int QU>
__global__ void __launch_bounds__(QT_THREADS) quantize_kernel(const T* __restrict__ x, long ldx, int M, int K,
                                                              unsigned ktiles, unsigned units,
                                                              uint8_t* __restrict__ data,
                                                              uint8_t* __restrict__ scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, seg = lane & 7;
  const unsigned u0 = (blockIdx.x * (QT_THREADS / 32) + (threadIdx.x >> 5)) * QU;
  unsigned rg = u0 / ktiles, kt = u0 - rg * ktiles;
  uint32_t raw[QU][4 * sizeof(T)];
  int row[QU], tile[QU];
#pragma unroll
  for (int i = 0; i < QU; ++i) {
    row[i] = u0 + i < units ? (int)(rg * 4 + (lane >> 3)) : -1;
    tile[i] = kt;
    if (++kt == ktiles) {
      kt = 0;
      ++rg;
    }
#pragma unroll
    for (int j = 0; j < 4 * (int)sizeof(T); ++j) raw[i][j] = 0u;
    const int col = tile[i] * 128 + seg * 16;
    if (row[i] >= 0 && row[i] < M && col < K) load16<T>(x + (long)row[i] * ldx + col, raw[i]);
  }
#pragma unroll
  for (int i = 0; i < QU; ++i) {
    float v[16];
    unpack16<T>(raw[i], v);
    uint32_t m = max(mx_amax8(v), mx_amax8(v + 8));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t byte = mx_scale_byte<F>(m);  // 0 for the zeros beyond the tensor
    uint32_t w = byte << (8 * (seg >> 1));
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    if (row[i] < 0) break;
    if (seg == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_word(row[i], tile[i], ktiles)) = w;
    const int col = tile[i] * 128 + seg * 16;
    if (row[i] < M && col < K) {
      const uint2 lo = mx_encode8<F>(v, byte), hi = mx_encode8<F>(v + 8, byte);
      const long at = (long)row[i] * K + col;
      if (F == MX_FP8)
        *reinterpret_cast<uint4*>(data + at) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      else
        *reinterpret_cast<uint2*>(data + at / 2) = make_uint2(lo.x, hi.x);
    }
  }
}

template <typename T, MxFormat F>
cudaError_t launch_quantize(const void* x, long ldx, int M, int K, uint8_t* data, uint8_t* scales, cudaStream_t st) {
  constexpr int QU = sizeof(T) == 2 ? 4 : 2;
  const long ktiles = (K + 127) / 128, units = ((long)M + 127) / 128 * 32 * ktiles;
  if (units > 0x7fffffffL) return cudaErrorInvalidValue;
  constexpr int per = QT_THREADS / 32 * QU;
  return launch_pdl(quantize_kernel<T, F, QU>, dim3((unsigned)((units + per - 1) / per)), dim3(QT_THREADS), 0, st,
                    (const T*)x, ldx, M, K, (unsigned)ktiles, (unsigned)units, data, scales);
}

// ------------------------------------------------------------------ dequantise
// One CTA per scale tile, 128 rows x 128 columns; sixteen lanes take a row, 8 values each, eight rows in
// flight. Bytes bound it: 8640 x 8960 mxfp8 to bf16 37.2 us (6.3 TB/s), to fp32 64 (86 with 16-byte stores,
// which leave half of each sector to the next).
template <typename T, MxFormat F>
__global__ void __launch_bounds__(QT_THREADS) dequantize_kernel(const uint8_t* __restrict__ data,
                                                                const uint8_t* __restrict__ scales, int M, int K,
                                                                bool wide, T* __restrict__ out) {
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
      store8w(out + r * K + col, v, wide);
    }
  }
}

// ------------------------------------------------------------------ residual + RMS norm
// s = x + res, kept in x's type; y = s / sqrt(mean(s^2) + eps) * g + c on s as it is kept, with
// g = a (plain gain) or 1 + a, and a, c the stream's own vectors. W warps share a row, which stays
// in registers (NC chunks of 8 values a lane) between the sum of squares and the output: x and res
// are read once, the sum and y written once, so bytes bound it. A lane's loads are all in flight
// together: they are predicated, not branched around, since a branch waits for its own. Four lanes
// make a microscaled block. Rows past M up to the end of the last scale tile only get zero scales.
// 23040 x 1536 fp32 + bf16 to mxfp8, 390 MB: 63 us, 6.2 TB/s.
enum NormOut { NO_F32 = 0, NO_BF16 = 1, NO_FP8 = 2, NO_FP4 = 3 };

// A row's 1 / rms as r + lo: the reciprocal root is good to 2 steps, and a Newton step on its
// residual, in the part that float32 would round away, keeps s * (r + lo) within about half a step
// (left out where r^2 would overflow).
__device__ __forceinline__ float2 inv_root(float m) {
  const float r = rsqrtf(m), p = r * r, perr = fmaf(r, r, -p);
  const float d = fmaf(-m, perr, fmaf(-m, p, 1.f));
  return make_float2(r, m > 1e-30f && m < INFINITY ? 0.5f * r * d : 0.f);
}

// A value of each of a row's W warps, joined; the same bits in all of them. One use per place in the code.
template <int W, typename F>
__device__ __forceinline__ float row_reduce(float x, F join) {
  if constexpr (W > 1) {
    __shared__ float part[W];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) x = join(x, part[w]);
  }
  return x;
}

// Rows whose squares leave float32's range (1e19 and above, or 1e-15 and below where eps is less than
// 1e-30): scales them by the power of two that takes the largest to [2, 4), or by 2^127, and returns
// mean(s^2) + eps of that, with eps scaled alike; `mean` as it was for rows of zeros, and for those with an
// infinity or a NaN. Only they take this way: the others' times are those without it (23040 x 1536 fp32
// and bf16 to mxfp8 63 us).
template <int W, int NC>
__device__ __forceinline__ float rescale_row(float (&v)[NC][8], float mean, int D, float eps) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; e += 2) m = amax3(m, v[i][e], v[i][e + 1]);
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  m = row_reduce<W>(m, [](float s, float t) { return amax3(s, t, 0.f); });
  if (!(m > 0.f && m < INFINITY)) return mean;
  const float scale = __uint_as_float(min(254u, 255u - (__float_as_uint(m) >> 23)) << 23);
  const float small = eps * scale * scale;
  if (!(small < INFINITY)) return mean;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[i][e] *= scale;
      q = fmaf(v[i][e], v[i][e], q);
    }
  q = row_reduce<W>(warp_sum(q), [](float s, float t) { return s + t; });
  return q / (float)D + small;
}

// Eight consecutive values as they lie in memory, zeros where `in` is false: fp32 in one access
// where `wide` says that they lie on 32 bytes
template <typename T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ void load(const T* p, bool in, bool wide) {
    if constexpr (sizeof(T) == 2) {
      asm volatile(
          "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
          "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
          "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
          : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3])
          : "l"(p), "r"((int)in)
          : "memory");
    } else {
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %9, 0;\n\tsetp.ne.b32 q, %10, 0;\n\t"
          "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
          "mov.b32 %4, 0;\n\tmov.b32 %5, 0;\n\tmov.b32 %6, 0;\n\tmov.b32 %7, 0;\n\t"
          "@p ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
          "@q ld.global.v4.b32 {%0, %1, %2, %3}, [%8];\n\t"
          "@q ld.global.v4.b32 {%4, %5, %6, %7}, [%8 + 16];\n\t}"
          : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3]), "=&r"(w[4]), "=&r"(w[5]), "=&r"(w[6]), "=&r"(w[7])
          : "l"(p), "r"((int)(in && wide)), "r"((int)(in && !wide))
          : "memory");
    }
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __uint_as_float(sizeof(T) == 4 ? w[i] : i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

template <typename TX, typename TR, int OUT, int W, int NC>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W)
    add_rms_norm_kernel(const TX* x, const TR* res, TX* sum, const float* __restrict__ a,
                        const float* __restrict__ c, long bstride, int rows_per_batch, int M, int rows, int D,
                        float eps, bool wide, void* __restrict__ out, uint8_t* __restrict__ scales) {
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
    Raw8<TX> xw[NC];
    Raw8<TR> rw[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int ch = t + i * 32 * W;
      xw[i].load(x + row * D + ch * 8, ch < chunks, wide);
      rw[i].load(res + row * D + ch * 8, ch < chunks, wide);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int ch = t + i * 32 * W;
      float r[8];
      xw[i].unpack(v[i]);
      rw[i].unpack(r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = to_f(from_f<TX>(v[i][e] + r[e]));
      if (ch < chunks) store8w(sum + row * D + ch * 8, v[i], wide);
    }
  }
  float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 s = make_float2(v[i][e], v[i][e + 1]);
      q2 = fma2(s, s, q2);
    }
  const float q = row_reduce<W>(warp_sum(q2.x + q2.y), [](float s, float t) { return s + t; });
  float mean = q / (float)D + eps;
  if (!(mean >= 1e-30f && mean < INFINITY)) mean = rescale_row<W>(v, mean, D, eps);
  const float2 rstd = inv_root(mean);
  const float2 r2 = make_float2(rstd.x, rstd.x), lo2 = make_float2(rstd.y, rstd.y);
  const long mb = ((int)row / rows_per_batch) * bstride;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int ch = t + i * 32 * W;
    const bool in = ch < chunks;
    float y[8], g[8], h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = h[e] = 0.f;
    if (in) {
      load8(a + mb + ch * 8, g);
      if (c) load8(c + mb + ch * 8, h);
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 s = make_float2(v[i][e], v[i][e + 1]), g2 = make_float2(g[e], g[e + 1]);
      const float2 n = fma2(s, r2, mul2(s, lo2));
      const float2 y2 = c ? add2(n, fma2(n, g2, make_float2(h[e], h[e + 1]))) : mul2(n, g2);
      y[e] = y2.x;
      y[e + 1] = y2.y;
    }
    if constexpr (OUT == NO_F32) {
      if (in) store8w(reinterpret_cast<float*>(out) + row * D + ch * 8, y, wide);
    } else if constexpr (OUT == NO_BF16) {
      if (in) store8w(reinterpret_cast<bf16*>(out) + row * D + ch * 8, y, wide);
    } else {
      constexpr MxFormat F = OUT == NO_FP8 ? MX_FP8 : MX_FP4;
      uint32_t m = mx_amax8(y);  // a block's four lanes are in the row or past it together
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t byte = mx_scale_byte<F>(m);
      uint32_t w = in ? byte << (8 * ((lane >> 2) & 3)) : 0u;
      w |= __shfl_xor_sync(0xffffffffu, w, 4);
      w |= __shfl_xor_sync(0xffffffffu, w, 8);
      if (in) {
        if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_word(row, ch >> 4, ktiles)) = w;
        const uint2 code = mx_encode8<F>(y, byte);
        if (F == MX_FP8)
          *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(out) + row * D + ch * 8) = code;
        else
          *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(out) + row * (D / 2) + ch * 4) = code.x;
      }
    }
  }
}

// Warps to a row and chunks to a lane, the first pair that the row fits. Measured at 128 to 160 MB: rows
// of fp32 are fastest at two chunks a lane, which keep enough bytes in flight without starving the SM of
// warps (1536 columns, fp32 and bf16: 36.0 us with 3 warps of 2, 37.8 with 2 of 3, 38.8 with 6 of 1; only 11
// or 12 warps of two leave the SM half empty: 6144 columns 43.4, 8 of 3 40.9); rows of bf16, half as many
// bytes, at three or four, whichever leaves fewer lanes idle (1536 columns: 26.2 us with 2 of 3, 28.1 with
// 3 of 2; 4000 columns: 28.5 with 4 of 4, 30.4 with 6 of 3). Up to 256 rows each is a latency (100 x 1536:
// 2.6 us with 8 of 1, 3.0 with 4 of 2). Above 8192 columns there is one pair, 16 of 4, and no other was
// measured (2440 x 10240 fp32 5.0 TB/s, x 16384 5.6). The pairs are compiled: with the count of warps known at run time only,
// a row's addresses cost up to a tenth (30000 x 1568 bf16 66 us, 59 compiled).
template <typename TX, typename TR, int OUT>
cudaError_t launch_norm(const void* x, const void* res, void* sum, const float* a, const float* c, long bstride,
                        int rows_per_batch, int M, int D, float eps, void* out, uint8_t* scales, cudaStream_t st) {
  const int rows = OUT >= NO_FP8 ? (M + 127) / 128 * 128 : M;
  const int chunks = D / 8;
  const bool wide = aligned32(x) && aligned32(res) && aligned32(sum) && aligned32(out);
#define FH_NORM(WV, NCV)                                                                                             \
  if (chunks <= 32 * WV * NCV)                                                                                        \
  return launch_pdl(add_rms_norm_kernel<TX, TR, OUT, WV, NCV>, dim3(WV == 1 ? (rows + 3) / 4 : rows),                 \
                    dim3(WV == 1 ? 128 : 32 * WV), 0, st, (const TX*)x, (const TR*)res, (TX*)sum, a, c, bstride,      \
                    rows_per_batch, M, rows, D, eps, wide, out, scales)
  FH_NORM(1, 1);
  if (M <= 256) {
    FH_NORM(2, 1);
    FH_NORM(4, 1);
    FH_NORM(8, 1);
    FH_NORM(16, 1);
  }
  FH_NORM(1, 2);
  if constexpr (sizeof(TX) == 2) {
    FH_NORM(1, 4);
    FH_NORM(2, 3);
    FH_NORM(2, 4);
    FH_NORM(3, 3);
    FH_NORM(4, 3);
    FH_NORM(4, 4);
    FH_NORM(5, 4);
    FH_NORM(8, 3);
    FH_NORM(8, 4);
  } else {
    FH_NORM(2, 2);
    FH_NORM(3, 2);
    FH_NORM(4, 2);
    FH_NORM(5, 2);
    FH_NORM(6, 2);
    FH_NORM(8, 2);
    FH_NORM(10, 2);
    FH_NORM(8, 3);
    FH_NORM(16, 2);
  }
  FH_NORM(16, 4);
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
  uint8_t *d = (uint8_t*)data, *s = (uint8_t*)scales;
  if (x_bf16)
    return fmt == MX_FP8 ? launch_quantize<bf16, MX_FP8>(x, ldx, M, K, d, s, st)
                         : launch_quantize<bf16, MX_FP4>(x, ldx, M, K, d, s, st);
  return fmt == MX_FP8 ? launch_quantize<float, MX_FP8>(x, ldx, M, K, d, s, st)
                       : launch_quantize<float, MX_FP4>(x, ldx, M, K, d, s, st);
}

cudaError_t mx_dequantize(const void* data, const void* scales, int M, int K, int fmt, void* out, bool out_bf16,
                          cudaStream_t st) {
  const long tiles = (long)((K + 127) / 128) * ((M + 127) / 128);
  if (tiles > 0x7fffffffL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)tiles);
  const bool wide = aligned32(out);
  const uint8_t *d = (const uint8_t*)data, *s = (const uint8_t*)scales;
  if (out_bf16)
    return fmt == MX_FP8 ? launch_pdl(dequantize_kernel<bf16, MX_FP8>, grid, dim3(QT_THREADS), 0, st, d, s, M, K, wide, (bf16*)out)
                         : launch_pdl(dequantize_kernel<bf16, MX_FP4>, grid, dim3(QT_THREADS), 0, st, d, s, M, K, wide, (bf16*)out);
  return fmt == MX_FP8 ? launch_pdl(dequantize_kernel<float, MX_FP8>, grid, dim3(QT_THREADS), 0, st, d, s, M, K, wide, (float*)out)
                       : launch_pdl(dequantize_kernel<float, MX_FP4>, grid, dim3(QT_THREADS), 0, st, d, s, M, K, wide, (float*)out);
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
