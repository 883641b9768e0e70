// gemm_mx.cu - block-scaled tensor-core product of two microscaled operands (format: mx.cuh):
// out[m, n] = act(sum_k A[m, k] W[n, k] + bias[n]), fp32 accumulation, sm_100a.
//
// tcgen05.mma ... block_scale multiplies the raw e4m3 or e2m1 codes and applies the e8m0 scales
// inside the tensor core, from TMEM: A's 128 rows x 4 blocks take 4 TMEM columns (row r in lane
// r % 32, column r / 32, the 4 blocks its 4 bytes, repeated in every lane quarter), the layout
// that tcgen05.cp.32x128b.warpx4 makes of one 512-byte scale tile. Both formats run the same
// loop on 128-byte rows of codes, 128 values of mxfp8 or 256 of mxfp4, four MMAs of 32 bytes:
//   warp 0     TMA producer: per stage the codes of A and W (128-byte swizzle) and their scale
//              tiles (zero past the tensor, so a scale that the codes' padding meets is finite).
//   warp 1     allocates TMEM, copies each stage's scales there and issues the MMAs.
//   warps 2-9  epilogue, two warps per TMEM lane quarter, each half of the tile's columns: bias,
//              GELU, and fp32 or bf16 rows, or the microscaled form again: a thread holds 32
//              consecutive values of a row, which is a block. Results leave by TMA from boxes
//              in shared memory.
// CTAs take tiles in rounds, alone or as pairs (cta_group::2, each loading half of the W tile); or
// the CTAs of a cluster share one tile's stages and join their sums in shared memory.
// Warps 0 and 1 run their loops whole and elect a lane to issue: with one lane in a divergent
// branch instead, issuing a stage's four MMAs took longer than running them (4096^3 mxfp8: 78.8 us
// against 59.3). What bounds the loop now is shared memory: a stage's 32 KB are written by TMA and
// read by the MMAs at 128 bytes a clock each SM, 512 of the about 600 clocks that a stage of a
// 256 x 256 tile takes: 4096^3 mxfp8 48.7 us (2820 TFLOP/s), 4096 x 4096 x 8192 mxfp4 48 (5700); for a
// second and longer the power cap holds the clock below that. With few stages a tile and GELU the epilogue
// bounds it: 8640 x 8960 x 1536 mxfp4 to bf16 67 us, 56 without GELU (and 73 to float32, whose boxes are half
// as wide, 49 to mxfp4).
// The tensor core cuts its float32 sums off where an addition does not fit: K = 1536 mxfp8 is off by 1.0e-7
// of the result's norm and 6e-8 low on average, a float32 product by 0.6e-7; mxfp4, whose products have
// fewer bits, by 0.3e-7 like the float32 one.
// Every wait is bounded (FH_WAIT_LIMIT_NS), as in gemm_tc.cu; one that ran out is latched in the
// device's error word of the operators.
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "mx.cuh"

namespace fh {

namespace {

constexpr int MXG_THREADS = 320;
constexpr int EPI_THREADS = 256;
constexpr uint32_t BOX_BYTES = 4096;   // an epilogue warp's staging box: 32 rows of up to 128 bytes
constexpr uint32_t BIAS_BYTES = 512;   // and its columns' bias

enum MxOut { MXO_F32 = 0, MXO_BF16 = 1, MXO_FP8 = 2, MXO_FP4 = 3 };

// Columns that an epilogue warp takes at a time, of its share `half` of the tile: 64 where that
// divides and a row of them fits the box.
constexpr int box_cols(int out, int half) { return out != MXO_F32 && half % 64 == 0 ? 64 : 32; }
constexpr int box_row_bytes(int out, int half) {
  return box_cols(out, half) * (out == MXO_F32 ? 8 : out == MXO_BF16 ? 4 : out == MXO_FP8 ? 2 : 1) / 2;
}

template <MxFormat F, int BN, bool PAIR>
struct MxShape {
  static constexpr int TM = PAIR ? 256 : 128;
  static constexpr int KB = F == MX_FP8 ? 128 : 256;  // values per 128-byte row of a stage
  static constexpr int ATOMS = KB / 128;              // scale tiles along K per stage
  static constexpr int WROWS = PAIR ? BN / 2 : BN;    // W rows each CTA loads
  static constexpr int SFBT = (BN + 127) / 128;       // scale row tiles of W
  static constexpr uint32_t A_BYTES = 128 * 128;
  static constexpr uint32_t B_BYTES = WROWS * 128;
  static constexpr uint32_t SFA_BYTES = ATOMS * 512;
  static constexpr uint32_t SFB_BYTES = SFBT * ATOMS * 512;
  static constexpr uint32_t OPER_BYTES = A_BYTES + B_BYTES;
  static constexpr uint32_t SF_BYTES = SFA_BYTES + SFB_BYTES;
  static constexpr uint32_t STAGE_BYTES = OPER_BYTES + SF_BYTES;
  static constexpr uint32_t TX_BYTES = STAGE_BYTES * (PAIR ? 2 : 1);
  // TMEM columns: two accumulators (at BN = 256 the second starts inside the first: see the
  // epilogue), then the scale buffers
  static constexpr int ACC1 = BN == 256 ? 192 : BN;
  static constexpr int OVERLAP = BN == 256 ? 64 : 0;
  static constexpr int SF_COL = ACC1 + BN;
  static constexpr int SFA_COLS = 4 * ATOMS;
  static constexpr int SF_COLS = SFA_COLS + 4 * ATOMS * SFBT;
  static constexpr int NSF_FIT = (512 - SF_COL) / SF_COLS;
  static constexpr uint32_t OUT_BYTES = 8 * (BOX_BYTES + BIAS_BYTES);  // the epilogue warps' staging
  static constexpr uint32_t AUX_BYTES = 1024;
  static constexpr int FIT = (int)((227u * 1024u - 1024u - AUX_BYTES - OUT_BYTES) / STAGE_BYTES);
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  // A scale buffer is free once the MMAs that read it are done. With one buffer per stage the
  // stage's own barriers say so; where TMEM has room for fewer, the copy waits for the MMAs of
  // the stage NSF before it.
  static constexpr int NSF = NSF_FIT < STAGES ? NSF_FIT : STAGES;
  static constexpr uint32_t OUT_OFF = STAGES * OPER_BYTES;
  static constexpr uint32_t SF_OFF = OUT_OFF + OUT_BYTES;
  static constexpr uint32_t AUX_OFF = SF_OFF + STAGES * SF_BYTES;
  static constexpr uint32_t SMEM = AUX_OFF + AUX_BYTES + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static_assert(NSF >= 2 && SF_COL + NSF * SF_COLS <= 512, "TMEM");
  static_assert(NSF <= STAGES, "a scale buffer's stage is still in the ring when it is reused");
};

// Matrix descriptor of a 512-byte scale tile for tcgen05.cp: 16-byte rows, no swizzle, groups
// of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(128u >> 4) << 32 | (uint64_t)1u << 46;
}

template <bool PAIR>
__device__ __forceinline__ void tc_cp_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// Instruction descriptor of the block-scaled kinds, e8m0 scales, shape M x N; `id` is the first
// of the scale bytes (of the 4 of a TMEM column) that this MMA uses, of A and of B.
__host__ __device__ constexpr uint32_t idesc_mx(MxFormat f, int M, int N, int id) {
  const uint32_t t = f == MX_FP8 ? 0u : 1u;  // e4m3 in kind::mxf8f6f4, e2m1 in kind::mxf4
  return (uint32_t)id << 4               // B's scale byte
         | t << 7 | t << 10              // A and B type
         | (uint32_t)(N >> 3) << 17      //
         | 1u << 23                      // scales: e8m0
         | (uint32_t)(M >> 7) << 27      //
         | (uint32_t)id << 29;           // A's scale byte
}

template <MxFormat F, bool PAIR>
__device__ __forceinline__ void tc_mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
#define FH_MMA_MX(G, KIND)                                                              \
  asm volatile(                                                                         \
      "{\n\t.reg .pred p;\n\t"                                                          \
      "setp.ne.b32 p, %6, 0;\n\t"                                                       \
      "tcgen05.mma.cta_group::" G "." KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), \
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                   \
      : "memory")
  if constexpr (F == MX_FP8) {
    if constexpr (PAIR)
      FH_MMA_MX("2", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    else
      FH_MMA_MX("1", "kind::mxf8f6f4.block_scale.scale_vec::1X");
  } else {
    if constexpr (PAIR)
      FH_MMA_MX("2", "kind::mxf4.block_scale.scale_vec::2X");
    else
      FH_MMA_MX("1", "kind::mxf4.block_scale.scale_vec::2X");
  }
#undef FH_MMA_MX
}

// Per-CTA TMA loads; in a pair the completion counts on the even CTA's barrier.
template <bool PAIR>
__device__ __forceinline__ void load_codes(const CUtensorMap* map, uint64_t* bar, void* dst, int c0, int c1) {
  if constexpr (PAIR)
    tma_load_2d_pair(map, mapa_shared(smem_u32(bar), 0), dst, c0, c1);
  else
    tma_load_2d(map, bar, dst, c0, c1);
}
template <bool PAIR>
__device__ __forceinline__ void load_scales(const CUtensorMap* map, uint64_t* bar, void* dst, int kt, int rt) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(mapa_shared(smem_u32(bar), 0)), "r"(0), "r"(kt), "r"(rt)
        : "memory");
  else
    tma_load_3d(map, bar, dst, 0, kt, rt);
}
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (PAIR)
    tc_commit_pair(bar, 0x3);
  else
    tc_commit(bar);
}

// The tanh form of GELU of four values, as x / (1 + 2^z) with z = -2 log2(e) sqrt(2/pi)
// (x + 0.044715 x^3), which is x (1 + tanh u) / 2. The special-function unit (an eighth of a
// warp instruction a clock and scheduler) would bound it at 2^z and a reciprocal per value; one
// reciprocal of the four denominators' product serves all of them: 10 clocks per value and scheduler
// instead of 16. For the product to stay finite x is raised to -5.6 first: every result below that
// is -2.7e-9, off by at most as much, 2^-28. Above it the largest relative error, of 2^20 arguments a
// range, is 37 x 2^-24 up to -4, where the roundings of z, of up to 31, pass into 2^z; 17 up to -3, 15 up
// to -2, 9 up to -1 and 6.2 beyond.
__device__ __forceinline__ void gelu4(float* v) {
  float2 x[2], d[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    asm("max.NaN.f32 %0, %1, 0fC0B33333;" : "=f"(x[i].x) : "f"(v[2 * i]));
    asm("max.NaN.f32 %0, %1, 0fC0B33333;" : "=f"(x[i].y) : "f"(v[2 * i + 1]));
    // a NaN stays in its factor x and out of the shared reciprocal
    const float2 w = make_float2(fmaxf(v[2 * i], -5.6f), fmaxf(v[2 * i + 1], -5.6f));
    const float2 k1 = make_float2(-2.3022082f, -2.3022082f), k3 = make_float2(-0.10294324f, -0.10294324f);
    const float2 z = mul2(fma2(mul2(w, w), k3, k1), w);
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(z.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(z.y));
    d[i] = add2(e, make_float2(1.f, 1.f));
  }
  const float ab = d[0].x * d[0].y, cd = d[1].x * d[1].y;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ab * cd));
  const float2 q = mul2(make_float2(r, r), make_float2(cd, ab));  // 1 / ab, 1 / cd
  const float2 y0 = mul2(x[0], mul2(make_float2(q.x, q.x), make_float2(d[0].y, d[0].x)));
  const float2 y1 = mul2(x[1], mul2(make_float2(q.y, q.y), make_float2(d[1].y, d[1].x)));
  v[0] = y0.x;
  v[1] = y0.y;
  v[2] = y1.x;
  v[3] = y1.y;
}

struct MxParams {
  const float* bias;  // or null
  void* out;
  uint8_t* oscales;  // of a microscaled output
  int M, N, nk;      // nk: stages along K
  int last;          // MMAs of the last stage
  int split;         // CTAs that share a tile
  uint32_t tx;       // bytes that fill a stage
  int num_m, ntiles;
  int wide;  // 256-column tiles: those from here on are taken as two halves each
  int gelu;
  int tma;        // rows of out are 16-byte aligned: boxes leave by TMA
  unsigned* err;  // where a wait that ran out is latched
};

// One row's 32 consecutive results: bias (of these columns, in shared memory), activation.
__device__ __forceinline__ void finish32(const MxParams& p, const float4* bias, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 b = bias[j / 4];
    const float2 lo = add2(make_float2(v[j], v[j + 1]), make_float2(b.x, b.y));
    const float2 hi = add2(make_float2(v[j + 2], v[j + 3]), make_float2(b.z, b.w));
    v[j] = lo.x;
    v[j + 1] = lo.y;
    v[j + 2] = hi.x;
    v[j + 3] = hi.y;
  }
  if (p.gelu) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) gelu4(v + j);
  }
}

// Columns col .. col + 4 of the bias; 0 past its end and where there is none
__device__ __forceinline__ float4 load_bias(const MxParams& p, int col) {
  float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.bias && col < p.N) {
    if (col + 4 <= p.N) return *reinterpret_cast<const float4*>(p.bias + col);
    b.x = p.bias[col];
    if (col + 1 < p.N) b.y = p.bias[col + 1];
    if (col + 2 < p.N) b.z = p.bias[col + 2];
  }
  return b;
}

// 16 bytes, unit `j` of a row of RB bytes, into a staging box as the TMA swizzle of that width has it
template <int RB>
__device__ __forceinline__ uint4* box_unit(uint8_t* box, int row, int j) {
  const int x = RB == 128 ? j ^ (row & 7) : RB == 64 ? j ^ ((row >> 1) & 3) : RB == 32 ? j ^ ((row >> 2) & 1) : j;
  return reinterpret_cast<uint4*>(box + row * RB + x * 16);
}

// A block of 32 values as codes, in 16-byte units at unit(0), unit(1) (e2m1: one); its scale byte
template <MxFormat F, typename Unit>
__device__ __forceinline__ uint32_t encode32(const float (&v)[32], Unit unit) {
  const uint32_t byte = mx_scale_byte<F>(mx_amax32(v));
  uint2 c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = mx_encode8<F>(v + 8 * j, byte);
  if constexpr (F == MX_FP8) {
    *unit(0) = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
    *unit(1) = make_uint4(c[2].x, c[2].y, c[3].x, c[3].y);
  } else {
    *unit(0) = make_uint4(c[0].x, c[1].x, c[2].x, c[3].x);
  }
  return byte;
}

// One row's 32 consecutive results into the warp's box, `c0` columns from its left; the block's
// scale byte for microscaled ones.
template <int OUT, int RB>
__device__ __forceinline__ uint32_t stage32(uint8_t* box, int row, int c0, const float (&v)[32]) {
  if constexpr (OUT == MXO_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<float4*>(box_unit<RB>(box, row, c0 / 4 + j)) =
          make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    return 0;
  } else if constexpr (OUT == MXO_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) store8(reinterpret_cast<bf16*>(box_unit<RB>(box, row, c0 / 8 + j)), v + 8 * j);
    return 0;
  } else {
    return encode32<OUT == MXO_FP8 ? MX_FP8 : MX_FP4>(
        v, [&](int j) { return box_unit<RB>(box, row, c0 / (OUT == MXO_FP8 ? 16 : 32) + j); });
  }
}

// A box's columns col .. col + COLS of rows row0 .. row0 + 32 to rows that are not 16-byte aligned:
// consecutive lanes take consecutive columns.
template <int OUT, int RB, int COLS>
__device__ __forceinline__ void copy_box(const MxParams& p, uint8_t* box, int row0, int col, int lane) {
  using T = typename std::conditional<OUT == MXO_F32, float, bf16>::type;
  constexpr int PER = 16 / (int)sizeof(T);
  const int rows = min(32, p.M - row0);
#pragma unroll 8
  for (int r = 0; r < rows; ++r) {
    T* dst = reinterpret_cast<T*>(p.out) + (long)(row0 + r) * p.N + col;
#pragma unroll
    for (int c = 0; c < COLS; c += 32)
      if (col + c + lane < p.N)
        dst[c + lane] = reinterpret_cast<const T*>(box_unit<RB>(box, r, (c + lane) / PER))[(c + lane) % PER];
  }
}

// ---- a tile shared by the CTAs of a cluster (64 columns): each CTA owns 128 / parts of the rows and
// takes all CTAs' sums of them in shared memory, [part][row][64], 16-byte units swizzled by the row.
__device__ __forceinline__ uint32_t sum_unit(int part, int rows, int i, int unit) {
  return (uint32_t)((part * rows + i) * 16 + (unit ^ (i & 15))) * 16u;
}
// Row r's columns 32 sub .. 32 sub + 32 to its owner
__device__ __forceinline__ void send_row(const uint8_t* sums, int part, int rows, int r, int sub, const float (&v)[32]) {
  const uint32_t to = mapa_shared(smem_u32(sums), (uint32_t)(r / rows));
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st_cluster_v4(to + sum_unit(part, rows, r % rows, sub * 8 + j), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
// The owned rows, from global row `row0` on, of the tile at column n0: sums over the parts in their
// order, a block of 32 columns a thread, and what follows them. `bias`: eight warps' columns.
template <int OUT>
__device__ __forceinline__ void join_rows(const MxParams& p, const uint8_t* sums, int parts, int row0, int n0,
                                          const float4* bias) {
  const int rows = 128 / parts;
  if ((int)threadIdx.x >= 2 * rows) return;
  const int i = threadIdx.x % rows, half = threadIdx.x / rows;
  const int row = row0 + i, col = n0 + 32 * half;
  const bool in = row < p.M && col < p.N;
  uint32_t byte = 0;
  if (in) {
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.f;
    for (int s = 0; s < parts; ++s) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 f = *reinterpret_cast<const float4*>(sums + sum_unit(s, rows, i, half * 8 + j));
        v[4 * j] += f.x;
        v[4 * j + 1] += f.y;
        v[4 * j + 2] += f.z;
        v[4 * j + 3] += f.w;
      }
    }
    finish32(p, bias + half * 4 * (BIAS_BYTES / 16), v);
    if constexpr (OUT == MXO_F32 || OUT == MXO_BF16) {
      using T = typename std::conditional<OUT == MXO_F32, float, bf16>::type;
      T* dst = reinterpret_cast<T*>(p.out) + (long)row * p.N + col;
      if (p.tma && col + 32 <= p.N) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) store8(dst + j, v + j);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (col + j < p.N) dst[j] = from_f<T>(v[j]);
      }
    } else {
      uint8_t* dst = reinterpret_cast<uint8_t*>(p.out) + ((long)row * p.N + col) / (OUT == MXO_FP8 ? 1 : 2);
      byte = encode32<OUT == MXO_FP8 ? MX_FP8 : MX_FP4>(v, [&](int j) { return reinterpret_cast<uint4*>(dst) + j; });
    }
  }
  if (OUT >= MXO_FP8) {  // 0 beyond the tensor, up to the end of its last scale tiles
    const int okt = (p.N + 127) >> 7, blk = col >> 5;
    if ((blk >> 2) < okt && row < ((p.M + 127) & ~127))
      p.oscales[mx_scale_word(row, blk >> 2, okt) + (blk & 3)] = (uint8_t)byte;
  }
}

// Where a tile lies, of the `ntiles` that are dealt out
template <int BN>
struct Tile {
  int mt, n0;   // tile along M, first column
  bool narrow;  // half of a 256-column tile
  __device__ __forceinline__ Tile(const MxParams& p, int i) {
    narrow = BN == 256 && i >= p.wide;
    const int t = narrow ? p.wide + ((i - p.wide) >> 1) : i;
    mt = t % p.num_m;
    n0 = t / p.num_m * BN + (narrow && ((i - p.wide) & 1) ? BN / 2 : 0);
  }
};

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// mbar_wait (common.cuh: bounded, false on giving up) by a whole warp, with one answer
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || mbar_wait(bar, parity, abort, err, ERRBIT_TIMEOUT_GEMM));
}

// Whether the phase is complete, without waiting
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A place in a ring of N barriers
template <int N>
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1u;
    }
  }
};

// The scale copies and the k-th of the four MMAs of a stage; `ad`, `bd`, `sd` describe its operands
// and its scale tiles in shared memory, `sf` its scale buffer in TMEM; `narrower`: what the
// instruction descriptor of a narrow tile is less.
template <MxFormat F, int BN, bool PAIR>
__device__ __forceinline__ void issue_scales(uint64_t sd, uint32_t sf) {
  using S = MxShape<F, BN, PAIR>;
  // columns: A's tiles by K, then W's by (K, row tile); in shared memory W's lie by (row tile, K)
#pragma unroll
  for (int a = 0; a < S::ATOMS; ++a) {
    tc_cp_scales<PAIR>(sf + 4 * a, sd + a * 32);
#pragma unroll
    for (int r = 0; r < S::SFBT; ++r)
      tc_cp_scales<PAIR>(sf + S::SFA_COLS + 4 * (a * S::SFBT + r), sd + (S::ATOMS + r * S::ATOMS + a) * 32);
  }
}
template <MxFormat F, int BN, bool PAIR>
__device__ __forceinline__ void issue_mma(int k, uint32_t d, uint64_t ad, uint64_t bd, uint32_t sf, uint32_t sfb_off,
                                          uint32_t narrower, uint32_t accumulate) {
  using S = MxShape<F, BN, PAIR>;
  // 32 code bytes: 32 values (one block) of mxfp8, 64 values (two blocks) of mxfp4
  const int atom = F == MX_FP8 ? 0 : k >> 1;
  const int id = F == MX_FP8 ? k : 2 * (k & 1);
  tc_mma_mx<F, PAIR>(d, ad + 2 * k, bd + 2 * k, idesc_mx(F, S::TM, BN, id) - narrower, sf + 4 * atom,
                     sf + S::SFA_COLS + 4 * S::SFBT * atom + sfb_off, accumulate);
}

template <MxFormat F, int BN, bool PAIR, int OUT, bool SPLIT>
__global__ void __launch_bounds__(MXG_THREADS, 1)
    gemm_mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSW,
                   const __grid_constant__ CUtensorMap tmO, MxParams p) {
  using S = MxShape<F, BN, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::AUX_OFF);
  uint64_t* empty = full + S::STAGES;
  uint64_t* tfull = empty + S::STAGES;  // [2] accumulator complete
  uint64_t* tempty = tfull + 2;         // [2] accumulator (its overlapped part at BN = 256) read
  uint64_t* dealloc_bar = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(dealloc_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  // SPLIT: the CTAs of a cluster share a tile, each a run of its stages, and join their sums below
  const int parts = SPLIT ? p.split : 1;
  const int part = SPLIT ? (int)cluster_ctarank() : 0;
  const int cl = PAIR ? blockIdx.x >> 1 : blockIdx.x / parts;
  const int ncl = PAIR ? gridDim.x >> 1 : gridDim.x / parts;
  const int kb0 = SPLIT ? (int)((long)p.nk * part / parts) : 0;
  const int kb1 = SPLIT ? (int)((long)p.nk * (part + 1) / parts) : p.nk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], EPI_THREADS * (PAIR ? 2 : 1));
    }
    mbar_init(dealloc_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmSA);
    prefetch_tmap(&tmSW);
    if (OUT >= MXO_FP8 || p.tma) prefetch_tmap(&tmO);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_holder, S::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, S::TMEM_COLS);
      tmem_relinquish();
    }
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (PAIR || SPLIT)
    cluster_sync_all();  // the cluster's CTAs run, with their barriers initialised, before any cross-CTA access
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    pdl_wait();  // codes and scales may be the preceding kernel's output
    Ring<S::STAGES> cur;
    int issues = 0;
    bool ok = true;
    for (int tile = cl; ok && tile < p.ntiles; tile += ncl) {
      const Tile<BN> at(p, tile);
      const int m0 = at.mt * S::TM + (int)rank * 128;
      // a narrow tile's box has W rows beyond it, which no MMA reads
      const int w0 = at.n0 + (int)rank * (at.narrow ? S::WROWS / 2 : S::WROWS);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait(&empty[cur.i], cur.phase ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* sa = smem + cur.i * S::OPER_BYTES;
          uint8_t* sf = smem + S::SF_OFF + cur.i * S::SF_BYTES;
          if (rank == 0) mbar_expect_tx(&full[cur.i], p.tx);
          load_codes<PAIR>(&tmA, &full[cur.i], sa, kb * 32, m0);
          load_codes<PAIR>(&tmW, &full[cur.i], sa + S::A_BYTES, kb * 32, w0);
          load_scales<PAIR>(&tmSA, &full[cur.i], sf, kb * S::ATOMS, m0 >> 7);
          load_scales<PAIR>(&tmSW, &full[cur.i], sf + S::SFA_BYTES, kb * S::ATOMS, at.n0 >> 7);
        }
        __syncwarp();
        ++issues;
        cur.next();
      }
    }
    pdl_launch_dependents();
    // tail: the MMA thread has released every stage filled last, so no arrival is in flight
    // towards this CTA when it exits
    for (int s = 0; ok && s < S::STAGES && s < issues; ++s) {
      int st = cur.i - 1 - s;
      uint32_t ph = cur.phase;
      if (st < 0) {
        st += S::STAGES;
        ph ^= 1u;
      }
      ok = warp_wait(&empty[st], ph, abort_flag, p.err);
    }
    if (!ok) {  // give copies already issued time to land
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 200000ull) {
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      Ring<S::STAGES> cur, done;  // the stage to issue, and the one whose MMAs free its scale buffer
      int sf_next = 0, local = 0;
      int pending = 0;  // stages issued, up to NSF
      bool ready = false;
      const uint64_t ad0 = sdesc_kmajor_sw128(smem_u32(smem));
      const uint64_t bd0 = sdesc_kmajor_sw128(smem_u32(smem) + S::A_BYTES);
      const uint64_t sd0 = sdesc_scales(smem_u32(smem) + S::SF_OFF);
      bool ok = true;
      for (int tile = cl; tile < p.ntiles; tile += ncl, ++local) {
        const int acc = local & 1;
        // BN < 256: the accumulator's previous tile (local - 2) has been read. BN = 256: the part
        // of the preceding tile's accumulator that this one overlaps has been read, by threads
        // that had finished tile local - 2 before.
        if (BN == 256) {
          if (local >= 1 && !warp_wait(&tempty[acc ^ 1], ((local - 1) >> 1) & 1, abort_flag, p.err)) break;
        } else {
          if (local >= 2 && !warp_wait(&tempty[acc], ((local - 2) >> 1) & 1, abort_flag, p.err)) break;
        }
        const uint32_t d_tmem = tmem_base + acc * S::ACC1;
        // the tile's first W row within its scale row tile (BN = 64, 192): 32 rows a column
        const Tile<BN> at(p, tile);
        const uint32_t sfb_off = BN % 128 != 0 ? (uint32_t)((at.n0 & 127) >> 5) : 0u;
        const uint32_t narrower = at.narrow ? idesc_mx(F, S::TM, BN, 0) - idesc_mx(F, S::TM, BN / 2, 0) : 0u;
        for (int kb = kb0; kb < kb1; ++kb) {
          if constexpr (S::NSF < S::STAGES) {
            if (pending == S::NSF) {
              ok = warp_wait(&empty[done.i], done.phase, abort_flag, p.err);
              done.next();
            } else {
              ++pending;
            }
          }
          ok = ok && (__all_sync(0xffffffffu, ready) || warp_wait(&full[cur.i], cur.phase, abort_flag, p.err));
          if (!ok) break;
          const int sfi = S::NSF < S::STAGES ? sf_next : cur.i, stage = cur.i;
          cur.next();
          ready = mbar_test(&full[cur.i], cur.phase);  // the next stage's, under this one's issue
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sf = tmem_base + S::SF_COL + sfi * S::SF_COLS;
            const uint64_t ad = ad0 + stage * (S::OPER_BYTES >> 4), bd = bd0 + stage * (S::OPER_BYTES >> 4);
            issue_scales<F, BN, PAIR>(sd0 + stage * (S::SF_BYTES >> 4), sf);
            issue_mma<F, BN, PAIR>(0, d_tmem, ad, bd, sf, sfb_off, narrower, kb > kb0);
            if (kb + 1 < p.nk || p.last == 4) {
#pragma unroll
              for (int k = 1; k < 4; ++k) issue_mma<F, BN, PAIR>(k, d_tmem, ad, bd, sf, sfb_off, narrower, 1u);
            } else {  // the last MMAs end with K: its padding meets at most the second block of one
              if (p.last > 1) issue_mma<F, BN, PAIR>(1, d_tmem, ad, bd, sf, sfb_off, narrower, 1u);
              if (p.last > 2) issue_mma<F, BN, PAIR>(2, d_tmem, ad, bd, sf, sfb_off, narrower, 1u);
            }
            commit<PAIR>(&empty[stage]);
            if (kb + 1 == kb1) commit<PAIR>(&tfull[acc]);
          }
          __syncwarp();
          if (++sf_next == S::NSF) sf_next = 0;
        }
        if (!ok) break;
      }
      // tail: the epilogues have released the last accumulators (no arrival left in flight)
      for (int i = 0; i < 2 && i < local; ++i) {
        const int t = local - 1 - i;
        if (!warp_wait(&tempty[t & 1], (t >> 1) & 1, abort_flag, p.err)) break;
      }
    }
  } else {
    const int quarter = warp & 3;
    const int sub = (warp - 2) >> 2;  // which half of the tile's columns
    constexpr int HALF = BN / 2;
    constexpr int NCH = HALF / 32;              // chunks of 32 columns
    constexpr int COLS = box_cols(OUT, HALF), RB = box_row_bytes(OUT, HALF);
    constexpr int PER = COLS / 32;              // chunks taken at a time
    const long okt = (p.N + 127) >> 7;
    const int mpad = (p.M + 127) & ~127;
    uint8_t* const box = smem + S::OUT_OFF + (warp - 2) * BOX_BYTES;
    float4* const bias = reinterpret_cast<float4*>(smem + S::OUT_OFF + 8 * BOX_BYTES + (warp - 2) * BIAS_BYTES);
    pdl_wait();
    int local = 0;
    for (int tile = cl; tile < p.ntiles; tile += ncl, ++local) {
      const int acc = local & 1;
      const Tile<BN> at(p, tile);
      const int m0 = at.mt * S::TM + (int)rank * 128;
      const int share = at.narrow ? HALF / 2 : HALF, nch = share / 32;
      const int n0 = at.n0 + sub * share;
      if (lane < share / 4) bias[lane] = load_bias(p, n0 + 4 * lane);  // while the MMAs run
      __syncwarp();
      const int row0 = m0 + quarter * 32, row = row0 + lane;
      if (!warp_wait(&tfull[acc], (local >> 1) & 1, abort_flag, p.err)) break;  // tcgen05.ld is warp-collective
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * S::ACC1 + sub * share;
      auto release = [&]() {
        tc_fence_before();
        if constexpr (PAIR)
          mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
        else
          mbar_arrive(&tempty[acc]);
      };
      // At BN = 256 the accumulators share columns 192-255: the last 64 of the first, the first
      // 64 of the second. The warps that hold them read them first and release them, so that the
      // next tile's MMAs run under the rest of this epilogue.
      // (A narrow tile is a CTA's last.)
      const bool overlaps = S::OVERLAP != 0 && !at.narrow;
      const bool holds = overlaps && sub == (acc ^ 1);
      const int first = overlaps && acc == 0 ? NCH / 2 : 0;  // chunk order: rotated for acc 0
      if (overlaps && !holds) release();
      uint32_t word = 0;
      if constexpr (SPLIT) {
        float v[32];
        tmem_ld32(tb, v);
        tc_wait_ld();
        release();
        if (row < p.M) send_row(smem + S::OUT_OFF, part, 128 / parts, quarter * 32 + lane, sub, v);
      } else if (row0 < mpad) {
#pragma unroll 1
        for (int i = 0; i < nch; i += PER) {
          const int ch0 = S::OVERLAP != 0 ? (i + first) & (NCH - 1) : i;
          const int col = n0 + ch0 * 32;
          float v[PER][32];
#pragma unroll
          for (int k = 0; k < PER; ++k) tmem_ld32(tb + (ch0 + k) * 32, v[k]);
          tc_wait_ld();
          if (holds && i + PER == NCH / 2) release();
          if (!overlaps && i + PER == nch) release();
          if (col >= p.N || row0 >= p.M) continue;  // nothing of the tensor
#pragma unroll
          for (int k = 0; k < PER; ++k) finish32(p, bias + (ch0 + k) * 8, v[k]);
          if (p.tma) {  // the box's last store has read it
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
          }
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const uint32_t byte = stage32<OUT, RB>(box, lane, 32 * k, v[k]);
            if (OUT >= MXO_FP8 && row < p.M && col + 32 * k < p.N) word |= byte << (8 * (ch0 + k));
          }
          if (OUT >= MXO_FP8 || p.tma) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmO, box, col / COLS * (RB / 4), row0);
              bulk_commit();
            }
          } else if constexpr (OUT < MXO_FP8) {
            __syncwarp();
            copy_box<OUT, RB, COLS>(p, box, row0, col, lane);
            __syncwarp();
          }
        }
        if constexpr (OUT == MXO_FP8 || OUT == MXO_FP4) {
          if constexpr (NCH == 3) {
            for (int ch = 0; ch < NCH; ++ch) {
              const int blk = (n0 >> 5) + ch;
              if ((blk >> 2) < okt) p.oscales[mx_scale_word(row, blk >> 2, okt) + (blk & 3)] = (uint8_t)(word >> (8 * ch));
            }
          } else if ((n0 >> 7) < okt) {  // scales of this warp's columns; 0 beyond the tensor
            uint8_t* dst = p.oscales + mx_scale_word(row, n0 >> 7, okt) + ((n0 >> 5) & 3);
            if (NCH == 4 && nch == 4) *reinterpret_cast<uint32_t*>(dst) = word;
            if (NCH == 2 || (NCH == 4 && nch == 2)) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)word;
            if (NCH == 1) *dst = (uint8_t)word;
          }
        }
      } else if (!overlaps || holds) {
        release();
      }
      __syncwarp();  // the bias is read
      if (*abort_flag) break;
    }
    if (lane == 0) bulk_wait_all();  // the boxes outlive the stores, and the results are in memory
  }

  // every role ends here with its warp converged again, so the barrier counts each warp once
  __syncwarp();
  tc_fence_before();
  if constexpr (SPLIT) {
    cluster_sync_all();  // all sums are here; nobody writes to this CTA any more
    join_rows<OUT>(p, smem + S::OUT_OFF, parts, (cl % p.num_m) * S::TM + part * (128 / parts), (cl / p.num_m) * BN,
                   reinterpret_cast<const float4*>(smem + S::OUT_OFF + 8 * BOX_BYTES));
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      // both CTAs are past their last TMEM access before the pair's allocation is released
      if (lane == 0) {
        mbar_arrive_cluster(mapa_shared(smem_u32(dealloc_bar), rank ^ 1u));
        drain_wait(dealloc_bar, 0);
      }
      __syncwarp();
      tc_fence_after();
      tmem_dealloc_pair(tmem_base, S::TMEM_COLS);
    } else {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem_base, S::TMEM_COLS);
    }
  }
}

// Of the 256-column tiles, those taken whole: where the last round would leave half of the CTA
// pairs idle, its tiles are taken as halves.
int wide_tiles(long tiles, int slots) {
  const long rest = tiles % slots;
  return (int)(2 * rest <= slots ? tiles - rest : tiles);
}

template <MxFormat F, int BN, bool PAIR, int OUT, bool SPLIT>
cudaError_t launch_mx(const MxMaps& maps, MxParams p, int K, int sms, cudaStream_t st) {
  using S = MxShape<F, BN, PAIR>;
  p.nk = (K + S::KB - 1) / S::KB;
  p.last = (K - (p.nk - 1) * S::KB + S::KB / 4 - 1) / (S::KB / 4);
  p.num_m = (p.M + S::TM - 1) / S::TM;
  p.tx = S::TX_BYTES - (128 - gemm_mx_a_rows({BN, PAIR, 1}, p.M)) * 128 * (PAIR ? 2 : 1);
  // a microscaled output's scale tiles are written whole: tiles up to the next multiple of 128
  const int ncols = OUT >= MXO_FP8 ? (p.N + 127) / 128 * 128 : p.N;
  const long tiles = (long)p.num_m * ((ncols + BN - 1) / BN);
  if (tiles > 0x3fffffffL) return cudaErrorInvalidValue;
  const int cluster = PAIR ? 2 : SPLIT ? p.split : 1;
  // a CTA that shares its tile takes no second one
  const int slots = SPLIT ? (int)tiles : sms / cluster;
  p.wide = BN == 256 ? wide_tiles(tiles, slots) : (int)tiles;
  p.ntiles = p.wide + 2 * ((int)tiles - p.wide);
  const int grid = p.ntiles < slots ? p.ntiles : slots;
  // the kernel's shared memory, once on each device; only kernels in use are loaded
  static std::atomic<uint64_t> prepared{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (e == cudaSuccess && !(prepared.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(gemm_mx_kernel<F, BN, PAIR, OUT, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)S::SMEM);
    if (e == cudaSuccess) prepared.fetch_or(bit, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster * grid);
  cfg.blockDim = dim3(MXG_THREADS);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemm_mx_kernel<F, BN, PAIR, OUT, SPLIT>, maps.a, maps.w, maps.sa, maps.sw, maps.o, p);
}

template <MxFormat F, int BN, bool PAIR, bool SPLIT>
cudaError_t launch_out(const MxMaps& maps, const MxParams& p, int K, int out, int sms, cudaStream_t st) {
  switch (out) {
    case MXO_F32: return launch_mx<F, BN, PAIR, MXO_F32, SPLIT>(maps, p, K, sms, st);
    case MXO_BF16: return launch_mx<F, BN, PAIR, MXO_BF16, SPLIT>(maps, p, K, sms, st);
    case MXO_FP8: return launch_mx<F, BN, PAIR, MXO_FP8, SPLIT>(maps, p, K, sms, st);
    default: return launch_mx<F, BN, PAIR, MXO_FP4, SPLIT>(maps, p, K, sms, st);
  }
}

}  // namespace

// Every tile shape, for X(BN, PAIR, SPLIT)
#define FH_MX_TILES(X) \
  X(64, false, true) X(64, false, false) X(128, false, false) X(128, true, false) X(192, true, false) X(256, true, false)

// The tile shape with the least estimated time. Tiles are dealt out in rounds, one per CTA or CTA
// pair; a round takes a fixed part and a part per stage, measured in back-to-back launches of
// 4096 x 4096 x {4096 mxfp8, 8192 mxfp4}, 8640 x 4608 x 1536 mxfp8 and 23040 x 8960 x 1536 mxfp4
// (us): wide tiles read fewer operand bytes per MMA and win where there are many rounds (the
// last shape: 146 us at 256 columns on pairs, 159 at 128), narrow ones where a round of wide ones
// would leave SMs idle (1280 x 1536 x 8960 mxfp4: 11.0 us at 128 columns, 14.4 at 256). Where even
// those leave most SMs idle, CTAs share a tile, which costs them 2.5 us, 3.5 where eight of one GPC
// have to start together (1 x 64 x 8960 mxfp8: 18.7 us on one CTA, 10.9, 7.5 and 5.5 on two, four
// and eight; 100 x 1536 x 8960: 18.9, 12.1 on two and 9.4 on four; but 437 x 1008 x 1568 5.8 on one
// and 6.9 on two, and 100 x 1000 x 2048 mxfp4 4.5 on one and 10.3 on eight, 128 CTAs in all).
MxTile gemm_mx_tile(int M, int N, int K, int fmt, int sms) {
  static const struct {
    MxTile t;
    float stage[2], fixed;
  } shapes[] = {{{64, false, 1}, {0.238f, 0.252f}, 0.33f},
                {{128, false, 1}, {0.270f, 0.283f}, 0.45f},
                {{128, true, 1}, {0.234f, 0.228f}, 0.52f},
                {{192, true, 1}, {0.281f, 0.324f}, 0.75f},
                {{256, true, 1}, {0.336f, 0.326f}, 1.45f}};
  const int kb = fmt == MX_FP8 ? 128 : 256, nk = (K + kb - 1) / kb;
  MxTile best = shapes[0].t;
  float least = 0.f;
  for (const auto& s : shapes) {
    const int tm = s.t.pair ? 256 : 128, slots = s.t.pair ? sms / 2 : sms;
    if (slots < 1 || (s.t.pair && M <= 128)) continue;  // a pair's second CTA would have no rows
    const long tiles = (long)((M + tm - 1) / tm) * ((N + s.t.bn - 1) / s.t.bn);
    float us = (float)((tiles + slots - 1) / slots) * (nk * s.stage[fmt] + s.fixed);
    if (s.t.bn == 256 && wide_tiles(tiles, slots) < tiles)  // the last round is one of 128 columns
      us = (float)(tiles / slots) * (nk * s.stage[fmt] + s.fixed) + nk * shapes[2].stage[fmt] + shapes[2].fixed;
    if (least == 0.f || us < least) {
      least = us;
      best = s.t;
    }
  }
  const long tiles = (long)((M + 127) / 128) * ((N + 127) / 128 * 2);
  for (int split = 2; split <= 8; split *= 2) {
    const float us = (float)((nk + split - 1) / split) * shapes[0].stage[fmt] + shapes[0].fixed + (split == 8 ? 3.5f : 2.5f);
    if (split <= nk && tiles * split <= (split == 8 ? sms / 2 : sms) && us < least) {
      least = us;
      best = MxTile{64, false, split};
    }
  }
  return best;
}

// Rows of A that a load brings: not the 127 past a single one, which take as long to fill with zeros
// as they would to read (1 x 9216 x 1536 mxfp8: 9.0 us with them). What lies in the other rows of
// shared memory makes results of rows that no one stores.
int gemm_mx_a_rows(MxTile t, int M) { return t.pair || M >= 128 ? 128 : (M + 7) / 8 * 8; }

int gemm_mx_out_row_bytes(MxTile t, int out_kind) { return box_row_bytes(out_kind, t.bn / 2); }

cudaError_t gemm_mx(const MxMaps& maps, MxTile t, const float* bias, void* out, void* oscales, int M, int N, int K,
                    int fmt, bool gelu, int out_kind, int sms, unsigned* err, cudaStream_t st) {
  MxParams p = {};
  p.err = err;
  p.bias = bias;
  p.out = out;
  p.oscales = (uint8_t*)oscales;
  p.M = M;
  p.N = N;
  p.gelu = gelu;
  p.tma = gemm_mx_tma_out(N, out_kind);
  p.split = t.split;
#define FH_X(BNV, PAIRV, SPLITV)                                                                      \
  if (t.bn == BNV && t.pair == PAIRV && (t.split > 1) == SPLITV)                                      \
    return fmt == MX_FP8 ? launch_out<MX_FP8, BNV, PAIRV, SPLITV>(maps, p, K, out_kind, sms, st)      \
                         : launch_out<MX_FP4, BNV, PAIRV, SPLITV>(maps, p, K, out_kind, sms, st);
  FH_MX_TILES(FH_X)
#undef FH_X
  return cudaErrorInvalidValue;
}

}  // namespace fh
