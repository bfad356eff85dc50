// Matrix product with bias, activation and residual in its epilogue, and its
// backward pass (gfx950):
//
//     u = x w^T + bias        y = act(u) + residual
//     du = dy act'(u)         dx = du w     dw = du^T x     dbias = sum over rows of du
//
// Every product is one form: C[m][n] = sum_r P[m][r] Q[n][r], each operand in
// memory either by its rows (r contiguous, as x and w in the forward) or by the
// reduction axis (m or n contiguous, as w, x and du in the backward), with rows
// a whole number of 16-byte vectors apart. Operands of other widths are first
// copied into the workspace, padded with zeros.
#include <cmath>
#include <type_traits>
#include <utility>

#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

// Most rows of rows_kernel; 16-bit weights above kFewRowsBytes half as many.
// Against the tiles with a split reduction (us): bf16 4096 x 4096, 16 rows 9.5
// and 12.5, 32 rows 13.1 and 13.5; bf16 4096 x 8192, 16 rows 18.4 and 18.2, 32
// rows 24.1 and 18.4; e4m3 16384 x 4096, 32 rows 14.4 and 17.9; fp32 4096 x
// 4096, 32 rows 25 and 40.
constexpr int kFewRows = 32;
constexpr int64_t kFewRowsBytes = int64_t{32} << 20;
constexpr int kStep = 128;  // bytes of the reduction axis per step

// ---------------------------------------------------------------------------
// epilogue

struct Epilogue {
  const float *x_scale, *w_scale, *bias;  // [M], [N], [N] or null
  const void *residual;                   // [M, N] out_dtype or null
  void *pre, *y;                          // [M, N] out_dtype; pre may be null
  int64_t M;
  int N;
  int act, out_dtype;
};

// 1 / (1 + exp(-u)), see sigmoid() for its ends
__device__ __forceinline__ float act_fwd(float u, int act) {
  switch (act) {
    case 1: return u * sigmoid(u);
    case 2: return 0.5f * u * (1.0f + erff(u * 0.70710678f));
    case 3: return sigmoid(u);
    default: return u;
  }
}

__device__ __forceinline__ float act_slope(float u, int act) {
  switch (act) {
    case 1: {
      const float p = sigmoid(u);
      return p * (1.0f + u * (1.0f - p));
    }
    case 2:  // the normal distribution's integral + u times its density
      return 0.5f * (1.0f + erff(u * 0.70710678f)) +
             u * 0.39894228f * __builtin_amdgcn_exp2f(-0.72134752f * u * u);
    case 3: {
      const float p = sigmoid(u);
      return p * (1.0f - p);
    }
    default: return 1.0f;
  }
}

template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
  typedef f32x4 raw;
  typedef f32x4 mem __attribute__((aligned(4)));
};
template <>
struct Vec4<_Float16> {
  typedef f16x4 raw;
  typedef f16x4 mem __attribute__((aligned(2)));
};
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
template <>
struct Vec4<bf16_t> {
  typedef bf16x4 raw;
  typedef bf16x4 mem __attribute__((aligned(2)));
};

// Four consecutive elements of a row at any alignment, or the first cnt < 4 of
// them (then one by one).
template <typename T>
__device__ __forceinline__ typename Vec4<T>::raw load4_raw(const T *p, int cnt) {
  if (cnt >= 4) return *reinterpret_cast<const typename Vec4<T>::mem *>(p);
  typename Vec4<T>::raw v = __builtin_convertvector(zero4(), typename Vec4<T>::raw);
  typedef decltype(v[0] + 0) any;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < cnt) v[i] = static_cast<any>(io<T>::to_f32(p[i]));
  return v;
}
template <typename T>
__device__ __forceinline__ f32x4 load4(const T *p, int cnt) {
  return __builtin_convertvector(load4_raw(p, cnt), f32x4);
}
template <typename T>
__device__ __forceinline__ void store4(T *p, f32x4 v, int cnt) {
  if (cnt >= 4) {
    *reinterpret_cast<typename Vec4<T>::mem *>(p) =
        __builtin_convertvector(v, typename Vec4<T>::raw);
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < cnt) p[i] = io<T>::from_f32(v[i]);
}

template <typename TO>
__device__ __forceinline__ void epilogue4_as(const Epilogue &e, int64_t m, int n, f32x4 v) {
  const int cnt = e.N - n;
  const size_t at = static_cast<size_t>(m) * e.N + n;
  if (e.w_scale) {
    const float xs = e.x_scale[m];
    const f32x4 ws = load4(e.w_scale + n, cnt);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= xs * ws[i];
  }
  if (e.bias) {
    const f32x4 b = load4(e.bias + n, cnt);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += b[i];
  }
  if (e.pre) store4(static_cast<TO *>(e.pre) + at, v, cnt);
  if (e.act) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_fwd(v[i], e.act);
  }
  if (e.residual) {
    const f32x4 r = load4(static_cast<const TO *>(e.residual) + at, cnt);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += r[i];
  }
  store4(static_cast<TO *>(e.y) + at, v, cnt);
}

// u[m][n .. n + 3] (n a multiple of 4, m < M, n < N) through the epilogue
__device__ __forceinline__ void epilogue4(const Epilogue &e, int64_t m, int n, f32x4 v) {
  if (e.out_dtype == 1) epilogue4_as<bf16_t>(e, m, n, v);
  else if (e.out_dtype == 2) epilogue4_as<_Float16>(e, m, n, v);
  else epilogue4_as<float>(e, m, n, v);
}

// ---------------------------------------------------------------------------
// tile kernel

// f(0), f(1), .. f(N - 1) with constant arguments, whatever the code's size
template <int... I, typename F>
__device__ __forceinline__ void unrolled_(std::integer_sequence<int, I...>, F &&f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unrolled(F &&f) {
  unrolled_(std::make_integer_sequence<int, N>{}, f);
}

// eight e4m3 values as fp16
__device__ __forceinline__ f16x8 widen_e4m3(uint32_t lo, uint32_t hi) {
  struct Quad {
    f16x2 v[4];
  } q;
  q.v[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  q.v[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  q.v[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  q.v[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return __builtin_bit_cast(f16x8, q);
}

// acc += A B over the 32 bytes of the reduction axis that the lane holds of
// one operand row, two 16-byte vectors, in PIECES matrix instructions. The
// lanes lg = 0..3 of a row hold bytes 16 lg and 64 + 16 lg of the 128-byte
// step; the matrix cores pair the operands slot by slot, so any assignment of
// reduction indices to slots that both operands share gives the product.
//
// The 8-bit matrix instructions take the products of a lane's 8 consecutive
// bytes together, each cut off 13 bits below the largest's exponent (observed
// on the card; the 16x16x32 and 16x16x128 forms alike): relative errors of
// about 1.5e-5 of the result, well under the rounding of a 16-bit output, but
// not of an fp32 one. EXACT widens e4m3 to fp16 (which holds every e4m3
// value) and uses the 16-bit instructions, whose sums are good to fp32.
template <typename T, bool EXACT>
struct Mma {
  static constexpr int PIECES = __is_same(T, float) ? 8 : !__is_same(T, e4m3_t) ? 2 : EXACT ? 4 : 1;
  __device__ static __forceinline__ f32x4 piece(const u32x4 (&a)[2], const u32x4 (&b)[2], f32x4 acc,
                                                int p) {
    if constexpr (__is_same(T, bf16_t)) {
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(bf16x8, a[p]), __builtin_bit_cast(bf16x8, b[p]), acc, 0, 0, 0);
    } else if constexpr (__is_same(T, _Float16)) {
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a[p]),
                                                    __builtin_bit_cast(f16x8, b[p]), acc, 0, 0, 0);
    } else if constexpr (__is_same(T, float)) {
      return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[p / 4][p % 4]),
                                                  __uint_as_float(b[p / 4][p % 4]), acc, 0, 0, 0);
    } else if constexpr (EXACT) {
      const int q = 2 * (p % 2);
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(widen_e4m3(a[p / 2][q], a[p / 2][q + 1]),
                                                    widen_e4m3(b[p / 2][q], b[p / 2][q + 1]), acc,
                                                    0, 0, 0);
    } else {
      struct Pair {
        u32x4 v[2];
      };
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          __builtin_bit_cast(i32x8, Pair{{a[0], a[1]}}),
          __builtin_bit_cast(i32x8, Pair{{b[0], b[1]}}), acc, 0, 0, 0, 0, 0, 0);  // no block scales
    }
  }
  __device__ static __forceinline__ f32x4 step(const u32x4 (&a)[2], const u32x4 (&b)[2], f32x4 acc) {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) acc = piece(a, b, acc, p);
    return acc;
  }
};

// One matrix instruction of Mma with the accumulator updated in place:
// part 0 or 1 (8-bit types have one part). Written in asm, with the
// accumulator in the accumulation registers: from the builtins the compiler
// moves accumulators between registers around a kernel that fills them all.
// The compiler knows no wait states around it: s_nop 1 covers operands that
// were just written by a VALU instruction, and settle() below has to stand
// between the last product and any other use of the accumulators.
template <typename T>
__device__ __forceinline__ void mma_part(const i32x8 &a, const i32x8 &b, f32x4 &acc, int part) {
  if constexpr (__is_same(T, e4m3_t)) {
    asm("s_nop 1\n\tv_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
  } else {
    const i32x4 a4 = part ? __builtin_shufflevector(a, a, 4, 5, 6, 7)
                          : __builtin_shufflevector(a, a, 0, 1, 2, 3);
    const i32x4 b4 = part ? __builtin_shufflevector(b, b, 4, 5, 6, 7)
                          : __builtin_shufflevector(b, b, 0, 1, 2, 3);
    if constexpr (__is_same(T, bf16_t))
      asm("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a4), "v"(b4));
    else
      asm("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a4), "v"(b4));
  }
}
__device__ __forceinline__ void settle(f32x4 (&c)[8]) {
  asm volatile("s_nop 15\n\ts_nop 3"
               : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3]), "+a"(c[4]), "+a"(c[5]),
                 "+a"(c[6]), "+a"(c[7]));
}

// Workgroups are dealt round robin to the 8 XCDs, each with an L2 of its own:
// XCD x takes a run of consecutive tiles, ordered so that the 32 tiles that
// its CUs work on at a time are 8 row tiles by 4 column tiles.
struct TileAt {
  int64_t m;
  int n;
};
__device__ __forceinline__ TileAt tile_at(int64_t tiles_m, int tiles_n) {
  const uint32_t total = gridDim.x, x = blockIdx.x % 8, slot = blockIdx.x / 8;
  const uint32_t q = total / 8, r = total % 8;
  const uint32_t t = x * q + (x < r ? x : r) + slot;
  const uint32_t group = t / (8 * tiles_n), in = t % (8 * tiles_n);
  const int64_t left = tiles_m - static_cast<int64_t>(group) * 8;
  const uint32_t rows = left < 8 ? static_cast<uint32_t>(left) : 8;
  return {static_cast<int64_t>(group) * 8 + in % rows, static_cast<int>(in / rows)};
}

struct GemmArgs {
  const char *p, *q;         // operands: [M] rows, [N] rows
  int64_t ldp, ldq;          // bytes between rows, multiples of 16
  int64_t M;
  int N;
  int64_t rbytes;            // bytes of the reduction axis (by rows: with padding, whole vectors)
  int64_t red;               // its indices
  int steps;                 // kStep-byte steps per split
  float *part;               // null: epilogue; else [splits][M][ldpart] sums
  int64_t ldpart;
  int64_t tiles_m;
  int tiles_n;
  Epilogue e;
};

// One operand of a tile: TILE rows (outputs) by a stage of 128 bytes of the
// reduction axis (64 16-bit or 32 fp32 indices), loaded straight to LDS by four
// waves, 1 KiB an instruction: lane L's 16 bytes land at byte 16 L. What lane L
// fetches is permuted so that the fragment reads touch all banks evenly.
//
// BYRED false: rows of 128 bytes, 8 an instruction; vector v of row r lies at
// v ^ (r % 8). BYRED true: reduction index k is a row of TILE elements; its
// 16-bit elements lie with 32-byte group u at u ^ (k % 4 + 4 (k / 8 % 2)), fp32
// ones with 64-byte group u at u ^ (k / 4 % 4).
//
// A lane's fragment of output row c (lane % 16 of a group of 16) holds, as
// vector `part` (0 or 1), the reduction bytes 64 part + 16 (lane / 16) .. + 15
// of the stage. By rows that is one 16-byte read; by the reduction axis, 16-bit
// elements come through the transposing LDS read, 4 indices of 16 outputs at a
// time, and fp32 ones one by one.
template <typename T, int TILE, bool BYRED>
struct Operand {
  static constexpr int ES = sizeof(T);
  static constexpr int BYTES = TILE * kStep;
  static constexpr int LOADS = TILE / 32;            // per wave and stage
  static constexpr int RB = BYRED ? TILE * ES : kStep;  // bytes of a row in LDS
  static constexpr int VPR = RB / 16;                // vectors of a row
  static constexpr int INDICES = kStep / ES;         // reduction indices of a stage
  static constexpr int GROUPS = TILE / 32;           // 16-row groups of a wave

  i32x4 rsrc;
  const char *base;
  int64_t ld, bytes;        // BYRED: pitch, bytes from base to the operand's end
  uint32_t off[LOADS];
  uint32_t vec, r;
  int rbytes;
  uint32_t at;              // LDS byte of the operand in stage 0
  uint32_t frag[BYRED && ES == 2 ? GROUPS : 1];
  uint32_t wbase;

  // rows [o0, o0 + TILE) of `outs`; w0: the wave's first row of the tile
  __device__ __forceinline__ void init(const char *p, int64_t pitch, int64_t o0, int64_t outs,
                                       int64_t red_bytes, int64_t red, uint32_t lds, int lane,
                                       int wave, int w0) {
    const int lc = lane % 16, lg = lane / 16;
    at = lds;
    ld = pitch;
    if constexpr (BYRED) {
      base = p + o0 * ES;
      bytes = red * pitch - o0 * ES;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int at16 = (wave + 4 * i) * 64 + lane, k = at16 / VPR, v = at16 % VPR;
        const int x = ES == 2 ? 2 * (k % 4 + 4 * (k / 8 % 2)) : 4 * (k / 4 % 4);
        off[i] = static_cast<uint32_t>(k * pitch + (v ^ x) * 16);
      }
      if constexpr (ES == 2) {
        const int f = lc / 4 + 4 * (lg & 1);
#pragma unroll
        for (int q = 0; q < GROUPS; ++q)
          frag[q] = (8 * lg + lc / 4) * RB + ((w0 / 16 + q) ^ f) * 32 + (lc % 4 / 2) * 16 +
                    (lc & 1) * 8;
      } else {
        frag[0] = 4 * lg * RB + lc * 4;
        wbase = w0 / 16;
      }
    } else {
      // rows past the operand's end lie past the resource's end and read as zeros
      const int64_t rows = outs - o0 < TILE ? outs - o0 : TILE;
      rsrc = buffer_rsrc(p + o0 * pitch, static_cast<uint32_t>(rows * pitch));
      vec = ((lane % 8) ^ (lane / 8)) * 16;
      rbytes = static_cast<int>(red_bytes);
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        off[i] = static_cast<uint32_t>(((wave + 4 * i) * 8 + lane / 8) * pitch);
      frag[0] = lc * 128 + ((lg ^ (lc & 7)) * 16);
      wbase = w0 * 128;
    }
  }
  // stage s is loaded next; `valid` false: zeros. So are bytes past the axis.
  __device__ __forceinline__ void stage(int s, bool valid) {
    if constexpr (BYRED) {
      const int64_t skip = static_cast<int64_t>(s) * INDICES * ld;
      const int64_t left = valid ? bytes - skip : 0;
      rsrc = buffer_rsrc(base + skip, static_cast<uint32_t>(
                                          left < 0 ? 0 : left < 0x40000000 ? left : 0x40000000));
    } else {
      r = s * kStep + vec;
      if (!valid || static_cast<int>(r) >= rbytes) r = 0x80000000u;
    }
  }
  __device__ __forceinline__ void load(int i, uint32_t stage_off, int wave) {
    dma16(rsrc, BYRED ? off[i] : off[i] + r, at + stage_off + (wave + 4 * i) * 1024);
  }
  // vector `part` of the fragment of the wave's row group q
  __device__ __forceinline__ i32x4 read(const char *smem, uint32_t stage_off, int q,
                                        int part) const {
    const char *from = smem + (at - lds_addr(smem)) + stage_off;
    if constexpr (!BYRED) {
      return *reinterpret_cast<const i32x4 *>(from + wbase + 16 * q * 128 + (frag[0] ^ (64 * part)));
    } else if constexpr (ES == 2) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4 lds4;
      struct Two {
        s16x4 v[2];
      } two;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        two.v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds4 *)(from + frag[q] + (32 * part + 4 * h) * RB));
      return __builtin_bit_cast(i32x4, two);
    } else {
      i32x4 x;
      const int lg = threadIdx.x % 64 / 16;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = *reinterpret_cast<const int32_t *>(from + frag[0] + (16 * part + e) * RB +
                                                  ((wbase + q) ^ lg) * 64);
      return x;
    }
  }
};

// Epilogue of a wave's 16 G x 16 G of C: the lane holds rows
// m + 16 j, columns n + 16 i .. + 3. All of the residual and the scales are
// requested first, so that their latency is paid once.
template <typename TO, int ACT, int G>
__device__ __forceinline__ void epilogue_tile_act(const Epilogue &e, f32x4 (&acc)[G][G], int64_t m,
                                                  int n) {
  typedef typename Vec4<TO>::raw raw;
  raw res[G][G];
  float xs[G];
  f32x4 ws[G], b[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int64_t row = m + 16 * j < e.M ? m + 16 * j : e.M - 1;
    if (e.w_scale) xs[j] = e.x_scale[row];
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (e.residual && n + 16 * i < e.N)
        res[i][j] = load4_raw(static_cast<const TO *>(e.residual) + row * e.N + n + 16 * i,
                              e.N - n - 16 * i);
  }
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const bool in = n + 16 * i < e.N;
    ws[i] = in && e.w_scale ? load4(e.w_scale + n + 16 * i, e.N - n - 16 * i) : zero4();
    b[i] = in && e.bias ? load4(e.bias + n + 16 * i, e.N - n - 16 * i) : zero4();
  }
#pragma unroll
  for (int j = 0; j < G; ++j) {
    if (m + 16 * j >= e.M) break;
    const size_t at = static_cast<size_t>(m + 16 * j) * e.N + n;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (n + 16 * i >= e.N) break;
      f32x4 v = acc[i][j];
      if (e.w_scale) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= xs[j] * ws[i][k];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += b[i][k];
      if (e.pre) store4(static_cast<TO *>(e.pre) + at + 16 * i, v, e.N - n - 16 * i);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = act_fwd(v[k], ACT);
      if (e.residual) {
        const f32x4 x = __builtin_convertvector(res[i][j], f32x4);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] += x[k];
      }
      store4(static_cast<TO *>(e.y) + at + 16 * i, v, e.N - n - 16 * i);
    }
  }
}
template <typename TO, int G>
__device__ __forceinline__ void epilogue_tile(const Epilogue &e, f32x4 (&acc)[G][G], int64_t m,
                                              int n) {
  switch (e.act) {
    case 1: epilogue_tile_act<TO, 1>(e, acc, m, n); break;
    case 2: epilogue_tile_act<TO, 2>(e, acc, m, n); break;
    case 3: epilogue_tile_act<TO, 3>(e, acc, m, n); break;
    default: epilogue_tile_act<TO, 0>(e, acc, m, n); break;
  }
}

// One TILE x TILE tile of C (times one split of the reduction) per workgroup
// of four waves, each a quarter of it in 16 x 16 accumulators. A wave reads the
// fragments of the next step, and requests the stage NST steps ahead, between
// the products of this one: read, multiplied and loaded one after the other a
// step took 0.7 us with one workgroup a CU, three times its products' time. At
// the barrier of step s, stage s + 1 has landed and stage s is fully read, so
// the new stage goes over it. Now 0.34 us a step: M1024 N4096 K4096 bf16 38 us
// (0.9 PFLOP/s), M2048 N2048 K8192 e4m3 35 us (2.0). fp32 at 4096^3: 138
// TFLOP/s, the library's rate.
template <typename T, bool EXACT, bool PRED, bool QRED, int TILE, int NST>
__global__ __launch_bounds__(256) void gemm_kernel(const GemmArgs g) {
  constexpr int STAGE = 2 * TILE * kStep, G = TILE / 32;
  __shared__ __attribute__((aligned(1024))) char smem[NST * STAGE];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lc = lane % 16, lg = lane / 16;
  const TileAt at = tile_at(g.tiles_m, g.tiles_n);
  const int64_t m0 = at.m * TILE;
  const int n0 = at.n * TILE;
  const int wm = (wave / 2) * 16 * G, wn = (wave % 2) * 16 * G;

  Operand<T, TILE, PRED> P;
  Operand<T, TILE, QRED> Q;
  P.init(g.p, g.ldp, m0, g.M, g.rbytes, g.red, lds_addr(smem), lane, wave, wm);
  Q.init(g.q, g.ldq, n0, g.N, g.rbytes, g.red, lds_addr(smem) + TILE * kStep, lane, wave, wn);
  const int s0 = blockIdx.y * g.steps;
  const int total = static_cast<int>((g.rbytes + kStep - 1) / kStep);
  const int s1 = s0 + g.steps < total ? s0 + g.steps : total;
  // load i of the stage set by next(), to buffer buf; past the split zeros are
  // loaded (without traffic), so that as many loads are in flight at every step
  constexpr int LOADS = 2 * G, READS = 4 * G;
  auto next = [&](int s) {
    P.stage(s, s < s1);
    Q.stage(s, s < s1);
  };
  auto load = [&](int buf, int i) {
    if (i % 2) Q.load(i / 2, buf * STAGE, wave);
    else P.load(i / 2, buf * STAGE, wave);
  };
  struct Frags {
    u32x4 a[G][2], b[G][2];
  } F[2];
  auto read = [&](Frags &f, int buf, int i) {
    const int q = i / 4, h = i % 2;
    if (i / 2 % 2) f.a[q][h] = __builtin_bit_cast(u32x4, Q.read(smem, buf * STAGE, q, h));
    else f.b[q][h] = __builtin_bit_cast(u32x4, P.read(smem, buf * STAGE, q, h));
  };

  f32x4 acc[G][G];  // [n tile][m tile]
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int j = 0; j < G; ++j) acc[i][j] = zero4();

  auto step = [&](int s, auto par) {
    constexpr int B = decltype(par)::value;  // stage s % NST
    const Frags &cur = F[B % 2];
    Frags &nxt = F[(B + 1) % 2];
    wait_vmcnt<(NST - 2) * LOADS>();
    wg_barrier();
    next(s + NST);
    constexpr int PIECES = Mma<T, EXACT>::PIECES, TOTAL = PIECES * G * G;
    unrolled<TOTAL>([&](auto at_k) {
      constexpr int k = decltype(at_k)::value;
      constexpr int p = k / (G * G), i = k / G % G, j = k % G;
      acc[i][j] = Mma<T, EXACT>::piece(cur.a[i], cur.b[j], acc[i][j], p);
      constexpr int R0 = k * READS / TOTAL, L0 = k * LOADS / TOTAL;
      unrolled<(k + 1) * READS / TOTAL - R0>(
          [&](auto r) { read(nxt, (B + 1) % NST, R0 + decltype(r)::value); });
      unrolled<(k + 1) * LOADS / TOTAL - L0>([&](auto r) { load(B, L0 + decltype(r)::value); });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  if (s0 < s1) {
#pragma unroll
    for (int s = 0; s < NST; ++s) {
      next(s0 + s);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) load(s, i);
    }
    wait_vmcnt<(NST - 1) * LOADS>();
    wg_barrier();
#pragma unroll
    for (int i = 0; i < READS; ++i) read(F[0], 0, i);
    // NST steps at a time; those past the end multiply zeros
    for (int s = s0; s < s1; s += NST) {
      step(s, std::integral_constant<int, 0>{});
      step(s + 1, std::integral_constant<int, 1>{});
      if constexpr (NST == 4) {
        step(s + 2, std::integral_constant<int, 2>{});
        step(s + 3, std::integral_constant<int, 3>{});
      }
    }
    wait_vmcnt<0>();  // no load may land in LDS that is no longer this workgroup's
  }

  const int64_t m = m0 + wm + lc;
  const int n = n0 + wn + 4 * lg;
  if (g.part) {
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (m + 16 * j < g.M && n + 16 * i < g.N)
          *reinterpret_cast<f32x4 *>(g.part +
                                     (static_cast<size_t>(blockIdx.y) * g.M + m + 16 * j) * g.ldpart +
                                     n + 16 * i) = acc[i][j];
  } else if (g.e.out_dtype == 1) {
    epilogue_tile<bf16_t>(g.e, acc, m, n);
  } else if (g.e.out_dtype == 2) {
    epilogue_tile<_Float16>(g.e, acc, m, n);
  } else {
    epilogue_tile<float>(g.e, acc, m, n);
  }
}

__device__ __forceinline__ float readlane(float x, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l));
}

// Epilogue of 8 rows of C, m .. m + 7, by one wave: columns n .. n + 3 of each
// per lane, the products in LDS at rows + r * ldc, the residual in registers.
// Rows are uniform, so their addresses are scalar.
template <typename TO, int ACT>
__device__ __forceinline__ void epilogue_rows8(const Epilogue &e, const float *rows, int ldc,
                                               int64_t m, int n, float xs, int xlane, f32x4 ws,
                                               f32x4 b, const typename Vec4<TO>::raw (&res)[8]) {
  f32x4 v[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) v[r] = *reinterpret_cast<const f32x4 *>(rows + r * ldc);
  // one branch a step for all rows: branches in every row took twice the time
  if (e.w_scale) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float x = readlane(xs, xlane + r);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[r][i] *= x * ws[i];
    }
  }
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[r][i] += b[i];
  const int cnt = e.N - n, left = e.M - m < 8 ? static_cast<int>(e.M - m) : 8;
  auto store_rows = [&](void *out) {
    TO *to = static_cast<TO *>(out) + m * e.N;
    if (left == 8 && cnt >= 4) {
#pragma unroll
      for (int r = 0; r < 8; ++r, to += e.N) store4(to + n, v[r], 4);
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r, to += e.N)
        if (r < left) store4(to + n, v[r], cnt);
    }
  };
  if (e.pre) store_rows(e.pre);
  if (ACT) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[r][i] = act_fwd(v[r][i], ACT);
      // two rows at a time: more side by side would spill
      if (r % 2) __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (e.residual) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const f32x4 x = __builtin_convertvector(res[r], f32x4);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[r][i] += x[i];
    }
  }
  store_rows(e.y);
}

// Epilogue of one wave's part of a tile: twice 32 rows, from row
// m + hstep * half, staged to LDS at `rows` by stage(half). The
// residual of 8 rows is requested two groups of 8 ahead.
template <typename TO, typename F>
__device__ __forceinline__ void epilogue_wave(const Epilogue &e, const float *rows, int ldc,
                                              int64_t m, int hstep, int n, F &&stage) {
  typedef typename Vec4<TO>::raw raw;
  const bool in = n < e.N;
  f32x4 ws = zero4(), b = zero4();
  if (in && e.w_scale) ws = load4(e.w_scale + n, e.N - n);
  if (in && e.bias) b = load4(e.bias + n, e.N - n);
  // x_scale of row r of half h in lane 32 h + r
  float xs = 0.0f;
  if (e.w_scale) {
    const int lane = threadIdx.x % 64;
    const int64_t row = m + hstep * (lane / 32) + lane % 32;
    xs = e.x_scale[row < e.M ? row : e.M - 1];
  }
  // the residual of the 8 rows at hand and of the next two groups of 8
  raw res[8], next[8], after[8];
  auto fetch = [&](int group) {  // 0 .. 7: four groups per half
    if (!e.residual || !in || group >= 8) return;
    const int64_t at = m + hstep * (group / 4) + 8 * (group % 4);
    const TO *from[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      from[r] = static_cast<const TO *>(e.residual) + (at + r < e.M ? at + r : e.M - 1) * e.N;
    if (e.N - n >= 4) {
#pragma unroll
      for (int r = 0; r < 8; ++r) after[r] = load4_raw(from[r] + n, 4);
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r) after[r] = load4_raw(from[r] + n, e.N - n);
    }
  };
  auto shift = [&]() {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      res[r] = next[r];
      next[r] = after[r];
    }
  };
  fetch(0);
  shift();
  fetch(1);
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    stage(half);
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const int64_t at = m + hstep * half + 8 * q;
      shift();
      fetch(4 * half + q + 2);
      if (!in) continue;
      const float *from = rows + 8 * q * ldc;
      const int xl = 32 * half + 8 * q;
      switch (e.act) {
        case 1: epilogue_rows8<TO, 1>(e, from, ldc, at, n, xs, xl, ws, b, res); break;
        case 2: epilogue_rows8<TO, 2>(e, from, ldc, at, n, xs, xl, ws, b, res); break;
        case 3: epilogue_rows8<TO, 3>(e, from, ldc, at, n, xs, xl, ws, b, res); break;
        default: epilogue_rows8<TO, 0>(e, from, ldc, at, n, xs, xl, ws, b, res); break;
      }
    }
  }
}

// Row groups 4 HALF .. 4 HALF + 3 of the accumulators to LDS, straight from
// the accumulation registers (the barrier that follows waits for it).
template <int HALF, int LDC>
__device__ __forceinline__ void store_half(uint32_t to, const f32x4 (&acc)[8][8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm volatile("ds_write_b128 %0, %1 offset:%2" ::"v"(to), "a"(acc[i][4 * HALF + j]),
                   "n"((16 * j * LDC + 16 * i) * 4)
                   : "memory");
}

// The large tile: 256 x 256 of C by four waves, each 128 x 128 of it (256
// accumulator registers), so that a step's LDS reads (4 x 32 KB) and direct
// loads (64 KB) take 1536 of the 2048 clocks its products take at the 128
// bytes a clock of LDS. One wave per SIMD: nothing hides a stall but the wave
// itself, so everything is ordered by hand. A step of 128 bytes of the
// reduction axis is four quadrants of 64 x 64; A0, A1 (halves of the wave's
// rows of q) and B0, B1 (of p) are read one quadrant before their first use,
// the halves of B in turn first and second so that no register is held twice:
//     (A0 Bf) read Bs | (A0 Bs) read A1 | barrier | (A1 Bs) read A0' | (A1 Bf) read Bs'
// where ' is the next step, whose Bf is this one's Bs. At the barrier the next
// stage has landed and this one is fully read: the stage after next is loaded
// over it, a whole step (about 1 us) ahead of its use. Measured: M16384 N8192
// K2048 bf16 with bias and silu 482 us (1.14 PFLOP/s; products alone 390 us),
// M16384 N4096 K4096 e4m3 with residual 250 us (2.20 PFLOP/s; alone 170 us):
// bound by the matrix cores, then by the epilogue, in which they rest.
struct Half {
  i32x8 v[4];
};

template <typename T, bool PRED, bool QRED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void
gemm256_kernel(const GemmArgs g) {
  constexpr int TILE = 256, STAGE = 2 * TILE * kStep, LDC = TILE + 4;
  constexpr int PARTS = __is_same(T, e4m3_t) ? 1 : 2;  // instructions per tile and step
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE + 128 * 16];
  static_assert(sizeof(smem) >= 128 * LDC * 4, "half a tile of fp32 for the epilogue");
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lc = lane % 16, lg = lane / 16;
  const TileAt at = tile_at(g.tiles_m, g.tiles_n);
  const int64_t m0 = at.m * TILE;
  const int n0 = at.n * TILE;
  const int wm = (wave / 2) * 128, wn = (wave % 2) * 128;

  const uint32_t lds0 = lds_addr(smem);
  Operand<T, TILE, PRED> OP;
  Operand<T, TILE, QRED> OQ;
  OP.init(g.p, g.ldp, m0, g.M, g.rbytes, g.red, lds0, lane, wave, wm);
  OQ.init(g.q, g.ldq, n0, g.N, g.rbytes, g.red, lds0 + TILE * kStep, lane, wave, wn);
  const int s0 = blockIdx.y * g.steps;
  const int total = static_cast<int>((g.rbytes + kStep - 1) / kStep);
  const int s1 = s0 + g.steps < total ? s0 + g.steps : total;
  // load i (0..7: p, 8..15: q) of the stage set by next(); past the split zeros
  auto next = [&](int s) {
    OP.stage(s, s < s1);
    OQ.stage(s, s < s1);
  };
  auto load = [&](int buf, int i) {
    if (i < 8) OP.load(i, buf * STAGE, wave);
    else OQ.load(i - 8, buf * STAGE, wave);
  };

  // 16 bytes of one half's fragments: vector i % 2 of row group i / 2, i = 0..7
  auto put = [&](Half &f, const i32x4 &x, int i) {
    i32x8 &d = f.v[i / 2];
#pragma unroll
    for (int e = 0; e < 4; ++e) d[4 * (i % 2) + e] = x[e];
  };
  auto read_a = [&](Half &f, int buf, int h, int i) {
    put(f, OQ.read(smem, buf * STAGE, 4 * h + i / 2, i % 2), i);
  };
  auto read_b = [&](Half &f, int buf, int h, int i) {
    put(f, OP.read(smem, buf * STAGE, 4 * h + i / 2, i % 2), i);
  };

  f32x4 acc[8][8];  // [n tile][m tile]
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = zero4();

  // one quadrant, with `side(0..7)` spread between its products
  auto quadrant = [&](const Half &a, const Half &b, int ia, int jb, auto &&side) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        mma_part<T>(a.v[t / 4], b.v[t % 4], acc[4 * ia + t / 4][4 * jb + t % 4], p);
        constexpr int EVERY = 2 * PARTS;
        if ((p * 16 + t) % EVERY == EVERY - 1) {
          side((p * 16 + t) / EVERY);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
  };

  Half A0, A1, B0, B1;
  auto step = [&](int s, auto par) {
    constexpr int P = decltype(par)::value;  // stage, and which half of B comes first
    Half &Bf = P ? B1 : B0, &Bs = P ? B0 : B1;
    quadrant(A0, Bf, 0, P, [&](int i) { read_b(Bs, P, 1 - P, i); });
    quadrant(A0, Bs, 0, 1 - P, [&](int i) { read_a(A1, P, 1, i); });
    wait_vmcnt<0>();
    wg_barrier();
    next(s + 2);
    quadrant(A1, Bs, 1, 1 - P, [&](int i) {
      read_a(A0, 1 - P, 0, i);
      load(P, i);
    });
    quadrant(A1, Bf, 1, P, [&](int i) {
      read_b(Bs, 1 - P, 1 - P, i);
      load(P, 8 + i);
    });
  };

  if (s0 < s1) {
    next(s0);
#pragma unroll
    for (int i = 0; i < 16; ++i) load(0, i);
    next(s0 + 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) load(1, i);
    wait_vmcnt<16>();
    wg_barrier();
#pragma unroll
    for (int i = 0; i < 8; ++i) read_a(A0, 0, 0, i);
#pragma unroll
    for (int i = 0; i < 8; ++i) read_b(B0, 0, 0, i);
    // an odd count ends with a step of zeros
    for (int s = s0; s < s1; s += 2) {
      step(s, std::integral_constant<int, 0>{});
      step(s + 1, std::integral_constant<int, 1>{});
    }
    wait_vmcnt<0>();  // no load may land in LDS that is used otherwise, or by others
  }

#pragma unroll
  for (int i = 0; i < 8; ++i) settle(acc[i]);

  // Half of the rows of C at a time through LDS, so that the stores (and the
  // reads of bias and residual) are whole rows of 256 columns: rows 0..63 of
  // the LDS tile are those of waves 0 and 1, 64..127 of waves 2 and 3, and
  // each wave then takes 32 of the 128.
  float *cs = reinterpret_cast<float *>(smem);
  auto stage = [&](int half) {
    wg_barrier();
    const uint32_t to = lds0 + ((wm / 2 + lc) * LDC + wn + 4 * lg) * 4;
    if (half == 0) store_half<0, LDC>(to, acc);
    else store_half<1, LDC>(to, acc);
    wg_barrier();
  };
  const int n = n0 + 4 * lane;
  const int64_t m = m0 + (wave / 2) * 128 + (wave % 2) * 32;  // row of `rows`, + 64 in half 1
  const float *rows = cs + 32 * wave * LDC + 4 * lane;
  if (g.part) {
    for (int half = 0; half < 2; ++half) {
      stage(half);
      if (n >= g.N) continue;
      float *out = g.part + (static_cast<size_t>(blockIdx.y) * g.M + m + 64 * half) * g.ldpart + n;
#pragma unroll 8
      for (int r = 0; r < 32; ++r)
        if (m + 64 * half + r < g.M)
          *reinterpret_cast<f32x4 *>(out + r * g.ldpart) =
              *reinterpret_cast<const f32x4 *>(rows + r * LDC);
    }
  } else if (g.e.out_dtype == 1) {
    epilogue_wave<bf16_t>(g.e, rows, LDC, m, 64, n, stage);
  } else if (g.e.out_dtype == 2) {
    epilogue_wave<_Float16>(g.e, rows, LDC, m, 64, n, stage);
  } else {
    epilogue_wave<float>(g.e, rows, LDC, m, 64, n, stage);
  }
}

// Few rows (decode): C is M <= 16 MT rows by 16 NT columns per workgroup, the
// reduction dealt to its waves in steps of 128 bytes and joined in LDS. Every
// weight byte goes to one wave only, so it is loaded straight to registers,
// 8 KiB a wave in flight; x comes from the L2, once for the NT groups of
// columns. Bound by the weights' HBM traffic: N16384 K4096 e4m3, one row, 15.4 us
// (4.4 TB/s); N4096 K4096 bf16, 8 rows, 8.2 us (the load latency shows).
template <typename T, int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void rows_kernel(const GemmArgs g) {
  constexpr int AHEAD = 4 / NT;
  __shared__ __attribute__((aligned(16))) float part[WAVES][MT * NT][64][4];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lc = lane % 16, lg = lane / 16;
  const int n0 = blockIdx.x * 16 * NT;
  const int nrows = g.N - n0 < 16 * NT ? g.N - n0 : 16 * NT;
  const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char *>(g.q + n0 * g.ldq), 0, static_cast<int>(nrows * g.ldq), 0x00020000);
  const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char *>(g.p), 0, static_cast<int>(g.M * g.ldp), 0x00020000);
  const int total = static_cast<int>((g.rbytes + kStep - 1) / kStep);
  f32x4 acc[NT][MT];
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[q][j] = zero4();
  // rows past N or M, and bytes past the axis, read as zeros
  auto fetch = [&](__amdgpu_buffer_rsrc_t from, int row, int64_t ld, uint32_t r) {
    const uint32_t at = r < g.rbytes ? static_cast<uint32_t>(row * ld) + r : 0x80000000u;
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, at, 0, 0));
  };
  for (int s = wave; s < total; s += WAVES * AHEAD) {
    u32x4 w[AHEAD][NT][2], x[AHEAD][MT][2];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t r = (s + WAVES * i) * kStep + 64 * h + 16 * lg;
#pragma unroll
        for (int q = 0; q < NT; ++q) w[i][q][h] = fetch(rq, 16 * q + lc, g.ldq, r);
#pragma unroll
        for (int j = 0; j < MT; ++j) x[i][j][h] = fetch(rp, 16 * j + lc, g.ldp, r);
      }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[q][j] = Mma<T, true>::step(w[i][q], x[i][j], acc[q][j]);
  }
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int j = 0; j < MT; ++j)
      *reinterpret_cast<f32x4 *>(part[wave][q * MT + j][lane]) = acc[q][j];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * MT * 64; i += 64 * WAVES) {
    const int t = i / 64, l = i % 64;
    f32x4 v = *reinterpret_cast<const f32x4 *>(part[0][t][l]);
#pragma unroll
    for (int k = 1; k < WAVES; ++k) v += *reinterpret_cast<const f32x4 *>(part[k][t][l]);
    const int64_t m = 16 * (t % MT) + l % 16;
    const int n = n0 + 16 * (t / MT) + 4 * (l / 16);
    if (m < g.M && n < g.N) epilogue4(g.e, m, n, v);
  }
}

// partial sums of the splits, added in order, through the epilogue
__global__ __launch_bounds__(256) void join_kernel(const float *__restrict__ part, int splits,
                                                   int64_t ldpart, const Epilogue e) {
  const int64_t quads = ldpart / 4;
  const int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (q >= e.M * quads) return;
  const int64_t m = q / quads;
  const int n = static_cast<int>(q % quads) * 4;
  f32x4 v = *reinterpret_cast<const f32x4 *>(part + m * ldpart + n);
  for (int s = 1; s < splits; ++s)
    v += *reinterpret_cast<const f32x4 *>(part + (static_cast<size_t>(s) * e.M + m) * ldpart + n);
  epilogue4(e, m, n, v);
}

// ---------------------------------------------------------------------------
// operand layout

// dst[r][0 .. pitch) = src[r][0 .. cols) and zeros (E: raw bits of an element):
// a wave takes rows, a lane their 16-byte vectors, read at any alignment
template <typename E>
__global__ __launch_bounds__(256) void pad_rows_kernel(const E *__restrict__ src, int64_t rows,
                                                       int cols, E *__restrict__ dst, int pitch) {
  constexpr int PER = 16 / sizeof(E);
  typedef u32x4 any __attribute__((aligned(1)));
  const int lane = threadIdx.x % 64;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64; r < rows;
       r += static_cast<int64_t>(gridDim.x) * 4) {
    const E *from = src + r * cols;
    E *to = dst + r * pitch;
#pragma unroll 4
    for (int c = lane * PER; c < pitch; c += 64 * PER) {
      if (c + PER <= cols) {
        *reinterpret_cast<u32x4 *>(to + c) = *reinterpret_cast<const any *>(from + c);
      } else {
        for (int i = 0; i < PER; ++i) to[c + i] = c + i < cols ? from[c + i] : E(0);
      }
    }
  }
}

// du[m][0 .. pitch) = dy act'(pre), zeros from N on (du may be null), and the
// column sums of the unrounded du over each run of `run` rows (part may be
// null). A workgroup owns 256 columns of one run: 8 columns of every eighth row
// a thread. HBM-bound: 16384 x 4096 bf16 78 us (5.1 TB/s).
template <typename TG, typename T>
__global__ __launch_bounds__(256) void du_kernel(const TG *__restrict__ dy,
                                                 const TG *__restrict__ pre, int64_t M, int N,
                                                 int act, T *__restrict__ du, int pitch, int run,
                                                 float *__restrict__ part) {
  __shared__ float s[8][257];
  const int g = threadIdx.x % 32, hi = threadIdx.x / 32;
  const int n = blockIdx.x * 256 + 8 * g;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * run;
  const int64_t m1 = m0 + run < M ? m0 + run : M;
  float sum[8] = {};
#pragma unroll 2
  for (int64_t m = m0 + hi; m < m1; m += 8) {
    float v[8];
    load8(dy + m * N, n, N, v);
    if (act) {
      float u[8];
      load8(pre + m * N, n, N, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= act_slope(u[i], act);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += v[i];
    // v is zero from N on (whatever act_slope gives there meets a zero dy)
    if (du) store8(du + m * pitch, n, pitch, v);
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[hi][8 * g + i] = sum[i];
  __syncthreads();
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col < N) {
    float t = s[0][threadIdx.x];
#pragma unroll
    for (int q = 1; q < 8; ++q) t += s[q][threadIdx.x];
    part[static_cast<size_t>(blockIdx.y) * N + col] = t;
  }
}

// ---------------------------------------------------------------------------
// plans

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
int esize(int t) { return t == 0 ? 4 : t == kE4m3 ? 1 : 2; }
int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

template <typename F>
hipError_t with_type(int code, F &&f) {
  switch (code) {
    case 1: return f(bf16_t{});
    case 2: return f(_Float16{});
    default: return f(float{});
  }
}

// One product: the kernel, how the reduction is split and what that needs.
struct GemmPlan {
  int tile;  // 0: rows_kernel
  int64_t tiles_m;
  int tiles_n;
  int splits, steps;
  int64_t ldpart;
  size_t part_bytes;
};

// What a tile kernel costs in us on the whole card: start + rounds of 256
// workgroups * (steps * step + tile), the last two less where part of the CUs
// is idle; a split adds the joining pass. Fitted to timings (bf16, M x N x K,
// us): 1024 x 4096 x 4096 128: 38, 256: 90; 4096 x 4096 x 4096 128: 145, 256:
// 110; 4096 x 4096 x 1024 128: 60, 256: 43; 4096 x 2048 x 8192 128: 131, 256:
// 166, 256 in two splits 123; 1024 x 1024 x 2048 128 in 1, 2, 4 splits: 19.3,
// 16.4, 17.5; 4096 x 512 x 512 128 in 1, 2 splits 10.7, 19.5; fp32 2531 x 1000
// x 520 64: 32, 128: 42.
struct TileCost {
  int tile;
  float start, step, each;
};
constexpr TileCost kCost64F32{64, 7.0f, 0.55f, 3.0f}, kCost128F32{128, 7.0f, 2.0f, 6.0f},
    kCost128{128, 7.0f, 0.44f, 6.0f}, kCost256{256, 4.0f, 1.4f, 18.0f};

GemmPlan plan_gemm(int64_t M, int N, int64_t rbytes, int es, bool large, bool by_rows) {
  GemmPlan best{};
  if (by_rows && M <= (es == 2 && N * rbytes > kFewRowsBytes ? kFewRows / 2 : kFewRows)) {
    best.splits = best.steps = 1;
    return best;
  }
  const int total = static_cast<int>((rbytes + kStep - 1) / kStep);
  const TileCost cand[2] = {es == 4 ? kCost64F32 : kCost128, es == 4 ? kCost128F32 : kCost256};
  float least = 0.0f;
  for (int c = 0; c < (es == 4 || large ? 2 : 1); ++c) {
    GemmPlan p;
    p.tile = cand[c].tile;
    p.tiles_m = (M + p.tile - 1) / p.tile;
    p.tiles_n = (N + p.tile - 1) / p.tile;
    const int64_t tiles = p.tiles_m * p.tiles_n;
    // 1, 2, 3, 4, 6, 8, 12, .. splits while they leave no more workgroups than
    // CUs, nor fewer than four steps each
    for (int want = 1; want == 1 || (want * tiles <= 256 && want * 4 <= total);
         want += want < 4 ? 1 : want % 3 ? want / 2 : want / 3) {
      p.steps = (total + want - 1) / want;
      if (p.steps < 1) p.steps = 1;
      p.splits = total > 0 ? (total + p.steps - 1) / p.steps : 1;
      const float full = static_cast<float>(tiles * p.splits) / 256.0f;
      const float busy = full < 1.0f ? full : 1.0f;
      const float rounds = full < 1.0f ? 1.0f : es == 4 ? full : std::ceil(full);
      float cost = cand[c].start + rounds * (cand[c].step * p.steps * (0.7f + 0.3f * busy) +
                                             cand[c].each * (0.35f + 0.65f * busy));
      if (p.splits > 1) cost += 1.5f + 0.6e-6f * p.splits * M * N;
      if (!best.tile || cost < least) {
        best = p;
        least = cost;
      }
    }
  }
  best.ldpart = (N + 3) / 4 * 4;
  best.part_bytes =
      best.splits > 1 ? align256(static_cast<size_t>(best.splits) * M * best.ldpart * 4) : 0;
  return best;
}

// whether the large tile exists for the types: 16-bit and 8-bit matrix
// instructions (fp32 sums of 8-bit operands are taken by the small one)
bool large_ok(int dtype, int out_dtype) { return dtype != 0 && !(dtype == kE4m3 && out_dtype == 0); }

struct Matrix {
  const void *p;
  int64_t ld;   // bytes
  bool by_red;  // the reduction axis is the slow one
};

// Column groups per workgroup: as many as leave every CU one; where even single
// groups leave CUs idle, more waves share the reduction.
template <typename T, int MT>
hipError_t start_rows(const GemmArgs &g, hipStream_t stream) {
  const int groups = (g.N + 15) / 16;
  if (groups >= 4 * 256)
    hipLaunchKernelGGL((rows_kernel<T, MT, 4, 8>), dim3((groups + 3) / 4), dim3(512), 0, stream, g);
  else if (groups >= 2 * 256)
    hipLaunchKernelGGL((rows_kernel<T, MT, 2, 8>), dim3((groups + 1) / 2), dim3(512), 0, stream, g);
  else if (groups >= 128)
    hipLaunchKernelGGL((rows_kernel<T, MT, 1, 8>), dim3(groups), dim3(512), 0, stream, g);
  else
    hipLaunchKernelGGL((rows_kernel<T, MT, 1, 16>), dim3(groups), dim3(1024), 0, stream, g);
  return hipGetLastError();
}

template <typename T, bool EXACT, bool PRED, bool QRED>
hipError_t start_gemm(const GemmArgs &g, const GemmPlan &p, hipStream_t stream) {
  if constexpr (!PRED && !QRED) {
    if (p.tile == 0)
      return g.M <= 16 ? start_rows<T, 1>(g, stream) : start_rows<T, 2>(g, stream);
  }
  const dim3 grid(static_cast<unsigned>(p.tiles_m * p.tiles_n), p.splits);
  if constexpr (!__is_same(T, float) && (!__is_same(T, e4m3_t) || !EXACT)) {
    if (p.tile == 256) {
      hipLaunchKernelGGL((gemm256_kernel<T, PRED, QRED>), grid, dim3(256), 0, stream, g);
      return hipGetLastError();
    }
  }
  if constexpr (__is_same(T, float)) {
    if (p.tile == 64)
      hipLaunchKernelGGL((gemm_kernel<T, EXACT, PRED, QRED, 64, 2>), grid, dim3(256), 0, stream, g);
    else
      hipLaunchKernelGGL((gemm_kernel<T, EXACT, PRED, QRED, 128, 2>), grid, dim3(256), 0, stream, g);
  } else {
    hipLaunchKernelGGL((gemm_kernel<T, EXACT, PRED, QRED, 128, 4>), grid, dim3(256), 0, stream, g);
  }
  return hipGetLastError();
}

// C = P Q^T through the epilogue: M by N outputs, `red` reduction indices, that
// operands by rows hold padded with zeros to `pitch` of them
hipError_t run_gemm(const Matrix &P, const Matrix &Q, int64_t M, int N, int64_t pitch, int64_t red,
                    int dtype, const Epilogue &e, char *part, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const int64_t rbytes = pitch * esize(dtype);
  const GemmPlan p = plan_gemm(M, N, rbytes, esize(dtype), large_ok(dtype, e.out_dtype), !Q.by_red);
  GemmArgs g;
  g.p = static_cast<const char *>(P.p);
  g.q = static_cast<const char *>(Q.p);
  g.ldp = P.ld;
  g.ldq = Q.ld;
  g.M = M;
  g.N = N;
  g.rbytes = rbytes;
  g.red = red;
  g.steps = p.steps;
  g.part = p.splits > 1 ? reinterpret_cast<float *>(part) : nullptr;
  g.ldpart = p.ldpart;
  g.tiles_m = p.tiles_m;
  g.tiles_n = p.tiles_n;
  g.e = e;
  hipError_t err;
  if (dtype == kE4m3) {
    err = e.out_dtype == 0 ? start_gemm<e4m3_t, true, false, false>(g, p, stream)
                           : start_gemm<e4m3_t, false, false, false>(g, p, stream);
  } else {
    err = with_type(dtype, [&](auto t) {
      using T = decltype(t);
      if (P.by_red) return start_gemm<T, true, true, true>(g, p, stream);
      if (Q.by_red) return start_gemm<T, true, false, true>(g, p, stream);
      return start_gemm<T, true, false, false>(g, p, stream);
    });
  }
  if (err != hipSuccess || !g.part) return err;
  const int64_t quads = M * (p.ldpart / 4);
  hipLaunchKernelGGL(join_kernel, dim3(static_cast<unsigned>((quads + 255) / 256)), dim3(256), 0,
                     stream, g.part, p.splits, p.ldpart, e);
  return hipGetLastError();
}

template <typename F>
void by_size(int es, F &&f) {
  if (es == 4) f(uint32_t{});
  else if (es == 2) f(uint16_t{});
  else f(uint8_t{});
}

hipError_t pad_rows(const void *src, int64_t rows, int cols, void *dst, int pitch, int es,
                    hipStream_t stream) {
  const int64_t blocks = (rows + 3) / 4;
  by_size(es, [&](auto e) {
    using E = decltype(e);
    hipLaunchKernelGGL(pad_rows_kernel<E>, dim3(static_cast<unsigned>(blocks < 8192 ? blocks : 8192)),
                       dim3(256), 0, stream, static_cast<const E *>(src), rows, cols,
                       static_cast<E *>(dst), pitch);
  });
  return hipGetLastError();
}

// forward workspace: padded copies of x and w where K is no whole vector,
// then the partial sums
struct FwdLayout {
  int64_t pitch;  // elements between rows of the operands in use
  bool pad;
  size_t x, w, part, total;
};
FwdLayout fwd_layout(int64_t M, int N, int K, int dtype) {
  const int es = esize(dtype);
  FwdLayout L;
  const int64_t rb = round16(static_cast<int64_t>(K) * es);
  L.pitch = rb / es;
  L.pad = L.pitch != K;
  size_t off = 0;
  L.x = off;
  if (L.pad) off += align256(static_cast<size_t>(M) * rb);
  L.w = off;
  if (L.pad) off += align256(static_cast<size_t>(N) * rb);
  L.part = off;
  // e4m3 inputs: whichever of the tiles for 16-bit and fp32 outputs needs more
  const size_t p1 = plan_gemm(M, N, rb, es, large_ok(dtype, 1), true).part_bytes;
  const size_t p2 = dtype == kE4m3 ? plan_gemm(M, N, rb, es, false, true).part_bytes : 0;
  off += p1 > p2 ? p1 : p2;
  L.total = off;
  return L;
}

constexpr int kDuRuns = 256;  // most runs of rows whose column sums are kept
int du_run(int64_t M) {
  const int64_t r = (M + kDuRuns - 1) / kDuRuns;
  return static_cast<int>(r < 16 ? 16 : r);
}

// backward workspace: du (when it is not dy itself), padded copies of x and w
// where K is no whole vector, partial sums of dbias, partial sums of one
// product at a time
struct BwdLayoutL {
  bool own_du, pad;
  int64_t pn, pk;  // elements between rows of du, and of x and w
  size_t du, x, w, db, part, total;
};
BwdLayoutL bwd_layout(int64_t M, int N, int K, int act, int in_dtype, int dy_dtype) {
  const int es = esize(in_dtype);
  BwdLayoutL L;
  const int64_t rn = round16(static_cast<int64_t>(N) * es);
  const int64_t rk = round16(static_cast<int64_t>(K) * es);
  L.pn = rn / es;
  L.pk = rk / es;
  L.own_du = act != 0 || dy_dtype != in_dtype || L.pn != N;
  L.pad = L.pk != K;
  size_t off = 0;
  L.du = off;
  if (L.own_du) off += align256(static_cast<size_t>(M) * rn);
  L.x = off;
  if (L.pad) off += align256(static_cast<size_t>(M) * rk);
  L.w = off;
  if (L.pad) off += align256(static_cast<size_t>(N) * rk);
  L.db = off;
  off += align256(static_cast<size_t>((M + du_run(M) - 1) / du_run(M)) * N * 4);
  L.part = off;
  const bool large = large_ok(in_dtype, in_dtype);
  const size_t p1 = plan_gemm(M, K, rn, es, large, false).part_bytes;
  const size_t p2 = plan_gemm(N, K, M * es, es, large, false).part_bytes;
  off += p1 > p2 ? p1 : p2;
  L.total = off;
  return L;
}

}  // namespace

size_t linear_workspace_size(int64_t M, int N, int K, int in_dtype) {
  return fwd_layout(M, N, K, in_dtype).total;
}

hipError_t launch_linear(const LinearArgs &a) {
  if (a.M == 0) return hipSuccess;
  const FwdLayout L = fwd_layout(a.M, a.N, a.K, a.in_dtype);
  const int es = esize(a.in_dtype);
  const void *x = a.x, *w = a.w;
  if (L.pad) {
    hipError_t err = pad_rows(a.x, a.M, a.K, a.ws + L.x, static_cast<int>(L.pitch), es, a.stream);
    if (err != hipSuccess) return err;
    err = pad_rows(a.w, a.N, a.K, a.ws + L.w, static_cast<int>(L.pitch), es, a.stream);
    if (err != hipSuccess) return err;
    x = a.ws + L.x;
    w = a.ws + L.w;
  }
  const Epilogue e{a.x_scale, a.w_scale, a.bias, a.residual, a.pre, a.y, a.M, a.N, a.act,
                   a.out_dtype};
  return run_gemm({x, L.pitch * es, false}, {w, L.pitch * es, false}, a.M, a.N, L.pitch,
                  a.K, a.in_dtype, e, a.ws + L.part, a.stream);
}

size_t linear_bwd_workspace_size(int64_t M, int N, int K, int act, int in_dtype, int dy_dtype) {
  return bwd_layout(M, N, K, act, in_dtype, dy_dtype).total;
}

hipError_t launch_linear_bwd(const LinearBwdArgs &a) {
  const BwdLayoutL L = bwd_layout(a.M, a.N, a.K, a.act, a.in_dtype, a.dy_dtype);
  const int es = esize(a.in_dtype);
  const int run = du_run(a.M);
  const int runs = static_cast<int>((a.M + run - 1) / run);
  const void *du = L.own_du ? a.ws + L.du : a.dy;
  // a single run's sums are dbias itself
  float *db = runs == 1 ? a.dbias : reinterpret_cast<float *>(a.ws + L.db);
  hipError_t err = hipSuccess;
  if (a.M > 0 && (L.own_du || a.dbias)) {
    err = with_type(a.in_dtype, [&](auto t) {
      return with_type(a.dy_dtype, [&](auto tg) {
        using T = decltype(t);
        using TG = decltype(tg);
        hipLaunchKernelGGL((du_kernel<TG, T>), dim3(static_cast<unsigned>((L.pn + 255) / 256), runs),
                           dim3(256), 0, a.stream, static_cast<const TG *>(a.dy),
                           static_cast<const TG *>(a.pre), a.M, a.N, a.act,
                           L.own_du ? reinterpret_cast<T *>(a.ws + L.du) : nullptr,
                           static_cast<int>(L.pn), run, a.dbias ? db : nullptr);
        return hipGetLastError();
      });
    });
    if (err != hipSuccess) return err;
  }
  if (a.dbias && runs != 1) {
    err = launch_colsum(db, runs, a.N, a.dbias, a.stream);
    if (err != hipSuccess) return err;
  }
  const int64_t ldn = L.pn * es, ldk = L.pk * es;
  Epilogue e{};
  e.N = a.K;
  e.out_dtype = a.in_dtype;
  if (a.dx && a.M > 0) {
    const void *w = a.w;
    if (L.pad) {
      err = pad_rows(a.w, a.N, a.K, a.ws + L.w, static_cast<int>(L.pk), es, a.stream);
      if (err != hipSuccess) return err;
      w = a.ws + L.w;
    }
    e.M = a.M;
    e.y = a.dx;
    // the reduction stops at N: past it du has zeros, but w no rows
    err = run_gemm({du, ldn, false}, {w, ldk, true}, a.M, a.K, L.pn, a.N, a.in_dtype, e,
                   a.ws + L.part, a.stream);
    if (err != hipSuccess) return err;
  }
  if (a.dw) {
    const void *x = a.x;
    if (L.pad && a.M > 0) {
      err = pad_rows(a.x, a.M, a.K, a.ws + L.x, static_cast<int>(L.pk), es, a.stream);
      if (err != hipSuccess) return err;
      x = a.ws + L.x;
    }
    e.M = a.N;
    e.y = a.dw;
    err = run_gemm({du, ldn, true}, {x, ldk, true}, a.N, a.K, a.M, a.M, a.in_dtype, e,
                   a.ws + L.part, a.stream);
  }
  return err;
}

}  // namespace gdn
