// Residual addition + RMSNorm, its backward pass and the row quantiser
// (gfx950).
//
//     r = x + residual                    y = r / sqrt(mean(r^2) + eps) * (1 + w)
//     e4m3 output: scale = max(max |y|, 1e-30) / 448 per row, q = y / scale
// and, for L = <dy, y> + <dr, r> with g = dy (1 + w), rs = 1 / sqrt(mean(r^2) + eps),
//     dL/dr = dr + rs (g - r rs^2 mean(g r)),   dL/dw = sum over rows of dy r rs
// (dL/dr is the gradient of x and of the residual alike). The weight is the
// zero-centred one of the output gate (gain 1 + w).
//
// All three are HBM streams of a few flops per byte. A row is held in the
// registers of the NT threads that own it (up to kChunks groups of 8 elements
// each), so every input is read once and every output written once; sums,
// maxima and the normalised values stay in fp32 and are rounded once, when
// they are stored. Measured: forward with residual, 16384 x 2048 bf16, 52 us
// (5.2 TB/s, a plain copy's rate); quantiser, 8192 x 4096 bf16, 20 us (4.9
// TB/s); backward, 16384 x 4096 bf16, 115 us (4.7 TB/s).
#include <type_traits>

#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kChunks = 4;          // 8-element groups per thread
constexpr int64_t kMaxBlocks = 1 << 21;  // 1024 threads each: under 2^32 threads
constexpr float kE4m3Max = 448.0f;  // largest finite e4m3 value
// Rows whose absolute maximum is below this (zero rows among them) take it as
// their maximum: the scale stays a normal number and its reciprocal finite.
constexpr float kTinyMax = 1e-30f;

// the larger of two values, NaN if either is (a NaN in a row reaches its scale)
__device__ __forceinline__ float max_nan(float m, float v) { return (v > m || v != v) ? v : m; }

struct Add {
  __device__ static __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {
  __device__ static __forceinline__ float of(float a, float b) { return max_nan(a, b); }
};

// All-reduce of K values over the NT threads of a row, in a fixed order. Rows
// wider than a wave are joined in `part` (NT / 64 entries per value).
template <int NT, int K, typename Op>
__device__ __forceinline__ void row_reduce(float (&v)[K], float *part) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int s = 1; s < (NT < 64 ? NT : 64); s *= 2) v[k] = Op::of(v[k], __shfl_xor(v[k], s));
  if constexpr (NT > 64) {
    constexpr int W = NT / 64;
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    __syncthreads();  // an earlier reduction's readers are done with `part`
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) part[k * W + wave] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = part[k * W];
#pragma unroll
      for (int w = 1; w < W; ++w) v[k] = Op::of(v[k], part[k * W + w]);
    }
  }
}

// NT threads own a row: a workgroup of its own, or 256 / NT rows of one wave or
// less each share one.
// NORM false: y = x (the row quantiser).
template <typename TI, typename TO, int NT, bool NORM>
__global__ __launch_bounds__(NT <= 64 ? 256 : NT) void rmsnorm_kernel(const NormArgs a) {
  constexpr int RPB = NT <= 64 ? 256 / NT : 1;
  __shared__ float part[NT > 64 ? NT / 64 : 1];
  const int t = threadIdx.x % NT;
  const int d = a.d;
  // one pass, but for more rows than a grid has workgroups
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * RPB; r0 < a.rows;
       r0 += static_cast<int64_t>(gridDim.x) * RPB) {
    const bool live = r0 + threadIdx.x / NT < a.rows;
    const int64_t row = live ? r0 + threadIdx.x / NT : a.rows - 1;
    const size_t base = static_cast<size_t>(row) * d;

    float v[kChunks][8];
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      load8(static_cast<const TI *>(a.x) + base, (c * NT + t) * 8, d, v[c]);
    if (NORM && a.residual) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        float s[8];
        load8(static_cast<const TI *>(a.residual) + base, (c * NT + t) * 8, d, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += s[i];
        if (a.r && live)
          store8(static_cast<TI *>(a.r) + base, (c * NT + t) * 8, d, v[c]);
      }
    }
    if constexpr (NORM) {
      // the norm takes the unrounded sum
      float ss[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(v[c][i], v[c][i], ss[0]);
      row_reduce<NT, 1, Add>(ss, part);
      const float rs = rsqrtf(ss[0] / static_cast<float>(d) + a.eps);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        float w[8] = {};
        if (a.norm_w) load8(a.norm_w, (c * NT + t) * 8, d, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * rs * (1.0f + w[i]);
      }
    }
    if constexpr (__is_same(TO, e4m3_t)) {
      float top[1] = {kTinyMax};
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) top[0] = max_nan(top[0], fabsf(v[c][i]));
      row_reduce<NT, 1, Max>(top, part);
      if (live && t == 0) a.y_scale[row] = top[0] / kE4m3Max;
      const float inv = kE4m3Max / top[0];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= inv;
    }
    if (live) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        store8(static_cast<TO *>(a.y) + base, (c * NT + t) * 8, d, v[c]);
    }
  }
}

// Backward: a workgroup takes rows block, block + gridDim, ... (RPB of them at
// a time, CH 8-element groups a thread) and keeps the weight gradient of its
// rows in registers; the per-workgroup sums go to a.part [gridDim][d], added in
// order by colsum_kernel. The next row is requested before this one is worked
// on: without that, 2 us of latency a row left half of the bandwidth unused.
// (Rows of 1024 threads have no registers for it, nor for the gain.)
template <typename TI, typename TG, int NT, int CH>
__global__ __launch_bounds__(NT <= 64 ? 256 : NT) void rmsnorm_bwd_kernel(const NormBwdArgs a) {
  constexpr int RPB = NT <= 64 ? 256 / NT : 1;
  constexpr bool AHEAD = NT < 1024;
  __shared__ float part[NT > 64 ? 2 * (NT / 64) : 1];
  __shared__ float join[RPB > 1 ? RPB * NT * CH * 8 : 1];
  const int t = threadIdx.x % NT, grp = threadIdx.x / NT;
  const int d = a.d;
  float acc[CH][8] = {}, gain[AHEAD ? CH : 1][8];
  auto load_gain = [&](int c, float *w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.0f;
    if (a.norm_w) load8(a.norm_w, (c * NT + t) * 8, d, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] += 1.0f;
  };
  struct Row {
    Raw8<TI> r[CH], dr[CH];
    Raw8<TG> dy[CH];
  } now, ahead;
  auto fetch = [&](int64_t r0, Row &row) {
    const size_t base = static_cast<size_t>(r0 + grp < a.rows ? r0 + grp : a.rows - 1) * d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * NT + t) * 8;
      row.r[c] = load_raw8(static_cast<const TI *>(a.r) + base, e0, d);
      row.dy[c] = load_raw8(static_cast<const TG *>(a.dy) + base, e0, d);
      if (a.dr) row.dr[c] = load_raw8(static_cast<const TI *>(a.dr) + base, e0, d);
    }
  };
  if constexpr (AHEAD) {
#pragma unroll
    for (int c = 0; c < CH; ++c) load_gain(c, gain[c]);
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x) * RPB;
  int64_t r0 = static_cast<int64_t>(blockIdx.x) * RPB;
  if (AHEAD && r0 < a.rows) fetch(r0, ahead);
  for (; r0 < a.rows; r0 += stride) {
    const bool live = r0 + grp < a.rows;
    if constexpr (AHEAD) {
      now = ahead;
      if (r0 + stride < a.rows) fetch(r0 + stride, ahead);
    } else {
      fetch(r0, now);
    }
    float sum[2] = {0.0f, 0.0f};  // sum r^2, sum g r
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float r[8], g[8], w[8];
      raw8_to_f32(now.r[c], r);
      raw8_to_f32(now.dy[c], g);
      if constexpr (!AHEAD) load_gain(c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = fmaf(r[i], r[i], sum[0]);
        sum[1] = fmaf(g[i] * (AHEAD ? gain[AHEAD ? c : 0][i] : w[i]), r[i], sum[1]);
      }
    }
    row_reduce<NT, 2, Add>(sum, part);
    const float rs = rsqrtf(sum[0] / static_cast<float>(d) + a.eps);
    const float along = rs * rs * sum[1] / static_cast<float>(d);
    if (live) {
      const size_t base = static_cast<size_t>(r0 + grp) * d;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float r[8], g[8], w[8], dx[8] = {};
        raw8_to_f32(now.r[c], r);
        raw8_to_f32(now.dy[c], g);
        if constexpr (!AHEAD) load_gain(c, w);
        if (a.dr) raw8_to_f32(now.dr[c], dx);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[c][i] = fmaf(g[i], r[i] * rs, acc[c][i]);
          dx[i] += rs * (g[i] * (AHEAD ? gain[AHEAD ? c : 0][i] : w[i]) - r[i] * along);
        }
        store8(static_cast<TI *>(a.dx) + base, (c * NT + t) * 8, d, dx);
      }
    }
  }
  if (!a.part) return;
  float *out = a.part + static_cast<size_t>(blockIdx.x) * d;
  if constexpr (RPB > 1) {
    constexpr int W = NT * CH * 8;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) join[grp * W + (c * NT + t) * 8 + i] = acc[c][i];
    __syncthreads();
    for (int e = threadIdx.x; e < d; e += 256) {
      float s = join[e];
      for (int q = 1; q < RPB; ++q) s += join[q * W + e];
      out[e] = s;
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) store8(out, (c * NT + t) * 8, d, acc[c]);
  }
}

// out[c] = sum over p of part[p][c], in order: 16 columns per workgroup, the
// rows dealt to 64 groups of threads and joined in order
__global__ __launch_bounds__(1024) void colsum_kernel(const float *__restrict__ part, int P, int d,
                                                      float *__restrict__ out) {
  __shared__ float s[64][17];
  const int c = threadIdx.x % 16, g = threadIdx.x / 16;
  const int col = blockIdx.x * 16 + c;
  float v = 0.0f;
  if (col < d) {
#pragma unroll 8
    for (int p = g; p < P; p += 64) v += part[static_cast<size_t>(p) * d + col];
  }
  s[g][c] = v;
  __syncthreads();
  if (g == 0 && col < d) {
#pragma unroll
    for (int q = 1; q < 64; ++q) v += s[q][c];
    out[col] = v;
  }
}

template <typename F>
hipError_t with_type(int code, F &&f) {
  switch (code) {
    case 1: return f(bf16_t{});
    case 2: return f(_Float16{});
    default: return f(float{});
  }
}

// threads per row: the fewest whose registers hold it
template <typename F>
hipError_t with_threads(int d, F &&f) {
  if (d <= 16 * 8 * kChunks) return f(std::integral_constant<int, 16>{});
  if (d <= 64 * 8 * kChunks) return f(std::integral_constant<int, 64>{});
  if (d <= 256 * 8 * kChunks) return f(std::integral_constant<int, 256>{});
  if (d <= 512 * 8 * kChunks) return f(std::integral_constant<int, 512>{});
  return f(std::integral_constant<int, 1024>{});
}
static_assert(kNormMaxD == 1024 * 8 * kChunks, "widest row");

template <bool NORM, typename TI, typename TO>
hipError_t launch_rows(const NormArgs &a) {
  return with_threads(a.d, [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    constexpr int RPB = NT <= 64 ? 256 / NT : 1;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    hipLaunchKernelGGL((rmsnorm_kernel<TI, TO, NT, NORM>),
                       dim3(static_cast<unsigned>(blocks < kMaxBlocks ? blocks : kMaxBlocks)),
                       dim3(NT <= 64 ? 256 : NT), 0, a.stream, a);
    return hipGetLastError();
  });
}

// the same for the backward: two 8-element groups a thread, four for the widest
template <typename F>
hipError_t with_threads_bwd(int d, F &&f) {
  using std::integral_constant;
  if (d <= 16 * 16) return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  if (d <= 64 * 16) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if (d <= 128 * 16) return f(integral_constant<int, 128>{}, integral_constant<int, 2>{});
  if (d <= 256 * 16) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (d <= 512 * 16) return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  if (d <= 1024 * 16) return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

// Workgroups of the backward, and so partial sums of the weight gradient: 1024
// threads a CU (16384 x 4096 bf16: 115 us with 1024 workgroups, 120 with 512),
// fewer for few rows, whose partial sums would cost as much as the rows.
int bwd_blocks(int64_t rows, int d) {
  int64_t b = 0;
  with_threads_bwd(d, [&](auto nt, auto) {
    constexpr int NT = decltype(nt)::value;
    constexpr int RPB = NT <= 64 ? 256 / NT : 1;
    constexpr int64_t MOST = NT <= 256 ? 1024 : 1024 * 256 / NT;
    const int64_t all = (rows + RPB - 1) / RPB;
    b = all / 2;  // at least two rows a group, once every CU has a workgroup
    if (b < 256) b = all < 256 ? all : 256;
    if (b > MOST) b = MOST;
    return hipSuccess;
  });
  return static_cast<int>(b);
}

}  // namespace

hipError_t launch_colsum(const float *part, int P, int d, float *out, hipStream_t stream) {
  hipLaunchKernelGGL(colsum_kernel, dim3((d + 15) / 16), dim3(1024), 0, stream, part, P, d, out);
  return hipGetLastError();
}

hipError_t launch_add_rmsnorm(const NormArgs &a) {
  if (a.rows == 0) return hipSuccess;
  return with_type(a.in_dtype, [&](auto ti) {
    using TI = decltype(ti);
    if (a.out_dtype == kE4m3) return launch_rows<true, TI, e4m3_t>(a);
    return with_type(a.out_dtype,
                     [&](auto to) { return launch_rows<true, TI, decltype(to)>(a); });
  });
}

hipError_t launch_quantize_rows(const NormArgs &a) {
  if (a.rows == 0) return hipSuccess;
  return with_type(a.in_dtype, [&](auto ti) { return launch_rows<false, decltype(ti), e4m3_t>(a); });
}

size_t add_rmsnorm_bwd_workspace_size(int64_t rows, int d) {
  return static_cast<size_t>(bwd_blocks(rows, d)) * d * 4;
}

hipError_t launch_add_rmsnorm_bwd(const NormBwdArgs &a) {
  const int P = bwd_blocks(a.rows, a.d);
  if (P > 0) {
    const hipError_t e = with_type(a.in_dtype, [&](auto ti) {
      return with_type(a.dy_dtype, [&](auto tg) {
        return with_threads_bwd(a.d, [&](auto nt, auto ch) {
          constexpr int NT = decltype(nt)::value, CH = decltype(ch)::value;
          hipLaunchKernelGGL((rmsnorm_bwd_kernel<decltype(ti), decltype(tg), NT, CH>), dim3(P),
                             dim3(NT <= 64 ? 256 : NT), 0, a.stream, a);
          return hipGetLastError();
        });
      });
    });
    if (e != hipSuccess) return e;
  }
  return a.dnorm_w ? launch_colsum(a.part, P, a.d, a.dnorm_w, a.stream) : hipSuccess;
}

}  // namespace gdn
