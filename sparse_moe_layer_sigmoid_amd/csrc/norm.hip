// moe_norm / moe_norm_backward: layer norm (or root mean square norm) of the rows that enter the
// layer, and its gradients.
//
//   mean = (1/d) sum_i x_i          (0 for the root mean square form)
//   rstd = (1/d sum_i (x_i - mean)^2 + eps)^(-1/2),   xhat = (x - mean) rstd,   y = xhat w + b
//   g = dy w;  dx = rstd (g - m1 - xhat m2),  m1 = (1/d) sum g (0 without the mean),
//   m2 = (1/d) sum g xhat;  dw = sum_rows dy xhat,  db = sum_rows dy
//
// Everything between the loads and the final rounding is fp32.  Both kernels are bound by HBM:
// each element is read once and written once.
//
//  * Forward: one workgroup holds a row in registers (chunks of 8 elements per lane), so the
//    variance is summed over x - mean in a second pass over registers, not from squares that
//    cancel.  With a checkpoint the normalised row is also stored as E4M3 with power-of-two 1x128
//    scales: 16 lanes are a tile, so its maximum is four lane rotations.  Stores are non-temporal
//    (4096 x 7168 bf16: 21.5 us, 5.5 TB/s, against 29 us; with the checkpoint 26 us, 5.6 TB/s,
//    against 38 us).  Walking several rows with the weights in registers measured slower (33 us).
//  * Backward: a workgroup owns all columns and walks rows b, b + grid, ...; each lane keeps dw
//    and db of its columns in registers over all its rows, and the next row's loads are issued
//    before the current row's two sums are exchanged (two rows ahead measured no faster).  The
//    workgroups' partial dw / db rows go to the workspace and a second kernel adds them in
//    workgroup order, so the result does not depend on timing.  4096 x 7168 from bf16 x, f32 dy and
//    dx: 61 us (4.8 TB/s); 16384 x 7168 from the checkpoint, bf16: 120 us (4.9 TB/s, the rate of a
//    large copy).
//  * Rows of up to 512 elements: 16, 32 or 64 lanes hold a row, so a workgroup takes several, their sums
//    stay inside a wave, and the backward adds its 16 to 64 rows' dw and db through LDS before it writes
//    one partial row.  65536 x 64 bf16: 7 us (24 us with a workgroup per row), x 256: 15 us (26 us);
//    backward 65536 x 128 bf16: 15 us (37 us), 32768 x 512: 24 us (32 us).  The backward takes rows of up
//    to 1024 that way, two chunks to a lane: 4096 x 768 bf16 14 us (29 us), 65536 x 640 f32 104 us (115
//    us), but 16384 x 1024 42 us (39.5 us).  A short last chunk is read element by element: as the row's
//    last 8 elements, shifted into place, the same kernels took 1.5 to 4 times as long.
#include "abi_common.h"
#include "device_common.h"
#include "rows_common.h"

namespace moe {
namespace {

constexpr int kMaxNormD = 16384;  // 1024 lanes x 2 chunks of 8
constexpr int kNarrow = 256;      // lanes of a forward workgroup of several rows

enum { SRC_BF16 = ROW_BF16, SRC_F32 = ROW_F32, SRC_CKPT = 2 };

// Sums v over the workgroup, the same value in every lane; `red` holds one float per wave.  The
// caller alternates between two arrays, so one barrier per sum is enough.
__device__ __forceinline__ float block_sum(float v, float* red, int nwaves) {
  v = wave_sum(v);
  if (nwaves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < nwaves; ++w) s += red[w];
  return s;
}

// Sums v over the L neighbouring lanes of a row (16: a DPP row, 32, or 64: the wave).
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L == 64) return wave_sum(v);
  v += __uint_as_float(row_ror<8>(__float_as_uint(v)));
  v += __uint_as_float(row_ror<4>(__float_as_uint(v)));
  v += __uint_as_float(row_ror<2>(__float_as_uint(v)));
  v += __uint_as_float(row_ror<1>(__float_as_uint(v)));
  return L == 16 ? v : v + __shfl_xor(v, 16, kWave);
}

// Largest v over the workgroup or, for L lanes, the row's lanes.
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red, int nwaves) {
#pragma unroll
  for (int o = (L ? L : kWave) / 2; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, kWave));
  if (L || nwaves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  for (int w = 0; w < nwaves; ++w) v = max(v, red[w]);
  return v;
}

struct NormArgs {
  int rows;
  const void* x;
  int64_t ldx_b;  // bytes
  const void* w;
  const void* b;
  int w_dtype;
  int d;
  float eps;
  int rms;
  void* y;
  int y_dtype;
  int64_t ldy_b;
  float* mean;
  float* rstd;
  uint8_t* q;
  uint8_t* q_scale;
  int tiles;  // scales per row: ceil(d / 128)
};

// L: lanes of a row, 0 for the whole workgroup.
template <int XT, int NV, bool FULL, int L>
__global__ __launch_bounds__(L ? kNarrow : 1024) void norm_kernel(NormArgs p) {
  __shared__ float red[2][16];
  __shared__ uint32_t red_max[16];
  constexpr int D = L ? L : 1;
  const int64_t r = L ? (int64_t)blockIdx.x * (kNarrow / D) + threadIdx.x / D : blockIdx.x;
  const int t = L ? threadIdx.x % D : threadIdx.x, G = L ? L : blockDim.x, nw = G >> 6;
  if (L && r >= p.rows) return;  // the row's lanes together
  auto row_sum = [&](float v, float* red) __attribute__((always_inline)) {
    if constexpr (L) return lanes_sum<L>(v);
    else return block_sum(v, red, nw);
  };
  const char* xr = static_cast<const char*>(p.x) + r * p.ldx_b;
  // values and squares are summed times 2^-k >= 1/d > 2^-k-1 (exact products), so a sum overflows only
  // where its mean nearly does
  const int k = 31 - __clz(p.d);
  const float down = pow2f(-k), up = pow2f(k) / (float)p.d;
  float f[NV][8], mean = 0.f;
  // loads the row times 2^-e, subtracts the mean and returns the variance, the same bits in every lane of the row
  auto take_row = [&](int e) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * G) * 8;
      if (c < p.d) {
        values8(load8<XT, FULL>(xr, c, p.d), f[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = 0.f;
      }
    }
    if (e != 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = ldexpf(f[i][j], -e);
    }
    if (!p.rms) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(f[i][e], down, s);
      mean = row_sum(s, red[0]) * up;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * G) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = c + e < p.d ? f[i][e] - mean : 0.f;
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[i][e] * down, f[i][e], ss);
    return row_sum(ss, red[1]) * up;
  };
  const float var = take_row(0);
  float rstd = 1.0f / sqrtf(var + p.eps);
  // Squares leave the float range where the values do not: above 2^64 they overflow, and below about 2^-56
  // their sum loses bits, which shows unless eps covers it (rows of 1e-21 and eps = 0: rstd off by 38%).
  // A row whose variance comes out that way is taken again times 2^-e, with largest value or eps^1/2 in [1/2, 1).
  int e = 0;
  if (__builtin_expect(!(var <= 0x1p120f) || (var < 0x1p-96f && p.eps < 0x1p-70f), 0)) {
    uint32_t top = 0;
    int at = t;
    asm volatile("" : "+v"(at));  // else its addresses are kept in registers from the loads above on
#pragma nounroll
    for (int c = at * 8; c < p.d; c += G * 8) {
      float v[8];
      values8(load8<XT, FULL>(xr, c, p.d), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    top = row_max<L>(top, red_max, nw);
    // a row with an infinity or NaN, and one of zeros without eps, keep what they have
    if (top < 0x7f800000u && (top != 0 || p.eps > 0.f)) {
      const int ex = top ? __builtin_amdgcn_frexp_expf(__uint_as_float(top)) : -1000;
      const int ee = p.eps > 0.f ? (__builtin_amdgcn_frexp_expf(p.eps) + 1) >> 1 : -1000;
      e = max(ex, ee);
      rstd = 1.0f / sqrtf(take_row(e) + ldexpf(p.eps, -2 * e));
    }
  }
  if (t == 0) {
    if (p.mean) p.mean[r] = ldexpf(mean, e);
    if (p.rstd) p.rstd[r] = ldexpf(rstd, -e);
  }
  char* yr = static_cast<char*>(p.y) + r * p.ldy_b;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = t + i * G, c = ch * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[i][e] *= rstd;
    if (p.q) {  // a whole 16-lane tile shares this test, and lanes past the row hold zeros
      uint32_t code;
      const u32x2 q = ckpt_encode8(f[i], code);
      if (c < p.d) {
        store_codes8<FULL, true>(p.q + r * p.d, c, p.d, q);
        if ((ch & 15) == 0) p.q_scale[r * p.tiles + ch / 16] = (uint8_t)code;
      }
    }
    if (c < p.d) {
      float w[8], b[8];
      if (p.w) {
        load8_any<FULL>(p.w_dtype, p.w, c, p.d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] *= w[e];
      }
      if (p.b) {
        load8_any<FULL>(p.w_dtype, p.b, c, p.d, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] += b[e];
      }
      store8_any<FULL, true>(p.y_dtype, yr, c, p.d, f[i]);
    }
  }
}

struct NormBwdArgs {
  const void* dy;
  int64_t lddy_b;
  const void* x;  // rows, or the checkpoint's codes
  int64_t ldx_b;
  const uint8_t* q_scale;
  int tiles;
  const float* mean;
  const float* rstd;
  const void* w;
  int w_dtype;
  int rows;
  int d;
  int rms;
  void* dx;
  int dx_dtype;
  int64_t lddx_b;
  float* part_w;  // [grid][d] partial sums (or the results themselves when grid == 1), or null
  float* part_b;
};

template <int SRC>
struct RawX {
  Raw8<SRC> v;
};
template <>
struct RawX<SRC_CKPT> {
  u32x2 q;
  uint32_t s;
};

// Makes the compiler take a row's raw values as new ones here (it would keep what it computed
// from them instead).
__device__ __forceinline__ void keep(Raw8<ROW_BF16>& r) { asm volatile("" : "+v"(r.v)); }
__device__ __forceinline__ void keep(Raw8<ROW_F32>& r) { asm volatile("" : "+v"(r.lo), "+v"(r.hi)); }
__device__ __forceinline__ void keep(RawX<SRC_CKPT>& r) { asm volatile("" : "+v"(r.q), "+v"(r.s)); }
template <int SRC>
__device__ __forceinline__ void keep(RawX<SRC>& r) { keep(r.v); }

// L: lanes of a row, 0 for the whole workgroup.  LANES: the largest workgroup.  Up to 512 lanes (d <= 8192) a wave may have more than 128 registers,
// which the kernel takes where x and dy are f32: 4096 x 7168 72 us, 95 us held to 128.
template <int SRC, int DYT, int NV, bool FULL, int L, int LANES>
__global__ __launch_bounds__(LANES) void norm_backward_kernel(NormBwdArgs p) {
  constexpr int D = L ? L : 1;
  constexpr int ROWS = L ? LANES / D : 1;  // of a workgroup at a time
  __shared__ float red[2][2][16];
  __shared__ float s_part[L ? ROWS : 1][L ? L * NV * 8 + 1 : 1];
  const int t = L ? threadIdx.x % D : threadIdx.x, G = L ? L : blockDim.x, nw = G >> 6;
  const float inv_d = 1.0f / (float)p.d;
  float w[NV][8], aw[NV][8], ab[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * G) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[i][e] = 1.f;
      aw[i][e] = ab[i][e] = 0.f;
    }
    if (p.w && c < p.d) load8_any<FULL>(p.w_dtype, p.w, c, p.d, w[i]);
  }
  Raw8<DYT> ndy[NV];
  RawX<SRC> nx[NV];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int64_t r) __attribute__((always_inline)) {
    const char* dyr = static_cast<const char*>(p.dy) + r * p.lddy_b;
    const char* xr = static_cast<const char*>(p.x) + r * p.ldx_b;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = t + i * G, c = ch * 8;
      if (c < p.d) {
        ndy[i] = load8<DYT, FULL>(dyr, c, p.d);
        if constexpr (SRC == SRC_CKPT) {
          nx[i].q = load_codes8<FULL>(reinterpret_cast<const uint8_t*>(xr), c, p.d);
          nx[i].s = p.q_scale[r * p.tiles + ch / 16];
        } else {
          nx[i].v = load8<SRC, FULL>(xr, c, p.d);
        }
      }
    }
    nmean = p.mean ? p.mean[r] : 0.f;
    nrstd = p.rstd[r];
  };
  int64_t r = L ? (int64_t)blockIdx.x * ROWS + threadIdx.x / D : blockIdx.x;
  const int step = gridDim.x * ROWS;
  if (r < p.rows) fetch(r);
  for (int it = 0; r < p.rows; r += step, ++it) {
    const float mean = nmean, rstd = nrstd;
    Raw8<DYT> dy[NV];
    RawX<SRC> x[NV];
    float s1 = 0.f, s2 = 0.f;
    // g = dy w and xhat of chunk i, from the row's raw values: taken twice, so that only the raw
    // values (8 registers a chunk in bf16, 16 for g and xhat) live across the exchange of the sums
    auto values = [&](int i, float(&g)[8], float(&xh)[8]) __attribute__((always_inline)) {
      values8(dy[i], g);
      if constexpr (SRC == SRC_CKPT) {
        ckpt_decode8(x[i].q, x[i].s, xh);
      } else {
        values8(x[i].v, xh);
#pragma unroll
        for (int e = 0; e < 8; ++e)  // past the row's end 0: there mean * rstd alone could overflow
          xh[e] = FULL || (t + i * G) * 8 + e < p.d ? (xh[e] - mean) * rstd : 0.f;
      }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * G) * 8;
      dy[i] = ndy[i];
      x[i] = nx[i];
      if (c < p.d) {
        float g[8], xh[8];
        values(i, g, xh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // past the row's end dy (and so g) reads as zero
          aw[i][e] = fmaf(g[e], xh[e], aw[i][e]);
          ab[i][e] += g[e];
          g[e] *= w[i][e];
          s1 += g[e];
          s2 = fmaf(g[e], xh[e], s2);
        }
      }
    }
    if (r + step < p.rows) fetch(r + step);
    s1 = lanes_sum<L ? L : 64>(s1);
    s2 = lanes_sum<L ? L : 64>(s2);
    if (!L && nw > 1) {
      float(*rd)[16] = red[it & 1];
      if ((t & 63) == 0) {
        rd[0][t >> 6] = s1;
        rd[1][t >> 6] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
      for (int k = 0; k < nw; ++k) {
        s1 += rd[0][k];
        s2 += rd[1][k];
      }
    }
    const float m1 = p.rms ? 0.f : s1 * inv_d, m2 = s2 * inv_d;
    char* dxr = static_cast<char*>(p.dx) + r * p.lddx_b;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * G) * 8;
      if (c < p.d) {
        keep(dy[i]);
        keep(x[i]);
        float g[8], xh[8];
        values(i, g, xh);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = rstd * (g[e] * w[i][e] - m1 - xh[e] * m2);
        store8_any<FULL>(p.dx_dtype, dxr, c, p.d, g);
      }
    }
  }
  if constexpr (L > 0) {  // the rows' sums through LDS, added in row order
    for (int which = 0; which < 2; ++which) {
      float* part = which ? p.part_b : p.part_w;
      if (!part) continue;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s_part[threadIdx.x / D][(t + i * L) * 8 + e] = which ? ab[i][e] : aw[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < p.d; c += LANES) {
        float v = 0.f;
#pragma unroll 8
        for (int k = 0; k < ROWS; ++k) v += s_part[k][c];
        part[(int64_t)blockIdx.x * p.d + c] = v;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * G) * 8;
    if (c < p.d) {
      if (p.part_w) store8_any<FULL>(ROW_F32, p.part_w + (int64_t)blockIdx.x * p.d, c, p.d, aw[i]);
      if (p.part_b) store8_any<FULL>(ROW_F32, p.part_b + (int64_t)blockIdx.x * p.d, c, p.d, ab[i]);
    }
  }
}

// out[c] = sum over the n partial rows in a fixed order: 16 strips of rows, 64 columns each, then the strips in order.
// With 16 columns and 64 strips the backward of 16384 x 4096 (1024 partial rows) takes 93.7 us, not 89.0, of 8208 x
// 2048 (513) 41.2, not 40.3, of 4096 x 7168 (256) 49.4, not 46.5; only many rows of few columns gain: 33000 x 1025
// (2048) 66.0, not 66.9 (bf16, dw and db, whole calls).
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* __restrict__ part_w,
                                                           const float* __restrict__ part_b, int n, int d,
                                                           float* __restrict__ dw, float* __restrict__ db) {
  constexpr int COLS = 64, STRIPS = 1024 / COLS;
  __shared__ float red[STRIPS][COLS + 1];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;  // the whole workgroup
  const int col = threadIdx.x % COLS, strip = threadIdx.x / COLS;
  const int c = blockIdx.x * COLS + col;
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int r = strip; r < n; r += STRIPS) s += part[(int64_t)r * d + c];
  }
  red[strip][col] = s;
  __syncthreads();
  if (strip == 0 && c < d) {
    float v = 0.f;
#pragma unroll 8
    for (int k = 0; k < STRIPS; ++k) v += red[k][col];
    out[c] = v;
  }
}

void launch_reduce(const float* pw, const float* pb, int n, int d, float* dw, float* db, hipStream_t stream) {
  norm_reduce_kernel<<<dim3((d + 63) / 64, db ? 2 : 1), 1024, 0, stream>>>(pw, pb, n, d, dw, db);
}

// Forward: chunks per lane.  Few rows: one, so that a row's loads are all in flight together (one row
// of 7168: 4.2 us against 5.0 us with four).  Many rows: a row in one wave while its chunks fit 4 to a
// lane, else 4 to a lane (4096 rows of 7168: 21 us, 28 us with two chunks).
int norm_chunks_per_lane(int rows, int d) {
  const int chunks = (d + 7) / 8;
  if (rows <= 256) return chunks <= 1024 ? 1 : 2;
  return chunks <= 128 ? 2 : 4;
}

// Rows of up to 64 chunks take 16, 32 or 64 lanes of one chunk each, several rows to a workgroup.
int narrow_lanes(int d) { return d <= 128 ? 16 : d <= 256 ? 32 : d <= 512 ? 64 : 0; }
// The backward's workgroups of several rows: up to 1024 elements, with two chunks to a lane past 512.
constexpr int kNarrowBwd = 1024, kNarrowBwd2 = 512;  // their lanes

int group_threads(int d, int nv) {
  const int chunks = (d + 7) / 8;
  return ((chunks + nv - 1) / nv + 63) / 64 * 64;
}

// Workgroups of the backward kernel.  Every one writes a partial row of dw and db that is read again,
// so each should walk 16 rows or more, down to four waves per CU: 4096 rows of 7168 (7 waves), 256
// workgroups 61 us, 512 70 us; 16384 rows, 256 143 us, 512 (32 rows each) 121 us; 4096 rows of 2048 (2
// waves), 256 28 us, 512 22.5 us, 1024 27 us.
int norm_bwd_grid(int rows, int d) {
  if (d <= 1024) {
    const int at_once = d <= 512 ? kNarrowBwd / narrow_lanes(d) : kNarrowBwd2 / 64, most = d <= 512 ? 256 : 512;
    return rows < most * at_once ? (rows + at_once - 1) / at_once : most;
  }
  const int threads = group_threads(d, 2);
  const int per_cu = threads >= 448 ? 2 : threads >= 256 ? 4 : 8;
  int n = rows / 16;
  const int least = threads < 256 ? 256 * 256 / threads : 256;
  n = n < least ? least : n > 256 * per_cu ? 256 * per_cu : n;
  return rows < n ? rows : n;
}

template <int SRC, int DYT, bool FULL>
void launch_norm_backward_as(const NormBwdArgs& a, int grid, hipStream_t stream) {
  const int lanes = narrow_lanes(a.d);
  const int threads = lanes ? kNarrowBwd : a.d <= 1024 ? kNarrowBwd2 : group_threads(a.d, 2);
  auto kernel = lanes == 16      ? norm_backward_kernel<SRC, DYT, 1, FULL, 16, kNarrowBwd>
                : lanes == 32    ? norm_backward_kernel<SRC, DYT, 1, FULL, 32, kNarrowBwd>
                : lanes == 64    ? norm_backward_kernel<SRC, DYT, 1, FULL, 64, kNarrowBwd>
                : a.d <= 1024    ? norm_backward_kernel<SRC, DYT, 2, FULL, 64, kNarrowBwd2>
                : threads <= 512 ? norm_backward_kernel<SRC, DYT, 2, FULL, 0, 512>
                                 : norm_backward_kernel<SRC, DYT, 2, FULL, 0, 1024>;
  kernel<<<grid, threads, 0, stream>>>(a);
}

template <int SRC, int DYT>
void launch_norm_backward(const NormBwdArgs& a, int grid, hipStream_t stream) {
  if (a.d % 8 == 0) launch_norm_backward_as<SRC, DYT, true>(a, grid, stream);
  else launch_norm_backward_as<SRC, DYT, false>(a, grid, stream);
}

template <int XT, bool FULL>
void launch_norm(const NormArgs& a, hipStream_t stream) {
  if (const int lanes = narrow_lanes(a.d)) {
    const int at_once = kNarrow / lanes, grid = (a.rows + at_once - 1) / at_once;
    if (lanes == 16) norm_kernel<XT, 1, FULL, 16><<<grid, kNarrow, 0, stream>>>(a);
    else if (lanes == 32) norm_kernel<XT, 1, FULL, 32><<<grid, kNarrow, 0, stream>>>(a);
    else norm_kernel<XT, 1, FULL, 64><<<grid, kNarrow, 0, stream>>>(a);
    return;
  }
  const int nv = norm_chunks_per_lane(a.rows, a.d);
  auto kernel = nv == 1   ? norm_kernel<XT, 1, FULL, 0>
                : nv == 2 ? norm_kernel<XT, 2, FULL, 0>
                          : norm_kernel<XT, 4, FULL, 0>;
  kernel<<<a.rows, group_threads(a.d, nv), 0, stream>>>(a);
}

bool row_dtype(int t) { return t == MOE_BF16 || t == MOE_F32; }
int row_esz(int t) { return t == MOE_BF16 ? 2 : 4; }
bool elem_aligned(const void* p, int esz) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(esz - 1)) == 0; }

}  // namespace
}  // namespace moe

extern "C" moe_status moe_norm(const void* x, int x_dtype, int64_t ldx, const void* weight, const void* bias,
                               int w_dtype, int rows, int d, float eps, int kind, void* y, int y_dtype, int64_t ldy,
                               float* mean, float* rstd, uint8_t* ck_q, uint8_t* ck_scale, hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(rows == 0 || (x && y), MOE_ERR_NULL, "moe_norm: a required pointer is NULL");
  MOE_REQUIRE(!ck_q == !ck_scale, MOE_ERR_NULL, "moe_norm: ck_q and ck_scale go together");
  MOE_REQUIRE(row_dtype(x_dtype) && row_dtype(y_dtype) && row_dtype(w_dtype), MOE_ERR_DTYPE,
              "moe_norm: x, y and weights must be MOE_BF16 or MOE_F32 (%d, %d, %d)", x_dtype, y_dtype, w_dtype);
  MOE_REQUIRE(kind == MOE_NORM_LAYER || kind == MOE_NORM_RMS, MOE_ERR_DTYPE, "moe_norm: unknown kind %d", kind);
  MOE_REQUIRE(rows >= 0 && d >= 1 && d <= kMaxNormD && eps >= 0.f && eps < 1e30f, MOE_ERR_SHAPE,
              "moe_norm: rows=%d d=%d (1..%d) eps=%g (finite, >= 0)", rows, d, kMaxNormD, (double)eps);
  MOE_REQUIRE((ldx >= d && ldy >= d) || rows <= 1, MOE_ERR_ALIGN, "moe_norm: ldx=%lld ldy=%lld must be >= d=%d",
              (long long)ldx, (long long)ldy, d);
  MOE_REQUIRE(elem_aligned(x, row_esz(x_dtype)) && elem_aligned(y, row_esz(y_dtype)) &&
                  elem_aligned(weight, row_esz(w_dtype)) && elem_aligned(bias, row_esz(w_dtype)) &&
                  elem_aligned(mean, 4) && elem_aligned(rstd, 4),
              MOE_ERR_ALIGN, "moe_norm: pointers must be aligned to their elements");
  if (rows > 0) {
    NormArgs a;
    a.rows = rows;
    a.x = x;
    a.ldx_b = ldx * row_esz(x_dtype);
    a.w = weight;
    a.b = bias;
    a.w_dtype = w_dtype;
    a.d = d;
    a.eps = eps;
    a.rms = kind == MOE_NORM_RMS;
    a.y = y;
    a.y_dtype = y_dtype;
    a.ldy_b = ldy * row_esz(y_dtype);
    a.mean = mean;
    a.rstd = rstd;
    a.q = ck_q;
    a.q_scale = ck_scale;
    a.tiles = (d + 127) / 128;
    const int lanes = narrow_lanes(d) ? narrow_lanes(d) : group_threads(d, norm_chunks_per_lane(rows, d));
    MOE_REQUIRE(rows <= kMaxLanes / lanes, MOE_ERR_SHAPE, "moe_norm: too many rows (%d)", rows);
    const bool full = d % 8 == 0;
    if (x_dtype == MOE_BF16) full ? launch_norm<ROW_BF16, true>(a, stream) : launch_norm<ROW_BF16, false>(a, stream);
    else full ? launch_norm<ROW_F32, true>(a, stream) : launch_norm<ROW_F32, false>(a, stream);
  }
  return check_launch("moe_norm");
}

extern "C" size_t moe_norm_backward_workspace_size(int rows, int d) {
  if (rows <= 0 || d < 1 || d > moe::kMaxNormD) return 0;
  const int grid = moe::norm_bwd_grid(rows, d);
  return grid == 1 ? 0 : (size_t)2 * grid * d * sizeof(float);  // one workgroup's sums are the results
}

extern "C" moe_status moe_norm_backward(const void* dy, int dy_dtype, int64_t lddy, const void* x, int x_dtype,
                                        int64_t ldx, const uint8_t* ck_q, const uint8_t* ck_scale, const float* mean,
                                        const float* rstd, const void* weight, int w_dtype, int rows, int d, int kind,
                                        void* dx, int dx_dtype, int64_t lddx, float* dweight, float* dbias, void* ws,
                                        size_t ws_bytes, hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(rows == 0 || (dy && rstd && dx), MOE_ERR_NULL, "moe_norm_backward: a required pointer is NULL");
  MOE_REQUIRE(!ck_q == !ck_scale, MOE_ERR_NULL, "moe_norm_backward: ck_q and ck_scale go together");
  MOE_REQUIRE(rows == 0 || !x == !!ck_q, MOE_ERR_NULL, "moe_norm_backward: either x or the checkpoint is given");
  MOE_REQUIRE(row_dtype(dy_dtype) && row_dtype(x_dtype) && row_dtype(w_dtype) && row_dtype(dx_dtype), MOE_ERR_DTYPE,
              "moe_norm_backward: tensors must be MOE_BF16 or MOE_F32 (%d, %d, %d, %d)", dy_dtype, x_dtype, w_dtype,
              dx_dtype);
  MOE_REQUIRE(kind == MOE_NORM_LAYER || kind == MOE_NORM_RMS, MOE_ERR_DTYPE, "moe_norm_backward: unknown kind %d", kind);
  MOE_REQUIRE(rows == 0 || ck_q || kind == MOE_NORM_RMS || mean, MOE_ERR_NULL,
              "moe_norm_backward: the layer norm's backward from x needs mean");
  MOE_REQUIRE(rows >= 0 && d >= 1 && d <= kMaxNormD, MOE_ERR_SHAPE, "moe_norm_backward: rows=%d d=%d (1..%d)", rows, d,
              kMaxNormD);
  MOE_REQUIRE((lddy >= d && lddx >= d && (ck_q || ldx >= d)) || rows <= 1, MOE_ERR_ALIGN,
              "moe_norm_backward: lddy=%lld ldx=%lld lddx=%lld must be >= d=%d", (long long)lddy, (long long)ldx,
              (long long)lddx, d);
  MOE_REQUIRE(elem_aligned(dy, row_esz(dy_dtype)) && elem_aligned(x, row_esz(x_dtype)) &&
                  elem_aligned(dx, row_esz(dx_dtype)) && elem_aligned(weight, row_esz(w_dtype)) &&
                  elem_aligned(mean, 4) && elem_aligned(rstd, 4) && elem_aligned(dweight, 4) && elem_aligned(dbias, 4),
              MOE_ERR_ALIGN, "moe_norm_backward: pointers must be aligned to their elements");
  const size_t need = moe_norm_backward_workspace_size(rows, d);
  MOE_REQUIRE(!(dweight || dbias) || need == 0 || (ws && ws_bytes >= need && aligned16(ws)), MOE_ERR_WORKSPACE,
              "moe_norm_backward: workspace %zu < %zu bytes (or NULL / unaligned)", ws_bytes, need);
  int grid = 0;
  float* pw = static_cast<float*>(ws);
  float* pb = nullptr;
  if (rows > 0) {
    grid = norm_bwd_grid(rows, d);
    if (pw) pb = pw + (size_t)grid * d;
    NormBwdArgs a;
    a.dy = dy;
    a.lddy_b = lddy * row_esz(dy_dtype);
    a.x = ck_q ? static_cast<const void*>(ck_q) : x;
    a.ldx_b = ck_q ? (int64_t)d : ldx * row_esz(x_dtype);
    a.q_scale = ck_scale;
    a.tiles = (d + 127) / 128;
    a.mean = ck_q || kind == MOE_NORM_RMS ? nullptr : mean;
    a.rstd = rstd;
    a.w = weight;
    a.w_dtype = w_dtype;
    a.rows = rows;
    a.d = d;
    a.rms = kind == MOE_NORM_RMS;
    a.dx = dx;
    a.dx_dtype = dx_dtype;
    a.lddx_b = lddx * row_esz(dx_dtype);
    a.part_w = dweight ? (grid == 1 ? dweight : pw) : nullptr;
    a.part_b = dbias ? (grid == 1 ? dbias : pb) : nullptr;
    if (ck_q) {
      if (dy_dtype == MOE_BF16) launch_norm_backward<SRC_CKPT, ROW_BF16>(a, grid, stream);
      else launch_norm_backward<SRC_CKPT, ROW_F32>(a, grid, stream);
    } else if (x_dtype == MOE_BF16) {
      if (dy_dtype == MOE_BF16) launch_norm_backward<SRC_BF16, ROW_BF16>(a, grid, stream);
      else launch_norm_backward<SRC_BF16, ROW_F32>(a, grid, stream);
    } else {
      if (dy_dtype == MOE_BF16) launch_norm_backward<SRC_F32, ROW_BF16>(a, grid, stream);
      else launch_norm_backward<SRC_F32, ROW_F32>(a, grid, stream);
    }
  }
  if (grid != 1 && (dweight || dbias))  // with no rows the sums are zero
    launch_reduce(pw, pb, grid, d, dweight, dbias, stream);
  return check_launch("moe_norm_backward");
}
