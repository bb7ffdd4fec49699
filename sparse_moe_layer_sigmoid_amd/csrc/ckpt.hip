// Activation checkpoints in 8 bits and the backward kernels that read them ("DeepSeek-V3 Technical
// Report" (wiki summary), "FP8 混合精度訓練", 低精度ストレージ・通信: activations are kept for the
// backward pass in low precision).
//
// Format: E4M3 codes [rows, cols] and one E8M0 scale code per 1x128 tile [rows, ceil(cols / 128)],
// the scale the least 2^k with amax <= 448 * 2^k.  A power of two, so that packing rounds once
// (the scaling is exact, whatever the input type), a value code * 2^k is exact in bf16 too (from k =
// -124 on; below, it can fall between bf16's subnormals and is rounded to them), and a scale costs one byte: 1.008 bytes per element against 4 (f32 gate | up products) or 2 (bf16).
//
//  * fp8_ckpt_pack / fp8_ckpt_unpack: streaming passes, 8 elements per lane, 16 lanes per tile, the
//    tile's maximum by lane rotations.  36864 x 4096 f32 packed in 128 us (5.9 TB/s of 755 MB), bf16
//    in 79 us (5.7 TB/s), unpacked to bf16 in 85 us (5.3 TB/s; 88 us with ordinary stores).
//  * moe_swiglu_backward_ckpt: moe_swiglu_backward from the packed a | c; it also gives back
//    h = silu(a) c, which the down projection's weight gradient needs, so h is not kept at all.
//    36864 x 2048: 153 us (5.9 TB/s; 156 us with ordinary stores, 160 us with 8-byte ones).
//  * moe_combine_backward_ckpt: moe_combine_backward from the packed expert outputs.  4096 tokens of
//    8 experts, 7168 columns: 175-180 us (4.65 TB/s, two thirds of it stores), alike with 256 lanes a
//    token or non-temporal stores, 273 us with 896 lanes.
// All are bound by HBM: a 2 GiB copy on the same card runs at 4.9 TB/s, a read-only stream at 6.1.
#include "abi_common.h"
#include "device_common.h"
#include "quant_common.h"
#include "rows_common.h"

namespace moe {
namespace {

constexpr int kMaxBwdK = 32;

template <int XT, bool FULL>
__global__ __launch_bounds__(256) void ckpt_pack_kernel(const void* __restrict__ x, int64_t ldx_b, int64_t rows,
                                                        int cols, RowSplit sp, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scale) {
  int64_t r;
  int ch;
  split_chunk(sp, r, ch);  // per_row is a multiple of 16: a tile is one 16-lane row
  if (r >= rows) return;   // whole tiles leave together
  const int c = ch * 8;
  float f[8];
  if (c < cols) {
    values8(load8<XT, FULL>(static_cast<const char*>(x) + r * ldx_b, c, cols), f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
  }
  uint32_t code;
  const u32x2 v = ckpt_encode8(f, code);
  if (c < cols) {
    store_codes8<FULL>(q + r * cols, c, cols, v);
    if ((ch & 15) == 0) scale[r * (sp.per_row / 16) + ch / 16] = (uint8_t)code;
  }
}

template <bool FULL>
__global__ __launch_bounds__(256) void ckpt_unpack_kernel(const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scale, int64_t rows, int cols,
                                                          int tiles, RowSplit sp, const void* __restrict__ w,
                                                          const void* __restrict__ b, int w_dtype, void* out,
                                                          int out_dtype, int64_t ldo_b) {
  int64_t r;
  int ch;
  split_chunk(sp, r, ch);
  if (r >= rows) return;
  const int c = ch * 8;
  float f[8];
  ckpt_decode8(load_codes8<FULL>(q + r * cols, c, cols), scale[r * tiles + ch / 16], f);
  if (w) {
    float v[8];
    load8_any<FULL>(w_dtype, w, c, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= v[e];
  }
  if (b) {
    float v[8];
    load8_any<FULL>(w_dtype, b, c, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += v[e];
  }
  store8_any<FULL, true>(out_dtype, static_cast<char*>(out) + r * ldo_b, c, cols, f);
}

// CH elements of h per lane: 8 where inter % 8 == 0, else 4; neither straddles a scale tile of
// a (columns [0, inter)) or of c (columns [inter, 2 inter)).
template <int CH>
__global__ __launch_bounds__(256) void swiglu_backward_ckpt_kernel(const uint8_t* __restrict__ q,
                                                                   const uint8_t* __restrict__ scale,
                                                                   const float* __restrict__ dh, int64_t rows, int I,
                                                                   int tiles, RowSplit sp, uint16_t* __restrict__ dac,
                                                                   uint8_t* __restrict__ dacq,
                                                                   float* __restrict__ dacs, uint16_t* __restrict__ h) {
  int64_t r;
  int ch;
  split_chunk(sp, r, ch);
  if (r >= rows) return;
  const int i = ch * CH;
  const uint8_t* qr = q + r * 2 * I;
  const uint8_t* sr = scale + r * tiles;
  const uint32_t sa = sr[i / 128], sc = sr[(I + i) / 128];
  float a[CH], c[CH], g[CH];
#pragma unroll
  for (int k = 0; k < CH / 4; ++k) {
    const f32x4 v = *(const f32x4*)(dh + r * I + i + 4 * k);
#pragma unroll
    for (int e = 0; e < 4; ++e) g[4 * k + e] = v[e];
  }
  if constexpr (CH == 8) {
    ckpt_decode8(*(const u32x2*)(qr + i), sa, a);
    ckpt_decode8(*(const u32x2*)(qr + I + i), sc, c);
  } else {
    ckpt_decode4(*(const uint32_t*)(qr + i), sa, a);
    ckpt_decode4(*(const uint32_t*)(qr + I + i), sc, c);
  }
  float da[CH], dc[CH], hv[CH];
#pragma unroll
  for (int e = 0; e < CH; ++e) {
    const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-a[e]));
    const float s = a[e] * sg;
    dc[e] = g[e] * s;
    da[e] = g[e] * c[e] * (sg * (1.0f + a[e] * (1.0f - sg)));
    hv[e] = s * c[e];
  }
  auto store = [&](uint16_t* p, const float(&v)[CH]) __attribute__((always_inline)) {
    if constexpr (CH == 8) {
      __builtin_nontemporal_store(pack_bf16x8(v), reinterpret_cast<u32x4*>(p));
    } else {
      *(u32x2*)p = u32x2{f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16),
                         f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16)};
    }
  };
  store(dac + r * 2 * I + i, da);
  store(dac + r * 2 * I + I + i, dc);
  if (h) store(h + r * I + i, hv);
  if constexpr (CH == 8) {
    if (dacq) {
      // the 1x128 E4M3 form of the stored bf16 da | dc, as fp8_quant_1x128 gives it (I % 128 == 0, so
      // a tile is 16 lanes of one row)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float f[8], amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = bf16_to_f32(f32_to_bf16_rne(half ? dc[e] : da[e]));
          amax = fmaxf(amax, fabsf(f[e]));
        }
        amax = max16(amax);
        const float s = (amax == 0.f) ? 1.0f : amax / 448.0f;
        const int col = half * I + i;
        *(u32x2*)(dacq + r * 2 * I + col) = encode8(f, s);
        if ((i & 127) == 0) dacs[r * (2 * I / 128) + col / 128] = s;
      }
    }
  }
}

// One workgroup per token, as moe_combine_backward: KT bounds the unrolled loop over the pairs.
template <int KT>
__global__ __launch_bounds__(512) void combine_backward_ckpt_kernel(
    const uint16_t* __restrict__ d_out, const uint8_t* __restrict__ yq, const uint8_t* __restrict__ ysc,
    const int32_t* __restrict__ idx, const float* __restrict__ gate, const float* __restrict__ scores,
    const int32_t* __restrict__ pair_pos, int T, int K, int d, int N, uint16_t* __restrict__ dy,
    float* __restrict__ du, float* __restrict__ du_row, uint8_t* __restrict__ dyq, float* __restrict__ dys) {
  __shared__ int s_p[KT];
  __shared__ float s_g[KT];
  __shared__ float s_part[KT][8];
  const int t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  if (tid < K) {
    s_p[tid] = pair_pos[(int64_t)t * K + tid];
    s_g[tid] = gate[(int64_t)t * K + tid];
  }
  __syncthreads();
  float dot[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k) dot[k] = 0.f;
  const int nc = d / 8, tiles = (d + 127) / 128;
  const uint16_t* orow = d_out + (int64_t)t * d;
  // with dyq: each dy row also as E4M3 with 1x128 scales, from its bf16 values as fp8_quant_1x128
  // (d % 128 == 0, so whole 16-lane groups share the loop's trip count)
  auto quant_row = [&](int64_t row, int c, const u32x4& bits) __attribute__((always_inline)) {
    float v[8], amax = 0.f;
    unpack_bf16x8(bits, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = max16(amax);
    const float s = (amax == 0.f) ? 1.0f : amax / 448.0f;
    *(u32x2*)(dyq + row * d + c * 8) = encode8(v, s);
    if ((c & 15) == 0) dys[row * (d / 128) + c / 16] = s;
  };
  for (int c = tid; c < nc; c += blockDim.x) {
    const u32x4 ov = *(const u32x4*)(orow + c * 8);
    u32x2 q[KT];
    uint32_t sc[KT];
    if constexpr (KT <= 8) {  // all of the pairs' loads first
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        q[k] = u32x2{0u, 0u};
        sc[k] = 0;
        if (k < K && s_p[k] >= 0) {
          q[k] = *(const u32x2*)(yq + (int64_t)s_p[k] * d + c * 8);
          sc[k] = ysc[(int64_t)s_p[k] * tiles + c / 16];
        }
      }
    }
    *(u32x4*)(dy + ((int64_t)T * K + t) * d + c * 8) = ov;  // the shared expert's row: d_out itself
    if (dyq) quant_row((int64_t)T * K + t, c, ov);
    float f[8];
    unpack_bf16x8(ov, f);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      if (k < K && s_p[k] >= 0) {  // pairs skipped by the permutation (p < 0) carry nothing
        const int64_t p = s_p[k];
        if constexpr (KT > 8) {
          q[k] = *(const u32x2*)(yq + p * d + c * 8);
          sc[k] = ysc[p * tiles + c / 16];
        }
        float yv[8];
        ckpt_decode8(q[k], sc[k], yv);
        float acc = dot[k];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = fmaf(f[i], yv[i], acc);
        dot[k] = acc;
        const float g = s_g[k];
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f32_to_bf16_rne(g * f[2 * i]) | (f32_to_bf16_rne(g * f[2 * i + 1]) << 16);
        *(u32x4*)(dy + p * d + c * 8) = o;
        if (dyq) quant_row(p, c, o);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < KT; ++k) {
    if (k < K) {
      const float v = wave_sum(dot[k]);
      if (lane == 0) s_part[k][wave] = v;
    }
  }
  __syncthreads();
  if (wave == 0) {
    // lane k < K: gate gradient, selected affinity; then the two sums over the K lanes
    float dg = 0.f, s = 0.f, g = 0.f;
    const int e = lane < K ? idx[(int64_t)t * K + lane] : -1;
    const bool valid = lane < K && s_p[lane] >= 0 && e >= 0 && e < N;
    if (valid) {
      for (int w = 0; w < nw; ++w) dg += s_part[lane][w];
      s = scores[(int64_t)t * N + e];
      g = s_g[lane];
    }
    const float S = wave_sum(s), gd = wave_sum(g * dg);
    if (lane < K) {
      const float u = valid ? (dg - gd) / S * (s * (1.0f - s)) : 0.f;
      du[(int64_t)t * K + lane] = u;
      if (valid) du_row[s_p[lane]] = u;
    }
  }
}

bool row_dtype(int t) { return t == MOE_BF16 || t == MOE_F32; }
int row_esz(int t) { return t == MOE_BF16 ? 2 : 4; }
bool elem_aligned(const void* p, int esz) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(esz - 1)) == 0; }
constexpr int kMaxCols = 1 << 24;

}  // namespace
}  // namespace moe

extern "C" moe_status fp8_ckpt_pack(const void* x, int x_dtype, int64_t rows, int cols, int64_t ldx, uint8_t* q,
                                    uint8_t* scale, hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(rows == 0 || (x && q && scale), MOE_ERR_NULL, "fp8_ckpt_pack: a required pointer is NULL");
  MOE_REQUIRE(row_dtype(x_dtype), MOE_ERR_DTYPE, "fp8_ckpt_pack: x must be MOE_BF16 or MOE_F32 (%d)", x_dtype);
  MOE_REQUIRE(rows >= 0 && cols >= 1 && cols <= kMaxCols, MOE_ERR_SHAPE, "fp8_ckpt_pack: rows=%lld cols=%d (1..%d)",
              (long long)rows, cols, kMaxCols);
  MOE_REQUIRE((ldx >= cols || rows <= 1) && elem_aligned(x, row_esz(x_dtype)), MOE_ERR_ALIGN,
              "fp8_ckpt_pack: ldx=%lld must be >= cols and x aligned to its elements", (long long)ldx);
  if (rows > 0) {
    const int tiles = (cols + 127) / 128;
    MOE_REQUIRE(rows <= kMaxLanes / (tiles * 16), MOE_ERR_SHAPE, "fp8_ckpt_pack: too many rows");
    const int64_t grid = (rows * tiles * 16 + 255) / 256;
    const RowSplit sp = make_row_split((uint32_t)tiles * 16);
    const bool full = cols % 8 == 0;
    auto kernel = x_dtype == MOE_BF16 ? (full ? ckpt_pack_kernel<ROW_BF16, true> : ckpt_pack_kernel<ROW_BF16, false>)
                                      : (full ? ckpt_pack_kernel<ROW_F32, true> : ckpt_pack_kernel<ROW_F32, false>);
    kernel<<<(unsigned)grid, 256, 0, stream>>>(x, ldx * row_esz(x_dtype), rows, cols, sp, q, scale);
  }
  return check_launch("fp8_ckpt_pack");
}

extern "C" moe_status fp8_ckpt_unpack(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols,
                                      const void* weight, const void* bias, int w_dtype, void* out, int out_dtype,
                                      int64_t ldo, hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(rows == 0 || (q && scale && out), MOE_ERR_NULL, "fp8_ckpt_unpack: a required pointer is NULL");
  MOE_REQUIRE(row_dtype(out_dtype) && row_dtype(w_dtype), MOE_ERR_DTYPE,
              "fp8_ckpt_unpack: out and weights must be MOE_BF16 or MOE_F32 (%d, %d)", out_dtype, w_dtype);
  MOE_REQUIRE(rows >= 0 && cols >= 1 && cols <= kMaxCols, MOE_ERR_SHAPE, "fp8_ckpt_unpack: rows=%lld cols=%d (1..%d)",
              (long long)rows, cols, kMaxCols);
  MOE_REQUIRE((ldo >= cols || rows <= 1) && elem_aligned(out, row_esz(out_dtype)) &&
                  elem_aligned(weight, row_esz(w_dtype)) && elem_aligned(bias, row_esz(w_dtype)),
              MOE_ERR_ALIGN, "fp8_ckpt_unpack: ldo=%lld must be >= cols and pointers aligned to their elements",
              (long long)ldo);
  if (rows > 0) {
    const int tiles = (cols + 127) / 128, chunks = (cols + 7) / 8;
    MOE_REQUIRE(rows <= kMaxLanes / chunks, MOE_ERR_SHAPE, "fp8_ckpt_unpack: too many rows");
    const int64_t grid = (rows * chunks + 255) / 256;
    auto kernel = cols % 8 == 0 ? ckpt_unpack_kernel<true> : ckpt_unpack_kernel<false>;
    kernel<<<(unsigned)grid, 256, 0, stream>>>(q, scale, rows, cols, tiles, make_row_split(chunks), weight, bias, w_dtype,
                                               out, out_dtype, ldo * row_esz(out_dtype));
  }
  return check_launch("fp8_ckpt_unpack");
}

extern "C" moe_status moe_swiglu_backward_ckpt(const uint8_t* ac_q, const uint8_t* ac_scale, const float* dh,
                                               int64_t rows, int inter, uint16_t* dac, uint8_t* dac_q,
                                               float* dac_scale, uint16_t* h, hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(rows == 0 || (ac_q && ac_scale && dh && dac), MOE_ERR_NULL,
              "moe_swiglu_backward_ckpt: a required pointer is NULL");
  MOE_REQUIRE(!dac_q == !dac_scale, MOE_ERR_NULL, "moe_swiglu_backward_ckpt: dac_q and dac_scale go together");
  MOE_REQUIRE(rows >= 0 && inter >= 4 && inter % 4 == 0 && inter <= kMaxCols && (!dac_q || inter % 128 == 0),
              MOE_ERR_SHAPE,
              "moe_swiglu_backward_ckpt: rows=%lld inter=%d (a positive multiple of 4; of 128 with dac_q)",
              (long long)rows, inter);
  MOE_REQUIRE(aligned16(ac_q) && aligned16(dh) && aligned16(dac) && aligned16(dac_q) && aligned16(h) &&
                  elem_aligned(dac_scale, 4),
              MOE_ERR_ALIGN, "moe_swiglu_backward_ckpt: ac_q, dh, dac, dac_q and h must be 16-byte aligned");
  if (rows > 0) {
    const bool wide = inter % 8 == 0;
    const int per_row = inter / (wide ? 8 : 4), tiles = (2 * inter + 127) / 128;
    MOE_REQUIRE(rows <= kMaxLanes / per_row, MOE_ERR_SHAPE, "moe_swiglu_backward_ckpt: too many rows");
    const unsigned grid = (unsigned)((rows * per_row + 255) / 256);
    const RowSplit sp = make_row_split(per_row);
    if (wide)
      swiglu_backward_ckpt_kernel<8><<<grid, 256, 0, stream>>>(ac_q, ac_scale, dh, rows, inter, tiles, sp, dac, dac_q,
                                                               dac_scale, h);
    else
      swiglu_backward_ckpt_kernel<4><<<grid, 256, 0, stream>>>(ac_q, ac_scale, dh, rows, inter, tiles, sp, dac, dac_q,
                                                               dac_scale, h);
  }
  return check_launch("moe_swiglu_backward_ckpt");
}

extern "C" moe_status moe_combine_backward_ckpt(const uint16_t* d_out, const uint8_t* y_q, const uint8_t* y_scale,
                                                const int32_t* topk_idx, const float* topk_gate, const float* scores,
                                                const int32_t* pair_pos, int T, int top_k, int d, int n_experts,
                                                uint16_t* dy, float* du, float* du_row, uint8_t* dy_q, float* dy_scale,
                                                hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(T == 0 || (d_out && y_q && y_scale && topk_idx && topk_gate && scores && pair_pos && dy && du && du_row),
              MOE_ERR_NULL, "moe_combine_backward_ckpt: a required pointer is NULL");
  MOE_REQUIRE(!dy_q == !dy_scale, MOE_ERR_NULL, "moe_combine_backward_ckpt: dy_q and dy_scale go together");
  MOE_REQUIRE(T >= 0 && top_k >= 1 && top_k <= kMaxBwdK && top_k <= n_experts && d >= 8 && d % 8 == 0 &&
                  (!dy_q || d % 128 == 0),
              MOE_ERR_SHAPE,
              "moe_combine_backward_ckpt: T=%d top_k=%d (1..%d) d=%d (a multiple of 8; of 128 with dy_q) n_experts=%d",
              T, top_k, kMaxBwdK, d, n_experts);
  MOE_REQUIRE(aligned16(d_out) && ((uintptr_t)y_q & 7u) == 0 && aligned16(dy) && ((uintptr_t)dy_q & 7u) == 0 &&
                  elem_aligned(dy_scale, 4),
              MOE_ERR_ALIGN, "moe_combine_backward_ckpt: d_out and dy must be 16-byte, y_q and dy_q 8-byte aligned");
  if (T > 0) {
    const int threads = d <= 512 ? 64 : d <= 2048 ? 256 : 448;
    MOE_REQUIRE(T <= kMaxLanes / threads, MOE_ERR_SHAPE, "moe_combine_backward_ckpt: too many tokens (%d)", T);
    if (top_k <= 8)
      combine_backward_ckpt_kernel<8><<<T, threads, 0, stream>>>(d_out, y_q, y_scale, topk_idx, topk_gate, scores,
                                                                 pair_pos, T, top_k, d, n_experts, dy, du, du_row, dy_q,
                                                                 dy_scale);
    else
      combine_backward_ckpt_kernel<kMaxBwdK><<<T, threads, 0, stream>>>(d_out, y_q, y_scale, topk_idx, topk_gate,
                                                                        scores, pair_pos, T, top_k, d, n_experts, dy,
                                                                        du, du_row, dy_q, dy_scale);
  }
  return check_launch("moe_combine_backward_ckpt");
}
