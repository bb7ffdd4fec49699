// i8_quant / i8_dequant / moe_i8_gemm: rows in 8-bit integers with one scale each, and the experts' products of them.
//
//   A = max(max_k |x_rk|, 127 * 2^-126),  s_r = A / 127,  q_rk = RNE(127 x_rk / A)
//   out[r, n] = (sum_k aq_rk wq_nk) (as_r ws_n)          (SwiGLU: silu of the gate column times the up column)
//
// Codes and weights multiply and add exactly in 32-bit integers, so the scales are all that rounds: a row's and a channel's
// scale are constant along K and meet the sum once, in the epilogue.
#include <type_traits>

#include "abi_common.h"
#include "device_common.h"
#include "group_rows.h"
#include "rows_common.h"

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

namespace moe {
namespace {

constexpr float kLeast = 127.0f * 1.17549435e-38f;  // 127 * 2^-126: below it a scale would be subnormal

// ---- rows to codes ----

// 8 values -> codes RNE(127 v / A).  Values and A go times 2^-e, e the exponent of A, so that 127 v stays in range (exact but
// for values that round to code 0 anyway).  Of bf16 values 127 v is exact, and a quotient that is not at a midpoint is further from
// it than the quotient's own rounding (254 v and (2 c + 1) A have 16 bits each): the corrected reciprocal gives the codes of an exact
// division.  Of f32 values 127 v and the quotient are each off by 2^-24 of themselves, together by less than 2^-16: where a
// midpoint is that near (a value in 32 thousand), the remainder decides, exact in 64 bits, for v and A are multiples of 2^-33 there.
template <int DT>
__device__ __forceinline__ u32x2 i8_encode8(const float f[8], int e, float a, float ra) {
  u32x2 q = {0u, 0u};
  float v[8], c[8], off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = ldexpf(f[i], -e);
    const float t = quotient(127.0f * v[i], a, ra);
    c[i] = __builtin_rintf(t);
    if constexpr (DT == ROW_F32) off = fmaxf(off, fabsf(t - c[i]));
  }
  if (DT == ROW_F32 && off >= 0.5f - 0x1p-16f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double rest = fma((double)-c[i], (double)a, 127.0 * (double)v[i]), half = 0.5 * (double)a;
      const bool odd = ((int)c[i] & 1) != 0;
      if (fabs(rest) > half || (fabs(rest) == half && odd)) c[i] += rest > 0.0 ? 1.0f : -1.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i / 4] |= ((uint32_t)(int)c[i] & 255u) << (8 * (i & 3));
  return q;
}

// A row by L lanes (64: a wave of a workgroup of four; else the whole workgroup), CH chunks of 8 elements in each lane's
// registers: one read of the row.  CH = 0: any width, the row read twice.
template <int DT, int L, int CH>
__global__ __launch_bounds__(L < 256 ? 256 : L) void i8_quant_kernel(const void* __restrict__ x, int64_t ldx_b, int64_t rows,
                                                                     int cols, int8_t* __restrict__ q,
                                                                     float* __restrict__ scale) {
  constexpr int PER = L < 256 ? 256 / L : 1;  // rows per workgroup
  __shared__ uint32_t red[L < 256 ? 1 : L / 64];
  const int lane = threadIdx.x % L;
  const int64_t r = (int64_t)blockIdx.x * PER + threadIdx.x / L;
  if (PER > 1 && r >= rows) return;  // whole waves
  const uint8_t* row = static_cast<const uint8_t*>(x) + r * ldx_b;
  uint32_t top = 0;
  Raw8<DT> v[CH > 0 ? CH : 1];
  auto reduce = [&](const Raw8<DT>& w) __attribute__((always_inline)) {
    float f[8];
    values8(w, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int j = 0; j < CH; ++j) v[j] = load8<DT, false>(row, (lane + j * L) * 8, cols);
#pragma unroll
    for (int j = 0; j < CH; ++j) reduce(v[j]);
  } else {
    for (int c = lane * 8; c < cols; c += L * 8) reduce(load8<DT, false>(row, c, cols));
  }
  top = max16_u32(top);
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < L / 64; ++w) top = max(top, red[w]);
  }
  const bool bad = top >= 0x7f800000u;  // an infinity or NaN: the scale says NaN, the codes are 0
  const float A = fmaxf(bad ? 1.0f : __uint_as_float(top), kLeast);
  if (lane == 0) scale[r] = bad ? __uint_as_float(0x7fc00000u) : A / 127.0f;
  const int e = __builtin_amdgcn_frexp_expf(A);
  const float a = ldexpf(A, -e), ra = recip_refined(a);
  uint8_t* out = reinterpret_cast<uint8_t*>(q) + r * cols;
  auto put = [&](const Raw8<DT>& w, int c) __attribute__((always_inline)) {
    float f[8];
    values8(w, f);
    const u32x2 code = i8_encode8<DT>(f, e, a, ra);
    if (c < cols) store_codes8<false>(out, c, cols, bad ? u32x2{0u, 0u} : code);
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int j = 0; j < CH; ++j) put(v[j], (lane + j * L) * 8);
  } else {
    for (int c = lane * 8; c < cols; c += L * 8) put(load8<DT, false>(row, c, cols), c);
  }
}

// ---- codes to values ----
__global__ __launch_bounds__(256) void i8_dequant_kernel(const int8_t* __restrict__ q, const float* __restrict__ scale,
                                                         int64_t rows, int cols, RowSplit sp, void* __restrict__ out,
                                                         int out_dtype, int64_t ldo_b) {
  int64_t r;
  int chunk;
  split_chunk(sp, r, chunk);
  if (r >= rows) return;
  const int c = chunk * 8;
  const u32x2 code = load_codes8<false>(reinterpret_cast<const uint8_t*>(q) + r * cols, c, cols);
  const float s = scale[r];
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)(int8_t)(code[i / 4] >> (8 * (i & 3))) * s;
  store8_any<false>(out_dtype, static_cast<uint8_t*>(out) + r * ldo_b, c, cols, f);
}

// ---- products ----

#define I8_BARRIER()                                                          \
  do {                                                                        \
    __builtin_amdgcn_s_waitcnt((15) | (7 << 4) | (0 << 8) | (3 << 14));       \
    __builtin_amdgcn_s_barrier();                                             \
    asm volatile("" ::: "memory");                                            \
  } while (0)

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void glb_void;

__device__ const __attribute__((aligned(16))) uint8_t kZeros[16] = {};

struct I8Args {
  GroupRows rows;
  const uint8_t* a;
  const float* a_scale;
  const int32_t* a_rows;
  int64_t lda;            // bytes per A row
  const uint8_t* w;
  const float* w_scale;
  int first_group;
  int N;                  // rows of each W[g]
  int K;
  int n_tiles;            // column blocks
  int out_cols;
  uint8_t* out;
  int out_dtype;
  int64_t ldo_b;
  uint8_t* out_tail;
  int64_t ldo_tail_b;
};

struct Tile {
  int g, nt, row0, nrows;
};

// Persistent workgroups of WGM x WGN waves, one to a CU, walk tiles of BM rows x BN weight rows (SwiGLU: BN/2 gate rows and
// their up rows).  Both operands come by direct-to-LDS loads in steps of 128 bytes of K (a cache line: steps of 64 ask L2 for
// twice as many), three steps in flight in a ring that runs on over tile boundaries; 16-byte chunks are XOR-swizzled by row so
// that operand reads meet distinct banks.  A tile's scales travel the same way, its row numbers a tile ahead.  Tiles go by
// expert, column block, row block, a contiguous range to each XCD.
//
// Few rows to an expert: the weights' bytes bound it (256 tokens' down projection: 3.4 GB at 5.9 TB/s, a copy has 5.1).  Many:
// 192 x 192 is the most products per loaded byte of which LDS holds three steps.  16384 tokens' down projection (147456 rows,
// 7168 x 2048) takes 2.62 ms, 1.65 Pop/s; the library's largest 8-bit product on this card has 2.14.  The clock is down to
// 1.8 GHz, and what is left is rows of short tiles (an eighth) and, at a tile's end, its stores, which the next step's wait for
// loads includes.
template <int BM, int BN, int WGM, int WGN, bool SWIGLU>
__global__ __launch_bounds__(WGM * WGN * 64) void i8_gemm_kernel(I8Args p) {
  constexpr int NW = WGM * WGN;
  constexpr int WM = BM / WGM, WN = BN / WGN;
  constexpr int TM = WM / 16, TN = WN / 16;
  constexpr int STAGES = 3, A_BYTES = BM * 128, STAGE = (BM + BN) * 128;
  constexpr int A_PW = BM / 8 / NW, B_PW = BN / 8 / NW, L_STAGE = A_PW + B_PW;
  constexpr int OC = SWIGLU ? BN / 2 : BN;
  constexpr int SC = BM + BN;  // scales of a tile
  static_assert(A_PW * NW * 8 == BM && B_PW * NW * 8 == BN, "loads split evenly over the waves");
  static_assert(SC % 4 == 0 && BM % 4 == 0, "a tile's scales and its column scales begin at 16 bytes");
  static_assert(SC / 64 <= NW, "one load of scales per wave at most");
  static_assert(!SWIGLU || TN % 2 == 0, "a wave holds gate columns and their up columns");
  __shared__ __attribute__((aligned(1024))) uint8_t slot0[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t slot1[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t slot2[STAGE];
  // row scales, then column scales, read four at a time; loads are up to two tiles ahead
  __shared__ __attribute__((aligned(16))) float s_scale[STAGES][SC];
  __shared__ int s_tstart[kMaxRowGroups + 1], s_off[kMaxRowGroups + 1];
  __shared__ int s_rows[NW][64], s_srows[BM / 64][64];  // row numbers of the next tile: of a wave's loads, and of scales
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave - wm * WGN;
  const int G = p.rows.n_groups;
  const int32_t* offs = p.rows.offs;
  const int limit = __builtin_amdgcn_readfirstlane(rows_end(p.rows));
  for (int g = tid; g <= G; g += NW * 64) s_off[g] = min(offs[g], limit);
  if (wave == 0) {  // tiles before each group
    const int per = (G + 63) >> 6, g0 = min(G, lane * per), g1 = min(G, g0 + per);
    auto tiles = [&](int g) { return (max(min(offs[g + 1], limit) - min(offs[g], limit), 0) + BM - 1) / BM * p.n_tiles; };
    int local = 0;
    for (int g = g0; g < g1; ++g) local += tiles(g);
    int incl = local;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    int run = incl - local;
    for (int g = g0; g < g1; ++g) {
      s_tstart[g] = run;
      run += tiles(g);
    }
    if (lane == 63) s_tstart[G] = incl;
  }
  __syncthreads();
  const int total = s_tstart[G];
  const int n_xcd = gridDim.x >= 8 ? 8 : 1;
  const int xcd = blockIdx.x % n_xcd, seat = blockIdx.x / n_xcd, seats = gridDim.x / n_xcd;
  const int t_begin = (int)((int64_t)total * xcd / n_xcd), t_end = (int)((int64_t)total * (xcd + 1) / n_xcd);
  const int n_my = t_end - t_begin > seat ? (t_end - t_begin - seat + seats - 1) / seats : 0;
  const int ksteps = max((p.K + 127) / 128, 2);  // steps past K are zeros
  const int k_chunks = p.K / 16;
  const int total_steps = n_my * ksteps;
  if (total_steps == 0) return;

  // Tile q of this workgroup, found from the group of an earlier one: tiles rise with q.  A lane each looks at the next 64 groups.
  auto tile_of = [&](int q, int from) __attribute__((always_inline)) {
    const int L = t_begin + seat + q * seats;
    Tile t;
    t.g = from;
    for (;;) {
      const int n = __popcll(__ballot(s_tstart[min(t.g + 1 + lane, G)] <= L && t.g + 1 + lane <= G));
      t.g += n;
      if (n < 64) break;
    }
    t.g = __builtin_amdgcn_readfirstlane(t.g);
    const int m0 = __builtin_amdgcn_readfirstlane(s_off[t.g]), m1 = __builtin_amdgcn_readfirstlane(s_off[t.g + 1]);
    const int local = L - __builtin_amdgcn_readfirstlane(s_tstart[t.g]), blocks = (m1 - m0 + BM - 1) / BM;
    t.nt = (int)((uint32_t)local / (uint32_t)blocks);
    t.row0 = m0 + (local - t.nt * blocks) * BM;
    t.nrows = min(BM, m1 - t.row0);
    return t;
  };

  // ---- loads ----
  const int cch = lane & 7, lrow = lane >> 3;
  const uint8_t* a_ptr[A_PW];
  const uint8_t* b_ptr[B_PW];
  const float* sc_ptr = p.a_scale;  // this lane's scale of the tile
  const int chunk_of_row = cch ^ lrow;  // rows of a load are a multiple of 8 plus lrow
  // Row numbers of a tile go to LDS a tile ahead: in registers they would have to be waited for with everything else in flight.
  // They are older than the loads of the step that they were asked in, so the next step's wait covers them.
  auto tile_row = [&](const Tile& t, int r) __attribute__((always_inline)) { return t.row0 + min(r, t.nrows - 1); };
  auto fetch_rows = [&](const Tile& t) __attribute__((always_inline)) {
    if (!p.a_rows) return;
    __builtin_amdgcn_global_load_lds((glb_void*)(p.a_rows + tile_row(t, wave * A_PW * 8 + min(lane, A_PW * 8 - 1))),
                                     (lds_void*)s_rows[wave], 4, 0, 0);
    if (wave < BM / 64)
      __builtin_amdgcn_global_load_lds((glb_void*)(p.a_rows + tile_row(t, wave * 64 + lane)), (lds_void*)s_srows[wave], 4, 0, 0);
  };
  auto row_number = [&](const Tile& t, int r, const int* at) __attribute__((always_inline)) {
    int v = tile_row(t, r);
    if (p.a_rows) {  // (of a plain read the compiler would wait for all loads into LDS)
      const uint32_t a = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const int*)at;
      asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(v) : "v"(a) : "memory");
    }
    return v;
  };
  auto weight_row = [&](int nt, int rr) __attribute__((always_inline)) {
    if constexpr (SWIGLU) {
      const int c = min(nt * (BN / 2) + (rr < BN / 2 ? rr : rr - BN / 2), p.N / 2 - 1);
      return rr < BN / 2 ? c : p.N / 2 + c;
    } else {
      return min(nt * BN + rr, p.N - 1);
    }
  };
  auto set_tile = [&](const Tile& t) __attribute__((always_inline)) {
    const int64_t first = (int64_t)(p.first_group + t.g) * p.N;
#pragma unroll
    for (int i = 0; i < A_PW; ++i) a_ptr[i] = p.a + (int64_t)row_number(t, 8 * (wave * A_PW + i) + lrow, &s_rows[wave][i * 8 + lrow]) * p.lda + chunk_of_row * 16;
#pragma unroll
    for (int i = 0; i < B_PW; ++i)
      b_ptr[i] = p.w + (first + weight_row(t.nt, 8 * (wave * B_PW + i) + lrow)) * p.K + chunk_of_row * 16;
    if (wave < BM / 64) sc_ptr = p.a_scale + row_number(t, wave * 64 + lane, &s_srows[min(wave, BM / 64 - 1)][lane]);
    else sc_ptr = p.w_scale + first + weight_row(t.nt, min((wave - BM / 64) * 64, BN - 64) + lane);
  };
  Tile ct = tile_of(0, 0), lt = ct;  // the tile at work; the next one to load
  int lq = -1, dma_kt = 0, ld_kt = ksteps;  // tile and step of the batch being issued
  bool dma_ragged = false, dma_first = false;
  auto issue_prep = [&](int js) __attribute__((always_inline)) {
    dma_first = false;
    if (js < total_steps) {  // past the end the last step is loaded again: the number in flight stays
      if (++ld_kt >= ksteps) {
        ld_kt = 0;
        ++lq;
        set_tile(lt);
        if (lq + 1 < n_my) {
          lt = tile_of(lq + 1, lt.g);
          fetch_rows(lt);
        }
        dma_first = true;
      }
    }
    dma_kt = ld_kt;
    dma_ragged = ld_kt * 8 + chunk_of_row >= k_chunks;
  };
  auto issue_one = [&](auto slot_c, int k) __attribute__((always_inline)) {
    constexpr int SL = decltype(slot_c)::value;
    uint8_t* st = SL == 0 ? slot0 : (SL == 1 ? slot1 : slot2);
    if (k < A_PW) {  // chunks past the row: zeros against whatever the weights hold there
      const uint8_t* src = dma_ragged ? kZeros : a_ptr[k] + dma_kt * 128;
      __builtin_amdgcn_global_load_lds((glb_void*)src, (lds_void*)(st + (wave * A_PW + k) * 1024), 16, 0, 0);
    } else {
      const int i = k - A_PW;
      const uint8_t* src = b_ptr[i] + (dma_ragged ? -chunk_of_row * 16 : dma_kt * 128);
      __builtin_amdgcn_global_load_lds((glb_void*)src, (lds_void*)(st + A_BYTES + (wave * B_PW + i) * 1024), 16, 0, 0);
    }
  };
  auto issue_scales = [&]() __attribute__((always_inline)) {
    if (dma_first && wave < SC / 64)
      __builtin_amdgcn_global_load_lds((glb_void*)sc_ptr, (lds_void*)(&s_scale[lq % STAGES][wave * 64]), 4, 0, 0);
  };
  auto issue = [&](auto slot_c, int js) __attribute__((always_inline)) {
    issue_prep(js);
#pragma unroll
    for (int k = 0; k < L_STAGE; ++k) issue_one(slot_c, k);
    issue_scales();
  };
  fetch_rows(ct);
  wait_vm<0>();
  issue(std::integral_constant<int, 0>(), 0);
  issue(std::integral_constant<int, 1>(), 1);
  if (ksteps == 2) wait_vm<0>();  // the second tile's rows
  issue(std::integral_constant<int, 2>(), 2);

  // ---- products: weights first, so a lane's four results are four columns of one token row ----
  const int lr = lane & 15, lg = lane >> 4;
  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  // a wave's blocks of 16 rows are every WGM-th one, so that a short tile's rows are shared out too
  const int sw_lo = (lg ^ (lr & 7)) << 4, sw_hi = sw_lo ^ 64;
  const int fa = (wm * 16 + lr) * 128;
  const int fb = (SWIGLU ? wn * (WN / 2) + lr : wn * WN + lr) * 128;
  const int base_row = __builtin_amdgcn_readfirstlane(s_off[0]);
  const int tail_row = __builtin_amdgcn_readfirstlane(s_off[p.rows.tail_first]);
  int c_q = 0, c_kt = 0;

  // A tile's results, as F32 or bf16; FULL: none of its columns is past the last one.
  auto store_tile = [&](const Tile& t, const float* sc, auto f32_c, auto full_c) __attribute__((always_inline)) {
    constexpr bool F32 = decltype(f32_c)::value, FULL = decltype(full_c)::value;
    constexpr int TO = SWIGLU ? TN / 2 : TN;
    const bool tail = t.g >= p.rows.tail_first;
    uint8_t* base = tail ? p.out_tail + (int64_t)(t.row0 - tail_row) * p.ldo_tail_b : p.out + (int64_t)(t.row0 - base_row) * p.ldo_b;
    const int64_t ldo_b = tail ? p.ldo_tail_b : p.ldo_b;
    const int c0 = (SWIGLU ? wn * (WN / 2) : wn * WN) + lg * 4;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = (i * WGM + wm) * 16 + lr;
      if (m >= t.nrows) continue;
      const float as = sc[m];
      uint8_t* o = base + m * ldo_b + (int64_t)(t.nt * OC + c0) * (F32 ? 4 : 2);
#pragma unroll
      for (int j = 0; j < TO; ++j) {
        const f32x4 ws = *(const f32x4*)(sc + BM + c0 + j * 16);
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = (float)acc[i][j][r] * (as * ws[r]);
        if constexpr (SWIGLU) {
          const f32x4 us = *(const f32x4*)(sc + BM + BN / 2 + c0 + j * 16);
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = silu(v[r]) * ((float)acc[i][j + TO][r] * (as * us[r]));
        }
        const u32x2 b = __builtin_bit_cast(u32x2, bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]});  // RNE
        const int left = FULL ? 4 : p.out_cols - (t.nt * OC + c0 + j * 16);
        if (left >= 4) {
          if constexpr (F32) *reinterpret_cast<f32x4_u*>(o + j * 64) = v;
          else *reinterpret_cast<u32x2_u*>(o + j * 32) = b;
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            if (e >= left) break;
            if constexpr (F32) reinterpret_cast<float*>(o + j * 64)[e] = v[e];
            else reinterpret_cast<uint16_t*>(o + j * 32)[e] = (uint16_t)(b[e / 2] >> (16 * (e & 1)));
          }
        }
      }
    }
  };
  auto epilogue = [&]() __attribute__((always_inline)) {
    const float* sc = s_scale[c_q % STAGES];
    const bool f32 = ct.g >= p.rows.tail_first || p.out_dtype == ROW_F32, full = (ct.nt + 1) * OC <= p.out_cols;
    if (full) {
      if (f32) store_tile(ct, sc, std::true_type(), std::true_type());
      else store_tile(ct, sc, std::false_type(), std::true_type());
    } else {
      if (f32) store_tile(ct, sc, std::true_type(), std::false_type());
      else store_tile(ct, sc, std::false_type(), std::false_type());
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    c_kt = 0;
    if (++c_q < n_my) ct = tile_of(c_q, ct.g);
  };

  // A step is two halves of 64 bytes of K.  A half's products run on operands in registers, and read the next half's between
  // them.  So at the barrier between step j's halves every wave has read all of slot j, and step j + 3 may be loaded into it; step
  // j + 1 has to be complete there.
  i32x4 af[2][TM], bf[2][TN];
  auto read_one = [&](auto slot_c, int half, int k) __attribute__((always_inline)) {
    constexpr int SL = decltype(slot_c)::value;
    const uint8_t* st = SL == 0 ? slot0 : (SL == 1 ? slot1 : slot2);
    const int sw = half ? sw_hi : sw_lo;
    if (k < TN) {
      const int row = SWIGLU && k >= TN / 2 ? BN / 2 + (k - TN / 2) * 16 : k * 16;
      bf[half][k] = *(const i32x4*)(st + A_BYTES + fb + sw + row * 128);
    } else {
      af[half][k - TN] = *(const i32x4*)(st + fa + sw + (k - TN) * (WGM * 16 * 128));
    }
  };
  auto half_step = [&](int half, auto read_c, auto load_c, bool load) __attribute__((always_inline)) {
    constexpr int n = TM * TN, reads = TM + TN;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int jj = 0; jj < TN; ++jj) {
        const int t = i * TN + jj;
        acc[i][jj] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[half][jj], af[half][i], acc[i][jj], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < reads; ++k)
          if (t == k * n / reads) read_one(read_c, half ^ 1, k);
        if (load) {
#pragma unroll
          for (int k = 0; k < L_STAGE; ++k)
            if (t == k * n / L_STAGE) issue_one(load_c, k);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  wait_vm<2 * L_STAGE>();
  I8_BARRIER();
#pragma unroll
  for (int k = 0; k < TM + TN; ++k) read_one(std::integral_constant<int, 0>(), 0, k);
  auto step = [&](auto slot_c, int j) __attribute__((always_inline)) {
    constexpr auto next = std::integral_constant<int, (decltype(slot_c)::value + 1) % 3>();
    half_step(0, slot_c, slot_c, false);
    wait_vm<L_STAGE>();
    I8_BARRIER();
    issue_prep(j + 3);
    half_step(1, next, slot_c, true);
    issue_scales();
    if (++c_kt == ksteps) epilogue();
  };
  int j = 0;
  for (; j + 3 <= total_steps; j += 3) {
    step(std::integral_constant<int, 0>(), j);
    step(std::integral_constant<int, 1>(), j + 1);
    step(std::integral_constant<int, 2>(), j + 2);
  }
  if (j < total_steps) step(std::integral_constant<int, 0>(), j);
  if (j + 1 < total_steps) step(std::integral_constant<int, 1>(), j + 1);
  wait_vm<0>();  // the repeated loads land before the workgroup's LDS is given away
}

int compute_units() {
  int dev = 0, v = 0;
  if (hipGetDevice(&dev) == hipSuccess && hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess &&
      v >= 8)
    return v / 8 * 8;
  return 256;
}

template <int BM, int BN, int WGM, int WGN, bool SWIGLU>
void launch_gemm(I8Args a, int64_t m_total, hipStream_t stream) {
  constexpr int OC = SWIGLU ? BN / 2 : BN;
  a.n_tiles = (a.out_cols + OC - 1) / OC;
  const int64_t full = m_total / BM + a.rows.n_groups;  // at most one short block a group, never more blocks than rows
  const int64_t tiles = (full < m_total ? full : m_total) * a.n_tiles;
  const int cus = compute_units();
  const int64_t grid = tiles < cus ? (tiles + 7) / 8 * 8 : cus;
  i8_gemm_kernel<BM, BN, WGM, WGN, SWIGLU><<<(unsigned)grid, WGM * WGN * 64, 0, stream>>>(a);
}

template <bool SWIGLU>
void dispatch_gemm(const I8Args& a, int64_t m_total, hipStream_t stream) {
  // By rows per expert: the low tile wastes fewer products where the weights' bytes are the time, the high one reads them fewer
  // times.  257 experts of 7168 x 2048, 8 to a token, 64 against 192 rows, ms (gate/up, down):
  //   even routing, 256 tokens (9 rows)     1.26 / 1.53, 0.66 / 0.78    2000 (70)  1.51 / 1.62, 0.85 / 0.88
  //                                         3000 (105)  1.85 / 1.70, 0.98 / 0.93
  //   popularity rank^-1.1, 256 tokens      1.15 / 1.41, 0.61 / 0.73    2000       1.61 / 1.81, 0.87 / 0.96
  //                                         3000        1.88 / 1.99, 0.99 / 1.08
  //   all tokens on the same 8, 256 tokens  0.13 / 0.11, 0.06 / 0.06    2000       0.74 / 0.51, 0.43 / 0.32
  //                                         3000        0.96 / 0.75, 0.56 / 0.46
  // The offsets are on the device, so the rule cannot see who is popular: skewed batches above 80 rows pay 6 to 10%, and a
  // collapse onto few experts below 80 pays up to 45%.
  if (m_total / a.rows.n_groups < 80) launch_gemm<64, 256, 1, 8, SWIGLU>(a, m_total, stream);
  else launch_gemm<192, 192, 4, 2, SWIGLU>(a, m_total, stream);
}

template <int DT, int L, int CH>
void launch_quant(const void* x, int64_t ldx_b, int64_t rows, int cols, int8_t* q, float* scale, hipStream_t stream) {
  constexpr int PER = L < 256 ? 256 / L : 1;
  i8_quant_kernel<DT, L, CH><<<(unsigned)((rows + PER - 1) / PER), L < 256 ? 256 : L, 0, stream>>>(x, ldx_b, rows, cols, q, scale);
}

template <int DT>
void dispatch_quant(const void* x, int64_t ldx, int64_t rows, int cols, int8_t* q, float* scale, hipStream_t stream) {
  const int64_t b = ldx * (DT == ROW_BF16 ? 2 : 4);
  if (cols <= 512) launch_quant<DT, 64, 1>(x, b, rows, cols, q, scale, stream);
  else if (cols <= 2048) launch_quant<DT, 256, 1>(x, b, rows, cols, q, scale, stream);
  else if (cols <= 4096) launch_quant<DT, 256, 2>(x, b, rows, cols, q, scale, stream);
  else if (cols <= 8192) launch_quant<DT, 1024, 1>(x, b, rows, cols, q, scale, stream);
  else if (cols <= 16384) launch_quant<DT, 1024, 2>(x, b, rows, cols, q, scale, stream);
  else launch_quant<DT, 1024, 0>(x, b, rows, cols, q, scale, stream);
}

constexpr int kMaxQuantCols = 1 << 24;
}  // namespace
}  // namespace moe

extern "C" moe_status i8_quant(const void* x, int x_dtype, int64_t rows, int cols, int64_t ldx, int8_t* q, float* scale,
                               hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(x_dtype == MOE_BF16 || x_dtype == MOE_F32, MOE_ERR_DTYPE, "i8_quant: x must be MOE_BF16 or MOE_F32 (%d)", x_dtype);
  MOE_REQUIRE(rows >= 0 && cols >= 1 && cols <= kMaxQuantCols, MOE_ERR_SHAPE, "i8_quant: rows=%lld cols=%d (1..%d)",
              (long long)rows, cols, kMaxQuantCols);
  MOE_REQUIRE(rows == 0 || (x && q && scale), MOE_ERR_NULL, "i8_quant: a required pointer is NULL");
  MOE_REQUIRE(ldx >= cols, MOE_ERR_ALIGN, "i8_quant: ldx=%lld < cols=%d", (long long)ldx, cols);
  MOE_REQUIRE(aligned_to(x, x_dtype == MOE_F32 ? 4 : 2) && aligned_to(scale, 4), MOE_ERR_ALIGN,
              "i8_quant: x and scale must be aligned to their elements");
  MOE_REQUIRE(rows <= kMaxLanes / 1024, MOE_ERR_SHAPE, "i8_quant: too many rows (%lld)", (long long)rows);
  if (rows > 0) {
    if (x_dtype == MOE_BF16) dispatch_quant<ROW_BF16>(x, ldx, rows, cols, q, scale, stream);
    else dispatch_quant<ROW_F32>(x, ldx, rows, cols, q, scale, stream);
  }
  return check_launch("i8_quant");
}

extern "C" moe_status i8_dequant(const int8_t* q, const float* scale, int64_t rows, int cols, void* out, int out_dtype,
                                 int64_t ldo, hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(out_dtype == MOE_BF16 || out_dtype == MOE_F32, MOE_ERR_DTYPE, "i8_dequant: out must be MOE_BF16 or MOE_F32 (%d)",
              out_dtype);
  MOE_REQUIRE(rows >= 0 && cols >= 1 && cols <= kMaxQuantCols, MOE_ERR_SHAPE, "i8_dequant: rows=%lld cols=%d (1..%d)",
              (long long)rows, cols, kMaxQuantCols);
  MOE_REQUIRE(rows == 0 || (q && scale && out), MOE_ERR_NULL, "i8_dequant: a required pointer is NULL");
  MOE_REQUIRE(ldo >= cols, MOE_ERR_ALIGN, "i8_dequant: ldo=%lld < cols=%d", (long long)ldo, cols);
  MOE_REQUIRE(aligned_to(out, out_dtype == MOE_F32 ? 4 : 2) && aligned_to(scale, 4), MOE_ERR_ALIGN,
              "i8_dequant: out and scale must be aligned to their elements");
  const int chunks = (cols + 7) / 8;
  MOE_REQUIRE(rows <= kMaxLanes / chunks, MOE_ERR_SHAPE, "i8_dequant: too many elements");
  if (rows > 0)
    i8_dequant_kernel<<<(unsigned)((rows * chunks + 255) / 256), 256, 0, stream>>>(
        q, scale, rows, cols, make_row_split(chunks), out, out_dtype == MOE_F32 ? ROW_F32 : ROW_BF16,
        ldo * (out_dtype == MOE_F32 ? 4 : 2));
  return check_launch("i8_dequant");
}

extern "C" moe_status moe_i8_gemm(const moe_i8_desc* d, hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(d != nullptr, MOE_ERR_NULL, "moe_i8_gemm: desc is NULL");
  MOE_REQUIRE(d->epilogue == MOE_EPI_NONE || d->epilogue == MOE_EPI_SWIGLU, MOE_ERR_DTYPE, "moe_i8_gemm: unknown epilogue %d",
              d->epilogue);
  MOE_REQUIRE(d->out_dtype == MOE_BF16 || d->out_dtype == MOE_F32, MOE_ERR_DTYPE,
              "moe_i8_gemm: out_dtype must be MOE_BF16 or MOE_F32 (%d)", d->out_dtype);
  const bool swiglu = d->epilogue == MOE_EPI_SWIGLU;
  MOE_REQUIRE(d->n_groups >= 1 && d->n_groups <= kMaxRowGroups && d->first_group >= 0, MOE_ERR_SHAPE,
              "moe_i8_gemm: n_groups=%d (1..%d) first_group=%d", d->n_groups, kMaxRowGroups, d->first_group);
  MOE_REQUIRE(d->m_total >= 0 && d->m_total < ((int64_t)1 << 31), MOE_ERR_SHAPE, "moe_i8_gemm: m_total=%lld",
              (long long)d->m_total);
  MOE_REQUIRE(d->sorted_rows >= 0 && d->out_rows >= 0 && d->tail_rows >= 0, MOE_ERR_SHAPE,
              "moe_i8_gemm: negative counts of rows (%lld sorted, %lld of out, %lld of out_tail)", (long long)d->sorted_rows,
              (long long)d->out_rows, (long long)d->tail_rows);
  MOE_REQUIRE(d->K >= 16 && d->K % 16 == 0 && d->K < 131072 && d->N >= 1 && (!swiglu || d->N % 2 == 0), MOE_ERR_SHAPE,
              "moe_i8_gemm: K=%d must be a positive multiple of 16 below 131072, N=%d positive%s", d->K, d->N,
              swiglu ? " and even" : "");
  MOE_REQUIRE((int64_t)d->N * d->K < ((int64_t)1 << 31), MOE_ERR_SHAPE, "moe_i8_gemm: one W[g] exceeds 2 GiB");
  MOE_REQUIRE(d->tail_groups >= 0 && d->tail_groups <= d->n_groups, MOE_ERR_SHAPE,
              "moe_i8_gemm: tail_groups=%d must be in [0, n_groups=%d]", d->tail_groups, d->n_groups);
  const bool all_tail = d->tail_groups == d->n_groups;
  const bool nothing = d->m_total == 0 || d->sorted_rows == 0;
  MOE_REQUIRE(d->w_q && d->w_scale && d->group_offsets &&
                  (nothing || (d->a && d->a_scale && (d->out || d->out_rows == 0 || all_tail))),
              MOE_ERR_NULL, "moe_i8_gemm: a, a_scale, w_q, w_scale, group_offsets and out are required");
  const int out_cols = swiglu ? d->N / 2 : d->N;
  const int osz = d->out_dtype == MOE_F32 ? 4 : 2;
  MOE_REQUIRE(d->lda >= d->K && d->lda % 16 == 0 && aligned16(d->a) && aligned16(d->w_q), MOE_ERR_ALIGN,
              "moe_i8_gemm: lda=%lld must be >= K and a multiple of 16, a and w_q 16-byte aligned", (long long)d->lda);
  MOE_REQUIRE(aligned_to(d->a_scale, 4) && aligned_to(d->w_scale, 4), MOE_ERR_ALIGN, "moe_i8_gemm: scales must be 4-byte aligned");
  MOE_REQUIRE(all_tail || (d->ldo >= out_cols && aligned_to(d->out, osz)), MOE_ERR_ALIGN,
              "moe_i8_gemm: ldo=%lld must be >= %d and out aligned to its elements", (long long)d->ldo, out_cols);
  if (d->tail_groups > 0) {
    MOE_REQUIRE(nothing || d->tail_rows == 0 || d->out_tail, MOE_ERR_NULL, "moe_i8_gemm: out_tail is NULL");
    MOE_REQUIRE(d->ldo_tail >= out_cols && aligned_to(d->out_tail, 4), MOE_ERR_ALIGN,
                "moe_i8_gemm: ldo_tail=%lld must be >= %d and out_tail 4-byte aligned", (long long)d->ldo_tail, out_cols);
  }
  if (nothing) return MOE_OK;
  I8Args a;
  a.rows.offs = d->group_offsets + d->first_group;
  a.rows.n_groups = d->n_groups;
  a.rows.tail_first = d->n_groups - d->tail_groups;
  a.rows.m_total = row_count(d->m_total);
  a.rows.sorted_rows = row_count(d->sorted_rows);
  a.rows.out_rows = all_tail ? INT32_MAX : row_count(d->out_rows);
  a.rows.tail_rows = d->tail_groups > 0 ? row_count(d->tail_rows) : INT32_MAX;
  a.a = reinterpret_cast<const uint8_t*>(d->a);
  a.a_scale = d->a_scale;
  a.a_rows = d->a_rows;
  a.lda = d->lda;
  a.w = reinterpret_cast<const uint8_t*>(d->w_q);
  a.w_scale = d->w_scale;
  a.first_group = d->first_group;
  a.N = d->N;
  a.K = d->K;
  a.n_tiles = 0;  // set with the tile shape
  a.out_cols = out_cols;
  a.out = static_cast<uint8_t*>(d->out);
  a.out_dtype = d->out_dtype == MOE_F32 ? ROW_F32 : ROW_BF16;
  a.ldo_b = d->ldo * osz;
  a.out_tail = static_cast<uint8_t*>(d->out_tail);
  a.ldo_tail_b = d->ldo_tail * 4;
  const int64_t rows = d->m_total < d->sorted_rows ? d->m_total : d->sorted_rows;
  if (swiglu) dispatch_gemm<true>(a, rows, stream);
  else dispatch_gemm<false>(a, rows, stream);
  return check_launch("moe_i8_gemm");
}
