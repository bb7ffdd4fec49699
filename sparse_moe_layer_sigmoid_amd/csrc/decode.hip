// moe_decode: the whole layer for a few tokens, in two launches.
//
//   xn = bf16(norm(x)),  u = xn . e_i,  s = sigmoid(u),  top-K of s + b,  gate = s / sum s
//   out = sum_k gate_k W2[e_k] h_k + W2[shared] h_shared,   h_e = silu(W1[e] xn) * (W3[e] xn)
//
// A token's experts are read once and hardly computed with, so the bytes of the active experts' weights are the floor
// (one token: 9 experts of 257) and everything else is latency: launches, the first loads, the hand-over of h.
//
//  1. decode_rows_kernel: a workgroup for up to four tokens and one routed expert (of more than four tokens: as many experts as
//     there are groups of four) normalises its tokens (they are a few KB in L2, so that is done once per workgroup), writes its
//     share of them as bf16 and sums its experts' logits in fp64.
//  2. decode_experts_kernel: one workgroup of 8 waves per CU.  Each selects the tokens' experts from the affinities by itself
//     (4 us for one token, while its first weights are on the way), then takes tiles of 8 gate rows and their 8 up rows of the
//     active experts, and then a block of output columns, which it sums over all experts: no atomics on values, no partial
//     outputs in memory, one order of sums.
//
// Columns are tokens: the matrix cores take 16 weight rows against 16 columns, and column t is token t whatever its experts
// are.  Products with experts that a token did not choose cost nothing that the weights' bytes do not hide and are left out
// of its sums, so no rows are sorted or gathered, and a token's bits do not depend on the others'.
//
// K is split over the 8 waves in blocks of 128 bytes of a weight row, dealt out in turn; each wave holds its inputs of all
// tokens in registers, and its weights come through a ring of its own in LDS by direct-to-LDS loads of 16 rows x 128 bytes a
// step, XOR-swizzled so that operand reads meet distinct banks.  The ring runs on across tiles and experts: with 8 steps to a
// wave the chip has 32 MB on the way, what 6.5 TB/s need at 5 us.
//
// The hand-over: gate/up tiles are taken from counters, the first two (three) of a workgroup at once, and every tile is in the
// hands of a running workgroup before any workgroup waits for h.  None waits for one that has not started: calls may overlap on
// the device.  h goes through to memory by its stores; the workgroup that finishes the last tile raises flags.
//
// Timeline of 7168 x 2048, 8 of 256 experts and the shared one, one token, bf16 (4 bits), us: first launch 6 (4); selected and
// the ring full 11 (11); gate/up 99 (41), the median workgroup 90 (39); h there 100 (42); end 142 (59).  That is 148 us, 5.4 TB/s,
// with 4 bits 65 us, 3.3 TB/s; 4 tokens in E4M3 245 us, 5.7 TB/s; 16 tokens in int8 720 to 780 us, 5.8 to 6.3 TB/s (a large
// copy reads and writes 5.1 TB/s).  With E8M0 scales in place of f32 ones 1, 4 and 16 tokens in E4M3 take 94, 265 and 857 us
// against 87, 252 and 816.
//
// A unit of the down projection takes about 1 us whatever it holds, and is filled only by rows of about 7168 and experts of 1024 and
// more (32 columns x 8 blocks of 128 bytes): 1024 x 512, 91 experts reached by 16 tokens, takes 151 us in bf16 and 225 us in 4
// bits, where the layer's own calls take 103 and 63 us.
#include <type_traits>

#include "abi_common.h"
#include "device_common.h"
#include "rows_common.h"
#include "select.h"
#include "weights.h"

namespace moe {
namespace {

enum { W_BF16 = 0, W_E4M3 = 1, W_E4M3_E8M0 = 2, W_I8 = 3, W_FP4 = 4 };

constexpr int kMaxT = 16;         // tokens: the columns of a matrix product
constexpr int kMaxTopK = 32;
constexpr int kMaxD = 8192;       // inputs a workgroup's waves hold in registers
constexpr int kNW = 8;            // waves of a workgroup
constexpr int kMaxActive = 257;
constexpr int kJoiners = 2;       // waves that add the waves' sums: a token's 8 columns of a tile to 8 lanes
constexpr int kRowThreads = 1024;
// Bound of the wait for h, in looks at its flag (each a sleep of 256 clocks and a load past the caches: seconds).  Looks and not time,
// which goes on while a queue that was switched out cannot look.
constexpr int kWaitLooks = 1 << 22;

// Workspace: counters, affinities, normalised rows, h.
constexpr int kFlags = 16;    // "h is complete", for a workgroup in 16 each
constexpr int kClasses = 16;  // counters of the workgroups that have started, for a workgroup in 16 each
constexpr int kCounters = 2 + kFlags + kClasses;  // the next tile, finished tiles, flags, classes: 128 bytes apart
constexpr size_t kCounterBytes = (kCounters * 128 + 255) & ~255;
constexpr size_t kScoreBytes = (size_t)kMaxT * 256 * sizeof(double);
struct DecodeWs {
  size_t scores, xn, h, total;
};
DecodeWs decode_ws(int T, int d, int inter, int n_shared, int top_k) {
  DecodeWs w;
  w.scores = kCounterBytes;
  w.xn = w.scores + kScoreBytes;
  w.h = w.xn + (((size_t)T * d * 2 + 255) & ~(size_t)255);
  w.total = w.h + (size_t)T * (top_k + n_shared) * inter * 4;
  return w;
}

// ---- first launch: norm and logits ----

struct RowsArgs {
  const uint8_t* x;
  int x_dtype;
  int64_t ldx_b;
  int T, d, N;
  int norm;  // MOE_NORM_*
  const void* weight;
  const void* bias;
  int w_dtype;
  double eps;
  int experts;  // per workgroup
  const uint16_t* wr;
  uint32_t* counters;
  double* scores;  // affinities, [T][256]
  uint16_t* xn;
};

// Sums by DPP moves (no LDS): over rows of 16 lanes, in lane 15 of each; over the wave, in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROWS, 0xf, false),
                                          (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROWS, 0xf, false)});
}
__device__ __forceinline__ double row_sum64(double v) {
  v += dpp_or_zero<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
  v += dpp_or_zero<0x112, 0xf>(v);
  v += dpp_or_zero<0x114, 0xf>(v);
  return v + dpp_or_zero<0x118, 0xf>(v);
}
__device__ __forceinline__ double wave_sum64(double v) {
  v = row_sum64(v);
  v += dpp_or_zero<0x142, 0xa>(v);  // lane 15 to the second row of each half, lane 31 to the upper half
  v += dpp_or_zero<0x143, 0xc>(v);
  return lane_value(v, 63);
}

// A workgroup takes up to four tokens, one chunk of 8 inputs to a lane, and p.experts routed experts, so that the rows are
// normalised 256 times whatever their number (they come from L2).
template <bool NORM>
__global__ __launch_bounds__(kRowThreads) void decode_rows_kernel(RowsArgs p) {
  constexpr int G = 4, W = kRowThreads / 64;
  static_assert(kMaxD <= 8 * kRowThreads, "one chunk per lane");
  static_assert(W == 16, "a row of lanes adds the waves' sums");
  __shared__ double s_sums[NORM ? W : 1][2 * G];
  __shared__ double s_stat[NORM ? G : 1][2];
  __shared__ double s_part[2][W][G];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = tid * 8;
  const bool busy = wave * 512 < p.d;  // a wave without inputs leaves the arithmetic to the others
  const int e0 = blockIdx.x * p.experts, e1 = min(e0 + p.experts, p.N);
  const int t0 = blockIdx.y * G, nt = min(G, p.T - t0);
  const bool in = c < p.d;
  if (e0 == 0 && t0 == 0 && tid < kCounters) p.counters[tid * 32] = 0;
  u32x4 wv = {0u, 0u, 0u, 0u};
  if (in) wv = *(const u32x4*)(p.wr + (int64_t)e0 * p.d + c);
  float f[G][8];
#pragma unroll
  for (int i = 0; i < G; ++i) {
#pragma unroll
    for (int q = 0; q < 8; ++q) f[i][q] = 0.f;
    if (in && i < nt) load8_any<true>(p.x_dtype, p.x + (t0 + i) * p.ldx_b, c, p.d, f[i]);
  }
  if constexpr (NORM) {
    float g[8], b[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      g[q] = 1.f;
      b[q] = 0.f;
    }
    if (p.weight && in) load8_any<true>(p.w_dtype, p.weight, c, p.d, g);
    if (p.bias && in) load8_any<true>(p.w_dtype, p.bias, c, p.d, b);
    // In fp64, statistics of x minus the row's first element: there is no range to leave, a mean far from zero cancels
    // nothing, and the rounding to bf16 is that of the exact value but for one in 2^20 or so.
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (i >= nt) break;
      const uint8_t* row = p.x + (t0 + i) * p.ldx_b;
      const double pivot = p.norm != MOE_NORM_LAYER ? 0.0
                           : p.x_dtype == ROW_F32   ? (double)*(const float*)row
                                                    : (double)bf16_to_f32(*(const uint16_t*)row);
      double s1 = 0.0, s2 = 0.0;
      if (busy) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const double v = in ? (double)f[i][q] - pivot : 0.0;
          s1 += v;
          s2 = fma(v, v, s2);
        }
        if (p.norm == MOE_NORM_LAYER) s1 = wave_sum64(s1);
        s2 = wave_sum64(s2);
      }
      if (lane == 0) {
        s_sums[wave][2 * i] = s1;
        s_sums[wave][2 * i + 1] = s2;
        if (wave == 0) s_stat[i][0] = pivot;
      }
    }
    __syncthreads();
    if (tid < 2 * G * W) {  // row of lanes v: the waves' sums of value v (token v / 2: sum, sum of squares)
      const int v = tid >> 4, i = v >> 1;
      const double sum = row_sum64(s_sums[tid & 15][v]);
      const double s1 = __shfl(sum, (lane & 32) + 15, kWave);
      if ((tid & 31) == 31 && i < nt) {
        double mean = 0.0, var = sum / p.d;
        if (p.norm == MOE_NORM_LAYER) {
          const double m1 = s1 / p.d;
          mean = s_stat[i][0] + m1;
          var -= m1 * m1;
          if (var < 0.0) var = 0.0;
        }
        s_stat[i][0] = mean;
        s_stat[i][1] = 1.0 / sqrt(var + p.eps);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (i >= nt || !busy) break;
      const double mean = s_stat[i][0], rstd = s_stat[i][1];
      float y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = (float)fma(((double)f[i][q] - mean) * rstd, (double)g[q], (double)b[q]);
      const u32x4 o = pack_bf16x8(y);
      if (in && (t0 + i) % gridDim.x == blockIdx.x) *(u32x4*)(p.xn + (int64_t)(t0 + i) * p.d + c) = o;
      unpack_bf16x8(o, f[i]);
    }
  }
  double x[G][8];
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) x[i][q] = in ? (double)f[i][q] : 0.0;
  for (int e = e0; e < e1; ++e) {
    float w[8];
    unpack_bf16x8(wv, w);
    double wd[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) wd[q] = in ? (double)w[q] : 0.0;
    if (in && e + 1 < e1) wv = *(const u32x4*)(p.wr + (int64_t)(e + 1) * p.d + c);
    double(*const part)[G] = s_part[e & 1];  // two in turn: a barrier lies between a sum's last reader and its next writer
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (i >= nt) break;
      double acc = 0.0;
      if (busy) {
#pragma unroll
        for (int q = 0; q < 8; ++q) acc = fma(x[i][q], wd[q], acc);
        acc = wave_sum64(acc);
      }
      if (lane == 0) part[wave][i] = acc;
    }
    __syncthreads();
    if (wave == (e & 15)) {
      const double u = row_sum64(part[lane & 15][lane >> 4]);
      if ((lane & 15) == 15 && (lane >> 4) < nt) p.scores[(t0 + (lane >> 4)) * 256 + e] = sigmoid_v<double>(u);
    }
  }
}

__global__ __launch_bounds__(256) void decode_zero_counts_kernel(int32_t* counts, int n) {
  if ((int)threadIdx.x < n) counts[threadIdx.x] = 0;
}

// ---- second launch: selection and experts ----

struct ExpertArgs {
  const uint16_t* xn;
  int64_t ldxn;
  int T, d, inter, N, n_shared, K, n_group, topk_group;
  const float* bias;
  const double* scores;
  uint32_t* counters;
  uint16_t* h;  // [T][K + n_shared][inter], upper and lower parts one after the other
  int ahead;    // tiles a workgroup holds: the one at work and those that its ring reaches into
  int lists;    // batches of `ahead` tiles that are dealt out: one to a workgroup, and more where some never start
  int looks;    // bound of the wait for h
  const uint8_t* w13;
  const uint8_t* s13;
  const uint8_t* w2;
  const uint8_t* s2;
  uint8_t* out;
  int out_dtype;
  int64_t ldo_b;
  int32_t* topk_idx;
  float* topk_gate;
  int32_t* counts;
};

typedef __attribute__((address_space(3))) void lds_void;

// 16 or 4 bytes per lane from base + v + off (v per lane, base and off uniform) to LDS at dst, lane after lane.  (The host
// pass does not know the builtin.)
__device__ __forceinline__ void load16_to_lds(const uint8_t* base, uint32_t v, uint32_t off, uint8_t* dst) {
#ifdef __HIP_DEVICE_COMPILE__
  const auto r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 0xffffffffu, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, v, off, 0, 0);
#endif
}
__device__ __forceinline__ void load4_to_lds(const uint8_t* base, uint32_t v, uint32_t off, uint8_t* dst) {
#ifdef __HIP_DEVICE_COMPILE__
  const auto r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 0xffffffffu, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, v, off, 0, 0);
#endif
}

// 16 bytes at base + v + off (off uniform); zeros, and no memory access, from `bytes` on, as for a lane whose v is kNoLoad.
constexpr uint32_t kNoLoad = 0xffffffffu;
__device__ __forceinline__ u32x4 load16_if(const void* base, uint32_t bytes, uint32_t v, uint32_t off) {
#ifdef __HIP_DEVICE_COMPILE__
  const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, v, off, 0));
#else
  return u32x4{v, off, bytes, 0u};
#endif
}

template <int FMT, bool WIDE = false>
struct Fmt {
  static constexpr bool kScaled = FMT != W_BF16;
  static constexpr int kBlock = FMT == W_BF16 ? 64 : FMT == W_FP4 ? 256 : 128;  // inputs in 128 bytes of a weight row
  static constexpr int kVec = kBlock / 64;              // operands of 8 inputs per lane in half a block
  static constexpr int kSteps = kMaxD / kBlock / kNW;   // blocks per wave of a gate/up tile at most
  static constexpr int kSlot = 2048 + (kScaled ? 128 : 0);  // a step's weights and scales
  static constexpr int kDepth = FMT == W_FP4 ? 6 : 8;   // steps in flight per wave: as many as LDS holds, an even number
  static constexpr int kLoads = kScaled ? 3 : 2;        // loads of a step
  static constexpr int kWaitUp = kLoads * (kDepth - 1);
  // down: a unit is an expert's next 8 blocks of inner columns, one per wave, two steps; each brings kParts * 2 * kVec loads of h
  static constexpr int kParts = WIDE ? 2 : 1;
  // Units that h is loaded ahead: as many as the ring holds, for loads end in order, and a wait for h of the unit before the
  // last would be one for all weights but the last unit's (4 bits and two parts: one less, there are no more registers).
  static constexpr int kSets = kDepth / 2 - (FMT == W_FP4 && WIDE ? 1 : 0);
  static constexpr int kWaitDown = (kDepth / 2 - 1) * (2 * kLoads + kParts * 2 * kVec);
};

// 8 weights of a step's half block: dword pairs (bf16: the 16 bytes), its operand `s`.
template <int FMT>
__device__ __forceinline__ bf16x8_t operand(const u32x4& q, int s, float scale) {
  if constexpr (FMT == W_BF16) return __builtin_bit_cast(bf16x8_t, q);
  else if constexpr (FMT == W_FP4) return decode_w4(q[s], scale);
  else if constexpr (FMT == W_I8) return decode_i8(q[2 * s], q[2 * s + 1]);
  else return decode_e4m3(q[2 * s], q[2 * s + 1]);
}

// WIDE: more than 8 tokens.  h is in two bf16 parts; of up to 8 tokens the lower parts are columns of their own, t + 8, else
// products of their own (the two sums meet at the end either way: the same bits).
template <int FMT, bool WIDE>
__global__ __launch_bounds__(kNW * 64, 2) void decode_experts_kernel(ExpertArgs p) {
  using F = Fmt<FMT, WIDE>;
  constexpr int D = F::kDepth, SLOT = F::kSlot, P = F::kParts;
  static_assert(D % 2 == 0 && F::kSteps >= D / 2, "the ring holds whole units, and at most two tiles ahead");
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kNW * D * SLOT];
  __shared__ __attribute__((aligned(16))) f32x4 s_red[2][kNW][64];
  __shared__ float s_gate[kMaxT * (kMaxTopK + 1)];  // gate of slot t (K + n_shared) + k
  __shared__ __attribute__((aligned(16))) uint8_t s_k[kMaxActive][kMaxT];  // k of a token's active expert, 255: not chosen
  __shared__ uint16_t s_exp[kMaxActive];            // active experts, the shared one first
  __shared__ int s_ctl[4];                          // tiles taken (two in turn), gave up waiting, batch or tile taken
  // of the selection, before the sums need the space
  uint32_t* const s_mask = reinterpret_cast<uint32_t*>(&s_red[0][0][0]);
  int32_t* const s_idx = reinterpret_cast<int32_t*>(&s_red[0][4][0]);
  int32_t* const s_pos = reinterpret_cast<int32_t*>(&s_red[1][0][0]);
  uint32_t* const s_cnt = reinterpret_cast<uint32_t*>(&s_red[1][4][0]);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int T = p.T, K = p.K, KS = p.K + p.n_shared;
  uint32_t* const next_tile = p.counters;
  uint32_t* const done = p.counters + 32;
  uint32_t* const flags = p.counters + 2 * 32;
  uint32_t* const classes = flags + kFlags * 32;
  const int grid = p.lists;
  uint32_t in_vgpr = 0;  // of a uniform address the compiler combines the wave's additions, and waits for the sum at once
  asm volatile("" : "+v"(in_vgpr));
  auto take = [&](uint32_t* counter) __attribute__((always_inline)) {
    return (int)__hip_atomic_fetch_add(counter + in_vgpr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  // The first p.ahead * grid tiles come in batches of p.ahead, a grid apart, so that everyone starts with the shared expert's.
  // The n-th workgroup of a class to start takes the class's n-th batch: one counter for all would keep the last ones waiting
  // for 5 us.
  auto claim = [&](int c) __attribute__((always_inline)) { return take(classes + c * 32) * kClasses + c; };
  if (tid == 0) s_ctl[3] = claim((int)blockIdx.x % kClasses);

  // ---- what is needed of the weights' layout ----
  const int nt = p.inter / 8;                                // tiles of an expert
  const int nb1 = (p.d + F::kBlock - 1) / F::kBlock;         // blocks of a gate/up row
  const int nb2 = (p.inter + F::kBlock - 1) / F::kBlock;     // blocks of a down row
  // steps of a tile; as many at least as leave the ring no more than two tiles ahead (a block that a wave does not have
  // is another one of the row again, unused)
  const int steps = max((nb1 + kNW - 1) / kNW, D / 2);
  const uint32_t row1_b = p.d / F::kBlock * 128 + p.d % F::kBlock * 128 / F::kBlock;
  const uint32_t row2_b = p.inter / F::kBlock * 128 + p.inter % F::kBlock * 128 / F::kBlock;
  const int lrow = lane >> 3;
  const int chunk = (lane & 7) ^ lrow;                       // 16-byte piece of a block that this lane loads
  const int srow = FMT == W_FP4 ? (lane >> 1) & 15 : lr;     // row of a step whose scale this lane loads
  constexpr int kScaleLanes = FMT == W_FP4 ? 32 : 16;
  // offset of row q's scales from row 0's (k inputs, nb blocks to a row)
  auto scale_row = [&](uint32_t q, uint32_t nb, uint32_t k) __attribute__((always_inline)) {
    if constexpr (FMT == W_FP4) return q * (k / 32);
    else if constexpr (FMT == W_E4M3) return q / 128 * nb * 4;
    else if constexpr (FMT == W_E4M3_E8M0) return q / 128 * nb;
    else return q * 4;
  };
  // bytes of one expert's scales (n rows)
  auto scale_bytes = [&](int64_t n, int64_t nb, int64_t k) __attribute__((always_inline)) {
    if constexpr (FMT == W_FP4) return n * (k / 32);
    else if constexpr (FMT == W_E4M3) return n / 128 * nb * 4;
    else if constexpr (FMT == W_E4M3_E8M0) return n / 128 * nb;
    else return n * 4;
  };
  uint8_t* const ring = s_ring + wave * (D * SLOT);
  // A step: 16 rows x 128 bytes (block b of rows of row_b bytes) and their scales.  This lane's pieces are at v0 and v1 + off1 of
  // w, its scales at vs of sc.
  struct Place {
    const uint8_t *w, *sc;
  };
  struct Source {
    Place at;
    uint32_t row_b, b, v0, v1, off1, vs;
  };
  // Buffer loads: for the compiler global loads into LDS are flat ones, behind which it waits for everything in flight before it
  // uses a register that a load of h fills.
  auto load_step = [&](int slot, const Source& q) __attribute__((always_inline)) {
    uint8_t* dst = ring + slot * SLOT;
    const bool half = FMT == W_FP4 && q.b * 128 + 128 > q.row_b;  // a last block of 64 bytes: its first half twice
    const uint32_t back = half && (chunk & 4) ? 64 : 0;
    load16_to_lds(q.at.w, q.v0 - back, q.b * 128, dst);
    load16_to_lds(q.at.w, q.v1 - back, q.b * 128 + q.off1, dst + 1024);
    if constexpr (F::kScaled) {
      const uint32_t off = FMT == W_FP4 ? q.b * 8 : FMT == W_E4M3 ? q.b * 4 : FMT == W_E4M3_E8M0 ? q.b & ~3u : 0u;
      uint32_t v = q.vs;
      if constexpr (FMT == W_FP4) v += half ? 0 : (lane & 1) * 4;
      if (lane < kScaleLanes) load4_to_lds(q.at.sc, v, off, dst + 2048);
    }
  };
  // Wave w's i-th block of a row is in the i-th eight blocks, rotated by i and (down) the expert: with the same place in every
  // eight, a wave would meet the same memory channels all along.
  auto own_block = [&](int i, int e) __attribute__((always_inline)) { return i * kNW + ((wave + i + e) & (kNW - 1)); };
  auto block_of = [&](int i, int e, int nb) __attribute__((always_inline)) {
    const int b = own_block(i, e);
    return (uint32_t)(b < nb ? b : min(wave, nb - 1));
  };
  // gate/up: tile `tile` of expert e is 8 gate rows and their 8 up rows
  auto up_place = [&](int64_t e, int tile) __attribute__((always_inline)) {
    Place q;
    q.w = p.w13 + (e * 2 * p.inter + tile * 8) * row1_b;
    q.sc = p.s13 + e * scale_bytes(2 * p.inter, nb1, p.d) + scale_row(tile * 8, nb1, p.d);
    return q;
  };
  const uint32_t up_v = lrow * row1_b + chunk * 16, up_off = p.inter * row1_b;
  uint32_t up_vs;  // tiles start at multiples of 8 rows: none crosses a block of 128
  if constexpr (FMT == W_E4M3 || FMT == W_E4M3_E8M0) up_vs = srow < 8 ? 0 : scale_row(p.inter, nb1, p.d);
  else up_vs = scale_row((srow & 7) + (srow < 8 ? 0 : p.inter), nb1, p.d);
  auto up_step = [&](const Place& q, int s) __attribute__((always_inline)) {
    return Source{q, row1_b, block_of(s, 0, nb1), up_v, up_v, up_off, up_vs};
  };

  // ---- the tokens' affinities and inputs, in flight before any weights ----
  double u[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) u[r] = wave < T && lane * 4 + r < p.N ? p.scores[wave * 256 + lane * 4 + r] : 0.0;
  float bias[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) bias[r] = lane * 4 + r < p.N ? p.bias[lane * 4 + r] : 0.f;
  bf16x8_t x[F::kSteps][2][F::kVec];  // this wave's blocks of all tokens (columns past T hold the last token again)
  {
    const uint16_t* xr = p.xn + (int64_t)min(lr, T - 1) * p.ldxn;
#pragma unroll
    for (int j = 0; j < F::kSteps; ++j)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int k0 = own_block(j, 0) * F::kBlock + hf * (F::kBlock / 2);
#pragma unroll
        for (int s = 0; s < F::kVec; ++s) {
          u32x4 v = {0u, 0u, 0u, 0u};
          if (k0 < p.d) v = *(const u32x4*)(xr + k0 + lg * (F::kBlock / 8) + s * 8);
          x[j][hf][s] = __builtin_bit_cast(bf16x8_t, v);
        }
      }
  }
  for (int i = tid; i < 256; i += kNW * 64) s_mask[i] = 0;
  for (int i = tid; i < kMaxActive * kMaxT / 4; i += kNW * 64) reinterpret_cast<uint32_t*>(&s_k[0][0])[i] = 0xffffffffu;
  __syncthreads();
  const int batch = __builtin_amdgcn_readfirstlane(s_ctl[3]);
  const int first = batch < grid ? batch : INT32_MAX;  // the class's batches may be in others' hands by now

  // the shared expert's tiles come first: their weights are on the way while the routed ones are being chosen
  int loaded = 0;
  if (p.n_shared && first < nt) {
    const Place q = up_place(p.N, first);
    loaded = min(D, steps);
#pragma unroll 1
    for (int s = 0; s < loaded; ++s) load_step(s, up_step(q, s));
  }

  // ---- selection ----
#pragma unroll 1
  for (int t = wave; t < T; t += kNW) {
    if (t >= kNW) {
#pragma unroll
      for (int r = 0; r < 4; ++r) u[r] = lane * 4 + r < p.N ? p.scores[t * 256 + lane * 4 + r] : 0.0;
    }
    float* const gate = s_gate + t * (KS - K);  // select_token writes at t * K + k; rows here are KS apart
    select_token<double, true>(u, bias, p.N, K, p.n_group, p.topk_group, t, true, s_idx, gate, nullptr);
    if (lane == 0 && p.n_shared) s_gate[t * KS + K] = 1.0f;
  }
  lds_barrier();
  for (int i = tid; i < T * K; i += kNW * 64) atomicOr(&s_mask[s_idx[i]], 1u << (i / K));
  lds_barrier();
  {
    const uint32_t mask = tid < p.N ? s_mask[tid] : 0u;
    const uint64_t any = __ballot(mask != 0);
    if (lane == 0 && wave < 4) s_cnt[wave] = (uint32_t)__popcll(any);
    lds_barrier();
    int at = p.n_shared;
    for (int w = 0; w < 4 && w < wave; ++w) at += (int)s_cnt[w];
    at += __popcll(any & ((1ull << lane) - 1));
    if (mask != 0) {
      s_exp[at] = (uint16_t)tid;
      s_pos[tid] = at;
    }
    if (tid == 0) {
      if (p.n_shared) s_exp[0] = (uint16_t)p.N;
      s_ctl[2] = 0;
    }
    if (blockIdx.x == 0) {  // one workgroup reports the routing
      if (p.counts && tid < p.N) p.counts[tid] = __popc(mask);
      for (int i = tid; i < T * K; i += kNW * 64) {
        if (p.topk_idx) p.topk_idx[i] = s_idx[i];
        if (p.topk_gate) p.topk_gate[i] = s_gate[i / K * KS + i % K];
      }
    }
  }
  const int A = __builtin_amdgcn_readfirstlane(p.n_shared + (int)(s_cnt[0] + s_cnt[1] + s_cnt[2] + s_cnt[3]));
  const int tiles = A * nt;
  lds_barrier();
  for (int i = tid; i < T * K; i += kNW * 64) s_k[s_pos[s_idx[i]]][i / K] = (uint8_t)(i % K);
  if (p.n_shared && tid < T) s_k[0][tid] = (uint8_t)K;

  // ---- down: blocks of R output columns, block `number` for this workgroup (and, were there more blocks than workgroups,
  // every grid-th from there): no other workgroup needs them, so they may wait for one that starts late ----
  const int number = (int)blockIdx.x;
  const int columns = (p.d + (int)gridDim.x - 1) / (int)gridDim.x;
  const int R = min(32, (columns + 3) & ~3);
  const int blocks = (p.d + R - 1) / R;
  const int slices = (nb2 + kNW - 1) / kNW;                  // units of an expert
  const int units = A * slices;
  uint32_t dn_v[4], dn_vs[2];  // this lane's rows of a block, two times 16
  auto set_block = [&](int block) __attribute__((always_inline)) {
    const int c0 = block * R, last = min(c0 + R, p.d) - 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) dn_v[i] = (uint32_t)min(c0 + i * 8 + lrow, last) * row2_b + chunk * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) dn_vs[i] = scale_row(min(c0 + i * 16 + srow, last), nb2, p.inter);
  };
  auto expert = [&](int a) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(s_exp[a]); };
  auto down_place = [&](int64_t e) __attribute__((always_inline)) {
    Place q;
    q.w = p.w2 + e * p.d * row2_b;
    q.sc = p.s2 + e * scale_bytes(p.d, nb2, p.inter);
    return q;
  };
  auto down_step = [&](const Place& q, int e, int sl, int i) __attribute__((always_inline)) {  // step i of unit sl of expert e
    Source r = {q, row2_b, block_of(sl, e, nb2), dn_v[0], dn_v[1], 0, dn_vs[0]};
    if (i) {
      r.v0 = dn_v[2];
      r.v1 = dn_v[3];
      r.vs = dn_vs[1];
    }
    return r;
  };
  auto down_step_at = [&](int c) __attribute__((always_inline)) {  // step c of the block (past its end: step 0's, unused)
    int un = c / 2;
    un = un < units ? un : 0;
    const int a = slices == 1 ? un : (int)((uint32_t)un / (uint32_t)slices);
    const int e = expert(a);
    return down_step(down_place(e), e, un - a * slices, c & 1);
  };
  set_block(number < blocks ? number : 0);

  // A step's operands from its slot: this lane's two 16-byte pieces of row lr and its scales.  The reads and their wait
  // are one block: the compiler does not order them against the loads into LDS, the waits on those do.
  const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)ring;
  const uint32_t rd = (lr >> 3) * 1024 + (lr & 7) * 128 + ((lg ^ (lr & 7)) << 4);
  struct Step {
    u32x4 lo, hi;
    u32x4 sc;  // FP4: two codes; else the scales of rows lg * 4 .. + 3
  };
  auto read_step = [&](int slot) __attribute__((always_inline)) {
    Step s;
    const uint32_t at = ring_at + slot * SLOT + rd, at2 = at ^ 64;
    if constexpr (FMT == W_FP4) {
      const uint32_t sa = ring_at + slot * SLOT + lr * 8 + lg;
      asm volatile(
          "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_u8 %2, %6 offset:2048\n\tds_read_u8 %3, %6 offset:2052\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(s.lo), "=&v"(s.hi), "=&v"(s.sc[0]), "=&v"(s.sc[1])
          : "v"(at), "v"(at2), "v"(sa)
          : "memory");
    } else if constexpr (F::kScaled) {
      const uint32_t sa = ring_at + slot * SLOT + lg * 16;
      asm volatile(
          "ds_read_b128 %0, %3\n\tds_read_b128 %1, %4\n\tds_read_b128 %2, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(s.lo), "=&v"(s.hi), "=&v"(s.sc)
          : "v"(at), "v"(at2), "v"(sa)
          : "memory");
    } else {
      asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                   : "=&v"(s.lo), "=&v"(s.hi)
                   : "v"(at), "v"(at2)
                   : "memory");
    }
    return s;
  };
  // The two steps of a unit, in an even slot and the next one.
  auto read_pair = [&](int slot, Step& s, Step& t) __attribute__((always_inline)) {
    const uint32_t at = ring_at + slot * SLOT + rd, at2 = at ^ 64, bt = at + SLOT, bt2 = at2 + SLOT;
    if constexpr (FMT == W_FP4) {
      static_assert(SLOT == 2176, "the offsets below");
      const uint32_t sa = ring_at + slot * SLOT + lr * 8 + lg;
      asm volatile(
          "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_u8 %2, %12 offset:2048\n\tds_read_u8 %3, %12 offset:2052\n\t"
          "ds_read_b128 %4, %10\n\tds_read_b128 %5, %11\n\tds_read_u8 %6, %12 offset:4224\n\tds_read_u8 %7, %12 offset:4228\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(s.lo), "=&v"(s.hi), "=&v"(s.sc[0]), "=&v"(s.sc[1]), "=&v"(t.lo), "=&v"(t.hi), "=&v"(t.sc[0]), "=&v"(t.sc[1])
          : "v"(at), "v"(at2), "v"(bt), "v"(bt2), "v"(sa)
          : "memory");
    } else if constexpr (F::kScaled) {
      static_assert(SLOT == 2176, "the offsets below");
      const uint32_t sa = ring_at + slot * SLOT + lg * 16;
      asm volatile(
          "ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\tds_read_b128 %2, %10 offset:2048\n\t"
          "ds_read_b128 %3, %8\n\tds_read_b128 %4, %9\n\tds_read_b128 %5, %10 offset:4224\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(s.lo), "=&v"(s.hi), "=&v"(s.sc), "=&v"(t.lo), "=&v"(t.hi), "=&v"(t.sc)
          : "v"(at), "v"(at2), "v"(bt), "v"(bt2), "v"(sa)
          : "memory");
    } else {
      asm volatile(
          "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\tds_read_b128 %3, %7\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(s.lo), "=&v"(s.hi), "=&v"(t.lo), "=&v"(t.hi)
          : "v"(at), "v"(at2), "v"(bt), "v"(bt2)
          : "memory");
    }
  };
  // scale of row lg * 4 + r of a step from block b (E4M3: of its block; int8: of the row)
  auto row_scale = [&](const Step& s, int b, int r) __attribute__((always_inline)) {
    if constexpr (FMT == W_E4M3_E8M0) {
      const uint32_t c = (s.sc[r] >> (8 * (b & 3))) & 255u;
      return c == 0 ? __uint_as_float(0x00400000u) : c == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(c << 23);
    } else {
      return __uint_as_float(s.sc[r]);
    }
  };
  // The 8 waves' partial sums of one value, in wave order: 1 KB apart from byte address `at` on.
  auto join8 = [](uint32_t at) __attribute__((always_inline)) {
    float v[8];
    asm volatile(
        "ds_read_b32 %0, %8\n\tds_read_b32 %1, %8 offset:1024\n\tds_read_b32 %2, %8 offset:2048\n\t"
        "ds_read_b32 %3, %8 offset:3072\n\tds_read_b32 %4, %8 offset:4096\n\tds_read_b32 %5, %8 offset:5120\n\t"
        "ds_read_b32 %6, %8 offset:6144\n\tds_read_b32 %7, %8 offset:7168\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(at)
        : "memory");
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNW; ++w) s += v[w];
    return s;
  };
  const uint32_t red_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const f32x4*)&s_red[0][0][0];

  int slot = 0;
  auto next_slot = [&]() __attribute__((always_inline)) { slot = slot + 1 == D ? 0 : slot + 1; };

  // ---- gate/up: tile q0 at work, q1 (deep: and q2) taken; those >= tiles do not exist ----
  auto place_of = [&](int id) __attribute__((always_inline)) {
    if (id >= tiles) return Place{p.w13, p.s13};
    const int a = (int)((uint32_t)id / (uint32_t)nt);
    return up_place(expert(a), id - a * nt);
  };
  const bool deep = p.ahead > 2;  // the ring reaches into the tile after next
  const int base = p.ahead * grid;  // from here on tiles are taken one at a time
  int q0, q1, q2;
  auto set_batch = [&](int v) __attribute__((always_inline)) {
    q0 = v < grid ? v : tiles;
    q1 = v < grid ? grid + v : tiles;
    q2 = v < grid && deep ? 2 * grid + v : tiles;
  };
  set_batch(batch);
  bool drained = tiles <= base;  // no tile is left but in others' batches
  Place p0 = place_of(q0), p1 = place_of(q1), p2 = place_of(q2);
  // The step `ahead` of tile q0's first one.  Past the last taken tile a step of the one at work again (it is in L2; the number in
  // flight stays): the down projection's weights would delay this workgroup's stores of h, which everyone waits for.
  auto load_ahead = [&](int slot, int ahead) __attribute__((always_inline)) {
    const int k = (ahead >= steps) + (ahead >= 2 * steps);
    int id = q2;
    Place q = p2;
    if (k == 0) {
      id = q0;
      q = p0;
    } else if (k == 1) {
      id = q1;
      q = p1;
    }
    // (one load_step behind both ways, so that the compiler can count its loads)
    Source r;
    if (id < tiles) {
      r = up_step(q, ahead - k * steps);
    } else {
      r = up_step(p0, 0);
    }
    load_step(slot, r);
  };
  __syncthreads();  // s_k; and the inputs are here: below, waits count the ring's loads alone
  wait_vm<0>();
#pragma unroll 1
  for (; loaded < D; ++loaded) load_ahead(loaded, loaded);

  int buf = 0, mine = 0, taken = 0;
  bool asked = (deep ? q2 : q1) < tiles && !drained;  // a tile's number is on the way
  if (asked && tid == 0) taken = base + take(next_tile);
  for (;;) {
    if (q0 >= tiles) {
      // Nothing left of what was taken.  Tiles may be left that workgroups would take which have not started, and may not start
      // before this one ends: take those.  (Counts only rise: a class that has given out its batches by now has none later.)
      uint32_t given = 0;
      const int ours = min(grid, tiles) - lane + kClasses - 1;  // batches of class `lane`, times kClasses
      if (wave == 0 && lane < kClasses) given = __hip_atomic_load(classes + lane * 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // This workgroup's h is in memory, past the XCD's L2, before it is counted: its stores went through and are waited for.
      // (A release fence would write the whole L2 back, one workgroup after the other: 13 us.)
      if (wave < kJoiners) wait_vm<0>();
      if (wave == 0) {
        const uint64_t left = __ballot(lane < kClasses && (int)given < ours / kClasses);
        if (lane == 0) {  // nothing; or a batch; or, from `grid` on, a tile taken alone
          int v = -1;
          if (!drained) v = grid + base + take(next_tile);
          else if (left != 0) v = claim(__builtin_ctzll(left));
          s_ctl[3] = v;
        }
      }
      lds_barrier();
      const int v = __builtin_amdgcn_readfirstlane(s_ctl[3]);
      // The last workgroup raises the flags, each for few enough that their reads do not hold it up (of one word, read by
      // everyone, the news took 6 us).
      if (wave == 0 && mine > 0) {
        uint32_t before = 0;
        if (lane == 0) before = __hip_atomic_fetch_add(done, (uint32_t)mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if ((int)__builtin_amdgcn_readfirstlane(before) + mine == tiles && lane < kFlags)
          __hip_atomic_store(flags + lane * 32, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      mine = 0;
      if (v < 0) break;
      lds_barrier();  // everyone has read what was taken
      if (drained) {
        set_batch(v);
      } else {
        q0 = v - grid;
        q1 = q2 = tiles;
        drained = q0 >= tiles;
      }
      asked = false;
      if (q0 >= tiles) continue;
      p0 = place_of(q0);
      p1 = place_of(q1);
      p2 = place_of(q2);
      wait_vm<0>();  // start over with an empty ring
      slot = 0;
#pragma unroll 1
      for (int s = 0; s < D; ++s) load_ahead(s, s);
    }
    const int a = (int)((uint32_t)q0 / (uint32_t)nt), tile = q0 - a * nt;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    u32x4 sc = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < F::kSteps; ++j) {
      if (j < D / 2 || j < steps) {
        wait_vm<F::kWaitUp>();
        const Step s = read_step(slot);
        load_ahead(slot, j + D);
        next_slot();
        const int b = own_block(j, 0);
        if (b < nb1) {
          f32x4 part = {0.f, 0.f, 0.f, 0.f};
          if constexpr (FMT != W_E4M3 && FMT != W_E4M3_E8M0) part = acc;
          const float s0 = __uint_as_float(s.sc[0] << 23), s1 = __uint_as_float(s.sc[1] << 23);
#pragma unroll
          for (int v = 0; v < F::kVec; ++v) part = mfma_bf16(operand<FMT>(s.lo, v, s0), x[j][0][v], part);
          if (FMT != W_FP4 || b * F::kBlock + F::kBlock / 2 < p.d) {
#pragma unroll
            for (int v = 0; v < F::kVec; ++v) part = mfma_bf16(operand<FMT>(s.hi, v, s1), x[j][1][v], part);
          }
          if constexpr (FMT == W_E4M3 || FMT == W_E4M3_E8M0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = fmaf(part[r], row_scale(s, b, r), acc[r]);
          } else {
            acc = part;
          }
        }
        if constexpr (FMT == W_I8) sc = s.sc;
      }
    }
    if constexpr (FMT == W_I8) {
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] *= __uint_as_float(sc[r]);
    }
    s_red[buf][wave][lane] = acc;
    if (asked && tid == 0) s_ctl[buf] = taken;
    lds_barrier();
    const int next = asked ? __builtin_amdgcn_readfirstlane(s_ctl[buf]) : tiles;
    drained = drained || (asked && next >= tiles);
    // The tile after the ones that are known by now is asked for here, where only the first wave will wait for the answer
    // (at the end of the next tile), not the others' loads.
    asked = next < tiles;
    if (asked && tid == 0) taken = base + take(next_tile);
    if (wave < kJoiners) {  // the waves' sums in wave order, SwiGLU, h
      const int t = tid >> 3, c = tid & 7;
      const uint32_t at = red_at + buf * (kNW * 1024) + (t + 16 * (c >> 2)) * 16 + (c & 3) * 4;
      const float g = join8(at), up = join8(at + 512);
      const int k = s_k[a][t];
      if (k != 255) {
        // h in two bf16 parts: the float's upper half and what is left of it, rounded (2^-16 of h at most is lost).  An even lane
        // stores its own and its neighbour's upper parts, an odd one the lower ones, through to memory.
        const float h = silu(g) * up;
        const uint32_t w = __float_as_uint(h);
        const float rest = fabsf(h) < INFINITY ? h - __uint_as_float(w & 0xffff0000u) : 0.f;
        const uint32_t both = (w >> 16) | (f32_to_bf16_rne(rest) << 16);
        const uint32_t next = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)both, 0xb1, 0xf, 0xf, false);  // quad_perm 1, 0, 3, 2
        const uint32_t pair = c & 1 ? (next >> 16) | (both & 0xffff0000u) : (both & 0xffffu) | (next << 16);
        uint16_t* o = p.h + (int64_t)(t * KS + k) * 2 * p.inter + (c & 1 ? p.inter : 0) + tile * 8 + (c & ~1);
        __hip_atomic_store(reinterpret_cast<uint32_t*>(o), pair, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    q0 = q1;
    p0 = p1;
    q1 = deep ? q2 : next;
    p1 = deep ? p2 : place_of(next);
    if (deep) {
      q2 = next;
      p2 = place_of(next);
    }
    buf ^= 1;
    ++mine;
  }
  // the down projection's first weights, while the others finish
  wait_vm<0>();
  slot = 0;
#pragma unroll 1
  for (int s = 0; s < D; ++s) load_step(s, down_step_at(s));

  // ---- down ----
  for (int block = number; block < blocks; block += gridDim.x) {
    const int c0 = block * R, cols = min(R, p.d - c0);
    if (block == number) {
      if (tid == 0) {
        const uint32_t* const flag = flags + number % kFlags * 32;
        int left = p.looks;
        while (left > 0 && __hip_atomic_load(flag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0) {
          __builtin_amdgcn_s_sleep(4);
          --left;
        }
        if (left <= 0) s_ctl[2] = 1;
      }
      // one wave's acquire clears what L1 and L2 hold for the others too (by all waves of all workgroups: 13 us)
      if (wave == 0) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      lds_barrier();
    } else {
      set_block(block);
      slot = 0;
#pragma unroll 1
      for (int s = 0; s < D; ++s) load_step(s, down_step_at(s));
    }
    f32x4 total[2][P];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < P; ++q) total[r][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    // This lane's h of a unit: its column's token's, zeros for a token that did not choose the expert.  What a unit needs from
    // tables in LDS is read an expert earlier: a chain of lookups would take longer than its products.
    const int col = WIDE ? lr : lr & 7;
    const uint32_t h_b = (uint32_t)(T * KS) * (uint32_t)p.inter * 4;
    const uint32_t hl = (WIDE || lr < 8 ? 0 : p.inter * 2) + lg * (F::kBlock / 4);
    auto after = [&](int a) __attribute__((always_inline)) { return a + 1 < A ? a + 1 : 0; };  // past the end the first units again
    auto h_at = [&](int k) __attribute__((always_inline)) {
      return k != 255 ? (uint32_t)(col * KS + k) * (uint32_t)p.inter * 4 + hl : kNoLoad;
    };
    u32x4 raw[F::kSets][2][F::kVec][P];  // of the next units
    int raw_k[F::kSets], raw_b[F::kSets];
    float raw_gate[F::kSets];
    int na = 0, ns = 0, ne = expert(0), nk = s_k[0][col];  // the unit whose h is loaded next
    uint32_t hv = h_at(nk);
    int ne2 = s_exp[after(0)], nk2 = s_k[after(0)][col];   // of the expert behind it
    auto load_next_h = [&](auto set_c) __attribute__((always_inline)) {
      constexpr int S = decltype(set_c)::value;
      raw_k[S] = nk;
      raw_gate[S] = s_gate[col * KS + min(nk, KS - 1)];
      raw_b[S] = own_block(ns, ne);
      const uint32_t off = block_of(ns, ne, nb2) * (F::kBlock * 2);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int v = 0; v < F::kVec; ++v)
#pragma unroll
          for (int q = 0; q < P; ++q) raw[S][hf][v][q] = load16_if(p.h, h_b, hv, off + q * p.inter * 2 + hf * F::kBlock + v * 16);
      if (++ns == slices) {
        ns = 0;
        na = after(na);
        ne = __builtin_amdgcn_readfirstlane(ne2);
        nk = nk2;
        hv = h_at(nk);
        ne2 = s_exp[after(na)];
        nk2 = s_k[after(na)][col];
      }
    };
    int la = D / 2 / slices, ls = D / 2 - la * slices;     // the unit whose weights are loaded next
    la = la < A ? la : 0;
    int le = expert(la), le2 = s_exp[after(la)];
    Place lp = down_place(le);
    load_next_h(std::integral_constant<int, 0>());
    load_next_h(std::integral_constant<int, 1>());
    if constexpr (F::kSets > 2) load_next_h(std::integral_constant<int, F::kSets == 2 ? 0 : 2>());
    if constexpr (F::kSets > 3) load_next_h(std::integral_constant<int, F::kSets == 4 ? 3 : 0>());
    wait_vm<0>();  // the compiler then counts the next units' loads against the ring's instead of waiting for all
    // (Every unit loads, also those that only round their number up: the waits count on it.)
    auto unit = [&](auto set_c, bool live) __attribute__((always_inline)) {
      constexpr int S = decltype(set_c)::value;
      const bool chosen = live && raw_k[S] != 255;
      const float gate = raw_gate[S];
      const int b = raw_b[S];
      wait_vm<F::kWaitDown>();
      Step st[2];
      read_pair(slot, st[0], st[1]);
      if (b < nb2) {
        f32x4 part[2][P];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int q = 0; q < P; ++q) part[r][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto products = [&](int hf) __attribute__((always_inline)) {
#pragma unroll
          for (int v = 0; v < F::kVec; ++v)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const bf16x8_t w = operand<FMT>(hf ? st[r].hi : st[r].lo, v, __uint_as_float(st[r].sc[hf] << 23));
#pragma unroll
              for (int q = 0; q < P; ++q) part[r][q] = mfma_bf16(w, __builtin_bit_cast(bf16x8_t, raw[S][hf][v][q]), part[r][q]);
            }
        };
        products(0);
        if (FMT != W_FP4 || b * F::kBlock + F::kBlock / 2 < p.inter) products(1);
        if (chosen) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float g = gate;
              if constexpr (FMT == W_E4M3 || FMT == W_E4M3_E8M0 || FMT == W_I8) g *= row_scale(st[r], b, i);
#pragma unroll
              for (int q = 0; q < P; ++q) total[r][q][i] = fmaf(g, part[r][q][i], total[r][q][i]);
            }
        }
      }
      load_next_h(set_c);
      load_step(slot, down_step(lp, le, ls, 0));
      load_step(slot + 1, down_step(lp, le, ls, 1));
      slot = slot + 2 == D ? 0 : slot + 2;
      if (++ls == slices) {
        ls = 0;
        la = after(la);
        le = __builtin_amdgcn_readfirstlane(le2);
        lp = down_place(le);
        le2 = s_exp[after(la)];
      }
    };
#pragma unroll 1
    for (int un = 0; un < units; un += F::kSets) {
      __builtin_amdgcn_s_barrier();  // the waves keep together: the last ones alone would not load at the full rate
      unit(std::integral_constant<int, 0>(), true);
      unit(std::integral_constant<int, 1>(), un + 1 < units);
      if constexpr (F::kSets > 2) unit(std::integral_constant<int, F::kSets == 2 ? 0 : 2>(), un + 2 < units);
      if constexpr (F::kSets > 3) unit(std::integral_constant<int, F::kSets == 4 ? 3 : 0>(), un + 3 < units);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // upper and lower parts: column t + 8 holds the latter, or the other sum
        total[r][0][i] += WIDE ? total[r][P - 1][i] : __uint_as_float(row_ror<8>(__float_as_uint(total[r][0][i])));
    lds_barrier();  // the sums' space is free
    s_red[0][wave][lane] = total[0][0];
    s_red[1][wave][lane] = total[1][0];
    lds_barrier();
    const int t = tid >> 5, c = tid & 31;
    float v = join8(red_at + (c >> 4) * (kNW * 1024) + (t + 16 * ((c & 15) >> 2)) * 16 + (c & 3) * 4);
    if (s_ctl[2]) v = __uint_as_float(0x7fc00000u);  // h was never complete
    if (t < T && c < cols) {
      uint8_t* o = p.out + t * p.ldo_b;
      if (p.out_dtype == ROW_F32) reinterpret_cast<float*>(o)[c0 + c] = v;
      else reinterpret_cast<uint16_t*>(o)[c0 + c] = (uint16_t)f32_to_bf16_rne(v);
    }
    wait_vm<0>();  // the ring is empty again
    lds_barrier();
  }
  wait_vm<0>();  // no load into LDS outlives the workgroup
}

int compute_units() {
  int dev = 0, v = 0;
  if (hipGetDevice(&dev) == hipSuccess && hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess &&
      v >= 1)
    return v;
  return 256;
}

template <int FMT>
void launch_experts(const ExpertArgs& a, int grid, hipStream_t stream) {
  if (a.T > 8) decode_experts_kernel<FMT, true><<<grid, kNW * 64, 0, stream>>>(a);
  else decode_experts_kernel<FMT, false><<<grid, kNW * 64, 0, stream>>>(a);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_decode_workspace_size(int T, int d, int inter, int n_experts, int n_shared, int top_k) {
  if (T < 0 || T > moe::kMaxT || d < 1 || d > moe::kMaxD || inter < 1 || n_experts < 1 || n_shared < 0 || n_shared > 1 ||
      top_k < 1 || top_k > moe::kMaxTopK)
    return 0;
  return moe::decode_ws(T, d, inter, n_shared, top_k).total;
}

namespace moe {
namespace {

moe_status decode(const moe_decode_desc* q, int workgroups, int lists, int looks, hipStream_t stream) {
  clear_error();
  MOE_REQUIRE(q != nullptr, MOE_ERR_NULL, "moe_decode: desc is NULL");
  MOE_REQUIRE(q->T >= 0 && q->T <= kMaxT, MOE_ERR_SHAPE, "moe_decode: T=%d must be in [0, %d]", q->T, kMaxT);
  MOE_REQUIRE(q->n_experts >= 4 && q->n_experts <= 256 && q->n_experts % 4 == 0, MOE_ERR_SHAPE,
              "moe_decode: n_experts=%d must be in [4, 256] and a multiple of 4", q->n_experts);
  MOE_REQUIRE(q->n_shared == 0 || q->n_shared == 1, MOE_ERR_SHAPE, "moe_decode: n_shared=%d must be 0 or 1", q->n_shared);
  MOE_REQUIRE(q->top_k >= 1 && q->top_k <= kMaxTopK && q->top_k <= q->n_experts, MOE_ERR_SHAPE,
              "moe_decode: top_k=%d must be in [1, %d] and at most n_experts=%d", q->top_k, kMaxTopK, q->n_experts);
  MOE_REQUIRE(q->n_group >= 1 && q->n_group <= 64 && q->n_experts % q->n_group == 0, MOE_ERR_SHAPE,
              "moe_decode: n_group=%d must divide n_experts=%d and be <= 64", q->n_group, q->n_experts);
  MOE_REQUIRE(q->topk_group >= 1 && q->topk_group <= q->n_group, MOE_ERR_SHAPE,
              "moe_decode: topk_group=%d must be in [1, n_group=%d]", q->topk_group, q->n_group);
  if (q->n_group > 1) {
    const int gs = q->n_experts / q->n_group;
    MOE_REQUIRE(gs >= 4 && (gs & (gs - 1)) == 0, MOE_ERR_SHAPE,
                "moe_decode: groups must hold a power of two >= 4 experts (n_experts/n_group=%d)", gs);
    MOE_REQUIRE(q->top_k <= q->topk_group * gs, MOE_ERR_SHAPE, "moe_decode: top_k=%d exceeds the %d experts of the kept groups",
                q->top_k, q->topk_group * gs);
  }
  int fmt;
  switch (q->w_dtype) {
    case MOE_BF16: fmt = W_BF16; break;
    case MOE_FP8_E4M3: fmt = q->scale_fmt == MOE_SCALE_E8M0 ? W_E4M3_E8M0 : W_E4M3; break;
    case MOE_I8: fmt = W_I8; break;
    case MOE_FP4_E2M1: fmt = W_FP4; break;
    default: fmt = -1;
  }
  MOE_REQUIRE(fmt >= 0, MOE_ERR_DTYPE, "moe_decode: unknown w_dtype %d", q->w_dtype);
  MOE_REQUIRE(q->scale_fmt == MOE_SCALE_F32 || (q->scale_fmt == MOE_SCALE_E8M0 && q->w_dtype == MOE_FP8_E4M3), MOE_ERR_DTYPE,
              "moe_decode: unknown scale_fmt %d", q->scale_fmt);
  MOE_REQUIRE(q->norm == MOE_NORM_NONE || q->norm == MOE_NORM_LAYER || q->norm == MOE_NORM_RMS, MOE_ERR_DTYPE,
              "moe_decode: unknown norm %d", q->norm);
  const bool norm = q->norm != MOE_NORM_NONE;
  MOE_REQUIRE(q->x_dtype == MOE_BF16 || (norm && q->x_dtype == MOE_F32), MOE_ERR_DTYPE,
              "moe_decode: x must be MOE_BF16, or MOE_F32 with a norm (%d)", q->x_dtype);
  MOE_REQUIRE(q->out_dtype == MOE_BF16 || q->out_dtype == MOE_F32, MOE_ERR_DTYPE,
              "moe_decode: out_dtype must be MOE_BF16 or MOE_F32 (%d)", q->out_dtype);
  MOE_REQUIRE(!norm || q->norm_dtype == MOE_BF16 || q->norm_dtype == MOE_F32, MOE_ERR_DTYPE, "moe_decode: unknown norm_dtype %d",
              q->norm_dtype);
  MOE_REQUIRE(!norm || (q->norm_eps >= 0.0f && q->norm_eps < 1e30f), MOE_ERR_SHAPE, "moe_decode: norm_eps=%g must be in [0, 1e30)",
              (double)q->norm_eps);
  const int gran = fmt == W_BF16 ? 64 : fmt == W_E4M3_E8M0 ? 512 : 128;
  MOE_REQUIRE(q->d >= gran && q->d <= kMaxD && q->d % gran == 0, MOE_ERR_SHAPE,
              "moe_decode: d=%d must be a positive multiple of %d up to %d", q->d, gran, kMaxD);
  MOE_REQUIRE(q->inter >= gran && q->inter % gran == 0, MOE_ERR_SHAPE, "moe_decode: inter=%d must be a positive multiple of %d",
              q->inter, gran);
  const int64_t esz2 = fmt == W_BF16 ? 4 : fmt == W_FP4 ? 1 : 2;  // half bytes per weight
  MOE_REQUIRE((int64_t)2 * q->inter * q->d * esz2 / 2 < ((int64_t)1 << 31), MOE_ERR_SHAPE,
              "moe_decode: one expert's weights exceed 2 GiB");
  MOE_REQUIRE(q->T == 0 || (q->x && q->w_router && q->bias && q->w13 && q->w2 && q->out &&
                            (fmt == W_BF16 || (q->w13_scale && q->w2_scale))),
              MOE_ERR_NULL, "moe_decode: x, w_router, bias, w13, w2 (with their scales) and out are required");
  const int xsz = q->x_dtype == MOE_F32 ? 4 : 2, osz = q->out_dtype == MOE_F32 ? 4 : 2, nsz = q->norm_dtype == MOE_F32 ? 4 : 2;
  MOE_REQUIRE(q->ldx >= q->d && (norm ? aligned_to(q->x, xsz) : q->ldx % 8 == 0 && aligned16(q->x)), MOE_ERR_ALIGN,
              "moe_decode: ldx=%lld must be >= d (without a norm: a multiple of 8, x 16-byte aligned)", (long long)q->ldx);
  MOE_REQUIRE(q->ldo >= q->d && aligned_to(q->out, osz), MOE_ERR_ALIGN,
              "moe_decode: ldo=%lld must be >= d and out aligned to its elements", (long long)q->ldo);
  MOE_REQUIRE(aligned16(q->w_router) && aligned16(q->w13) && aligned16(q->w2), MOE_ERR_ALIGN,
              "moe_decode: w_router, w13 and w2 must be 16-byte aligned");
  MOE_REQUIRE(aligned_to(q->w13_scale, 4) && aligned_to(q->w2_scale, 4) && aligned_to(q->bias, 4) && aligned_to(q->topk_idx, 4) &&
                  aligned_to(q->topk_gate, 4) && aligned_to(q->expert_counts, 4) &&
                  (!norm || (aligned_to(q->norm_weight, nsz) && aligned_to(q->norm_bias, nsz))),
              MOE_ERR_ALIGN, "moe_decode: scales, bias, norm vectors and routing outputs must be aligned to their elements");
  if (q->T == 0) {
    if (q->expert_counts) decode_zero_counts_kernel<<<1, 256, 0, stream>>>(q->expert_counts, q->n_experts);
    return check_launch("moe_decode");
  }
  MOE_REQUIRE((int64_t)q->T * (q->top_k + q->n_shared) * q->inter * 4 < ((int64_t)1 << 32) - 256, MOE_ERR_SHAPE,
              "moe_decode: T * (top_k + n_shared) * inter = %lld values of h exceed 4 GiB",
              (long long)q->T * (q->top_k + q->n_shared) * q->inter);
  const DecodeWs L = decode_ws(q->T, q->d, q->inter, q->n_shared, q->top_k);
  MOE_REQUIRE(q->ws && q->ws_bytes >= L.total && aligned16(q->ws), MOE_ERR_WORKSPACE,
              "moe_decode: workspace %zu < %zu bytes (or NULL / unaligned)", q->ws_bytes, L.total);
  uint8_t* ws = static_cast<uint8_t*>(q->ws);
  RowsArgs r;
  r.x = static_cast<const uint8_t*>(q->x);
  r.x_dtype = q->x_dtype == MOE_F32 ? ROW_F32 : ROW_BF16;
  r.ldx_b = q->ldx * xsz;
  r.T = q->T;
  r.d = q->d;
  r.N = q->n_experts;
  r.norm = q->norm;
  r.weight = q->norm_weight;
  r.bias = q->norm_bias;
  r.w_dtype = q->norm_dtype == MOE_F32 ? ROW_F32 : ROW_BF16;
  r.eps = q->norm_eps;
  r.wr = q->w_router;
  r.counters = reinterpret_cast<uint32_t*>(ws);
  r.scores = reinterpret_cast<double*>(ws + L.scores);
  r.xn = reinterpret_cast<uint16_t*>(ws + L.xn);
  const int token_groups = (q->T + 3) / 4;
  r.experts = token_groups;  // as many workgroups as experts: all at once on the card
  const dim3 rows_grid((q->n_experts + r.experts - 1) / r.experts, token_groups);
  if (norm) decode_rows_kernel<true><<<rows_grid, kRowThreads, 0, stream>>>(r);
  else decode_rows_kernel<false><<<rows_grid, kRowThreads, 0, stream>>>(r);
  ExpertArgs a;
  a.xn = norm ? r.xn : static_cast<const uint16_t*>(q->x);
  a.ldxn = norm ? q->d : q->ldx;
  a.T = q->T;
  a.d = q->d;
  a.inter = q->inter;
  a.N = q->n_experts;
  a.n_shared = q->n_shared;
  a.K = q->top_k;
  a.n_group = q->n_group;
  a.topk_group = q->topk_group;
  a.bias = q->bias;
  a.scores = r.scores;
  a.counters = r.counters;
  a.h = reinterpret_cast<uint16_t*>(ws + L.h);
  a.w13 = static_cast<const uint8_t*>(q->w13);
  a.s13 = static_cast<const uint8_t*>(q->w13_scale);
  a.w2 = static_cast<const uint8_t*>(q->w2);
  a.s2 = static_cast<const uint8_t*>(q->w2_scale);
  a.out = static_cast<uint8_t*>(q->out);
  a.out_dtype = q->out_dtype == MOE_F32 ? ROW_F32 : ROW_BF16;
  a.ldo_b = q->ldo * osz;
  a.topk_idx = q->topk_idx;
  a.topk_gate = q->topk_gate;
  a.counts = q->expert_counts;
  const int block = fmt == W_BF16 ? 64 : fmt == W_FP4 ? 256 : 128, depth = fmt == W_FP4 ? Fmt<W_FP4>::kDepth : Fmt<W_BF16>::kDepth;
  const int per_wave = ((q->d + block - 1) / block + kNW - 1) / kNW;
  a.ahead = per_wave < depth ? 3 : 2;
  a.lists = lists;
  a.looks = looks;
  switch (fmt) {
    case W_BF16: launch_experts<W_BF16>(a, workgroups, stream); break;
    case W_E4M3: launch_experts<W_E4M3>(a, workgroups, stream); break;
    case W_E4M3_E8M0: launch_experts<W_E4M3_E8M0>(a, workgroups, stream); break;
    case W_I8: launch_experts<W_I8>(a, workgroups, stream); break;
    default: launch_experts<W_FP4>(a, workgroups, stream); break;
  }
  return check_launch("moe_decode");
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_decode(const moe_decode_desc* q, hipStream_t stream) {
  const int cus = moe::compute_units();
  return moe::decode(q, cus, cus, moe::kWaitLooks, stream);
}

// For the tests, not in moe.h: moe_decode as a smaller or a busy device runs it.  `workgroups` of the second launch start, and tiles
// are dealt out as for `lists` of them, so that those which start take over the rest; they also walk more than one block of columns
// each, where moe_decode's workgroups have one at most on 256 CUs.  Each gives up waiting for h after `looks` at its flag (0: none).
extern "C" moe_status moe_decode_shaped(const moe_decode_desc* q, int workgroups, int lists, int looks, hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(workgroups >= 1 && workgroups <= lists && lists <= 1024, MOE_ERR_SHAPE,
              "moe_decode_shaped: workgroups=%d must be in [1, lists=%d], lists at most 1024", workgroups, lists);
  MOE_REQUIRE(looks >= 0 && looks <= kWaitLooks, MOE_ERR_SHAPE, "moe_decode_shaped: looks=%d must be in [0, %d]", looks, kWaitLooks);
  return decode(q, workgroups, lists, looks, stream);
}
