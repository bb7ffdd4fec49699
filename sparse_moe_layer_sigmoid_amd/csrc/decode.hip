// moe_decode: the whole layer for a few tokens, in two launches.
//
//   xn = bf16(norm(x)),  u = xn . e_i,  s = sigmoid(u),  top-K of s + b,  gate = s / sum s
//   out = sum_k gate_k W2[e_k] h_k + W2[shared] h_shared,   h_e = silu(W1[e] xn) * (W3[e] xn)
//
// A token's experts are read once and hardly computed with, so the bytes of the active experts' weights are the floor
// (one token: 9 experts of 257) and everything else is latency: launches, the first loads, the hand-over of h.
//
//  1. decode_rows_kernel: a workgroup per routed expert normalises the tokens (each workgroup all of them: the rows are a
//     few KB in L2), writes its share of them as bf16 and sums its expert's logits in fp64 (bf16 products are exact in fp32).
//  2. decode_experts_kernel: one workgroup of 8 waves per CU.  Each selects the tokens' experts from the logits by itself
//     (a microsecond or two, while its first weights are on the way), then takes tiles of 8 gate rows and their 8 up rows of the
//     active experts, and then blocks of output columns, which it sums over all experts: no atomics on values, no partial
//     outputs in memory, one order of sums.
//
// Columns are tokens: the matrix cores take 16 weight rows against 16 columns, and column t is token t whatever its experts
// are.  Products with experts that a token did not choose cost nothing that the weights' bytes do not hide and are left out
// of its sums, so no rows are sorted or gathered.
//
// K is split over the 8 waves in blocks of 128 bytes of a weight row, dealt out in turn; each wave holds its inputs of all
// tokens in registers, and its weights come through a ring of its own in LDS by direct-to-LDS loads of 16 rows x 128 bytes a
// step, XOR-swizzled so that operand reads meet distinct banks.  The ring runs on across tiles, experts and from the gate/up
// tiles into the down projection, whose weights do not depend on h: while the workgroups wait for each other's h, the chip
// has up to 32 MB of the next weights in LDS or on the way.
//
// The hand-over: gate/up tiles are dealt out in lists, one per workgroup, by a ticket; a workgroup that has finished its list
// takes further lists while there are any, so that every list is in the hands of a running workgroup before any workgroup
// waits for the count of finished lists.  None waits for one that has not started: calls may overlap on the device.
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
constexpr int kRowThreads = 512;
constexpr uint64_t kWaitTicks = 500000000ull;  // 5 s of the 100 MHz clock: bound of the wait for h

// Workspace: counters, logits, normalised rows, h.
constexpr size_t kCounterBytes = 512;  // the next list, the next block of columns, finished lists: 128 bytes apart
constexpr size_t kLogitBytes = (size_t)kMaxT * 256 * sizeof(double);
struct DecodeWs {
  size_t logits, xn, h, total;
};
DecodeWs decode_ws(int T, int d, int inter, int n_shared, int top_k) {
  DecodeWs w;
  w.logits = kCounterBytes;
  w.xn = w.logits + kLogitBytes;
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
  const uint16_t* wr;
  uint32_t* counters;
  double* logits;  // [T][256]
  uint16_t* xn;
};

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

__global__ __launch_bounds__(kRowThreads) void decode_rows_kernel(RowsArgs p) {
  constexpr int CH = kMaxD / 8 / kRowThreads;  // chunks of 8 inputs per lane
  __shared__ double s_mean[kMaxT], s_rstd[kMaxT], s_red[kRowThreads / 64][kMaxT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x, chunks = p.d / 8;
  if (e == 0 && tid < 3) p.counters[tid * 32] = 0;
  u32x4 wv[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    wv[j] = u32x4{0u, 0u, 0u, 0u};
    const int c = tid + j * kRowThreads;
    if (c < chunks && e < p.N) wv[j] = *(const u32x4*)(p.wr + (int64_t)e * p.d + c * 8);
  }
  if (p.norm != MOE_NORM_NONE) {
    // statistics in fp64, of x minus the row's first element: no range to leave, and a mean far from zero cancels nothing
    for (int t = wave; t < p.T; t += kRowThreads / 64) {
      const uint8_t* row = p.x + t * p.ldx_b;
      float f[8];
      double pivot = 0.0, s1 = 0.0, s2 = 0.0;
      if (p.norm == MOE_NORM_LAYER)
        pivot = p.x_dtype == ROW_F32 ? (double)*(const float*)row : (double)bf16_to_f32(*(const uint16_t*)row);
      for (int c = lane; c < chunks; c += 64) {
        load8_any<true>(p.x_dtype, row, c * 8, p.d, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double v = (double)f[i] - pivot;
          s1 += v;
          s2 += v * v;
        }
      }
      s1 = wave_sum64(s1) / p.d;
      s2 = wave_sum64(s2) / p.d;
      if (lane == 0) {
        const bool layer = p.norm == MOE_NORM_LAYER;
        s_mean[t] = layer ? pivot + s1 : 0.0;
        s_rstd[t] = 1.0 / sqrt(fmax(layer ? s2 - s1 * s1 : s2, s2 - s2) + p.eps);
      }
    }
    __syncthreads();
  }
  float g[CH][8], b[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = tid + j * kRowThreads;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[j][i] = 1.f;
      b[j][i] = 0.f;
    }
    if (p.norm != MOE_NORM_NONE && c < chunks) {
      if (p.weight) load8_any<true>(p.w_dtype, p.weight, c * 8, p.d, g[j]);
      if (p.bias) load8_any<true>(p.w_dtype, p.bias, c * 8, p.d, b[j]);
    }
  }
  for (int t = 0; t < p.T; ++t) {
    const uint8_t* row = p.x + t * p.ldx_b;
    double acc = 0.0;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = tid + j * kRowThreads;
      if (c >= chunks) continue;
      float f[8], w[8];
      load8_any<true>(p.x_dtype, row, c * 8, p.d, f);
      if (p.norm != MOE_NORM_NONE) {
        const double mean = s_mean[t], rstd = s_rstd[t];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)(((double)f[i] - mean) * rstd * (double)g[j][i] + (double)b[j][i]);
        const u32x4 o = pack_bf16x8(f);
        if (t % gridDim.x == e) *(u32x4*)(p.xn + (int64_t)t * p.d + c * 8) = o;
        unpack_bf16x8(o, f);
      }
      unpack_bf16x8(wv[j], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc += (double)(f[i] * w[i]);
    }
    acc = wave_sum64(acc);
    if (lane == 0) s_red[wave][t] = acc;
  }
  __syncthreads();
  if (tid < p.T && e < p.N) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kRowThreads / 64; ++w) sum += s_red[w][tid];
    p.logits[tid * 256 + e] = sum;
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
  const double* logits;
  uint32_t* counters;
  float* h;  // [T][K + n_shared][inter]
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

template <int N>
__device__ __forceinline__ void wait_vm() {  // at most N of the newest vector-memory operations in flight
  static_assert(N >= 0 && N <= 63, "six bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// Workgroup barrier that waits for this wave's LDS operations but not for its loads in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 or 4 bytes per lane from base + v + off (v per lane, base and off uniform; `bytes` from base on may be read) to LDS at
// dst, lane after lane.  (The host pass does not know the builtin.)
__device__ __forceinline__ void load16_to_lds(const uint8_t* base, uint32_t bytes, uint32_t v, uint32_t off, uint8_t* dst) {
#ifdef __HIP_DEVICE_COMPILE__
  const auto r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, v, off, 0, 0);
#endif
}
__device__ __forceinline__ void load4_to_lds(const uint8_t* base, uint32_t bytes, uint32_t v, uint32_t off, uint8_t* dst) {
#ifdef __HIP_DEVICE_COMPILE__
  const auto r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, v, off, 0, 0);
#endif
}

__device__ __forceinline__ float silu(float a) { return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }

template <int FMT>
struct Fmt {
  static constexpr bool kScaled = FMT != W_BF16;
  static constexpr int kBlock = FMT == W_BF16 ? 64 : FMT == W_FP4 ? 256 : 128;  // inputs in 128 bytes of a weight row
  static constexpr int kVec = kBlock / 64;              // operands of 8 inputs per lane in half a block
  static constexpr int kSteps = kMaxD / kBlock / kNW;   // blocks per wave of a gate/up tile at most
  static constexpr int kUnit = 256 / kBlock;            // blocks per wave of a unit of the down projection
  static constexpr int kSlot = 2048 + (kScaled ? 128 : 0);  // a step's weights and scales
  // Steps in flight per wave: as many as LDS holds, and in the down projection a whole number of units (of 2 * kUnit steps)
  // whose loads, with the 16 loads of h that each unit adds, can still be counted (see wait_step)
  static constexpr int kDepth = FMT == W_FP4 ? 6 : 8;
  static constexpr int kLoads = kScaled ? 3 : 2;        // loads of a step
  static constexpr int kWaitUp = kLoads * (kDepth - 1);
  static constexpr int kWaitDown = kWaitUp + kDepth / (2 * kUnit) * 16;
};

// 8 weights of a step's half block: dword pairs (bf16: the 16 bytes), its operand `s`.
template <int FMT>
__device__ __forceinline__ bf16x8_t operand(const u32x4& q, int s, float scale) {
  if constexpr (FMT == W_BF16) return __builtin_bit_cast(bf16x8_t, q);
  else if constexpr (FMT == W_FP4) return decode_w4(q[s], scale);
  else if constexpr (FMT == W_I8) return decode_i8(q[2 * s], q[2 * s + 1]);
  else return decode_e4m3(q[2 * s], q[2 * s + 1]);
}

// h in two bf16 parts: the upper half of the float and what is left, rounded (2^-16 of h at most is lost).
__device__ __forceinline__ void split8(const f32x4& a, const f32x4& b, bf16x8_t& hi, bf16x8_t& lo) {
  u32x4 h, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v0 = i < 2 ? a[2 * i] : b[2 * i - 4], v1 = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
    const uint32_t u0 = __float_as_uint(v0), u1 = __float_as_uint(v1);
    h[i] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
    const float r0 = v0 - __uint_as_float(u0 & 0xffff0000u), r1 = v1 - __uint_as_float(u1 & 0xffff0000u);
    const float l0 = fabsf(v0) < INFINITY ? r0 : 0.f, l1 = fabsf(v1) < INFINITY ? r1 : 0.f;
    l[i] = f32_to_bf16_rne(l0) | (f32_to_bf16_rne(l1) << 16);
  }
  hi = __builtin_bit_cast(bf16x8_t, h);
  lo = __builtin_bit_cast(bf16x8_t, l);
}

template <int FMT>
__global__ __launch_bounds__(kNW * 64, 2) void decode_experts_kernel(ExpertArgs p) {
  using F = Fmt<FMT>;
  constexpr int D = F::kDepth, SLOT = F::kSlot;
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kNW * D * SLOT];
  __shared__ __attribute__((aligned(16))) f32x4 s_red[2][kNW][64];
  __shared__ float s_gate[kMaxT * (kMaxTopK + 1)];  // gate of slot t (K + n_shared) + k
  __shared__ __attribute__((aligned(16))) uint8_t s_k[kMaxActive][kMaxT];  // k of a token's active expert, 255: not chosen
  __shared__ uint16_t s_exp[kMaxActive];            // active experts, the shared one first
  __shared__ uint8_t s_first[kMaxActive];           // a token that chose it
  __shared__ int s_ctl[4];                          // list, block of columns, active experts, gave up waiting
  // of the selection, before the sums need the space
  uint32_t* const s_mask = reinterpret_cast<uint32_t*>(&s_red[0][0][0]);
  int32_t* const s_idx = reinterpret_cast<int32_t*>(&s_red[0][4][0]);
  int32_t* const s_pos = reinterpret_cast<int32_t*>(&s_red[1][0][0]);
  uint32_t* const s_cnt = reinterpret_cast<uint32_t*>(&s_red[1][4][0]);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int T = p.T, K = p.K, KS = p.K + p.n_shared;
  uint32_t* const list_ticket = p.counters;
  uint32_t* const block_ticket = p.counters + 32;
  uint32_t* const done = p.counters + 64;
  auto take = [](uint32_t* c) {
    return (int)__hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  int first_list = 0;
  if (tid == 0) first_list = take(list_ticket);

  // ---- this wave's inputs of all tokens (columns past T hold the last token again and are never stored) ----
  const int nb1 = (p.d + F::kBlock - 1) / F::kBlock;        // blocks of a gate/up row
  const int steps1 = (nb1 + kNW - 1) / kNW;
  bf16x8_t x[F::kSteps][2][F::kVec];
  {
    const uint16_t* xr = p.xn + (int64_t)min(lr, T - 1) * p.ldxn;
#pragma unroll
    for (int j = 0; j < F::kSteps; ++j)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int k0 = (wave + j * kNW) * F::kBlock + hf * (F::kBlock / 2);
#pragma unroll
        for (int s = 0; s < F::kVec; ++s) {
          u32x4 v = {0u, 0u, 0u, 0u};
          if (k0 < p.d) v = *(const u32x4*)(xr + k0 + lg * (F::kBlock / 8) + s * 8);
          x[j][hf][s] = __builtin_bit_cast(bf16x8_t, v);
        }
      }
  }

  // ---- selection ----
  for (int i = tid; i < 256; i += kNW * 64) s_mask[i] = 0;
  for (int t = wave; t < T; t += kNW) {
    double u[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) u[r] = lane * 4 + r < p.N ? p.logits[t * 256 + lane * 4 + r] : 0.0;
    float* const gate = s_gate + t * (KS - K);  // select_token writes at t * K + k; rows here are KS apart
    select_token<double>(u, p.bias, p.N, K, p.n_group, p.topk_group, t, true, s_idx, gate, nullptr);
    if (lane == 0 && p.n_shared) s_gate[t * KS + K] = 1.0f;
  }
  if (tid == 0) s_ctl[0] = first_list;
  __syncthreads();
  for (int i = tid; i < T * K; i += kNW * 64) atomicOr(&s_mask[s_idx[i]], 1u << (i / K));
  for (int i = tid; i < kMaxActive * kMaxT / 4; i += kNW * 64) reinterpret_cast<uint32_t*>(&s_k[0][0])[i] = 0xffffffffu;
  __syncthreads();
  {
    const uint32_t mask = tid < p.N ? s_mask[tid] : 0u;
    const uint64_t any = __ballot(mask != 0);
    if (lane == 0 && wave < 4) s_cnt[wave] = (uint32_t)__popcll(any);
    __syncthreads();
    int at = p.n_shared;
    for (int w = 0; w < 4 && w < wave; ++w) at += (int)s_cnt[w];
    at += __popcll(any & ((1ull << lane) - 1));
    if (mask != 0) {
      s_exp[at] = (uint16_t)tid;
      s_first[at] = (uint8_t)__builtin_ctz(mask);
      s_pos[tid] = at;
    }
    if (tid == 0) {
      if (p.n_shared) {
        s_exp[0] = (uint16_t)p.N;
        s_first[0] = 0;
      }
      s_ctl[2] = p.n_shared + (int)(s_cnt[0] + s_cnt[1] + s_cnt[2] + s_cnt[3]);
      s_ctl[3] = 0;
    }
    if (s_ctl[0] == 0) {  // the first workgroup reports the routing
      if (p.counts && tid < p.N) p.counts[tid] = __popc(mask);
      for (int i = tid; i < T * K; i += kNW * 64) {
        if (p.topk_idx) p.topk_idx[i] = s_idx[i];
        if (p.topk_gate) p.topk_gate[i] = s_gate[i / K * KS + i % K];
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < T * K; i += kNW * 64) s_k[s_pos[s_idx[i]]][i / K] = (uint8_t)(i % K);
  if (p.n_shared && tid < T) s_k[0][tid] = (uint8_t)K;
  __syncthreads();
  const int A = __builtin_amdgcn_readfirstlane(s_ctl[2]);

  // ---- the work: lists of gate/up tiles, then blocks of output columns ----
  const int nt = p.inter / 8;                                // tiles of an expert
  const int tiles = A * nt;
  const int lists = min((int)gridDim.x, tiles);              // list v: tiles v, v + lists, ...
  const int R = min(32, (((p.d + (int)gridDim.x - 1) / (int)gridDim.x) + 3) & ~3);  // columns of a block
  const int blocks = (p.d + R - 1) / R;
  const int nb2 = (p.inter + F::kBlock - 1) / F::kBlock;     // blocks of a down row
  const int slices = (nb2 + kNW * F::kUnit - 1) / (kNW * F::kUnit);
  constexpr int U = 2 * F::kUnit;                            // steps of a unit (expert, slice)
  const uint32_t row1_b = p.d / F::kBlock * 128 + p.d % F::kBlock * 128 / F::kBlock;
  const uint32_t row2_b = p.inter / F::kBlock * 128 + p.inter % F::kBlock * 128 / F::kBlock;

  const int lrow = lane >> 3;
  const int chunk = (lane & 7) ^ lrow;  // 16-byte piece of a block that this lane loads

  // Where the next step is loaded from: `w` and `sc` are one expert's weights and scales; this lane's rows of them are at
  // v[0], v[1] (down: v[2], v[3] in the second 16 rows of the block), its scales at vs[0] (vs[1]).  Buffer loads: for
  // the compiler global loads into LDS are flat ones, behind which it waits for everything in flight before it uses a register
  // that a load of h fills.
  enum { UP, DOWN, NOTHING };
  struct Cursor {
    int kind, a, tile, id, j, sl, steps;
    uint32_t row_b, nb;
    const uint8_t *w, *sc;
    uint32_t w_bytes, sc_bytes;
    uint32_t v[4], vs[2];
  } cu;
  const uint8_t* ring = s_ring + wave * (D * SLOT);
  const int srow = FMT == W_FP4 ? (lane >> 1) & 15 : lr;  // row of a step whose scale this lane loads
  const uint32_t half_back = FMT == W_FP4 && (chunk & 4) ? 64 : 0;
  int next_kind = NOTHING, next_id = 0;  // what is loaded after the list's last step
  // offset of row q's scales within its expert's (k inputs to a row)
  auto scale_row = [&](uint32_t q, uint32_t nb, uint32_t k) __attribute__((always_inline)) {
    if constexpr (FMT == W_FP4) return q * (k / 32) + (lane & 1) * 4;
    else if constexpr (FMT == W_E4M3) return q / 128 * nb * 4;
    else if constexpr (FMT == W_E4M3_E8M0) return q / 128 * nb;
    else return q * 4;
  };
  auto set_expert = [&]() __attribute__((always_inline)) {
    const int64_t e = __builtin_amdgcn_readfirstlane(s_exp[cu.a]);
    const bool up = cu.kind == UP;
    const int64_t n = up ? 2 * p.inter : p.d;
    cu.w = (up ? p.w13 : p.w2) + e * n * cu.row_b;
    cu.w_bytes = (uint32_t)n * cu.row_b;
    const uint32_t k = up ? p.d : p.inter;
    const int64_t sn = FMT == W_FP4 ? n * (k / 32) : FMT == W_I8 ? n * 4 : n / 128 * cu.nb * (FMT == W_E4M3 ? 4 : 1);
    cu.sc = (up ? p.s13 : p.s2) + e * sn;
    cu.sc_bytes = (uint32_t)sn;
  };
  auto set_tile = [&]() __attribute__((always_inline)) {
    const uint32_t q = cu.tile * 8 + lrow;
    cu.v[0] = q * cu.row_b + chunk * 16;
    cu.v[1] = cu.v[0] + p.inter * cu.row_b;
    cu.vs[0] = scale_row(cu.tile * 8 + (srow & 7) + (srow < 8 ? 0 : p.inter), cu.nb, p.d);
  };
  auto start = [&](int kind, int id) __attribute__((always_inline)) {
    cu.kind = kind;
    cu.j = 0;
    cu.sl = 0;
    cu.id = id;
    cu.a = 0;
    if (kind == UP) {
      cu.a = (int)((uint32_t)id / (uint32_t)nt);
      cu.tile = id - cu.a * nt;
      cu.steps = steps1;
      cu.row_b = row1_b;
      cu.nb = nb1;
      set_expert();
      set_tile();
    } else {
      const int c0 = kind == DOWN ? id * R : 0, last = min(c0 + R, p.d) - 1;
      cu.steps = U;
      cu.row_b = row2_b;
      cu.nb = nb2;
      set_expert();
#pragma unroll
      for (int i = 0; i < 4; ++i) cu.v[i] = (uint32_t)min(c0 + i * 8 + lrow, last) * row2_b + chunk * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) cu.vs[i] = scale_row(min(c0 + i * 16 + srow, last), nb2, p.inter);
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {  // to the step after a tile's or a unit's last one
    cu.j = 0;
    if (cu.kind == UP) {
      cu.id += lists;
      if (cu.id >= tiles) {
        start(next_kind, next_id);
      } else {
        cu.tile += lists;
        while (cu.tile >= nt) {
          cu.tile -= nt;
          ++cu.a;
        }
        set_expert();
        set_tile();
      }
    } else if (cu.kind == DOWN && ++cu.sl == slices) {
      cu.sl = 0;
      if (++cu.a == A) {  // past the end the first steps again, so that the number of loads in flight stays
        cu.a = 0;
        cu.kind = NOTHING;
      }
      set_expert();
    }
  };
  // Load the next step, 16 weight rows x 128 bytes and its scales, into `slot`.
  auto issue = [&](int slot) __attribute__((always_inline)) {
    uint8_t* dst = const_cast<uint8_t*>(ring) + slot * SLOT;
    const bool up = cu.kind == UP, second = !up && (cu.j & 1);
    uint32_t b = up ? wave + cu.j * kNW : (cu.sl * F::kUnit + (cu.j >> 1)) * kNW + wave;
    b = b < cu.nb ? b : min((uint32_t)wave, cu.nb - 1);  // a wave without a block of its own here loads another, unused
    const uint32_t off = b * 128;
    const uint32_t back = FMT == W_FP4 && off + 128 > cu.row_b ? half_back : 0;  // a last block of 64 bytes
    load16_to_lds(cu.w, cu.w_bytes, (second ? cu.v[2] : cu.v[0]) - back, off, dst);
    load16_to_lds(cu.w, cu.w_bytes, (second ? cu.v[3] : cu.v[1]) - back, off, dst + 1024);
    if constexpr (F::kScaled) {
      const uint32_t vs = second ? cu.vs[1] : cu.vs[0];
      if (lane < (FMT == W_FP4 ? 32 : 16)) {
        uint32_t at = FMT == W_FP4 ? b * 8 : FMT == W_E4M3 ? b * 4 : FMT == W_E4M3_E8M0 ? b & ~3u : 0u;
        if constexpr (FMT == W_FP4) at -= off + 128 > cu.row_b ? (lane & 1) * 4 : 0;
        load4_to_lds(cu.sc, cu.sc_bytes, vs + at, 0, dst + 2048);
      }
    }
    if (++cu.j == cu.steps) advance();
  };

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

  // ---- gate/up ----
  // A list's successor has to be known when its last steps are being loaded, D steps ahead of its last tile's end: it is taken
  // `early` tiles before the last one (a short list's at its start).  Taking it sooner would keep lists from workgroups
  // that have yet to start.
  const int early = 1 + (D - 1) / steps1;
  // Lists so short that the ring holds all of one do not run on into each other: the one after next would have to be known.
  const bool chained = tiles / max(lists, 1) * steps1 > D;
  int list = __builtin_amdgcn_readfirstlane(s_ctl[0]);
  int next_list = lists, column_block = blocks;
  bool prefilled = false;
  auto take_next = [&]() __attribute__((always_inline)) {  // one lane: what follows
    const int v = take(list_ticket);
    if (v < lists) {
      s_ctl[0] = v;
    } else {
      s_ctl[0] = lists;
      s_ctl[1] = take(block_ticket);
    }
  };
  auto read_next = [&]() __attribute__((always_inline)) {
    const int v = __builtin_amdgcn_readfirstlane(s_ctl[0]);
    next_list = v;
    if (v < lists) {
      next_kind = chained ? UP : NOTHING;
      next_id = v;
    } else {
      column_block = __builtin_amdgcn_readfirstlane(s_ctl[1]);
      next_kind = column_block < blocks ? DOWN : NOTHING;
      next_id = column_block;
    }
  };
  __syncthreads();  // every lane has read the first list
  if (list >= lists) {
    if (tid == 0) s_ctl[1] = take(block_ticket);
    __syncthreads();
    column_block = __builtin_amdgcn_readfirstlane(s_ctl[1]);
  }
  wait_vm<0>();  // the inputs are here: below, waits count the ring's loads alone
  int buf = 0;
  while (list < lists) {
    const int n = (tiles - list + lists - 1) / lists;
    const int when = n - 1 - early;  // tile before which the successor is taken
    if (when < 1) {
      if (tid == 0) take_next();
      __syncthreads();
      read_next();
    }
    if (!prefilled) {
      start(UP, list);
      for (int s = 0; s < D; ++s) issue(s);
      prefilled = true;
    }
    int a = (int)((uint32_t)list / (uint32_t)nt), tile = list - a * nt;
    for (int i = 0; i < n; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      u32x4 sc = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < F::kSteps; ++j) {
        if (j < steps1) {
          wait_vm<F::kWaitUp>();
          const Step s = read_step(slot);
          issue(slot);
          next_slot();
          const int b = wave + j * kNW;
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
      if (when >= 1 && i + 1 == when && tid == 0) take_next();
      lds_barrier();
      if (when >= 1 && i + 1 == when) read_next();
      if (tid < 128) {  // the waves' sums in wave order, SwiGLU, h
        const int t = tid >> 3, c = tid & 7;
        const uint32_t at = red_at + buf * (kNW * 1024) + (t + 16 * (c >> 2)) * 16 + (c & 3) * 4;
        const float g = join8(at), u = join8(at + 512);
        const int k = s_k[a][t];
        if (k != 255) p.h[(int64_t)(t * KS + k) * p.inter + tile * 8 + c] = silu(g) * u;
      }
      buf ^= 1;
      tile += lists;
      while (tile >= nt) {
        tile -= nt;
        ++a;
      }
    }
    // this list's h is in memory, for every XCD to see, before it is counted
    if (tid < 128) __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    __syncthreads();
    if (tid == 0) __hip_atomic_fetch_add(done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    list = next_list;
    if (list < lists && !chained) {
      wait_vm<0>();  // start over with an empty ring
      slot = 0;
      prefilled = false;
    }
  }

  // ---- down ----
  bool waited = false;
  while (column_block < blocks) {
    const int c0 = column_block * R, cols = min(R, p.d - c0);
    if (!prefilled || waited) {
      start(DOWN, column_block);
      for (int s = 0; s < D; ++s) issue(s);
      slot = 0;
      prefilled = true;
    }
    if (!waited) {
      if (tid == 0) {
        const uint64_t t0 = wall_clock64();
        while (__hip_atomic_load(done, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < (uint32_t)lists) {
          __builtin_amdgcn_s_sleep(1);
          if (wall_clock64() - t0 > kWaitTicks) {
            s_ctl[3] = 1;
            break;
          }
        }
      }
      __syncthreads();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      waited = true;
    }
    const int units = A * slices;
    f32x4 total[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    // this lane's h of a unit: token lr's, or for a token that did not choose the expert one that did (not used)
    f32x4 raw[F::kUnit][2][F::kVec][2];
    auto load_h = [&](int a, int sl) __attribute__((always_inline)) {
      const int t = s_k[a][lr] != 255 ? lr : s_first[a];
      const float* hr = p.h + (int64_t)(t * KS + s_k[a][t]) * p.inter;
#pragma unroll
      for (int u = 0; u < F::kUnit; ++u) {
        int b = (sl * F::kUnit + u) * kNW + wave;
        b = b < nb2 ? b : min(wave, nb2 - 1);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int k0 = b * F::kBlock + (FMT == W_FP4 && b * F::kBlock + F::kBlock / 2 >= p.inter ? 0 : hf * (F::kBlock / 2));
#pragma unroll
          for (int v = 0; v < F::kVec; ++v)
#pragma unroll
            for (int q = 0; q < 2; ++q) raw[u][hf][v][q] = *(const f32x4*)(hr + k0 + lg * (F::kBlock / 8) + v * 8 + q * 4);
        }
      }
    };
    int a = 0, sl = 0;
    load_h(0, 0);
    wait_vm<0>();  // the compiler then counts the next unit's loads against the ring's instead of waiting for all
    for (int un = 0; un < units; ++un) {
      bf16x8_t hh[F::kUnit][2][F::kVec], hl[F::kUnit][2][F::kVec];
#pragma unroll
      for (int u = 0; u < F::kUnit; ++u)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int v = 0; v < F::kVec; ++v) split8(raw[u][hf][v][0], raw[u][hf][v][1], hh[u][hf][v], hl[u][hf][v]);
      // the conversion waits for h here, not among the loads below
#pragma unroll
      for (int u = 0; u < F::kUnit; ++u)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int v = 0; v < F::kVec; ++v) asm volatile("" : "+v"(hh[u][hf][v]), "+v"(hl[u][hf][v]));
      const int kk = s_k[a][lr], first = sl * F::kUnit * kNW + wave;
      const float gate = kk != 255 ? s_gate[lr * KS + kk] : 0.f;
      if (++sl == slices) {
        sl = 0;
        a = a + 1 < A ? a + 1 : 0;
      }
      load_h(a, sl);  // the next unit's (after the last one: the first one's again, not used)
      f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int u = 0; u < F::kUnit; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          wait_vm<F::kWaitDown>();
          const Step s = read_step(slot);
          issue(slot);
          next_slot();
          const int b = first + u * kNW;
          if (b < nb2) {
            f32x4 part = {0.f, 0.f, 0.f, 0.f};
            if constexpr (FMT != W_E4M3 && FMT != W_E4M3_E8M0) part = acc[r];
            const float s0 = __uint_as_float(s.sc[0] << 23), s1 = __uint_as_float(s.sc[1] << 23);
#pragma unroll
            for (int v = 0; v < F::kVec; ++v) {
              const bf16x8_t w = operand<FMT>(s.lo, v, s0);
              part = mfma_bf16(w, hh[u][0][v], part);
              part = mfma_bf16(w, hl[u][0][v], part);
            }
            if (FMT != W_FP4 || b * F::kBlock + F::kBlock / 2 < p.inter) {
#pragma unroll
              for (int v = 0; v < F::kVec; ++v) {
                const bf16x8_t w = operand<FMT>(s.hi, v, s1);
                part = mfma_bf16(w, hh[u][1][v], part);
                part = mfma_bf16(w, hl[u][1][v], part);
              }
            }
            if constexpr (FMT == W_E4M3 || FMT == W_E4M3_E8M0) {
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[r][q] = fmaf(part[q], row_scale(s, b, q), acc[r][q]);
            } else {
              acc[r] = part;
            }
          }
          if constexpr (FMT == W_I8) {
            if (u == F::kUnit - 1) {
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[r][q] *= __uint_as_float(s.sc[q]);
            }
          }
        }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) total[r][q] = kk != 255 ? fmaf(gate, acc[r][q], total[r][q]) : total[r][q];
    }
    lds_barrier();  // the sums' space is free
    s_red[0][wave][lane] = total[0];
    s_red[1][wave][lane] = total[1];
    if (tid == 0) s_ctl[1] = take(block_ticket);
    lds_barrier();
    {
      const int t = tid >> 5, c = tid & 31;
      float v = join8(red_at + (c >> 4) * (kNW * 1024) + (t + 16 * ((c & 15) >> 2)) * 16 + (c & 3) * 4);
      if (s_ctl[3]) v = __uint_as_float(0x7fc00000u);  // h was never complete
      if (t < T && c < cols) {
        uint8_t* o = p.out + t * p.ldo_b;
        if (p.out_dtype == ROW_F32) reinterpret_cast<float*>(o)[c0 + c] = v;
        else reinterpret_cast<uint16_t*>(o)[c0 + c] = (uint16_t)f32_to_bf16_rne(v);
      }
      column_block = __builtin_amdgcn_readfirstlane(s_ctl[1]);
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

bool aligned_to(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(n - 1)) == 0; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_decode_workspace_size(int T, int d, int inter, int n_experts, int n_shared, int top_k) {
  if (T < 0 || T > moe::kMaxT || d < 1 || d > moe::kMaxD || inter < 1 || n_experts < 1 || n_shared < 0 || n_shared > 1 ||
      top_k < 1 || top_k > moe::kMaxTopK)
    return 0;
  return moe::decode_ws(T, d, inter, n_shared, top_k).total;
}

extern "C" moe_status moe_decode(const moe_decode_desc* q, hipStream_t stream) {
  using namespace moe;
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
  r.logits = reinterpret_cast<double*>(ws + L.logits);
  r.xn = reinterpret_cast<uint16_t*>(ws + L.xn);
  decode_rows_kernel<<<q->n_experts, kRowThreads, 0, stream>>>(r);
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
  a.logits = r.logits;
  a.counters = r.counters;
  a.h = reinterpret_cast<float*>(ws + L.h);
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
  const int grid = compute_units(), threads = kNW * 64;
  switch (fmt) {
    case W_BF16: decode_experts_kernel<W_BF16><<<grid, threads, 0, stream>>>(a); break;
    case W_E4M3: decode_experts_kernel<W_E4M3><<<grid, threads, 0, stream>>>(a); break;
    case W_E4M3_E8M0: decode_experts_kernel<W_E4M3_E8M0><<<grid, threads, 0, stream>>>(a); break;
    case W_I8: decode_experts_kernel<W_I8><<<grid, threads, 0, stream>>>(a); break;
    default: decode_experts_kernel<W_FP4><<<grid, threads, 0, stream>>>(a); break;
  }
  return check_launch("moe_decode");
}
