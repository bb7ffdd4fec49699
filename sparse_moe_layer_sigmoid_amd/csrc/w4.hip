// w4_quant / moe_w4_gemm: the experts' products with 4-bit weights, for batches of few tokens.
//
// A weight is an E2M1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; two codes a byte, the
// even column in the low nibble) times a power of two shared by 32 consecutive inputs of its row
// (an E8M0 code): 4.25 bits.  With few rows per expert the products are bound by the bytes of the
// active experts' weights, so a 4-bit weight is worth 3.8 bf16 ones and nothing else matters much.
//
// Both kernels put the weights on the matrix cores as the first operand (16 weight rows x 32 inputs
// against 16 token rows): 16 bytes of a weight row are 32 inputs, exactly one scale group, and four
// K steps of the MFMA for the lane that holds them, so nothing is shuffled along K.  gfx950 converts
// two codes and applies the group's power of two in one instruction, exact in bf16, so scales cost
// no product of their own and every product accumulates in fp32.  K is split over the waves of a
// workgroup, whose sums are added through LDS in wave order (deterministic).  Work items (expert,
// row block, weight tile) come from the device-side offsets, as in moe_grouped_gemm: only experts
// that hold rows are read.
//
//  * w4_stream_kernel (K up to 8192, N a multiple of 16): the weights stream at 5.0-6.2 TB/s.  Widths
//    7168 -> 4096 (SwiGLU), 257 experts of 2048: one token 32-33 us (140 MB; about 9 us of that is the
//    start of the launch and its first loads), 64 tokens 566 us (3.5 GB, 6.2 TB/s), 256 tokens 700-724
//    us (3.6 GB, 5.0-5.2 TB/s); the down projection of 16 tokens 137-146 us (806 MB, 5.5-5.9 TB/s).  An expert with more than 16
//    rows is read by several workgroups, at the same time and on one XCD (802 us when they followed
//    each other); 256 tokens with skewed routing have 310 row blocks of 229 experts.  Sharing the
//    XCDs' work out by what a set costs instead of by units gained 2% there and lost 3% elsewhere.
//  * w4_gemm_kernel takes the other shapes, operands loaded straight into registers, up to 32
//    token rows an item: 2.2-2.5 TB/s on the sizes above.
#include <type_traits>

#include "abi_common.h"
#include "device_common.h"
#include "rows_common.h"

namespace moe {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int kMaxGroups = 1024;
constexpr int kGroup = 32;      // inputs per scale
constexpr int kRowBlock = 32;   // token rows of a work item
constexpr int kWaves = 4;

// E2M1 code of |v| rounded to nearest, ties to the even code, saturating at 6.
__device__ __forceinline__ uint32_t e2m1_code(float v) {
  const float a = fabsf(v);
  uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
  return c | ((__float_as_uint(v) >> 28) & 8u);
}

// One lane per 8 inputs, 4 lanes per scale group.
__global__ __launch_bounds__(256) void w4_quant_kernel(const uint16_t* __restrict__ w, int64_t n8,
                                                       uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;  // n8 is a multiple of 4: whole groups leave together
  float f[8];
  unpack_bf16x8(*(const u32x4*)(w + i * 8), f);
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1, kWave));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2, kWave));
  // the least 2^k with amax <= 6 * 2^k = 1.5 * 2^(k + 2); 0 for a group of zeros
  const int e = (int)(top >> 23) - 127;
  int k = e - 2 + ((top & 0x7fffffu) > 0x400000u ? 1 : 0);
  k = top == 0 ? 0 : top < 0x00800000u ? -127 : max(-127, k);
  const bool bad = top >= 0x7f800000u;  // an infinity or NaN: E2M1 holds neither, the scale says NaN
  const float inv = pow2f(-(bad ? 0 : k));
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) o |= e2m1_code(bad ? 0.f : f[j] * inv) << (4 * j);
  *(uint32_t*)(q + i * 4) = o;
  if ((i & 3) == 0) scale[i / 4] = bad ? 255 : (uint8_t)(k + 127);
}

struct W4Args {
  const uint8_t* a;  // bf16 token rows
  const int32_t* a_rows;
  int64_t lda_b;
  const uint8_t* q;
  const uint8_t* s;
  const int32_t* offs;  // group_offsets + first_group
  int first_group;
  int n_groups;
  // row counts, below 2^31 (an offset and a count add up in 32 bits): see row_limit
  uint32_t m_total;
  uint32_t sorted_rows;
  uint32_t out_rows;
  uint32_t tail_rows;
  int N;  // weight rows per group
  int K;
  int n_tiles;
  int out_cols;
  uint8_t* out;
  int out_dtype;
  int64_t ldo_b;
  int tail_first;  // first group (relative) of the f32 tail output; n_groups if none
  uint8_t* out_tail;
  int64_t ldo_tail_b;
};

__device__ __forceinline__ float silu(float a) { return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }

// 8 codes -> 8 bf16 weights (code * scale, exact unless it overflows).
__device__ __forceinline__ bf16x8_t decode_w4(uint32_t q, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The sorted row from which nothing is read or written: the first one that the caller did not vouch for.  Where the
// groups before the tail hold more rows than out does, that is the first row past out, and the tail is empty.
__device__ __forceinline__ int row_limit(const W4Args& p) {
  const uint32_t first = p.offs[0], tail = p.offs[p.tail_first];
  const uint32_t room = tail - first > p.out_rows ? first + p.out_rows : tail + p.tail_rows;
  return (int)min(min(first + p.m_total, p.sorted_rows), room);  // sorted_rows < 2^31
}
// Group offset i, held to that.
__device__ __forceinline__ int group_offset(const W4Args& p, int limit, int i) { return min(p.offs[i], limit); }

// Row blocks before each group (s_pre[g], of kMaxGroups + 1 entries) for row blocks of RB rows, built by a workgroup of THREADS lanes.
template <int RB, int THREADS>
__device__ __forceinline__ void row_block_prefix(const W4Args& p, int limit, int* s_pre, int* s_wsum) {
  constexpr int PER = kMaxGroups / THREADS;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int c[PER], sum = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int g = tid * PER + j;
    const int len = g < p.n_groups ? group_offset(p, limit, g + 1) - group_offset(p, limit, g) : 0;
    c[j] = (max(len, 0) + RB - 1) / RB;
    sum += c[j];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o, kWave);
    if (lane >= o) incl += v;
  }
  if (lane == 63) s_wsum[wave] = incl;
  __syncthreads();
  int base = incl - sum;
  for (int w = 0; w < wave; ++w) base += s_wsum[w];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    s_pre[tid * PER + j] = base;
    base += c[j];
  }
  if (tid == THREADS - 1) s_pre[kMaxGroups] = base;
  __syncthreads();
}

// The group whose row blocks, `per` work units each, hold unit L: the last one that starts at or before L.
__device__ __forceinline__ int find_group(const int* s_pre, int n_groups, int64_t per, int64_t L) {
  int lo = 0, hi = n_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)s_pre[mid] * per <= L) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Stores four consecutive output columns (those below out_cols) of sorted row `row` of group g.
__device__ __forceinline__ void store_columns(const W4Args& p, int limit, int g, int row, int base_row, int col, const f32x4& v) {
  const int left = p.out_cols - col;
  if (left <= 0) return;
  const bool tail = g >= p.tail_first;
  uint8_t* orow = tail ? p.out_tail + (int64_t)(row - group_offset(p, limit, p.tail_first)) * p.ldo_tail_b
                       : p.out + (int64_t)(row - base_row) * p.ldo_b;
  if (tail || p.out_dtype == ROW_F32) {
    float* o = reinterpret_cast<float*>(orow) + col;
    if (left >= 4) {
      *reinterpret_cast<f32x4_u*>(o) = v;
    } else {
      for (int e = 0; e < left; ++e) o[e] = v[e];
    }
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(orow) + col;
    const u32x2 b = {f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16),
                     f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16)};
    if (left >= 4) {
      *reinterpret_cast<u32x2_u*>(o) = b;
    } else {
      for (int e = 0; e < left; ++e) o[e] = (uint16_t)(b[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Workgroup barrier that waits for this wave's LDS operations but not for its loads in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The streaming kernel: K at most 128 * NW * KPW, N a multiple of 16.  A
// workgroup walks weight tiles (16 rows; SwiGLU: 8 gate rows and their 8 up rows) against a block of
// up to 16 token rows, whose values it holds in registers as matrix operands for as long as its
// tiles stay in that block, so that its loads are the weights alone.  A tile's bytes come by loads
// of whole 64-byte row pieces (the operand order, 16 rows to a load at 16 bytes each, measured 25%
// slower) and pass through LDS into operand order.  The code is kept short: a launch starts with
// a cold instruction cache, which for one token costs about a microsecond per kilobyte executed.
template <bool SWIGLU, int NW, int KPW>
__global__ __launch_bounds__(NW * 64, 2) void w4_stream_kernel(W4Args p) {
  constexpr int D = KPW > 4 ? 2 : 4;         // ring: weight tiles in flight per wave
  constexpr int SR = (KPW + 3) / 4;          // scale loads (4 dwords of each row) per tile
  constexpr int STRIDE = KPW * 64 + 16;      // bytes of a tile row in LDS, spread over the banks
  constexpr int SSTRIDE = SR * 4 + 1;        // dwords of a tile row's scales in LDS
  constexpr int THREADS = NW * 64;
  __shared__ int s_off[kMaxGroups + 1];      // the groups' offsets
  __shared__ int s_pre[kMaxGroups + 1];      // row blocks before each group
  __shared__ int s_wsum[NW];
  __shared__ int s_first;
  __shared__ __attribute__((aligned(16))) uint8_t s_w[NW][16 * STRIDE];
  __shared__ uint32_t s_s[NW][16 * SSTRIDE];
  __shared__ __attribute__((aligned(16))) f32x4 s_red[NW > 1 ? 2 * D : 1][NW][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int G = p.n_groups, n_tiles = p.n_tiles, limit = row_limit(p);

  // prefix of the groups' row blocks, `per` consecutive groups to a lane; the lane whose groups hold
  // the workgroup's first unit says which one
  int64_t u0;
  int step, count;  // units of this workgroup: u0, u0 + step, ...
  {
    const int per = (G + THREADS - 1) / THREADS, g0 = min(tid * per, G), g1 = min(g0 + per, G);
    int sum = 0, o = group_offset(p, limit, g0);
    for (int g = g0; g < g1; ++g) {
      const int next = group_offset(p, limit, g + 1);
      s_off[g] = o;
      sum += (max(next - o, 0) + 15) >> 4;
      o = next;
    }
    if (g1 == G) s_off[G] = o;  // the same value from every lane that ends there
    int incl = sum;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const int v = __shfl_up(incl, k, kWave);
      if (lane >= k) incl += v;
    }
    if (lane == 63) s_wsum[wave] = incl;
    __syncthreads();
    int base = incl - sum, all = 0;
    for (int w = 0; w < NW; ++w) {
      if (w < wave) base += s_wsum[w];
      all += s_wsum[w];
    }
    // Workgroup b runs on XCD b mod 8; `slice` numbers them XCD by XCD.  Few row blocks (one or two
    // tokens): each gets `share` workgroups of its own, every one a contiguous run of its tiles, so
    // none meets a second block and an XCD touches most of its 2 MiB pages of weights at once.
    // Else (less than 8 workgroups to a block, where whole shares would leave up to 1 / share of
    // them idle) the units are cut into equal slices, each for `step` neighbouring workgroups of one
    // XCD that take its tiles in turn.  `step` is as many as leave each 8 tiles of a block, or 16 where
    // there are more blocks than groups, so that blocks of one expert read the same weights: fetching a
    // block's token rows costs about as much as two tiles.  Gate/up of one token: 42 us dealt in turn, 33
    // us in shares; down of 16 tokens (114 blocks): 142 us in turn, 151 us in contiguous runs.  2048 -> 768
    // of 129 experts, 256 tokens: gate/up 106 us when all of an XCD's workgroups shared a block, 61 us
    // with 8 tiles each, 59 us with 16; down 73, 41 and 39 us; 16 tiles for 16 tokens above: 144 us.
    const int xcd = blockIdx.x & 7, seat = blockIdx.x >> 3, seats = gridDim.x >> 3;
    if (all * 8 <= (int)gridDim.x) {
      const uint32_t share = gridDim.x / max(all, 1), slice = xcd * seats + seat;
      const uint32_t rb = slice / share, part = slice - rb * share;
      const uint32_t t0 = (uint32_t)((uint64_t)n_tiles * part / share);
      u0 = (int64_t)rb * n_tiles + t0;
      step = 1;
      count = (int)rb < all ? (int)((uint32_t)((uint64_t)n_tiles * (part + 1) / share) - t0) : 0;
    } else {
      const int64_t units = (int64_t)all * n_tiles;
      step = min(seats, 1 << (31 - __clz(max(n_tiles / (all > G ? 16 : 8), 1))));  // powers of two
      const int lg_step = __builtin_ctz(step), lg_slices = __builtin_ctz(gridDim.x) - lg_step;
      const int slice = (xcd * seats + seat) >> lg_step;
      u0 = (units * slice >> lg_slices) + (seat & (step - 1));
      const int64_t left = (units * (slice + 1) >> lg_slices) - u0;
      count = left > 0 ? (int)((left + step - 1) >> __builtin_ctz(step)) : 0;
    }
    if (count == 0) return;  // the whole workgroup
    for (int g = g0; g < g1; ++g) {
      s_pre[g] = base;
      const int upto = base + ((max(s_off[g + 1] - s_off[g], 0) + 15) >> 4);
      if ((int64_t)base * n_tiles <= u0 && u0 < (int64_t)upto * n_tiles) s_first = g;
      base = upto;
    }
    if (g1 == G) s_pre[G] = all;
    __syncthreads();
  }
  const int base_row = s_off[0];
  const uint32_t w_row_b = p.K / 2, s_row_b = p.K / kGroup;
  const int kblocks = (p.K + 127) / 128, kper = (kblocks + NW - 1) / NW;
  const int kb0 = wave * kper;                             // this wave's K blocks
  const int nkb = min(max(kblocks - kb0, 0), kper);

  // A position in the unit order; everything uniform.  A group's row blocks go in sets of a power
  // of two (14 blocks: 8 + 4 + 2), and a set's units run over the blocks first, then the tiles: a
  // slice's workgroups (a multiple of the set) each keep to one block while they read a tile's
  // weights together, so that they come over the fabric once per set instead of once per block.
  struct Cursor {
    int g, base, size, idx;  // row blocks [base, base + size) of group g, unit idx of that set
    __device__ __forceinline__ int rb() const { return base + (idx & (size - 1)); }
    __device__ __forceinline__ int tile() const { return idx >> __builtin_ctz(size); }
  };
  const int max_set = min(step, 32);
  auto set_size = [&](int blocks) __attribute__((always_inline)) { return min(max_set, 1 << (31 - __clz(blocks))); };
  auto settle = [&](Cursor& c) __attribute__((always_inline)) {  // idx past the set: on to the set it is in
    int span = c.size * n_tiles;
    while (c.idx >= span) {
      c.idx -= span;
      c.base += c.size;
      int blocks = s_pre[c.g + 1] - s_pre[c.g];
      if (c.base >= blocks) {
        c.base = 0;
        do {
          ++c.g;
          blocks = s_pre[c.g + 1] - s_pre[c.g];
        } while (blocks == 0);
      }
      c.size = __builtin_amdgcn_readfirstlane(set_size(blocks - c.base));
      span = c.size * n_tiles;
    }
    c.g = __builtin_amdgcn_readfirstlane(c.g);
    c.base = __builtin_amdgcn_readfirstlane(c.base);
    c.idx = __builtin_amdgcn_readfirstlane(c.idx);
  };
  auto advance = [&](Cursor& c) __attribute__((always_inline)) {  // by `step` units, to one that exists
    c.idx += step;
    settle(c);
  };
  Cursor cur;
  {
    cur.g = __builtin_amdgcn_readfirstlane(s_first);
    const int local = (int)(u0 - (int64_t)s_pre[cur.g] * n_tiles), blocks = s_pre[cur.g + 1] - s_pre[cur.g];
    const int span = max_set * n_tiles;  // past the whole sets at once
    const int whole = min((int)((uint32_t)local / (uint32_t)span), blocks >> __builtin_ctz(max_set));
    cur.base = __builtin_amdgcn_readfirstlane(whole * max_set);
    cur.size = __builtin_amdgcn_readfirstlane(set_size(blocks - cur.base));
    cur.idx = local - whole * span;
    settle(cur);
  }

  // loads of a tile: load j reads K block j, four neighbouring lanes the 64 bytes of one row
  const int r4 = lane >> 2, c4 = lane & 3;
  const uint32_t row_in_tile = SWIGLU && r4 >= 8 ? p.N / 2 + r4 - 8 : r4;
  const uint32_t off_q = row_in_tile * w_row_b + kb0 * 64 + c4 * 16;
  const uint32_t off_s = row_in_tile * s_row_b + (kb0 + c4) * 4;
  // Buffer loads from one group's weights: past its end they read zero and touch no memory, so the
  // loop runs without branches around its loads (at a join the compiler waits for the path with
  // the fewest loads in flight): a tile that does not exist is fetched from a buffer of no bytes, and
  // inputs past a wave's last one or the row's end are what follows there, codes that meet zeros
  // of x under a scale of 1.
  const uint32_t q_bytes = p.N * w_row_b, s_bytes = p.N * s_row_b;
  uint32_t sc_keep[SR];  // the bytes of this lane's scale dwords that are its own
#pragma unroll
  for (int j = 0; j < SR; ++j) {
    const int groups = min(max(p.K / kGroup - (kb0 + c4 + j * 4) * 4, 0), 4);
    sc_keep[j] = c4 + j * 4 < nkb ? (groups == 4 ? 0xffffffffu : (1u << (8 * groups)) - 1u) : 0u;
  }
  u32x4 rq[D][KPW];
  uint32_t rs[D][SR];
  auto fetch = [&](int slot, const Cursor& c, bool exists) __attribute__((always_inline)) {
    const int64_t first = (int64_t)(p.first_group + c.g) * p.N;
    const uint32_t row = c.tile() * (SWIGLU ? 8 : 16);
    const uint32_t row_b = row * w_row_b;
    const auto bq = __builtin_amdgcn_make_buffer_rsrc((void*)(p.q + (first * w_row_b + row_b)), 0,
                                                      exists ? q_bytes - row_b : 0u, 0x00020000);
    const auto bs = __builtin_amdgcn_make_buffer_rsrc((void*)(p.s + first * s_row_b), 0, exists ? s_bytes : 0u, 0x00020000);
    uint32_t o = off_q;
    asm volatile("" : "+v"(o));  // else the KPW sums below are kept in registers instead of the instructions
#pragma unroll
    for (int j = 0; j < KPW; ++j) rq[slot][j] = __builtin_amdgcn_raw_buffer_load_b128(bq, o + j * 64, 0, 0);
#pragma unroll
    for (int j = 0; j < SR; ++j)  // a dword that would straddle the group's end is its last one instead
      rs[slot][j] = __builtin_amdgcn_raw_buffer_load_b32(bs, min(off_s + row * s_row_b + j * 16, s_bytes - 4), 0, 0);
  };

  // the token rows of a block; lanes past its last row hold its first one again and store nothing
  u32x4 x[KPW][4];
  auto load_x = [&](const Cursor& c) __attribute__((always_inline)) {
    const int row0 = s_off[c.g] + c.rb() * 16;
    const int r = row0 + (lr < s_off[c.g + 1] - row0 ? lr : 0);
    const uint8_t* xr = p.a + (int64_t)(p.a_rows ? p.a_rows[r] : r) * p.lda_b;
    if (nkb == KPW && (kb0 + KPW) * 128 <= p.K) {
      const uint8_t* xk = xr + kb0 * 256 + lg * 64;
#pragma unroll
      for (int k = 0; k < KPW; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[k][j] = *(const u32x4*)(xk + k * 256 + j * 16);
    } else {  // past this wave's K blocks or the row: zeros
#pragma unroll
      for (int k = 0; k < KPW; ++k) {
        const int at = (kb0 + k) * 128 + lg * 32;
        const bool in = k < nkb && at < p.K;
        const uint8_t* xk = xr + (in ? at : 0) * 2;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[k][j] = u32x4{0u, 0u, 0u, 0u};
          if (in) x[k][j] = *(const u32x4*)(xk + j * 16);
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): nothing of x is pending where the paths join
  };

  uint8_t* lw = s_w[wave];
  uint32_t* ls = s_s[wave];
  // one tile: the ring's registers to LDS (the slot then takes the tile D ahead), back in operand
  // order, decode and multiply.  LDS operations of one wave execute in order, so its lanes need no
  // barrier to see each other's bytes.
  auto tile = [&](int slot, const Cursor& next, bool exists) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < KPW; ++j) *(u32x4*)(lw + r4 * STRIDE + c4 * 16 + j * 64) = rq[slot][j];
    if (s_row_b & 3) {  // rows of scales at odd bytes: move the bytes of such a dword into place
#pragma unroll
      for (int j = 0; j < SR; ++j) {
        const uint32_t at = off_s + cur.tile() * (SWIGLU ? 8 : 16) * s_row_b + j * 16;
        rs[slot][j] >>= (at - min(at, s_bytes - 4)) * 8 & 31;
      }
    }
#pragma unroll
    for (int j = 0; j < SR; ++j)  // past this wave's K blocks or the row: 1
      ls[r4 * SSTRIDE + c4 + j * 4] = (rs[slot][j] & sc_keep[j]) | (0x7f7f7f7fu & ~sc_keep[j]);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    fetch(slot, next, exists);
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int k = 0; k < KPW; ++k) {
      const u32x4 q = *(const u32x4*)(lw + lr * STRIDE + k * 64 + lg * 16);
      const uint32_t sc = reinterpret_cast<const uint8_t*>(ls)[(lr * SSTRIDE + k) * 4 + lg];
      const float s = __uint_as_float(sc << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j & 1] = mfma_bf16(decode_w4(q[j], s), __builtin_bit_cast(bf16x8_t, x[k][j]), acc[j & 1]);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = acc[0][e] + acc[1][e];
    return v;
  };

  // a summed tile: SwiGLU's gate columns sit in lanes 0..31, the up columns of the same token row in
  // lanes 32..63; a lane stores four consecutive columns
  auto store = [&](f32x4 v, const Cursor& c) __attribute__((always_inline)) {
    const int row = s_off[c.g] + c.rb() * 16 + lr;
    int col = c.tile() * 16 + lg * 4;
    bool live = row < s_off[c.g + 1];
    if constexpr (SWIGLU) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = silu(v[e]) * __shfl_xor(v[e], 32, kWave);
      live = live && lg < 2;
      col = c.tile() * 8 + lg * 4;
    }
    if (!live) return;
    const bool tail = c.g >= p.tail_first;
    uint8_t* orow = tail ? p.out_tail + (int64_t)(row - s_off[p.tail_first]) * p.ldo_tail_b
                         : p.out + (int64_t)(row - base_row) * p.ldo_b;
    if (tail || p.out_dtype == ROW_F32) {
      *reinterpret_cast<f32x4_u*>(orow + col * 4) = v;
    } else {
      *reinterpret_cast<u32x2_u*>(orow + col * 2) = u32x2{f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16),
                                                           f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16)};
    }
  };

  Cursor pre = cur, done = cur;  // the next tile to fetch, the first one whose sums are not joined
  int ahead = 0;                 // tiles fetched
  int xg = -1, xrb = 0, buf = 0;
#pragma unroll
  for (int d = 0; d < D; ++d) {
    fetch(d, pre, ahead < count);
    if (++ahead < count) advance(pre);
  }
  // the waves' sums of tiles u .. u + n, in wave order.  D tiles' sums change hands at a time.  Two
  // sets of buffers alternate: a wave writes a set again only after the barrier of the other, which
  // the waves that read it have then passed.
  auto join = [&](int u, int n) __attribute__((always_inline)) {
    lds_barrier();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      if (wave == ((u + i) & (NW - 1))) {
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int w = 0; w < NW; ++w) {
          const f32x4 o = s_red[buf + i][w][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] += o[e];
        }
        store(sum, done);
      }
      if (u + i + 1 < count) advance(done);
    }
    buf ^= D;
  };
  // EARLY: leave after the last tile.  Else the ring's turn is finished with tiles that do not exist
  // (zeros, not stored): with two tiles to a turn that costs at most one, and the exit between them
  // costs more (gate/up of 256 tokens, 7168 inputs: 699 us, 733 us with it).  With four it is up to 20 KB
  // of cold code that a short run does not execute (8 us calls of one to four tiles: 6 us).
  constexpr bool EARLY = D > 2;
  int u = 0, n = 0;
  for (; EARLY || u < count; u += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (cur.g != xg || cur.rb() != xrb) {
        load_x(cur);
        xg = cur.g;
        xrb = cur.rb();
      }
      const f32x4 v = tile(d, pre, ahead < count);
      if (++ahead < count) advance(pre);
      if constexpr (NW > 1) s_red[buf + d][wave][lane] = v;
      else if (EARLY || u + d < count) store(v, cur);
      if (EARLY && u + d + 1 >= count) {
        n = d + 1;
        break;
      }
      if (EARLY || u + d + 1 < count) advance(cur);
    }
    if (EARLY && n > 0) break;
    if constexpr (NW > 1) join(u, EARLY ? D : min(D, count - u));
  }
  if constexpr (EARLY && NW > 1) join(u, n);
}

template <bool SWIGLU, int NT>
__global__ __launch_bounds__(256, 4) void w4_gemm_kernel(W4Args p) {
  constexpr int BN = NT * 16;                   // weight rows per item
  constexpr int OC = SWIGLU ? BN / 2 : BN;      // output columns per item
  __shared__ int s_pre[kMaxGroups + 1];         // row blocks before each group
  __shared__ int s_wsum[kWaves];
  __shared__ __attribute__((aligned(16))) float s_red[kWaves][16][BN + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lg = lane >> 4;

  const int limit = row_limit(p);
  row_block_prefix<kRowBlock, 256>(p, limit, s_pre, s_wsum);
  const int64_t total = (int64_t)s_pre[kMaxGroups] * p.n_tiles;
  const int base_row = p.offs[0];
  const int kblocks = (p.K + 127) / 128;
  const uint32_t w_row_b = p.K / 2, s_row_b = p.K / kGroup;

  for (int64_t L = blockIdx.x; L < total; L += gridDim.x) {
    const int g = find_group(s_pre, p.n_groups, p.n_tiles, L);
    const int blocks = s_pre[g + 1] - s_pre[g];
    const int local = (int)(L - (int64_t)s_pre[g] * p.n_tiles);
    const int nt = local / blocks, rb = local - nt * blocks;
    const int row0 = group_offset(p, limit, g) + rb * kRowBlock;
    const int rows = min(kRowBlock, group_offset(p, limit, g + 1) - row0);

    // weight rows of this lane (past N: the last one again, not stored)
    const int half = p.N / 2;
    const uint8_t* wq = p.q + (int64_t)(p.first_group + g) * p.N * w_row_b;  // uniform; offsets fit 32 bits
    const uint8_t* ws = p.s + (int64_t)(p.first_group + g) * p.N * s_row_b;
    uint32_t oq[NT], os[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      int r;
      if constexpr (SWIGLU) {
        const int c = min(nt * OC + (n % (NT / 2)) * 16 + lr, half - 1);
        r = n < NT / 2 ? c : half + c;
      } else {
        r = min(nt * OC + n * 16 + lr, p.N - 1);
      }
      oq[n] = (uint32_t)r * w_row_b + lg * 16;
      os[n] = (uint32_t)r * s_row_b + lg;
    }

    auto run = [&](auto mt_c) __attribute__((always_inline)) {
      constexpr int MT = decltype(mt_c)::value;
      constexpr int kRing = MT == 1 ? 4 : 3;  // weight loads in flight per wave and weight tile
      const uint8_t* xr[MT];
      bool live[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        live[m] = m * 16 + lr < rows;
        const int r = row0 + (live[m] ? m * 16 + lr : 0);
        const int64_t ar = p.a_rows ? p.a_rows[r] : r;
        xr[m] = p.a + ar * p.lda_b + lg * 64;
      }
      f32x4 acc[NT][MT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = f32x4{0.f, 0.f, 0.f, 0.f};
      u32x4 q[kRing][NT];
      uint32_t sc[kRing][NT];
      auto fetch = [&](int slot, int kb) __attribute__((always_inline)) {
        const bool ok = kb * 128 + lg * 32 < p.K;  // K is a multiple of 32: a lane's inputs are all in or all out
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          q[slot][n] = u32x4{0u, 0u, 0u, 0u};
          sc[slot][n] = 127;
          if (ok) {
            q[slot][n] = *(const u32x4*)(wq + (oq[n] + (uint32_t)kb * 64u));
            sc[slot][n] = ws[os[n] + (uint32_t)kb * 4u];
          }
        }
      };
#pragma unroll
      for (int d = 0; d < kRing; ++d) fetch(d, wave + d * kWaves);
      for (int kb0 = wave; kb0 < kblocks; kb0 += kRing * kWaves) {
#pragma unroll
        for (int d = 0; d < kRing; ++d) {
          const int kb = kb0 + d * kWaves;
          const bool ok = kb * 128 + lg * 32 < p.K;
          u32x4 x[MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[m][j] = u32x4{0u, 0u, 0u, 0u};
              if (ok && live[m]) x[m][j] = *(const u32x4*)(xr[m] + (int64_t)kb * 256 + j * 16);
            }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float s = __uint_as_float(sc[d][n] << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bf16x8_t w = decode_w4(q[d][n][j], s);
#pragma unroll
              for (int m = 0; m < MT; ++m) acc[n][m] = mfma_bf16(w, __builtin_bit_cast(bf16x8_t, x[m][j]), acc[n][m]);
            }
          }
          fetch(d, kb + kRing * kWaves);
        }
      }
      // add the waves' sums in wave order, 16 token rows at a time, and store
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int mrows = min(16, rows - m * 16);
        if (mrows <= 0) break;
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) *(f32x4*)&s_red[wave][lr][n * 16 + lg * 4] = acc[n][m];
        __syncthreads();
        for (int i = tid; i < mrows * (OC / 4); i += 256) {
          const int r = i / (OC / 4), c4 = (i - r * (OC / 4)) * 4;
          f32x4 v = *(const f32x4*)&s_red[0][r][c4];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) v += *(const f32x4*)&s_red[w][r][c4];
          if constexpr (SWIGLU) {
            f32x4 u = *(const f32x4*)&s_red[0][r][OC + c4];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) u += *(const f32x4*)&s_red[w][r][OC + c4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = silu(v[e]) * u[e];
          }
          store_columns(p, limit, g, row0 + m * 16 + r, base_row, nt * OC + c4, v);
        }
      }
    };
    if (rows <= 16) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 2>{});
  }
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// K blocks of 128 inputs that the streaming kernel can hold: 8 waves of 8.
constexpr int kMaxStreamBlocks = 64;

template <int NW, int KPW>
void launch_stream_as(const W4Args& a, bool swiglu, hipStream_t stream) {
  const int grid = 256 * (8 / NW);  // two waves per SIMD: every workgroup resident
  if (swiglu) w4_stream_kernel<true, NW, KPW><<<grid, NW * 64, 0, stream>>>(a);
  else w4_stream_kernel<false, NW, KPW><<<grid, NW * 64, 0, stream>>>(a);
}

// As few waves as hold K in 4 blocks each (fewer partial sums to add), then more blocks.
void launch_stream(const W4Args& a, bool swiglu, hipStream_t stream) {
  const int kb = (a.K + 127) / 128;
  if (kb <= 4) launch_stream_as<1, 4>(a, swiglu, stream);
  else if (kb <= 8) launch_stream_as<2, 4>(a, swiglu, stream);
  else if (kb <= 16) launch_stream_as<4, 4>(a, swiglu, stream);
  else if (kb <= 32) launch_stream_as<8, 4>(a, swiglu, stream);
  else if (kb <= 48) launch_stream_as<8, 6>(a, swiglu, stream);
  else if (kb <= 56) launch_stream_as<8, 7>(a, swiglu, stream);
  else launch_stream_as<8, 8>(a, swiglu, stream);
}

}  // namespace
}  // namespace moe

extern "C" moe_status w4_quant(const uint16_t* w, int n_mats, int n, int k, uint8_t* q, uint8_t* scale,
                               hipStream_t stream) {
  using namespace moe;
  clear_error();
  const bool empty = n_mats == 0;
  MOE_REQUIRE(empty || (w && q && scale), MOE_ERR_NULL, "w4_quant: a required pointer is NULL");
  MOE_REQUIRE(n_mats >= 0 && n >= 1 && k >= kGroup && k % kGroup == 0, MOE_ERR_SHAPE,
              "w4_quant: n_mats=%d n=%d k=%d (k a positive multiple of %d)", n_mats, n, k, kGroup);
  MOE_REQUIRE(aligned16(w) && aligned16(q), MOE_ERR_ALIGN, "w4_quant: w and q must be 16-byte aligned");
  const int64_t rows = (int64_t)n_mats * n;
  MOE_REQUIRE(rows <= kMaxLanes / (k / 8), MOE_ERR_SHAPE, "w4_quant: too many weights");
  const int64_t n8 = rows * (k / 8);
  if (n8 > 0) w4_quant_kernel<<<(unsigned)((n8 + 255) / 256), 256, 0, stream>>>(w, n8, q, scale);
  return check_launch("w4_quant");
}

extern "C" moe_status moe_w4_gemm(const moe_w4_desc* d, hipStream_t stream) {
  return moe_w4_gemm_bounded(d, INT64_MAX, INT64_MAX, INT64_MAX, stream);
}

extern "C" moe_status moe_w4_gemm_bounded(const moe_w4_desc* d, int64_t sorted_rows, int64_t out_rows, int64_t tail_rows,
                                          hipStream_t stream) {
  using namespace moe;
  clear_error();
  MOE_REQUIRE(d != nullptr, MOE_ERR_NULL, "moe_w4_gemm: desc is NULL");
  MOE_REQUIRE(d->w_q && d->w_scale && d->group_offsets && (d->m_total == 0 || sorted_rows == 0 ||
                  (d->a && (d->out || out_rows == 0 || d->tail_groups == d->n_groups))),
              MOE_ERR_NULL, "moe_w4_gemm: a, w_q, w_scale, group_offsets and out are required");
  MOE_REQUIRE(d->epilogue == MOE_EPI_NONE || d->epilogue == MOE_EPI_SWIGLU, MOE_ERR_DTYPE,
              "moe_w4_gemm: unknown epilogue %d", d->epilogue);
  MOE_REQUIRE(d->out_dtype == MOE_BF16 || d->out_dtype == MOE_F32, MOE_ERR_DTYPE,
              "moe_w4_gemm: out_dtype must be MOE_BF16 or MOE_F32 (%d)", d->out_dtype);
  const bool swiglu = d->epilogue == MOE_EPI_SWIGLU;
  MOE_REQUIRE(d->n_groups >= 1 && d->n_groups <= kMaxGroups && d->first_group >= 0, MOE_ERR_SHAPE,
              "moe_w4_gemm: n_groups=%d (1..%d) first_group=%d", d->n_groups, kMaxGroups, d->first_group);
  MOE_REQUIRE(d->m_total >= 0 && d->m_total < ((int64_t)1 << 31), MOE_ERR_SHAPE, "moe_w4_gemm: m_total=%lld",
              (long long)d->m_total);
  MOE_REQUIRE(sorted_rows >= 0 && out_rows >= 0 && tail_rows >= 0, MOE_ERR_SHAPE,
              "moe_w4_gemm: negative counts of rows (%lld sorted, %lld of out, %lld of out_tail)", (long long)sorted_rows,
              (long long)out_rows, (long long)tail_rows);
  MOE_REQUIRE(d->K >= kGroup && d->K % kGroup == 0 && d->N >= 1 && (!swiglu || d->N % 2 == 0), MOE_ERR_SHAPE,
              "moe_w4_gemm: K=%d must be a positive multiple of %d, N=%d positive%s", d->K, kGroup, d->N,
              swiglu ? " and even" : "");
  MOE_REQUIRE(d->tail_groups >= 0 && d->tail_groups <= d->n_groups, MOE_ERR_SHAPE,
              "moe_w4_gemm: tail_groups=%d must be in [0, n_groups=%d]", d->tail_groups, d->n_groups);
  const int out_cols = swiglu ? d->N / 2 : d->N;
  const int osz = d->out_dtype == MOE_F32 ? 4 : 2;
  MOE_REQUIRE(d->lda >= d->K && d->lda % 8 == 0 && aligned16(d->a), MOE_ERR_ALIGN,
              "moe_w4_gemm: lda=%lld must be >= K, a multiple of 8, and a 16-byte aligned", (long long)d->lda);
  MOE_REQUIRE(aligned16(d->w_q), MOE_ERR_ALIGN, "moe_w4_gemm: w_q must be 16-byte aligned");
  MOE_REQUIRE((d->ldo >= out_cols || d->tail_groups == d->n_groups) && (reinterpret_cast<uintptr_t>(d->out) & (uintptr_t)(osz - 1)) == 0, MOE_ERR_ALIGN,
              "moe_w4_gemm: ldo=%lld must be >= %d and out aligned to its elements", (long long)d->ldo, out_cols);
  if (d->tail_groups > 0) {
    MOE_REQUIRE(d->m_total == 0 || sorted_rows == 0 || tail_rows == 0 || d->out_tail, MOE_ERR_NULL, "moe_w4_gemm: out_tail is NULL");
    MOE_REQUIRE(d->ldo_tail >= out_cols && (reinterpret_cast<uintptr_t>(d->out_tail) & 3u) == 0, MOE_ERR_ALIGN,
                "moe_w4_gemm: ldo_tail=%lld must be >= %d and out_tail 4-byte aligned", (long long)d->ldo_tail, out_cols);
  }
  MOE_REQUIRE((int64_t)d->N * (d->K / 2) < ((int64_t)1 << 31), MOE_ERR_SHAPE, "moe_w4_gemm: one W[g] exceeds 2 GiB");
  if (d->m_total == 0 || sorted_rows == 0) return MOE_OK;
  W4Args a;
  a.a = static_cast<const uint8_t*>(d->a);
  a.a_rows = d->a_rows;
  a.lda_b = d->lda * 2;
  a.q = d->w_q;
  a.s = d->w_scale;
  a.offs = d->group_offsets + d->first_group;
  a.first_group = d->first_group;
  a.n_groups = d->n_groups;
  const auto count = [](int64_t n) { return (uint32_t)(n < INT32_MAX ? n : INT32_MAX); };  // no offset is larger
  a.m_total = count(d->m_total);
  a.sorted_rows = count(sorted_rows);
  a.out_rows = count(out_rows);
  a.tail_rows = d->tail_groups > 0 ? count(tail_rows) : INT32_MAX;
  a.N = d->N;
  a.K = d->K;
  a.out_cols = out_cols;
  a.out = static_cast<uint8_t*>(d->out);
  a.out_dtype = d->out_dtype == MOE_F32 ? ROW_F32 : ROW_BF16;
  a.ldo_b = d->ldo * osz;
  a.tail_first = d->n_groups - d->tail_groups;
  a.out_tail = static_cast<uint8_t*>(d->out_tail);
  a.ldo_tail_b = d->ldo_tail * 4;
  if (d->K <= 128 * kMaxStreamBlocks && d->N % 16 == 0 && aligned4(d->w_scale)) {
    a.n_tiles = d->N / 16;
    launch_stream(a, swiglu, stream);
    return check_launch("moe_w4_gemm");
  }
  constexpr int NT = 2;
  const int oc = swiglu ? NT * 8 : NT * 16;
  a.n_tiles = (out_cols + oc - 1) / oc;
  // row blocks: at most one short one per group that holds rows, and never more than rows
  const int64_t full = d->m_total / kRowBlock + d->n_groups;
  const int64_t items = (full < d->m_total ? full : d->m_total) * a.n_tiles;
  const int grid = (int)(items < 256 * 5 ? items : 256 * 5);
  if (swiglu) w4_gemm_kernel<true, NT><<<grid, 256, 0, stream>>>(a);
  else w4_gemm_kernel<false, NT><<<grid, 256, 0, stream>>>(a);
  return check_launch("moe_w4_gemm");
}
