// The router's selection for one token by one wave: sigmoid, bias, group limit, top-K, gates.
#pragma once

#include <math.h>

#include "device_common.h"

namespace moe {

constexpr uint32_t kNone = 0x7fffffffu;

// The wave's largest value, in every lane: DPP moves (no LDS) of its 32-bit words; lanes without a source keep their own.
template <int CTRL, typename V>
__device__ __forceinline__ V dpp_move(V v) {
  if constexpr (sizeof(V) == 4) {
    const int w = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(w, w, CTRL, 0xf, 0xf, false));
  } else {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(V, u32x2{(uint32_t)__builtin_amdgcn_update_dpp((int)w[0], (int)w[0], CTRL, 0xf, 0xf, false),
                                       (uint32_t)__builtin_amdgcn_update_dpp((int)w[1], (int)w[1], CTRL, 0xf, 0xf, false)});
  }
}
// v of one lane (uniform), in every lane.
template <typename V>
__device__ __forceinline__ V lane_value(V v, int lane) {
  if constexpr (sizeof(V) == 4) {
    return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  } else {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(V, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)w[0], lane),
                                       (uint32_t)__builtin_amdgcn_readlane((int)w[1], lane)});
  }
}
template <typename V>
__device__ __forceinline__ V wave_top(V v) {
  auto larger = [](V a, V b) { return b > a ? b : a; };
  v = larger(v, dpp_move<0x111>(v));  // row_shr 1, 2, 4, 8: lane 15 of each row of 16 has the row's
  v = larger(v, dpp_move<0x112>(v));
  v = larger(v, dpp_move<0x114>(v));
  v = larger(v, dpp_move<0x118>(v));
  v = larger(v, dpp_move<0x142>(v));  // lane 15 of a row to the next row, then lane 31 to the upper half
  v = larger(v, dpp_move<0x143>(v));
  return lane_value(v, 63);
}

__device__ __forceinline__ uint32_t wave_top_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xf, 0xf, true));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The best candidate of the wave, ties to the lower index (candidates' indices rise with the lane; kNone: no candidate here).
// NaN counts as -infinity.
template <typename V>
__device__ __forceinline__ void wave_argmax(V& bv, uint32_t& bi) {
  const V mine = bi == kNone || bv != bv ? (V)-INFINITY : bv;
  const V top = wave_top<V>(mine);
  const uint64_t at = __ballot(bi != kNone && mine == top);
  bv = top;
  bi = at == 0 ? kNone : (uint32_t)__builtin_amdgcn_readlane((int)bi, __builtin_ctzll(at));
}

template <typename V>
__device__ __forceinline__ V sigmoid_v(V u);
template <>
__device__ __forceinline__ float sigmoid_v<float>(float u) { return 1.0f / (1.0f + expf(-u)); }
template <>
__device__ __forceinline__ double sigmoid_v<double>(double u) { return 1.0 / (1.0 + exp(-u)); }

// Selection for one token by one wave.  u[r] is the logit (AFFINITY: the affinity) of expert 4*lane + r, bias[r] its bias.  Writes the
// outputs when `write`; returns the decision margin (min of the expert gap and half the
// group gap), +inf when nothing competes.
template <typename V, bool AFFINITY = false>
__device__ __forceinline__ V select_token(const V u[4], const float bias[4], int N, int K, int n_group, int topk_group, int64_t t,
                                          bool write, int32_t* __restrict__ topk_idx, float* __restrict__ topk_gate,
                                          float* __restrict__ scores) {
  const int lane = threadIdx.x & 63;
  const V inf = (V)INFINITY;
  V s4[4], z4[4];
  bool av[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int e = lane * 4 + r;
    if (e < N) {
      const V s = AFFINITY ? u[r] : sigmoid_v<V>(u[r]);
      V z = s + (V)bias[r];
      if (z != z) z = -inf;  // NaN ranks below every number
      s4[r] = s;
      z4[r] = z;
      av[r] = true;
    } else {
      s4[r] = (V)0;
      z4[r] = -inf;
      av[r] = false;
    }
  }
  if (write && scores != nullptr && lane * 4 < N)
    *(f32x4*)(scores + t * N + lane * 4) = f32x4{(float)s4[0], (float)s4[1], (float)s4[2], (float)s4[3]};

  V margin = inf;
  if (n_group > 1) {
    const int gs = N / n_group;  // a power of two >= 4: a lane's four experts share a group
    const int lanes_per_group = gs >> 2;
    const int g = (lane * 4) / gs;
    V m1 = -inf, m2 = -inf;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const V v = z4[r];
      if (v > m1) {
        m2 = m1;
        m1 = v;
      } else if (v > m2) {
        m2 = v;
      }
    }
    for (int o = 1; o < lanes_per_group; o <<= 1) {
      const V p1 = __shfl_xor(m1, o, kWave), p2 = __shfl_xor(m2, o, kWave);
      const V lo = m1 < p1 ? m1 : p1;
      const V hi2 = m2 > p2 ? m2 : p2;
      m1 = m1 > p1 ? m1 : p1;
      m2 = lo > hi2 ? lo : hi2;
    }
    const bool leader = (lane % lanes_per_group) == 0 && g < n_group;
    const V gscore = m1 + m2;
    bool gav = leader;
    uint64_t kept = 0;
    V last = (V)0;
    for (int rr = 0; rr <= topk_group; ++rr) {
      if (rr == n_group) break;
      V bv = gscore;
      uint32_t bi = gav ? (uint32_t)g : kNone;
      wave_argmax(bv, bi);
      if (bi == kNone) break;
      if (rr == topk_group) {
        margin = (last - bv) * (V)0.5;  // a group score moves twice as much as one z
        break;
      }
      kept |= 1ull << bi;
      last = bv;
      if (gav && (uint32_t)g == bi) gav = false;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (av[r] && !((kept >> g) & 1ull)) av[r] = false;
  }

  // Each lane sorts its four candidates (descending, equal ones by index; the ones out of play last), then the wave takes the
  // best of the lanes' heads K times.  Heads are compared by the bits of their float, in order as unsigned numbers: rounding
  // keeps their order, and where several lanes share the best one the exact values decide among them.
  int e4[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) e4[r] = lane * 4 + r;
  auto order = [&](int i, int j) __attribute__((always_inline)) {
    const bool swap = av[j] && (!av[i] || z4[j] > z4[i]);
    const V z = z4[i], s = s4[i];
    const int e = e4[i];
    const bool v = av[i];
    z4[i] = swap ? z4[j] : z;
    s4[i] = swap ? s4[j] : s;
    e4[i] = swap ? e4[j] : e;
    av[i] = swap ? av[j] : v;
    z4[j] = swap ? z : z4[j];
    s4[j] = swap ? s : s4[j];
    e4[j] = swap ? e : e4[j];
    av[j] = swap ? v : av[j];
  };
  order(0, 1);
  order(2, 3);
  order(1, 2);
  order(0, 1);
  order(2, 3);
  order(1, 2);
  uint32_t key[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t w = __float_as_uint((float)z4[r]);
    key[r] = av[r] ? w ^ ((uint32_t)((int32_t)w >> 31) | 0x80000000u) : 0u;  // -infinity is above 0
  }

  V sum = (V)0, zk = (V)0;
  int my_idx[4] = {0, 0, 0, 0};
  V my_s[4] = {(V)0, (V)0, (V)0, (V)0};
  for (int k = 0; k <= K; ++k) {
    const uint32_t top = wave_top_u32(key[0]);
    if (top == 0) break;
    const uint64_t heads = __ballot(key[0] == top);
    int owner = __builtin_ctzll(heads);
    if (sizeof(V) > 4 && (heads & (heads - 1)) != 0) {
      V bv = z4[0];
      uint32_t bi = key[0] == top ? (uint32_t)lane : kNone;
      wave_argmax(bv, bi);
      owner = (int)bi;
    }
    const V z = lane_value(z4[0], owner);
    if (k == K) {  // the best expert left out: the decision margin
      const V gap = zk - z;
      margin = gap < margin ? gap : margin;
      break;
    }
    zk = z;
    const V sk = lane_value(s4[0], owner);
    const int ek = __builtin_amdgcn_readlane(e4[0], owner);
    if (lane == owner) {
#pragma unroll
      for (int r = 0; r < 3; ++r) {
        z4[r] = z4[r + 1];
        s4[r] = s4[r + 1];
        e4[r] = e4[r + 1];
        key[r] = key[r + 1];
      }
      key[3] = 0u;
    }
    sum += sk;
    if (lane == (k & 63)) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((k >> 6) == q) {
          my_idx[q] = ek;
          my_s[q] = sk;
        }
    }
  }
  if (write) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = q * 64 + lane;
      if (k < K) {
        topk_idx[t * K + k] = my_idx[q];
        topk_gate[t * K + k] = (float)(my_s[q] / sum);
      }
    }
  }
  return margin;
}

}  // namespace moe
