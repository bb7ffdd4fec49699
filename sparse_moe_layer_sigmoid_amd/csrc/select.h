// The router's selection for one token by one wave: sigmoid, bias, group limit, top-K, gates.
#pragma once

#include <math.h>

#include "device_common.h"

namespace moe {

constexpr uint32_t kNone = 0x7fffffffu;

template <typename V>
__device__ __forceinline__ bool beats(V v, uint32_t i, V bv, uint32_t bi) {
  if (i == kNone) return false;
  if (bi == kNone) return true;
  return v > bv || (v == bv && i < bi);
}

template <typename V>
__device__ __forceinline__ void wave_argmax(V& bv, uint32_t& bi) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const V ov = __shfl_xor(bv, o, kWave);
    const uint32_t oi = (uint32_t)__shfl_xor((int)bi, o, kWave);
    if (beats(ov, oi, bv, bi)) {
      bv = ov;
      bi = oi;
    }
  }
}

template <typename V>
__device__ __forceinline__ V sigmoid_v(V u);
template <>
__device__ __forceinline__ float sigmoid_v<float>(float u) { return 1.0f / (1.0f + expf(-u)); }
template <>
__device__ __forceinline__ double sigmoid_v<double>(double u) { return 1.0 / (1.0 + exp(-u)); }

// Selection for one token by one wave.  u[r] is the logit of expert 4*lane + r.  Writes the
// outputs when `write`; returns the decision margin (min of the expert gap and half the
// group gap), +inf when nothing competes.
template <typename V>
__device__ __forceinline__ V select_token(const V u[4], const float* __restrict__ bias, int N, int K, int n_group,
                          int topk_group, int64_t t, bool write, int32_t* __restrict__ topk_idx,
                          float* __restrict__ topk_gate, float* __restrict__ scores) {
  const int lane = threadIdx.x & 63;
  const V inf = (V)INFINITY;
  V s4[4], z4[4];
  bool av[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int e = lane * 4 + r;
    if (e < N) {
      const V s = sigmoid_v<V>(u[r]);
      V z = s + (V)bias[e];
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

  V sum = (V)0, zk = (V)0;
  int my_idx[4] = {0, 0, 0, 0};
  V my_s[4] = {(V)0, (V)0, (V)0, (V)0};
  for (int k = 0; k <= K; ++k) {
    V bv = (V)0;
    uint32_t bi = kNone;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (av[r] && beats(z4[r], (uint32_t)(lane * 4 + r), bv, bi)) {
        bv = z4[r];
        bi = (uint32_t)(lane * 4 + r);
      }
    wave_argmax(bv, bi);
    if (bi == kNone) break;
    if (k == K) {  // the best expert left out: the decision margin
      const V gap = zk - bv;
      margin = gap < margin ? gap : margin;
      break;
    }
    zk = bv;
    const int owner = (int)(bi >> 2), slot = (int)(bi & 3u);
    V mine = s4[0];
#pragma unroll
    for (int r = 1; r < 4; ++r)
      if (slot == r) mine = s4[r];
    const V sk = __shfl(mine, owner, kWave);
    if (lane == owner) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (slot == r) av[r] = false;
    }
    sum += sk;
    if (lane == (k & 63)) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((k >> 6) == q) {
          my_idx[q] = (int)bi;
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
