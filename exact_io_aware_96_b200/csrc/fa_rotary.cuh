// fa_rotary.cuh — rotary positions with several axes on q and k (fa_rotary).
//
// The first 2R columns of a head hold R pairs (x_a, x_b): columns (j, j + R),
// or (2j, 2j + 1) when interleaved. Pair j belongs to one position axis
// (sections: the first n_0 pairs to axis 0, the next n_1 to axis 1, ...) and
// turns by the angle theta = position[axis] * inv_freq[j]:
//   (x_a, x_b) -> (x_a cos - x_b sin, x_a sin + x_b cos),
// a rotation, so the gradient is the rotation by -theta (sign = -1). Columns
// from 2R on are copied.
//
// The angle is reduced in fp64: position * (inv_freq / 2 pi) turns, minus the
// nearest integer, is exact to about 2^-52 * |turns|, whereas an fp32 product
// is off by 6e-3 rad at position 100,000. The sine and cosine of the reduced
// angle, and the rotation, are fp32; the result is rounded once.
//
// Bound by memory: every element is read and written once. One block takes a
// few tokens, computes their R sines and cosines once into shared memory (all
// heads of q and k share them) and streams q's and k's heads past them,
// VEC elements of both halves of a pair group per thread, the first loads on
// their way while the angles are computed. A pair is read and written by one
// thread, so the output may be the input. Measured: q and k of 8 x 8192 tokens,
// 16 heads each of 128 columns in a packed projection, 96 of them turned, bf16:
// 203 us, 5.3 TB/s, 82% of the copy rate (293 us with the loads after the
// angles and divisions by the hardware).
#pragma once

#include <cstdint>

#include "fa_common.cuh"

namespace fa {

constexpr int kRotMaxAxes = 8;
constexpr int kRotMaxTokens = 64;  // tokens of one block

struct RotArgs {
  const uint16_t* x[2];  // q and k (k's heads may be 0)
  uint16_t* y[2];
  int64_t xs[2][3], ys[2][3];  // element strides: batch, sequence, head
  int heads[2];
  const void* pos;  // int32 or int64 [axes][B][S] with element strides pos_s
  int64_t pos_s[3];
  int pos64;
  const void* inv_freq;  // fp32 or fp64 [R]
  int freq64;
  int end[kRotMaxAxes];  // pair index past each axis' section
  int axes;
  int B, S, D, R;
  int tokens;  // tokens per block
  float sign;  // +1 forward, -1 gradient
  // Items of a head (see the kernel) and of a token, and their reciprocals.
  int n_rot, n_item, per_tok;
  uint32_t inv_item, inv_tok;
};

// x / d for x d < 2^32 with inv = floor(2^32 / d) + 1: x inv / 2^32 is above x / d
// by at most x / 2^32 < 1 / d, too little to reach the next integer. inv = 0
// stands for d = 1; inv = 1 gives 0 (x < d).
__device__ __forceinline__ int div_by(int x, uint32_t inv) {
  return inv == 0 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), inv));
}

// VEC 16-bit values as they are loaded.
template <int VEC>
struct alignas(VEC * 2) RotPack {
  uint32_t w[VEC / 2];
};
template <>
struct alignas(2) RotPack<1> {
  uint16_t w[1];
};

// (cos, sin) of token t (of the block) and pair j.
__device__ __forceinline__ float2 rot_angle(const RotArgs& a, int b, int s, int j) {
  int axis = 0;
  while (axis < a.axes - 1 && j >= a.end[axis]) ++axis;
  const int64_t pa = axis * a.pos_s[0] + b * a.pos_s[1] + s * a.pos_s[2];
  const int64_t p = a.pos64 ? static_cast<const int64_t*>(a.pos)[pa] : static_cast<const int32_t*>(a.pos)[pa];
  const double f = a.freq64 ? static_cast<const double*>(a.inv_freq)[j]
                            : static_cast<double>(static_cast<const float*>(a.inv_freq)[j]);
  const double turns = static_cast<double>(p) * (f * 0.15915494309189533577);  // 1 / (2 pi)
  float sn, cn;
  sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &sn, &cn);
  return make_float2(cn, sn * a.sign);
}

// INTER: pairs are neighbours; VEC = elements per load (8: four pairs).
// Otherwise VEC pairs per thread from two loads of VEC elements, VEC the
// largest power of two up to 8 that divides R (so both loads are aligned).
template <bool BF16, bool INTER, int VEC>
__global__ void __launch_bounds__(256) fa_rotary_kernel(const RotArgs a) {
  using namespace sm100;
  using Pack = RotPack<VEC>;
  constexpr int U = 4;  // items of a thread whose loads are in flight together
  extern __shared__ float4 cs4[];  // (cos, sin) of [token][R]
  float2* cs = reinterpret_cast<float2*>(cs4);
  const int64_t total = static_cast<int64_t>(a.B) * a.S;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(a.tokens), total - tok0));
  const int b0 = static_cast<int>(tok0 / a.S);
  const int s0 = static_cast<int>(tok0 - static_cast<int64_t>(b0) * a.S);
  // Work items of a head: n_rot groups of VEC rotated pairs (INTER: VEC / 2),
  // then groups of VEC copied columns.
  const int items = nt * a.per_tok;
  Pack va[U], vb[U];
  uint16_t* out[U];
  int c0[U];    // first (cos, sin) of a rotated group; -1: copied; -2: none
  int left[U];  // INTER: the head's pairs from there on
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 256 * u;
      c0[u] = -2;
      if (i >= items) continue;
      const int t = div_by(i, a.inv_tok), r = i - t * a.per_tok;
      const int hh = div_by(r, a.inv_item), it = r - hh * a.n_item;
      const int w = hh >= a.heads[0];
      const int h = w ? hh - a.heads[0] : hh;
      int b = b0, s = s0 + t;
      while (s >= a.S) s -= a.S, ++b;
      const bool rot = it < a.n_rot;
      const int col = INTER || rot ? it * VEC : 2 * a.R + (it - a.n_rot) * VEC;
      const uint16_t* x = a.x[w] + b * a.xs[w][0] + s * a.xs[w][1] + h * a.xs[w][2] + col;
      out[u] = a.y[w] + b * a.ys[w][0] + s * a.ys[w][1] + h * a.ys[w][2] + col;
      c0[u] = rot ? t * a.R + (INTER ? it * (VEC / 2) : it * VEC) : -1;
      left[u] = a.R - it * (VEC / 2);
      va[u] = *reinterpret_cast<const Pack*>(x);
      if (!INTER && rot) vb[u] = *reinterpret_cast<const Pack*>(x + a.R);
    }
  };
  load(threadIdx.x);  // on its way while the angles are computed
  for (int i = threadIdx.x; i < nt * a.R; i += 256) {
    const int t = i / a.R;
    int b = b0, s = s0 + t;
    while (s >= a.S) s -= a.S, ++b;
    cs[i] = rot_angle(a, b, s, i - t * a.R);
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < items;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0[u] >= 0) {
        const float2* c = cs + c0[u];
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e)
            if (e < left[u]) {
              const float2 q = c[e], x = unpack2<BF16>(va[u].w[e]);
              va[u].w[e] = pack2<BF16>(x.x * q.x - x.y * q.y, x.x * q.y + x.y * q.x);
            }
        } else if constexpr (VEC == 1) {
          const float2 q = c[0];
          const float xa = unpack2<BF16>(va[u].w[0]).x, xb = unpack2<BF16>(vb[u].w[0]).x;
          const uint32_t o = pack2<BF16>(xa * q.x - xb * q.y, xa * q.y + xb * q.x);
          va[u].w[0] = static_cast<uint16_t>(o & 0xffffu);
          vb[u].w[0] = static_cast<uint16_t>(o >> 16);
        } else {
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) {
            const float2 q0 = c[2 * e], q1 = c[2 * e + 1];
            const float2 xa = unpack2<BF16>(va[u].w[e]), xb = unpack2<BF16>(vb[u].w[e]);
            va[u].w[e] = pack2<BF16>(xa.x * q0.x - xb.x * q0.y, xa.y * q1.x - xb.y * q1.y);
            vb[u].w[e] = pack2<BF16>(xa.x * q0.y + xb.x * q0.x, xa.y * q1.y + xb.y * q1.x);
          }
        }
        if (!INTER) *reinterpret_cast<Pack*>(out[u] + a.R) = vb[u];
      }
      if (c0[u] != -2) *reinterpret_cast<Pack*>(out[u]) = va[u];
    }
    i0 += 256 * U;
    load(i0);
  }
}

}  // namespace fa
