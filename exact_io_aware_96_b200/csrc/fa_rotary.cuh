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
// VEC elements of both halves of a pair group per thread. A pair is read and
// written by one thread, so the output may be the input.
#pragma once

#include <cstdint>

#include "fa_common.cuh"

namespace fa {

constexpr int kRotMaxAxes = 8;

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
};

// INTER: pairs are neighbours; VEC = elements per load (8: four pairs).
// Otherwise VEC pairs per thread from two loads of VEC elements, VEC the
// largest power of two up to 8 that divides R (so both loads are aligned).
template <bool BF16, bool INTER, int VEC>
__global__ void __launch_bounds__(256) fa_rotary_kernel(const RotArgs a) {
  using namespace sm100;
  extern __shared__ float2 cs[];  // [token][R]: (cos, sin)
  const int64_t total = static_cast<int64_t>(a.B) * a.S;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(a.tokens), total - tok0));
  for (int i = threadIdx.x; i < nt * a.R; i += 256) {
    const int t = i / a.R, j = i - t * a.R;
    const int64_t tok = tok0 + t;
    const int64_t b = tok / a.S, s = tok - b * a.S;
    int axis = 0;
    while (axis < a.axes - 1 && j >= a.end[axis]) ++axis;
    const int64_t at = axis * a.pos_s[0] + b * a.pos_s[1] + s * a.pos_s[2];
    const int64_t p = a.pos64 ? static_cast<const int64_t*>(a.pos)[at] : static_cast<const int32_t*>(a.pos)[at];
    const double f = a.freq64 ? static_cast<const double*>(a.inv_freq)[j]
                              : static_cast<double>(static_cast<const float*>(a.inv_freq)[j]);
    const double turns = static_cast<double>(p) * (f * 0.15915494309189533577);  // 1 / (2 pi)
    float sn, cn;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &sn, &cn);
    cs[i] = make_float2(cn, sn * a.sign);
  }
  __syncthreads();

  // Work items of a head: groups of VEC rotated pairs (INTER: VEC / 2), then
  // groups of VEC copied columns.
  const int n_rot = INTER ? (2 * a.R + VEC - 1) / VEC : a.R / VEC;
  const int n_item = INTER ? a.D / VEC : n_rot + (a.D - 2 * a.R) / VEC;
  const int heads = a.heads[0] + a.heads[1];
  const int per_tok = heads * n_item;
  struct alignas(VEC * 2) Pack {
    uint16_t e[VEC];
  };
  auto to_f = [](uint16_t v) {
    if constexpr (BF16)
      return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else
      return __half2float(__ushort_as_half(v));
  };
  auto from_f = [](float v) { return static_cast<uint16_t>(pack2<BF16>(v, 0.f) & 0xffffu); };
#pragma unroll 2
  for (int i = threadIdx.x; i < nt * per_tok; i += 256) {
    const int t = i / per_tok, r = i - t * per_tok;
    const int hh = r / n_item, it = r - hh * n_item;
    const int w = hh >= a.heads[0];
    const int h = w ? hh - a.heads[0] : hh;
    const int64_t tok = tok0 + t;
    const int64_t b = tok / a.S, s = tok - b * a.S;
    const uint16_t* x = a.x[w] + b * a.xs[w][0] + s * a.xs[w][1] + h * a.xs[w][2];
    uint16_t* y = a.y[w] + b * a.ys[w][0] + s * a.ys[w][1] + h * a.ys[w][2];
    const float2* c = cs + t * a.R;
    if constexpr (INTER) {
      Pack v = *reinterpret_cast<const Pack*>(x + it * VEC);
#pragma unroll
      for (int u = 0; u < VEC / 2; ++u) {
        const int j = it * (VEC / 2) + u;
        if (j < a.R) {
          const float2 q = c[j];
          const float xa = to_f(v.e[2 * u]), xb = to_f(v.e[2 * u + 1]);
          v.e[2 * u] = from_f(xa * q.x - xb * q.y);
          v.e[2 * u + 1] = from_f(xa * q.y + xb * q.x);
        }
      }
      *reinterpret_cast<Pack*>(y + it * VEC) = v;
    } else if (it < n_rot) {
      const int j0 = it * VEC;
      Pack va = *reinterpret_cast<const Pack*>(x + j0);
      Pack vb = *reinterpret_cast<const Pack*>(x + a.R + j0);
#pragma unroll
      for (int u = 0; u < VEC; ++u) {
        const float2 q = c[j0 + u];
        const float xa = to_f(va.e[u]), xb = to_f(vb.e[u]);
        va.e[u] = from_f(xa * q.x - xb * q.y);
        vb.e[u] = from_f(xa * q.y + xb * q.x);
      }
      *reinterpret_cast<Pack*>(y + j0) = va;
      *reinterpret_cast<Pack*>(y + a.R + j0) = vb;
    } else {
      const int col = 2 * a.R + (it - n_rot) * VEC;
      *reinterpret_cast<Pack*>(y + col) = *reinterpret_cast<const Pack*>(x + col);
    }
  }
}

}  // namespace fa
