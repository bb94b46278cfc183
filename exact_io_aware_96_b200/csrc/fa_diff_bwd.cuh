// fa_diff_bwd.cuh — differential attention backward for sm_100a (fa_diff_bwd).
//
// With P_c = softmax(scale Q_c K_c^T), O_c = P_c V, O = O_1 - lambda O_2 and
// W = P_1 - lambda P_2:
//   dV = W^T dO,   dP = dO V^T (one product serves both maps),
//   Delta_c = rowsum(P_c dP) = dO . O_c   (O_1 = O + lambda O_2),
//   dS_1 = P_1 (dP - Delta_1),   dS_2 = -lambda P_2 (dP - Delta_2),
//   dQ_c = scale dS_c K_c,   dK_c = scale dS_c^T Q_c,
//   dlambda = -dO . O_2 = -Delta_2.
// Two plain attention backwards would run dP and dV twice; taken together a
// 128 x 128 block costs 2 x 128 x 128 x (6 x 64 + 2 DV) flops, 640 columns of
// products at DV = 128 instead of 896.
//
// Kernels on the caller's stream:
//  1. fa_diff_pre: per row Delta_1, Delta_2, both LSEs in base 2 (+inf for rows
//     with no key and padding rows) and -lambda, packed per 64 rows; zeroes
//     the fp32 dQ accumulators; writes dlambda, or the terms of its sums.
//  2. fa_diff_bwd_main: one CTA per (batch, key head, 128-key block); walks the
//     query blocks of every query head that shares the key head, so dK and dV
//     of shared heads are summed in the CTA's fp32 accumulators, in a fixed
//     order. Where the longest such list would outlast the rest of the grid
//     (few key heads, many query heads, a causal mask), the lists are cut into
//     parts, a CTA each, whose fp32 dK and dV fa_diff_dkv adds in order.
//  3. fa_diff_dq: dq_c = scale * accumulator, rounded to the input dtype.
//  4. fa_diff_lam_few, or fa_diff_lam_part and fa_diff_lam_sum: dlambda summed
//     over the axes lambda is broadcast over, in a fixed order.
//
// Main kernel. Query rows go through the softmax 64 at a time ("chunks", two
// per 128-row query block): S_1^T, S_2^T and dP^T of a chunk then take 3 x 64
// columns of tensor memory beside the accumulators dV, dK_1, dK_2 (256) and a
// dQ block of one map (64 columns), 512 in all. dQ is a product over whole
// 128-row blocks (M = 128 is the tensor core's full rate), taken from the dS^T
// halves of both chunks in shared memory.
//
// Warp roles (448 threads):
//   warps 0-7   P and dS of 32 keys x 32 query columns per warp (warps 0-3 take
//               the chunk's columns [0, 32), warps 4-7 [32, 64)), in matrix-
//               fragment order. P_1 and -lambda P_2 stay in fp32 registers
//               between the two phases of a chunk. At the end warps 0-3 write
//               dK_1 and dK_2, warps 4-7 dV.
//   warps 8-11  read the dQ blocks out of tensor memory (one query row per
//               thread) and add them into the fp32 accumulators through the
//               TMA; deterministic mode stores them into their own slots.
//   warp  12    TMA loader: K_1, K_2, V once; per chunk Q_1 and Q_2, dO, and
//               the row terms
//   warp  13    MMA issuer
// MMA order per chunk i: dV(i), S_1(i+1), S_2(i+1), [dQ], dK_1(i), dK_2(i),
// dP(i+1), with dQ_1 in odd chunks and dQ_2 in the even ones after them: the
// softmax of chunk i+1 starts while dK(i), dP(i+1) and dQ run.
//
// What bounds it. A chunk's products take 1650 tensor cycles alone (1280 at
// the full rate: with N = 64 both operands from shared memory are read at 128
// bytes a cycle, 48 cycles an instruction instead of 32, which is why W^T and
// dS^T go to dV and dK through tensor memory). The softmax's two phases take
// about 2300 cycles a chunk and overlap the products except for the hand-offs
// (W ready -> dV, S ready -> exponentials, dS ready -> dK). Measured at B = 1,
// H = 8, S = 8192, D = 64, DV = 128, bf16, causal, all kernels of the call in
// bursts at 1965 MHz: 422 us, 814 TFLOP/s, tensor pipe 39% active; 480 when
// launched for a second without a pause (1700 MHz under the power cap). Of 474 us
// at an earlier step: without the exponentials 440, without the dQ reductions
// 459; no single part carries the rest. Tried and slower, against 455 to 490: 16
// softmax warps of 16 columns (550 us), dQ_2 over dP's columns with dK from shared
// memory (602), dQ by red.global instead of the TMA (604). At DV = 128 three
// registers of a thread spill (12 bytes, once each way).
//
// Rounded to 16 bits, as operands of the tensor cores: W before dV, dS_c before
// dQ_c and dK_c. Delta_c and dlambda come from O and O_2, which the forward has
// rounded to 16 bits (once as P's, once as their own): a sum over P_2 dP in fp32
// would spare dlambda that, at a row sum over the lanes in every chunk's softmax.
// Relative errors in norm, bf16 (rounding the result alone: 1.7e-3): dQ and dK
// 2.5e-3, dV 2.4e-3, dlambda 2.7e-3; fp16 (2.1e-4): 3.0e-4, 2.9e-4, 3.6e-4. An fp32
// dlambda of every row keeps 2.1e-3 (fp16: 2.9e-4); summed over 4,000 rows and
// more, one of a head is off by less than 1e-4 of its terms' magnitudes.
#pragma once

#include <type_traits>

#include "fa_common.cuh"
#include "fa_diff_fwd.cuh"

namespace fa {

struct DiffBwdArgs {
  const void* o;
  const void* o2;
  const void* dO;
  const float* lse;  // [2][B][H][Sq]
  const void* lam;
  int64_t lam_s[3];
  int lam_kind;
  void* dq[2];
  void* dk[2];
  void* dv;
  int64_t o_s[3], o2_s[3], do_s[3], dq_s[2][3], dk_s[2][3], dv_s[3];
  float* dq_acc;   // fp32 [2][B*H][Sq_pad][64]
  float* vec;      // fp32 [B*H][Sq_pad / 64][5][64]: -lse2_1, -lse2_2, -lambda, -Delta_1, -Delta_2
  float* drow;     // fp32 [B][H][Sq]: -Delta_2, where lambda is broadcast
  void* dlam;      // dlambda [B][Sq][H], where it is not; else null
  float* dkv_part;  // parts > 1: fp32 [parts][B*Hk][Sk_pad][128 + DV]: a part's dK_1, dK_2, dV; else null
  float* dq_part;  // deterministic mode: fp32 [B*H][nqb][nkb][2][128][64] slots; else null
  int B, H, Hk, Sq, Sk, Sq_pad;
  int nqb, nkb;    // ceil(Sq / 128), ceil(Sk / 128)
  int group;       // H / Hk
  int parts;       // CTAs that share a key block's (head, query block) list
  int d, dv_cols;  // head_dim of q and k; columns of v
  float scale, scale_log2;
  int causal;
  Div by_H, by_Sq, by_Sq_pad, by_Sk, by_Hk, by_parts;
  Div by_order;  // the faster dimension of the grid order: B x Hk with a causal mask, nkb without
};

constexpr int kDiffVec = 5 * 64;  // floats of one chunk's row terms

__device__ __forceinline__ void store_lam(void* p, int kind, int64_t at, float v) {
  if (kind == kLamF32)
    static_cast<float*>(p)[at] = v;
  else
    static_cast<uint16_t*>(p)[at] =
        static_cast<uint16_t>((kind == kLamBF16 ? sm100::pack2<true>(v, 0.f) : sm100::pack2<false>(v, 0.f)) & 0xffffu);
}

// Tensor memory in matrix-fragment order: of a warp's 32 lanes x 8 columns,
// thread t gets rows t / 4 + {0, 8, 16, 24} and columns 2 (t % 4) + {0, 1}, where
// the 32x32b form gives it all columns of row t. A thread then needs only a
// quarter of the per-column constants (for four rows each).
// 16 lanes x 32 columns (32-bit): v[4 j + 2 e + x] = row t / 4 + 8 e, column 8 j + 2 (t % 4) + x.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 16 lanes x 16 columns (32-bit words of two 16-bit values): r[2 j + e] = row t / 4 + 8 e, column 4 j + t % 4.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// The backward's kernels follow each other as programmatic dependent launches:
// a grid's blocks start as the grid before it runs out of them, and stop here
// until all of that grid's memory is written and visible. Every block waits, so
// the end of one grid implies the end of all before it.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Whether phase `parity` of `bar` has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(sm100::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The 64-bit descriptor of a 128-byte-swizzled operand from its low word
// (address >> 4 and lbo >> 4 << 16); the high word is the same for all: 1024
// bytes between 8-row groups, the sm_100 version and the swizzle mode.
__device__ __forceinline__ uint64_t desc_words(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((1024u >> 4) | (1u << 14) | (2u << 29)));
  return d;
}

// Four 8 x 8 matrices of 16-bit values; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void stsm_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// ------------------------------------------------------------- preprocess
// DV / 8 threads per (b, h, i) row, i in [0, Sq_pad).
template <int DV, bool BF16>
__global__ void __launch_bounds__(256) fa_diff_pre(const DiffBwdArgs a) {
  constexpr int G = DV / 8;
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = gid / G;
  const int part = static_cast<int>(gid % G);
  const int64_t nrows = static_cast<int64_t>(a.B) * a.H * a.Sq_pad;
  if (row >= nrows) return;  // whole groups leave together: G divides 32, nrows * G is a multiple of 256
  int i, h;
  const int bh = static_cast<int>(quo_rem(row, a.by_Sq_pad, &i));
  const int b = static_cast<int>(quo_rem(bh, a.by_H, &h));
  float d_o = 0.f, d_2 = 0.f;  // dO . O, dO . O_2
  if (i < a.Sq && part * 8 < a.dv_cols && checked(b < a.B && h < a.H, 501)) {
    auto at = [&](const void* p, const int64_t(&s)[3]) {
      return *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + b * s[0] + i * s[1] + h * s[2] +
                                             part * 8);
    };
    const uint4 ov = at(a.o, a.o_s), o2v = at(a.o2, a.o2_s), gv = at(a.dO, a.do_s);
    const uint32_t* o32 = reinterpret_cast<const uint32_t*>(&ov);
    const uint32_t* p32 = reinterpret_cast<const uint32_t*>(&o2v);
    const uint32_t* g32 = reinterpret_cast<const uint32_t*>(&gv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = sm100::unpack2<BF16>(o32[k]);
      const float2 z = sm100::unpack2<BF16>(p32[k]);
      const float2 y = sm100::unpack2<BF16>(g32[k]);
      d_o = fmaf(x.x, y.x, d_o);
      d_o = fmaf(x.y, y.y, d_o);
      d_2 = fmaf(z.x, y.x, d_2);
      d_2 = fmaf(z.y, y.y, d_2);
    }
  }
#pragma unroll
  for (int s = G / 2; s > 0; s >>= 1) {
    d_o += __shfl_xor_sync(0xffffffffu, d_o, s);
    d_2 += __shfl_xor_sync(0xffffffffu, d_2, s);
  }
  if (a.dq_part == nullptr && checked(row < nrows, 502)) {  // the atomic accumulators start from zero
    constexpr int F4 = 64 * 2 / 4 / G;  // float4s per thread over both maps
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < F4; ++u) {
      const int f = part + u * G;  // 0 .. 31: map f / 16, float4 f % 16
      reinterpret_cast<float4*>(a.dq_acc)[((f >> 4) * nrows + row) * 16 + (f & 15)] = z;
    }
  }
  if (part == 0 && checked(row < nrows, 503)) {
    float l1 = INFINITY, l2 = INFINITY, lam = 0.f;
    if (i < a.Sq) {
      const int64_t at = static_cast<int64_t>(bh) * a.Sq + i;
      const float e1 = a.lse[at], e2 = a.lse[static_cast<int64_t>(a.B) * a.H * a.Sq + at];
      if (e1 != -INFINITY) {  // a row with no key has -inf in both
        l1 = e1 * 1.4426950408889634f;
        l2 = e2 * 1.4426950408889634f;
        lam = load_lam(a.lam, a.lam_kind, b * a.lam_s[0] + i * a.lam_s[1] + h * a.lam_s[2]);
        // A NaN logsumexp has to reach every -lambda P_2 of the row: the exponentials
        // on the FMA pipe drop it, this factor does not.
        if (e2 != e2) lam = e2;
      } else {
        d_o = d_2 = 0.f;
      }
      if (a.dlam != nullptr)
        store_lam(a.dlam, a.lam_kind, (static_cast<int64_t>(b) * a.Sq + i) * a.H + h, -d_2);
      else
        a.drow[at] = -d_2;
    }
    float* v = a.vec + (static_cast<int64_t>(bh) * (a.Sq_pad / 64) + i / 64) * kDiffVec + (i & 63);
    v[0] = -l1;
    v[64] = -l2;
    v[128] = -lam;
    v[192] = -(lam == 0.f ? d_o : fmaf(lam, d_2, d_o));
    v[256] = -d_2;
  }
}

// ------------------------------------------------------------- dq convert
// dq_c = scale * accumulator (or the key blocks' slots, added in key-block
// order). 8 columns per thread; map in blockIdx.y.
template <bool BF16, bool DET>
__global__ void __launch_bounds__(256) fa_diff_dq(const DiffBwdArgs a) {
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = gid / 8;  // (b, h, i) with i < Sq
  const int part = static_cast<int>(gid % 8);
  const int c = blockIdx.y;
  const int64_t bhs = static_cast<int64_t>(a.B) * a.H;
  grid_wait();
  if (row >= bhs * a.Sq || part * 8 >= a.d) return;
  int i, h;
  const int bh = static_cast<int>(quo_rem(row, a.by_Sq, &i));
  const int b = static_cast<int>(quo_rem(bh, a.by_H, &h));
  float acc[8];
  if constexpr (DET) {
    const int qb = i / 128;
    const float* slot =
        a.dq_part + ((static_cast<int64_t>(bh) * a.nqb + qb) * a.nkb * 2 + c) * (128 * 64) + (i % 128) * 64 + part * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int kvb = 0; kvb < a.nkb; ++kvb) {
      if (qb < bwd_first_qblock(kvb, a.Sq, a.Sk, a.causal)) break;  // later key blocks start later still
      const float4* src = reinterpret_cast<const float4*>(slot + static_cast<int64_t>(kvb) * (2 * 128 * 64));
      const float4 x = src[0], y = src[1];
      acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
      acc[4] += y.x, acc[5] += y.y, acc[6] += y.z, acc[7] += y.w;
    }
  } else {
    const float4* src = reinterpret_cast<const float4*>(a.dq_acc + ((c * bhs + bh) * a.Sq_pad + i) * 64 + part * 8);
    const float4 x = src[0], y = src[1];
    acc[0] = x.x, acc[1] = x.y, acc[2] = x.z, acc[3] = x.w;
    acc[4] = y.x, acc[5] = y.y, acc[6] = y.z, acc[7] = y.w;
  }
  const float s = a.scale;
  uint4 out;
  out.x = sm100::pack2<BF16>(acc[0] * s, acc[1] * s);
  out.y = sm100::pack2<BF16>(acc[2] * s, acc[3] * s);
  out.z = sm100::pack2<BF16>(acc[4] * s, acc[5] * s);
  out.w = sm100::pack2<BF16>(acc[6] * s, acc[7] * s);
  if (checked(b < a.B && h < a.H && i < a.Sq, 504))
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.dq[c]) + b * a.dq_s[c][0] + i * a.dq_s[c][1] +
                              h * a.dq_s[c][2] + part * 8) = out;
}

// ------------------------------------------------------------ dk, dv join
// dk_c and dv of key blocks whose query blocks were cut into parts: the parts'
// sums are added in order. 8 columns per thread of a row of dK_1 | dK_2 | dV.
template <int DV, bool BF16>
__global__ void __launch_bounds__(256) fa_diff_dkv(const DiffBwdArgs a) {
  constexpr int G = (128 + DV) / 8;
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = gid / G;  // (b, hk, key)
  const int part = static_cast<int>(gid % G);
  const int64_t bhs = static_cast<int64_t>(a.B) * a.Hk;
  grid_wait();
  if (row >= bhs * a.Sk) return;
  int key, hk;
  const int bh = static_cast<int>(quo_rem(row, a.by_Sk, &key));
  const int b = static_cast<int>(quo_rem(bh, a.by_Hk, &hk));
  const bool is_k = part < 16;
  const int c = part >> 3;  // map, for dK
  const int col = is_k ? (part & 7) * 8 : (part - 16) * 8;
  if (col >= (is_k ? a.d : a.dv_cols)) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int64_t step = bhs * a.nkb * 128 * (128 + DV);
  const float* src = a.dkv_part + (static_cast<int64_t>(bh) * a.nkb * 128 + key) * (128 + DV) + part * 8;
  for (int p = 0; p < a.parts; ++p) {
    const float4 x = reinterpret_cast<const float4*>(src + p * step)[0];
    const float4 y = reinterpret_cast<const float4*>(src + p * step)[1];
    acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
    acc[4] += y.x, acc[5] += y.y, acc[6] += y.z, acc[7] += y.w;
  }
  const float s = is_k ? a.scale : 1.f;
  uint4 out;
  out.x = sm100::pack2<BF16>(acc[0] * s, acc[1] * s);
  out.y = sm100::pack2<BF16>(acc[2] * s, acc[3] * s);
  out.z = sm100::pack2<BF16>(acc[4] * s, acc[5] * s);
  out.w = sm100::pack2<BF16>(acc[6] * s, acc[7] * s);
  uint16_t* dst = is_k ? reinterpret_cast<uint16_t*>(a.dk[c]) + b * a.dk_s[c][0] + key * a.dk_s[c][1] + hk * a.dk_s[c][2]
                       : reinterpret_cast<uint16_t*>(a.dv) + b * a.dv_s[0] + key * a.dv_s[1] + hk * a.dv_s[2];
  if (checked(b < a.B && key < a.Sk, 505)) *reinterpret_cast<uint4*>(dst + col) = out;
}

// ----------------------------------------------------------- dlambda sums
// dlambda has lambda's extents (each 1 or the full axis; order batch, row, head)
// and is dense. Element x sums drow over the axes with extent 1: `count` terms,
// cut into `parts` runs. One block per (element, run) writes its sum to
// part[element * parts + run], in a fixed order.
constexpr int kLamThreads = 512;
struct LamSumArgs {
  const float* drow;  // [B][H][Sq]
  float* part;
  void* dlam;
  int dlam_kind;
  int B, H, Sq;
  Div by_s, by_h;    // lambda's extents along rows and heads
  Div by_ns, by_nh;  // rows and heads that one of its elements sums over
  int64_t n_out, count;
  int parts;
};

template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.f;
  for (int w = 0; w < THREADS / 32; ++w) r += sm[w];
  __syncthreads();
  return r;
}

// Element x's place, and term k of its sum. The summed axes, innermost first:
// rows, heads, batch.
__device__ __forceinline__ const float* lam_base(const LamSumArgs& a, int64_t x) {
  int eh, es;
  const int64_t eb = quo_rem(quo_rem(x, a.by_h, &eh), a.by_s, &es);
  return a.drow + (eb * a.H + eh) * a.Sq + es;
}
__device__ __forceinline__ float lam_term(const LamSumArgs& a, const float* base, int64_t k) {
  int s, h;
  const int64_t b = quo_rem(quo_rem(k, a.by_ns, &s), a.by_nh, &h);
  return base[(b * a.H + h) * a.Sq + s];
}
__device__ __forceinline__ float lam_term(const LamSumArgs& a, const float* base, int k) {
  const int z = quo(k, a.by_ns), b = quo(z, a.by_nh);
  const int s = k - z * a.by_ns.d, h = z - b * a.by_nh.d;
  return base[(static_cast<int64_t>(b) * a.H + h) * a.Sq + s];
}
// Terms lo + first, lo + first + step, ... below hi, in this order.
__device__ __forceinline__ float lam_terms(const LamSumArgs& a, const float* base, int64_t lo, int64_t hi, int first,
                                           int step) {
  float v = 0.f;
  if (hi < (int64_t(1) << 31) - step) {
#pragma unroll 8
    for (int k = static_cast<int>(lo) + first; k < static_cast<int>(hi); k += step) v += lam_term(a, base, k);
  } else {
    for (int64_t k = lo + first; k < hi; k += step) v += lam_term(a, base, k);
  }
  return v;
}

// Few terms: one thread per element.
__global__ void __launch_bounds__(256) fa_diff_lam_few(const LamSumArgs a) {
  const int64_t x = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  grid_wait();
  if (x < a.n_out) store_lam(a.dlam, a.dlam_kind, x, lam_terms(a, lam_base(a, x), 0, a.count, 0, 1));
}

__global__ void __launch_bounds__(kLamThreads) fa_diff_lam_part(const LamSumArgs a) {
  __shared__ float sm[kLamThreads / 32];
  const int64_t x = blockIdx.x / a.parts;
  const int run = static_cast<int>(blockIdx.x % a.parts);
  const int64_t len = (a.count + a.parts - 1) / a.parts;
  const int64_t lo = run * len, hi = min(a.count, lo + len);
  const float* base = lam_base(a, x);
  grid_wait();
  const float v = block_sum<kLamThreads>(lam_terms(a, base, lo, hi, threadIdx.x, kLamThreads), sm);
  if (threadIdx.x == 0) {
    if (a.parts == 1)
      store_lam(a.dlam, a.dlam_kind, x, v);
    else
      a.part[blockIdx.x] = v;
  }
}

__global__ void __launch_bounds__(256) fa_diff_lam_sum(const LamSumArgs a) {
  __shared__ float sm[8];
  float v = 0.f;
  grid_wait();
  for (int k = threadIdx.x; k < a.parts; k += 256) v += a.part[static_cast<int64_t>(blockIdx.x) * a.parts + k];
  v = block_sum<256>(v, sm);
  if (threadIdx.x == 0) store_lam(a.dlam, a.dlam_kind, blockIdx.x, v);
}

// ------------------------------------------------------------- main kernel
template <int DV>
struct DiffBwdLayout {
  static constexpr int kThreads = 448;
  static constexpr int BLK = 128 * 128;   // [128 rows][64 columns] of 16 bits
  static constexpr int HBLK = 64 * 128;   // [64 rows][64 columns]
  static constexpr int VB = DV / 64;
  // A stage of Q is in use from S(i) to dK(i), nearly two chunks; dO(i) is done
  // with at dV(i), early enough for one stage.
  static constexpr int QS = 3;            // stages of (Q_1, Q_2)
  static constexpr int VS = 2;            // stages of the row terms
  static constexpr int OFF_K = 0;                       // K_1, K_2
  static constexpr int OFF_V = OFF_K + 2 * BLK;
  static constexpr int OFF_Q = OFF_V + VB * BLK;        // [stage][map][64 rows]
  static constexpr int OFF_DO = OFF_Q + QS * 2 * HBLK;  // [column block][64 rows]
  static constexpr int OFF_DS = OFF_DO + VB * HBLK;  // dS_1^T: [chunk half][128 keys][64 queries]
  // dS_2^T's first half alternates between blocks 0 and 2, so that dQ_2 of a
  // block may still read its dS while the next block's is written.
  static constexpr int OFF_DS2 = OFF_DS + 2 * BLK;
  static constexpr int OFF_DQS = OFF_DS2 + 3 * BLK;     // dQ staging: 4 KB per drain warp
  static constexpr int OFF_VEC = OFF_DQS + 4 * 4096;
  static constexpr int OFF_BAR = OFF_VEC + VS * kDiffVec * 4;
  // kv_full, q_full/q_empty[QS], v_full[VS], o_full, o_empty, s_full, w_ready, dp_full, ds_ready, dq_full,
  // dq_free, mma_done, drain
  static constexpr int NBAR = 1 + 2 * QS + VS + 10;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static constexpr int SMEM_MAX = 232448;
  // Room to align the base to 1024 bytes where there is some; else the kernel
  // requires (and checks) an aligned base.
  static constexpr int SMEM_ALLOC = BYTES + 1024 <= SMEM_MAX ? BYTES + 1024 : BYTES;
  static constexpr int TMEM_COLS = 512;
  static constexpr int COL_DV = 0;
  static constexpr int COL_DK = 128;  // dK_1, dK_2: 64 columns each
  static constexpr int COL_S = 256;   // S_1^T, S_2^T: 64 columns each; W^T over S_1^T
  static constexpr int COL_DP = 384;
  static constexpr int COL_DQ = 448;
};

template <int DV, bool BF16>
__global__ void __launch_bounds__(448, 1)
    fa_diff_bwd_main(const __grid_constant__ CUtensorMap tmQ1, const __grid_constant__ CUtensorMap tmQ2,
                     const __grid_constant__ CUtensorMap tmK1, const __grid_constant__ CUtensorMap tmK2,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                     const __grid_constant__ CUtensorMap tmDQ, const DiffBwdArgs a) {
  using L = DiffBwdLayout<DV>;
  using namespace sm100;
  constexpr int QS = L::QS, VS = L::VS;
  static_assert(L::BYTES <= L::SMEM_MAX, "smem budget");

  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024 - (smem_u32(smem_raw) & 1023)) & 1023;
  uint8_t* smem = smem_raw + pad;
  if (L::BYTES + pad > L::SMEM_ALLOC) {
    if (threadIdx.x == 0) atomicCAS(&g_status[0], 0, -2);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = kv_full + 1;
  uint64_t* q_empty = q_full + QS;
  uint64_t* v_full = q_empty + QS;
  uint64_t* o_full = v_full + VS;
  uint64_t* o_empty = o_full + 1;
  uint64_t* s_full = o_empty + 1;
  uint64_t* w_ready = s_full + 1;
  uint64_t* dp_full = w_ready + 1;
  uint64_t* ds_ready = dp_full + 1;
  uint64_t* dq_full = ds_ready + 1;
  uint64_t* dq_free = dq_full + 1;
  uint64_t* mma_done = dq_free + 1;
  uint64_t* drain = mma_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const float* s_vec = reinterpret_cast<const float*>(smem + L::OFF_VEC);
  constexpr int kLoaderWarp = 12, kMmaWarp = 13;

  // Grid order as the plain backward's: with a causal mask key-block-major,
  // the first key blocks (the most query blocks) first; without one
  // head-major.
  int part, inner, hk;
  const int cta = static_cast<int>(quo_rem(blockIdx.x, a.by_parts, &part));
  const int outer = static_cast<int>(quo_rem(cta, a.by_order, &inner));
  const int kvb = a.causal ? outer : inner;
  const int b = static_cast<int>(quo_rem(a.causal ? inner : outer, a.by_Hk, &hk));
  const int group = a.group;
  const int n0 = kvb * 128;
  const int off = a.Sk - a.Sq;
  const int i_start = bwd_first_qblock(kvb, a.Sq, a.Sk, a.causal);
  const int nb = max(0, a.nqb - i_start);  // query blocks of one head
  // This CTA's part of the list of (head, query block) pairs; two chunks each.
  const int64_t listed = static_cast<int64_t>(nb) * group;
  int drop;
  const int blk0 = static_cast<int>(quo_rem(listed * part, a.by_parts, &drop));
  const int n = 2 * (static_cast<int>(quo_rem(listed * (part + 1), a.by_parts, &drop)) - blk0);
  // Where chunk 0 lies; the roles walk on from there: its head's (b, h) row base
  // and its block's first query row.
  const int head0 = blk0 == 0 ? 0 : blk0 / nb;
  const int bh0 = b * a.H + hk * group + head0, row0 = (i_start + blk0 - head0 * nb) * 128;
  auto next_block = [&](int& bh, int& r0) {
    r0 += 128;
    if (r0 == a.nqb * 128) r0 = i_start * 128, ++bh;
  };
  const int64_t acc_rows = static_cast<int64_t>(a.B) * a.H * a.Sq_pad;  // of one map's dQ accumulator

  // The loader's thread sets the barriers up itself and asks for the keys at
  // once: before tensor memory is allocated, and while fa_diff_pre still runs.
  if (warp == kLoaderWarp && lane == 0) {
    prefetch_tmap(&tmQ1);
    prefetch_tmap(&tmQ2);
    prefetch_tmap(&tmK1);
    prefetch_tmap(&tmK2);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmdO);
    mbar_init(kv_full, 1);
    for (int s = 0; s < QS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) mbar_init(&v_full[s], 1);
    mbar_init(o_full, 1);
    mbar_init(o_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(w_ready, 8);  // one arrival per softmax warp
    mbar_init(dp_full, 1);
    mbar_init(ds_ready, 8);
    mbar_init(dq_full, 1);
    mbar_init(dq_free, 4);
    mbar_init(mma_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (n > 0) {
      checked(n0 < a.Sk && b < a.B && hk < a.Hk, 510);
      mbar_arrive_expect_tx(kv_full, (2 + L::VB) * L::BLK);
      tma_load_4d(smem + L::OFF_K, &tmK1, kv_full, 0, n0, hk, b);
      tma_load_4d(smem + L::OFF_K + L::BLK, &tmK2, kv_full, 0, n0, hk, b);
      for (int vb = 0; vb < L::VB; ++vb)
        tma_load_4d(smem + L::OFF_V + vb * L::BLK, &tmV, kv_full, vb * 64, n0, hk, b);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();  // fa_diff_pre's row terms and cleared accumulators are there

  if (warp == kLoaderWarp) {
    // ------------------------------------------------------------------ loader
    if (lane == 0 && n > 0) {
      int nq = 0, nv = 0, no = 0;  // loads issued
      int bh = bh0, blk_row = row0;
      auto load = [&](int i) -> bool {
        const int qs = i % QS, vs = i % VS;
        const int r0 = blk_row + (i & 1) * 64, h = bh - b * a.H;
        // Row terms: free once the softmax warps are through with chunk i - 2.
        if (i >= VS && !wait_bar(ds_ready, (i - VS) & 1, abort_flag, kRoleLoader, i)) return false;
        mbar_arrive_expect_tx(&v_full[vs], kDiffVec * 4);
        // Skipped on a failed check: its wait then runs out (FA_ERR_BOUNDS stays recorded).
        if (checked(r0 + 64 <= a.Sq_pad && h < a.H, 511))
          bulk_load(smem + L::OFF_VEC + vs * kDiffVec * 4,
                    a.vec + (static_cast<int64_t>(bh) * (a.Sq_pad / 64) + r0 / 64) * kDiffVec, kDiffVec * 4,
                    &v_full[vs]);
        ++nv;
        if (!wait_bar(&q_empty[qs], ((i / QS) & 1) ^ 1, abort_flag, kRoleLoader, i)) return false;
        mbar_arrive_expect_tx(&q_full[qs], 2 * L::HBLK);
        tma_load_4d(smem + L::OFF_Q + qs * 2 * L::HBLK, &tmQ1, &q_full[qs], 0, r0, h, b);
        tma_load_4d(smem + L::OFF_Q + (qs * 2 + 1) * L::HBLK, &tmQ2, &q_full[qs], 0, r0, h, b);
        ++nq;
        if (!wait_bar(o_empty, (i & 1) ^ 1, abort_flag, kRoleLoader, i)) return false;
        mbar_arrive_expect_tx(o_full, L::VB * L::HBLK);
        for (int vb = 0; vb < L::VB; ++vb)
          tma_load_4d(smem + L::OFF_DO + vb * L::HBLK, &tmdO, o_full, vb * 64, r0, h, b);
        ++no;
        if (i & 1) next_block(bh, blk_row);
        return true;
      };
      for (int i = 0; i < n && load(i); ++i) {
      }
      if (*abort_flag) {
        drain_wait(kv_full, 0);
        for (int i = max(0, nq - QS); i < nq; ++i) drain_wait(&q_full[i % QS], (i / QS) & 1);
        for (int i = max(0, nv - VS); i < nv; ++i) drain_wait(&v_full[i % VS], (i / VS) & 1);
        if (no > 0) drain_wait(o_full, (no - 1) & 1);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- MMA issuer
    if (n > 0) {
      auto wait = [&](uint64_t* bar, uint32_t parity, int iter) {
        return __all_sync(0xffffffffu, wait_bar_c(bar, parity, abort_flag, kRoleMma, iter));
      };
      // S_c^T = K_c Q_c^T, dP^T = V dO^T: M = 128 keys, N = 64 queries (both K-major).
      constexpr uint32_t id_s = idesc_f16(BF16, 128, 64, 0, 0);
      // dV += W^T dO, dK_c += dS_c^T Q_c (A in TMEM); B MN-major, K = 64 queries.
      constexpr uint32_t id_v = idesc_f16(BF16, 128, DV, 0, 1);
      constexpr uint32_t id_k = idesc_f16(BF16, 128, 64, 0, 1);
      // dQ_c = dS_c K_c: M = 128 queries, N = 64, K = 128 keys; A = dS_c^T viewed MN-major, B = K_c MN-major.
      constexpr uint32_t id_q = idesc_f16(BF16, 128, 64, 1, 1);
      // Operand descriptors differ in their low words only (address and lbo):
      // every operand is one addition away.
      const uint32_t base = smem_u32(smem) >> 4;
      auto desc = [&](uint32_t off, uint32_t lbo) { return desc_words(base + (off >> 4) + ((lbo >> 4) << 16)); };
      auto issue_S = [&](int qs) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint64_t ad[4], bd[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            ad[u] = desc(L::OFF_K + c * L::BLK + u * 32, 16);
            bd[u] = desc(L::OFF_Q + (qs * 2 + c) * L::HBLK + u * 32, 16);
          }
          mma_ss_x4(tmem + L::COL_S + 64 * c, ad, bd, id_s, 0);
        }
      };
      auto issue_dP = [&]() {
#pragma unroll
        for (int vb = 0; vb < L::VB; ++vb) {
          uint64_t ad[4], bd[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            ad[u] = desc(L::OFF_V + vb * L::BLK + u * 32, 16);
            bd[u] = desc(L::OFF_DO + vb * L::HBLK + u * 32, 16);
          }
          mma_ss_x4(tmem + L::COL_DP, ad, bd, id_s, vb > 0);
        }
      };
      auto issue_dV = [&](uint32_t acc) {
        uint32_t pa[4];
        uint64_t bd[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          pa[u] = tmem + L::COL_S + (u >> 1) * 32 + (u & 1) * 8;  // W^T of queries 16u .. 16u + 15
          bd[u] = desc(L::OFF_DO + u * 2048, L::HBLK);
        }
        mma_ts_x4(tmem + L::COL_DV, pa, bd, id_v, acc);
      };
      auto issue_dK = [&](int qs, uint32_t acc) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pa[4];
          uint64_t bd[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            pa[u] = tmem + L::COL_DP + (u >> 1) * 32 + 16 * c + (u & 1) * 8;  // dS_c^T of queries 16u .. 16u + 15
            bd[u] = desc(L::OFF_Q + (qs * 2 + c) * L::HBLK + u * 2048, L::HBLK);
          }
          mma_ts_x4(tmem + L::COL_DK + 64 * c, pa, bd, id_k, acc);
        }
      };
      // dQ_1; dQ_2 of a block with dS_2's first half in block 0, or (alt) in
      // block 2: then the second half comes first, and the rows change places.
      auto issue_dQ = [&](int c, uint32_t alt) {
        const uint32_t a0 = (c == 0 ? L::OFF_DS : L::OFF_DS2) + alt * L::BLK;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint64_t ad[4], bd[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            ad[u] = desc(a0 + (4 * hf + u) * 2048, L::BLK);
            bd[u] = desc(L::OFF_K + c * L::BLK + (4 * hf + u) * 2048, L::BLK);
          }
          mma_ss_x4(tmem + L::COL_DQ, ad, bd, id_q, hf > 0);
        }
        mma_commit_w(dq_full);
      };
      bool ok = wait(kv_full, 0, -1) && wait(&q_full[0], 0, 0);
      if (ok) {
        tc_fence_after();
        issue_S(0);
        mma_commit_w(s_full);
        ok = wait(o_full, 0, 0);
      }
      if (ok) {
        tc_fence_after();
        issue_dP();
        mma_commit_w(dp_full);
      }
      int qs = 0;             // Q's stage of the chunk
      uint32_t q_phase = 0;   // and its phase
      auto chunk = [&](int blk, auto half) -> bool {  // chunk i = 2 blk + half
        constexpr int hf = decltype(half)::value;
        const int i = 2 * blk + hf;
        const bool more = i + 1 < n;
        const int qn = qs == QS - 1 ? 0 : qs + 1;
        const uint32_t q_phase_n = q_phase ^ (qn == 0);
        if (!wait(w_ready, hf, i)) return false;
        // The loads and the drain that the products below need are looked at
        // ahead of them: a wait between two groups of products, even for what is
        // there, lets the tensor core run dry (476 -> 468 us at S = 8192).
        const bool q_in = mbar_test(&q_full[qn], q_phase_n), dq_out = mbar_test(dq_free, hf);
        tc_fence_after();
        issue_dV(i > 0);
        mma_commit_w(o_empty);  // dP(i), issued before, and dV(i) are dO(i)'s readers
        if (more) {
          // S(i+1) goes over S(i) and W(i): the softmax warps have read S(i)
          // (w_ready) and dV(i), issued before, reads W(i) first.
          if (!__all_sync(0xffffffffu, q_in) && !wait(&q_full[qn], q_phase_n, i + 1)) return false;
          issue_S(qn);
          mma_commit_w(s_full);
        }
        if (hf == 0 && blk > 0) {
          // dQ_2 of the block before, once dQ_1 has been drained.
          if (!__all_sync(0xffffffffu, dq_out) && !wait(dq_free, 0, i)) return false;
          tc_fence_after();
          issue_dQ(1, (blk - 1) & 1);
        }
        if (!wait(ds_ready, hf, i)) return false;
        const bool o_in = mbar_test(o_full, hf ^ 1);
        tc_fence_after();
        if (hf) {
          if (blk > 0 && !__all_sync(0xffffffffu, dq_out) && !wait(dq_free, 1, i)) return false;  // the block before's dQ_2 has been drained
          tc_fence_after();
          issue_dQ(0, 0);
        }
        issue_dK(qs, i > 0);
        mma_commit_w(&q_empty[qs]);
        if (more) {
          if (!__all_sync(0xffffffffu, o_in) && !wait(o_full, hf ^ 1, i + 1)) return false;
          issue_dP();
          mma_commit_w(dp_full);
        }
        qs = qn;
        q_phase = q_phase_n;
        return true;
      };
      const int blocks = n / 2;
      for (int blk = 0; ok && blk < blocks; ++blk)
        ok = chunk(blk, std::integral_constant<int, 0>{}) && chunk(blk, std::integral_constant<int, 1>{});
      if (ok && (ok = wait(dq_free, 0, n))) {
        tc_fence_after();
        issue_dQ(1, (blocks - 1) & 1);
      }
      mma_commit_w(mma_done);
      mma_commit_w(drain);
      drain_wait(drain, 0);
    }
  } else if (warp < 8) {
    // ------------------- P and dS: 32 keys per warp, 32 query columns per warpgroup, in fragment order
    const int g = warp >> 2;
    const int wq = warp & 3;
    const int kr = wq * 32 + lane;  // this lane's row where a lane owns one (stores, epilogue)
    const int key = n0 + kr;
    const int fr = lane >> 2, fc = 2 * (lane & 3);  // fragment row and column pair
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS1 = tmem + lane_base + L::COL_S + 32 * g;
    const uint32_t tDP = tmem + lane_base + L::COL_DP + 32 * g;
    constexpr uint32_t kUpper = 16u << 16;  // the warp's lanes 16-31
    const float sl2 = a.scale_log2;
    bool ok = true;
    int bh = bh0, blk_row = row0;
    for (int i = 0; i < n; ++i) {
      const int vs = i % VS;
      ok = __all_sync(0xffffffffu, wait_bar_c(s_full, i & 1, abort_flag, kRoleSoftmax, i) &&
                                       wait_bar_c(&v_full[vs], (i / VS) & 1, abort_flag, kRoleSoftmax, i));
      if (!ok) break;
      tc_fence_after();
      // Query column e of this warpgroup's 32 is masked for key k if e < k + cm0
      // (causal), or if k is past the end.
      const int cm0 = a.causal ? n0 + wq * 32 - off - blk_row - (i & 1) * 64 - 32 * g : -256;
      if (i & 1) next_block(bh, blk_row);
      const bool masked = cm0 + 31 > 0 || n0 + wq * 32 + 31 >= a.Sk;
      const float* vec = s_vec + vs * kDiffVec + 32 * g + fc;
      // Phase A: p1 = P_1^T, p2 = -lambda P_2^T (fp32, kept), W^T = p1 + p2 in
      // 16 bits over S_1^T.
      uint32_t p1[2][16], p2[2][16];
      tmem_ld_frag(tS1, p1[0]);
      tmem_ld_frag(tS1 + kUpper, p1[1]);
      tmem_ld_frag(tS1 + 64, p2[0]);
      tmem_ld_frag(tS1 + 64 + kUpper, p2[1]);
      tmem_ld_wait();
      reg_fence(p1[0]);
      reg_fence(p1[1]);
      reg_fence(p2[0]);
      reg_fence(p2[1]);
      {
        uint32_t w[2][8];
        auto block = [&](auto masked_t) {
          const uint64_t sl2x2 = f2(sl2, sl2);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t nla = *reinterpret_cast<const uint64_t*>(vec + 8 * j);
            const uint64_t nlb = *reinterpret_cast<const uint64_t*>(vec + 64 + 8 * j);
            const uint64_t nl = *reinterpret_cast<const uint64_t*>(vec + 128 + 8 * j);
#pragma unroll
            for (int re = 0; re < 4; ++re) {  // rows fr + 8 re
              const int hh = re >> 1, e = re & 1, at = 4 * j + 2 * e;
              float x0 = __uint_as_float(p1[hh][at]), x1 = __uint_as_float(p1[hh][at + 1]);
              float y0 = __uint_as_float(p2[hh][at]), y1 = __uint_as_float(p2[hh][at + 1]);
              if constexpr (decltype(masked_t)::value) {
                // Masked entries are exactly 0 (MUFU of -inf).
                const int k = fr + 8 * re;
                const int cm = n0 + wq * 32 + k >= a.Sk ? 32 : k + cm0;
                const bool h0 = 8 * j + fc < cm, h1 = 8 * j + fc + 1 < cm;
                x0 = h0 ? -INFINITY : x0;
                x1 = h1 ? -INFINITY : x1;
                y0 = h0 ? -INFINITY : y0;
                y1 = h1 ? -INFINITY : y1;
              }
              const uint64_t tx = fma2(f2(x0, x1), sl2x2, nla);
              const uint64_t ty = fma2(f2(y0, y1), sl2x2, nlb);
              uint64_t ey;
              f2_split(tx, x0, x1);
              const uint64_t ex = f2(ex2(x0), ex2(x1));
              if (!decltype(masked_t)::value && (re & 1)) {  // one pair in four on the FMA pipe
                ey = exp2_poly2(ty);
              } else {
                f2_split(ty, y0, y1);
                ey = f2(ex2(y0), ex2(y1));
              }
              ey = mul2(ey, nl);
              const uint64_t ww = add2(ex, ey);
              f2_split(ex, x0, x1);
              f2_split(ey, y0, y1);
              p1[hh][at] = __float_as_uint(x0), p1[hh][at + 1] = __float_as_uint(x1);
              p2[hh][at] = __float_as_uint(y0), p2[hh][at + 1] = __float_as_uint(y1);
              f2_split(ww, x0, x1);
              w[hh][2 * j + e] = pack2<BF16>(x0, x1);
            }
          }
        };
        if (masked)
          block(std::true_type{});
        else
          block(std::false_type{});
        tmem_st_frag(tS1, w[0]);  // this warpgroup's own columns of S_1, read above
        tmem_st_frag(tS1 + kUpper, w[1]);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(w_ready);
      // Phase B: dS_1 = p1 (dP - Delta_1), dS_2 = p2 (dP - Delta_2) in 16 bits,
      // into tensor memory over dP (the A operands of dK: 16 columns each) and
      // into swizzled shared memory (the A operands of dQ).
      ok = __all_sync(0xffffffffu, wait_bar_c(dp_full, i & 1, abort_flag, kRoleSoftmax, i));
      if (!ok) break;
      tc_fence_after();
      uint32_t dp[2][16];
      tmem_ld_frag(tDP, dp[0]);
      tmem_ld_frag(tDP + kUpper, dp[1]);
      tmem_ld_wait();
      reg_fence(dp[0]);
      reg_fence(dp[1]);
      // (dP(i) was issued after the dQ products that last read these buffers.)
      const uint32_t row1 = smem_u32(smem + L::OFF_DS + (i & 1) * L::BLK) + kr * 128;
      const uint32_t row2 = smem_u32(smem + L::OFF_DS2 + ((i & 1) ? 1 : (i & 2)) * L::BLK) + kr * 128;
      uint32_t d1[2][8], d2[2][8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t nda = *reinterpret_cast<const uint64_t*>(vec + 192 + 8 * j);
        const uint64_t ndb = *reinterpret_cast<const uint64_t*>(vec + 256 + 8 * j);
#pragma unroll
        for (int re = 0; re < 4; ++re) {
          const int hh = re >> 1, e = re & 1, at = 4 * j + 2 * e;
          auto two = [&](const uint32_t(&r)[2][16]) {
            return f2(__uint_as_float(r[hh][at]), __uint_as_float(r[hh][at + 1]));
          };
          const uint64_t g2 = two(dp);
          float x0, x1, y0, y1;
          f2_split(mul2(two(p1), add2(g2, nda)), x0, x1);
          f2_split(mul2(two(p2), add2(g2, ndb)), y0, y1);
          d1[hh][2 * j + e] = pack2<BF16>(x0, x1);
          d2[hh][2 * j + e] = pack2<BF16>(y0, y1);
        }
        const uint32_t sw = ((4 * g + j) ^ (kr & 7)) << 4;
        stsm_x4(row1 + sw, d1[0][2 * j], d1[0][2 * j + 1], d1[1][2 * j], d1[1][2 * j + 1]);
        stsm_x4(row2 + sw, d2[0][2 * j], d2[0][2 * j + 1], d2[1][2 * j], d2[1][2 * j + 1]);
      }
      tmem_st_frag(tDP, d1[0]);
      tmem_st_frag(tDP + kUpper, d1[1]);
      tmem_st_frag(tDP + 16, d2[0]);
      tmem_st_frag(tDP + 16 + kUpper, d2[1]);
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_ready);
    }
    // Epilogue: warpgroup 0 writes dK_c = scale * accumulator, warpgroup 1 dV
    // (or, of several parts, the fp32 accumulators: fa_diff_dkv joins them).
    if (ok && !*abort_flag) {
      const bool have = n > 0;
      if (!have || __all_sync(0xffffffffu, wait_bar(mma_done, 0, abort_flag, kRoleSoftmax, n))) {
        tc_fence_after();
#pragma unroll 1
        for (int x = 0; x < (g == 0 ? 4 : DV / 32); ++x) {  // 32 accumulator columns
          const int c = x >> 1;
          const int col = g == 0 ? 32 * (x & 1) : 32 * x;  // first column of the tensor
          uint16_t* dst = g == 0 ? reinterpret_cast<uint16_t*>(a.dk[c]) + b * a.dk_s[c][0] + key * a.dk_s[c][1] +
                                       hk * a.dk_s[c][2] + col
                                 : reinterpret_cast<uint16_t*>(a.dv) + b * a.dv_s[0] + key * a.dv_s[1] +
                                       hk * a.dv_s[2] + col;
          const int cols = g == 0 ? a.d : a.dv_cols;
          const float mul = g == 0 ? a.scale : 1.f;
          uint32_t v[32];
          if (have) {
            tmem_ld32(tmem + lane_base + (g == 0 ? L::COL_DK : L::COL_DV) + 32 * x, v);
            tmem_ld_wait();
            reg_fence(v);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
          if (a.dkv_part != nullptr) {
            // Keys past Sk have rows here too (Sk_pad).
            float4* f = reinterpret_cast<float4*>(
                a.dkv_part +
                (((static_cast<int64_t>(part) * a.B + b) * a.Hk + hk) * a.nkb * 128 + key) * (128 + DV) +
                (g == 0 ? 0 : 128) + 32 * x);
            if (checked(part < a.parts && key < a.nkb * 128, 515)) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                f[u] = make_float4(__uint_as_float(v[4 * u]), __uint_as_float(v[4 * u + 1]),
                                   __uint_as_float(v[4 * u + 2]), __uint_as_float(v[4 * u + 3]));
            }
          } else if (key < a.Sk && checked(b < a.B && hk < a.Hk, 512)) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2<BF16>(__uint_as_float(v[8 * u + 2 * e]) * mul, __uint_as_float(v[8 * u + 2 * e + 1]) * mul);
              if (col + 8 * u < cols) reinterpret_cast<uint4*>(dst)[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------- dQ drain (warps 8-11)
    const int wq = warp & 3;
    const int tr = wq * 32 + lane;  // TMEM lane = query row of the block
    const uint32_t tDQ = tmem + (static_cast<uint32_t>(wq * 32) << 16) + L::COL_DQ;
    int bh = bh0, r0 = row0;
    for (int u = 0; u < n; ++u) {  // one use of the dQ buffer per map and block
      if (!__all_sync(0xffffffffu, wait_bar_c(dq_full, u & 1, abort_flag, kRoleSoftmax, u))) break;
      tc_fence_after();
      const int c = u & 1;
      const int swap = (c & (u >> 1)) * 64;  // dQ_2 of an odd block: its halves have changed places
      uint32_t v[2][32];
      tmem_ld32(tDQ, v[0]);
      tmem_ld32(tDQ + 32, v[1]);
      tmem_ld_wait();
      reg_fence(v[0]);
      reg_fence(v[1]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dq_free);
      if (a.dq_part != nullptr) {
        if (checked(bh < a.B * a.H && r0 / 128 < a.nqb && kvb < a.nkb, 513)) {
          float4* dst = reinterpret_cast<float4*>(
              a.dq_part +
              (((static_cast<int64_t>(bh) * a.nqb + r0 / 128) * a.nkb + kvb) * 2 + c) * (128 * 64) + (tr ^ swap) * 64);
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[8 * p + e] = make_float4(__uint_as_float(v[p][4 * e]), __uint_as_float(v[p][4 * e + 1]),
                                           __uint_as_float(v[p][4 * e + 2]), __uint_as_float(v[p][4 * e + 3]));
        }
      } else {
        // Two boxes of 32 rows x 32 floats, one after the other through this
        // warp's 4 KB, in the 128-byte swizzled layout that tmDQ reads: row
        // r's 16-byte chunk e at r * 128 + ((e ^ (r % 8)) * 16), so a store
        // phase's eight lanes hit eight different bank groups.
        uint8_t* buf = smem + L::OFF_DQS + wq * 4096;
        const uint32_t rbase = smem_u32(buf) + lane * 128;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (lane == 0) bulk_wait_read0();  // the reduction that read this buffer last
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            st_shared_v4(rbase + ((e ^ (lane & 7)) << 4), v[p][4 * e], v[p][4 * e + 1], v[p][4 * e + 2],
                         v[p][4 * e + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int64_t row = c * acc_rows + static_cast<int64_t>(bh) * a.Sq_pad + r0 + ((32 * wq) ^ swap);
            if (checked(row + 32 <= 2 * acc_rows, 514)) tma_reduce_add_2d(&tmDQ, buf, 32 * p, static_cast<int>(row));
            bulk_commit();
          }
        }
      }
      if (c == 1) next_block(bh, r0);
    }
    // Let the TMA finish the last reductions before shared memory goes away.
    if (lane == 0) bulk_wait0();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

}  // namespace fa
