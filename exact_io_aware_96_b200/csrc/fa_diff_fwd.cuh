// fa_diff_fwd.cuh — differential attention forward for sm_100a (fa_diff_fwd):
//   P_c = softmax(scale Q_c K_c^T [+ mask]), c = 1, 2
//   O   = (P_1 - lambda P_2) V,
// with two query/key projections of head_dim D <= 64 per head, one value
// projection of width Dv <= 128, and a weight lambda per (batch, row, head)
// (or broadcast over any of them). Heads of q may share a key/value head.
//
// The two maps have row maxima and sums of their own, so the difference can
// only be taken at the end: O = O_1 / l_1 - lambda O_2 / l_2 with
// unnormalised O_c = sum_j 2^(x_cj - m_c) v_j. One CTA takes 128 query rows of
// one (batch, head) and runs both maps side by side, map c where the plain
// forward has its query tile t = c: while one map's softmax runs, the tensor
// core works on the other map's products, and V is read from memory and
// shared memory once for both. The difference is formed in the epilogue from
// the two accumulators in tensor memory; nothing of either map reaches device
// memory. For training, O_2 (16 bits) and both logsumexps are written too:
// with O they give both row terms of the backward.
//
// The online softmax and the exponentials (one pair in four on the FMA pipe
// where no entry is masked) are those of fa_fwd.cuh. The running maximum is
// raised in few blocks: the exponentials go ahead with the maximum of the blocks
// before, in one pass over S, and the two warps that share a row meet after
// them. The block's own maximum is not even taken: a half's sum of at most 256
// says that no P is above 2^8. A block that does ask for a raise (the first one
// always does) has its maximum taken and is passed over again.
//
// P_c is rounded to 16 bits as P V's operand (a second 16-bit term, as in the
// few-row form, would cost a second product). O's relative error in norm is then
// 2.4e-3 in bf16 and 3.2e-4 in fp16; rounding O alone gives 1.7e-3 and 2.1e-4.
//
// Warp roles (576 threads):
//   warps 8t + 4c + r  softmax of map t, key half c of every block, TMEM lanes
//              32r .. 32r + 31, one query row per thread
//   warp  16   TMA loader: Q_1, Q_2 once, then (K_1, K_2)_j and V_j into rings
//   warp  17   MMA issuer
// Tensor memory: [128t, 128t + 64) S_t of keys 0 .. 63, [128t + 64, 128t + 128)
//   S_t of keys 64 .. 127, then P_t of the whole block  [256 + t DV, + DV) O_t
// P_t lies over the second half's scores alone. The first half's are free once
// their warps have read them, so S_t(j + 1) of that half is made before P V(j),
// and its softmax runs under P V(j) and the second half's S_t(j + 1).
//
// What bounds it: per 128 x 128 block the products take 1820 tensor cycles (S in
// four N = 64 products of 195, P V in two of 520) and the softmax 2 x 128 x 128
// exponentials (2048 MUFU cycles, 1536 with a quarter of them moved to the FMA
// pipe) and 1500 issue slots per scheduler; a block takes about 2700. A map's
// chain of P V, the second half's S and softmax, and the hand-offs between them
// (a wake-up is about 300 cycles) overlaps the other map's and the first half's
// only. Measured at B = 1, H = 8, S = 8192, D = 64, DV = 128, bf16, causal, in
// bursts of launches at 1965 MHz: 198 to 203 us on several GPUs, 1015 to 1041
// TFLOP/s. (Launched for a second without a pause it takes 230 us: the power cap
// brings the clock to 1700 MHz.) Against 198: 208 with the maximum of every block
// taken, 212 with the first block's exponentials computed twice, 214 with the
// first half's next S made when all of P is there, 225 with S in one N = 128
// product after P V. Slower: 64-key
// blocks in two buffers per map (356 us), an issuing warp per map (299), the first
// half's warps taking 80 keys of the 128 (213 against 212), waits out of line (222
// against 208), P in columns of its own where DV = 64 leaves room (60 against 56),
// no exponentials on the FMA pipe, or three pairs in eight (210 and 215 against
// 208).
#pragma once

#include <type_traits>

#include "fa_common.cuh"
#include "fa_fwd.cuh"

namespace fa {

// Division by a number known at launch. With s = ceil(log2 d) and
// mul = ceil(2^(31 + s) / d) the error mul * d - 2^(31 + s) is below d <= 2^s,
// so floor(x * mul / 2^(31 + s)) = floor(x / d) for 0 <= x < 2^31. The index
// arithmetic at the head of the kernels took 1,600 cycles (0.8 us of a call)
// with the compiled integer division.
struct Div {
  uint32_t mul;
  int shift;
  int d;
};
__host__ __device__ inline Div make_div(int d) {
  int s = 0;
  while ((int64_t(1) << s) < d) ++s;
  return {static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d - 1) / d), 31 + s, d};
}
__host__ __device__ __forceinline__ int quo(int x, const Div& v) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(x)) * v.mul) >> v.shift);
}
// x = quotient * d + remainder; 64-bit indexes past 2^31 take the long way.
__host__ __device__ __forceinline__ int64_t quo_rem(int64_t x, const Div& v, int* rem) {
  const int64_t q = x >> 31 == 0 ? quo(static_cast<int>(x), v) : x / v.d;
  *rem = static_cast<int>(x - q * v.d);
  return q;
}

enum LamKind : int { kLamF16 = 0, kLamBF16 = 1, kLamF32 = 2 };

__device__ __forceinline__ float load_lam(const void* lam, int kind, int64_t at) {
  if (kind == kLamF32) return static_cast<const float*>(lam)[at];
  const uint16_t v = static_cast<const uint16_t*>(lam)[at];
  return kind == kLamBF16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
}

struct DiffFwdArgs {
  void* o;
  void* o2;  // may be null
  float* lse;  // fp32 [2][B][H][Sq]
  int64_t o_s[3], o2_s[3];  // element strides: batch, sequence, head
  const void* lam;
  int64_t lam_s[3];  // 0 where lambda is broadcast
  int lam_kind;
  const int* k_lens;  // keys of each batch entry (null: Sk for all)
  int B, H, Hk, Sq, Sk;
  int d, dv;  // columns of q and k (<= 64); of v and o (<= the kernel's DV)
  float scale_log2;
  int causal;
  int n_qblocks;  // ceil(Sq / 128)
  Div by_order;   // the faster dimension of the grid order: B x H with a causal mask, n_qblocks without
  Div by_H, by_group;
};

__device__ __forceinline__ int diff_keys(const int* k_lens, int b, int Sk) {
  return k_lens == nullptr ? Sk : max(0, min(k_lens[b], Sk));
}

// wait_bar with everything after the first try out of line: the roles' loops
// stay short enough to be fetched without a pause.
__device__ __noinline__ bool wait_bar_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int role,
                                           int iter) {
  return wait_bar(bar, parity, abort_flag, role, iter);
}
__device__ __forceinline__ bool wait_bar_c(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int role,
                                           int iter) {
  return sm100::mbar_try_wait(bar, parity) || wait_bar_slow(bar, parity, abort_flag, role, iter);
}

template <int DV>
struct DiffFwdLayout {
  static constexpr int kThreads = 576;
  static constexpr int kLoaderWarp = 16;
  static constexpr int kMmaWarp = 17;
  static constexpr int BLK = 128 * 128;  // one 128-row x 128-byte block
  static constexpr int VB = DV / 64;     // column blocks of V
  static constexpr int KS = 3;           // stages of (K_1, K_2)
  static constexpr int VS = DV == 128 ? 2 : 3;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * BLK;
  static constexpr int OFF_V = OFF_K + KS * 2 * BLK;
  static constexpr int OFF_PMAX = OFF_V + VS * VB * BLK;      // [parity][map][half][row]
  static constexpr int OFF_LSUM = OFF_PMAX + 2 * 2 * 2 * 128 * 4;  // [map][half][row]
  static constexpr int OFF_M = OFF_LSUM + 2 * 2 * 128 * 4;    // [map][row]
  static constexpr int OFF_BAR = OFF_M + 2 * 128 * 4;
  // q_full, k_full/k_empty[KS], v_full/v_empty[VS], s_full[2][2], s_free[2], p_full[2], o_final[2], drain
  static constexpr int NBAR = 1 + 2 * KS + 2 * VS + 10 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static constexpr int SMEM_ALLOC = BYTES + 1024;
  static constexpr int TMEM_COLS = 512;
  static constexpr int OBASE = 256;
};

template <int DV, bool BF16>
__global__ void __launch_bounds__(576, 1)
    fa_diff_fwd_kernel(const __grid_constant__ CUtensorMap tmQ1, const __grid_constant__ CUtensorMap tmQ2,
                       const __grid_constant__ CUtensorMap tmK1, const __grid_constant__ CUtensorMap tmK2,
                       const __grid_constant__ CUtensorMap tmV, const DiffFwdArgs a) {
  using L = DiffFwdLayout<DV>;
  using namespace sm100;
  constexpr int KS = L::KS, VS = L::VS;
  static_assert(L::SMEM_ALLOC <= 232448, "smem budget");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + KS;
  uint64_t* v_full = k_empty + KS;
  uint64_t* v_empty = v_full + VS;
  uint64_t* s_full = v_empty + VS;
  uint64_t* s_free = s_full + 4;
  uint64_t* p_full = s_free + 2;
  uint64_t* o_final = p_full + 2;
  uint64_t* drain = o_final + 2;
  float* pmax = reinterpret_cast<float*>(smem + L::OFF_PMAX);
  float* lsum = reinterpret_cast<float*>(smem + L::OFF_LSUM);
  float* msm = reinterpret_cast<float*>(smem + L::OFF_M);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // Grid order as the plain forward's: with a causal mask rank-major over
  // (b, h), the last query blocks (the most key blocks) first; without one
  // head-major, so that the running CTAs share a few heads' K and V in L2.
  const int outer = quo(blockIdx.x, a.by_order), inner = static_cast<int>(blockIdx.x) - outer * a.by_order.d;
  const int rank = a.causal ? outer : inner;
  const int hb = a.causal ? inner : outer;
  const int b = quo(hb, a.by_H);
  const int h = hb - b * a.H;
  const int hk = quo(h, a.by_group);
  const int q0 = (a.causal ? a.n_qblocks - 1 - rank : rank) * 128;
  const int sk = diff_keys(a.k_lens, b, a.Sk);
  const int n = fwd_kv_blocks(q0, a.Sq, sk, a.causal);
  checked(q0 < a.Sq && b < a.B && hk < a.Hk, 401);

  // The loader's thread sets the barriers up itself and asks for Q and the
  // first keys at once, while the MMA warp allocates tensor memory.
  if (warp == L::kLoaderWarp && lane == 0) {
    prefetch_tmap(&tmQ1);
    prefetch_tmap(&tmQ2);
    prefetch_tmap(&tmK1);
    prefetch_tmap(&tmK2);
    prefetch_tmap(&tmV);
    mbar_init(q_full, 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[2 * t], 1);
      mbar_init(&s_full[2 * t + 1], 1);
      mbar_init(&s_free[t], 4);  // one arrival per warp of the first half
      mbar_init(&p_full[t], 8);  // one arrival per softmax warp of the map
      mbar_init(&o_final[t], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (n > 0) {
      mbar_arrive_expect_tx(q_full, 2 * L::BLK);
      tma_load_4d(smem + L::OFF_Q, &tmQ1, q_full, 0, q0, h, b);
      tma_load_4d(smem + L::OFF_Q + L::BLK, &tmQ2, q_full, 0, q0, h, b);
      mbar_arrive_expect_tx(&k_full[0], 2 * L::BLK);
      tma_load_4d(smem + L::OFF_K, &tmK1, &k_full[0], 0, 0, hk, b);
      tma_load_4d(smem + L::OFF_K + L::BLK, &tmK2, &k_full[0], 0, 0, hk, b);
    }
  }
  if (warp == L::kMmaWarp) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == L::kLoaderWarp) {
    // ------------------------------------------------------------ loader
    if (lane == 0 && n > 0) {
      int nk = 0, nv = 0;  // loads issued
      for (int j = 0; j < n; ++j) {
        const int ks = j % KS, vs = j % VS;
        checked(j * 128 < sk, 402);
        if (j > 0) {
          if (!wait_bar(&k_empty[ks], ((j / KS) & 1) ^ 1, abort_flag, kRoleLoader, j)) break;
          mbar_arrive_expect_tx(&k_full[ks], 2 * L::BLK);
          tma_load_4d(smem + L::OFF_K + ks * 2 * L::BLK, &tmK1, &k_full[ks], 0, j * 128, hk, b);
          tma_load_4d(smem + L::OFF_K + (ks * 2 + 1) * L::BLK, &tmK2, &k_full[ks], 0, j * 128, hk, b);
        }
        ++nk;
        if (!wait_bar(&v_empty[vs], ((j / VS) & 1) ^ 1, abort_flag, kRoleLoader, j)) break;
        mbar_arrive_expect_tx(&v_full[vs], L::VB * L::BLK);
        for (int vb = 0; vb < L::VB; ++vb)
          tma_load_4d(smem + L::OFF_V + (vs * L::VB + vb) * L::BLK, &tmV, &v_full[vs], vb * 64, j * 128, hk, b);
        ++nv;
      }
      if (*abort_flag) {
        // Let the copies already issued land before the CTA exits.
        drain_wait(q_full, 0);
        for (int j = max(0, nk - KS); j < nk; ++j) drain_wait(&k_full[j % KS], (j / KS) & 1);
        for (int j = max(0, nv - VS); j < nv; ++j) drain_wait(&v_full[j % VS], (j / VS) & 1);
      }
    }
  } else if (warp == L::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (n > 0) {
      auto wait = [&](uint64_t* bar, uint32_t parity, int iter) {
        return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, kRoleMma, iter));
      };
      constexpr uint32_t idS = idesc_f16(BF16, 128, 64, 0, 0);
      // Narrow heads: S over the 16-column steps that D reaches, P V for the
      // columns that Dv reaches (D = 40, Dv = 80: a third less tensor time).
      const int d_steps = (a.d + 15) / 16;
      const uint32_t idO = idesc_f16(BF16, 128, (a.dv + 15) & ~15, 0, 1);
      const uint32_t sQ = smem_u32(smem + L::OFF_Q);
      const uint32_t sK = smem_u32(smem + L::OFF_K);
      const uint32_t sV = smem_u32(smem + L::OFF_V);
      auto issue_S = [&](int t, int hf, int ks) {
        const uint64_t qd = desc_sw128(sQ + t * L::BLK, 16, 1024);
        const uint64_t kd = desc_sw128(sK + (ks * 2 + t) * L::BLK + hf * (L::BLK / 2), 16, 1024);
        uint64_t ad[4], bd[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          ad[u] = desc_add(qd, u * 32);
          bd[u] = desc_add(kd, u * 32);
        }
        mma_ss_up_to_4(tmem + 128 * t + 64 * hf, ad, bd, idS, 0, d_steps);
        mma_commit_w(&s_full[2 * t + hf]);
      };
      auto issue_PV = [&](int t, int vs, int acc) {
        const uint64_t vd = desc_sw128(sV + vs * L::VB * L::BLK, L::BLK, 1024);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pa[4];
          uint64_t vb[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            pa[u] = tmem + 128 * t + 64 + 32 * hf + u * 8;
            vb[u] = desc_add(vd, (4 * hf + u) * 2048);
          }
          mma_ts_x4(tmem + L::OBASE + t * DV, pa, vb, idO, (acc || hf > 0) ? 1u : 0u);
        }
      };
      bool ok = wait(q_full, 0, -1) && wait(&k_full[0], 0, 0);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < 2; ++t) {
          issue_S(t, 0, 0);
          issue_S(t, 1, 0);
        }
        mma_commit_w(&k_empty[0]);
      }
      for (int j = 0; ok && j < n; ++j) {
        const int vs = j % VS;
        const int jn = j + 1, ksn = jn % KS;
        if (!(ok = wait(&v_full[vs], (j / VS) & 1, j))) break;
        if (jn < n && !(ok = wait(&k_full[ksn], (jn / KS) & 1, jn))) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok) break;
          if (jn < n) {
            if (!(ok = wait(&s_free[t], j & 1, j))) break;
            tc_fence_after();
            issue_S(t, 0, ksn);
          }
          if (!(ok = wait(&p_full[t], j & 1, j))) break;
          tc_fence_after();
          issue_PV(t, vs, j > 0);
          if (j == n - 1) mma_commit_w(&o_final[t]);
          if (t == 1) mma_commit_w(&v_empty[vs]);
          if (jn < n) {
            issue_S(t, 1, ksn);
            if (t == 1) mma_commit_w(&k_empty[ksn]);
          }
        }
      }
      // Wait for every MMA this warp issued before TMEM is released.
      mma_commit_w(drain);
      drain_wait(drain, 0);
    }
  } else {
    // ------------------------------------------------------- softmax / epilogue
    const int t = warp >> 3;            // map
    const int c = (warp >> 2) & 1;      // key half of every block
    const int quarter = warp & 3;       // TMEM lane quarter
    const int r = quarter * 32 + lane;  // row within the tile
    const int row = q0 + r;
    const int pair_bar = 1 + t * 4 + quarter;  // named barrier of the two warps that share these rows
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + 128 * t + 64 * c;
    const uint32_t tP = tmem + lane_base + 128 * t + 64 + 32 * c;
    const uint32_t tO = tmem + lane_base + L::OBASE + t * DV + c * (DV / 2);  // the half this warp rescales
    const float sl2 = a.scale_log2;
    const int off = sk - a.Sq;
    float m = -INFINITY;  // running max of x = s * scale * log2(e), the same in both halves
    float l = 0.f;        // this half's running sum of 2^(x - m)
    bool ok = true;

    for (int j = 0; j < n; ++j) {
      // `ok` false here: a wait of the previous block ran out; this warp goes
      // straight to the pair barrier, which then ends both warps.
      const bool ready = ok && __all_sync(0xffffffffu, wait_bar(&s_full[2 * t + c], j & 1, abort_flag, kRoleSoftmax, j));
      const int k0 = j * 128 + 64 * c;  // first key of this half
      const bool masked = k0 + 64 > sk || (a.causal && k0 + 63 > q0 + off);
      int lim = sk - 1 - k0;  // last allowed column of this half
      if (a.causal) lim = min(lim, row + off - k0);
      float* slot = pmax + (((j & 1) * 2 + t) * 2) * 128;
      const uint64_t sl2x2 = f2(sl2, sl2);
      float add = 0.f;
      uint32_t pw[2][16];  // P, two keys to a word
      // P and its sum in one pass over this half's S, 32 columns at a time, with
      // the maximum of the blocks before; returns whether that maximum will do.
      auto pass = [&](auto masked_t) -> bool {
        constexpr bool M = decltype(masked_t)::value;
        const float mu = (m == -INFINITY) ? 0.f : m;
        const uint64_t negmu2 = f2(-mu, -mu);
        uint64_t acc0 = f2(0.f, 0.f), acc1 = f2(0.f, 0.f);
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t sv[32];
          tmem_ld32(tS + 32 * q, sv);
          tmem_ld_wait();
          reg_fence(sv);
          if constexpr (!M) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (fwd_pair_on_fma(i)) mx = max3(mx, __uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
          }
          fwd_exp32<BF16, M, true>(sv, 32 * q, lim, sl2x2, negmu2, acc0, acc1, pw[q]);
        }
        float a0, a1;
        f2_split(add2(acc0, acc1), a0, a1);
        add = a0 + a1;
        return m != -INFINITY && fabsf(add) <= 256.f && !(mx * sl2 > m + 8.f);
      };
      bool keep = false;  // the first block has no maximum to go ahead with
      if (ready && j > 0) {
        tc_fence_after();
        keep = masked ? pass(std::true_type{}) : pass(std::false_type{});
      }
      // The maximum is raised in few blocks. So the exponentials above have gone
      // ahead with the old one, and the two warps meet afterwards, when neither
      // has to wait long. While a half's sum is at most 256, each of its P is: no
      // row maximum is needed to know that the old one will do. (A pair on the
      // FMA pipe may be anything past 2^128; its scores are looked at. A NaN there
      // makes the sum huge, one elsewhere makes it NaN.) If a row of either half
      // asks for a raise, the block's maximum is taken, O_t is rescaled and the
      // pass is made again, on the MUFU unit alone, which keeps a NaN.
      tc_fence_before();
      if (!named_bar_and(pair_bar, 64, keep)) {
        const bool in = ready && __all_sync(0xffffffffu, wait_bar(&s_full[2 * t + 1], j & 1, abort_flag, kRoleSoftmax, j));
        tc_fence_after();
        float pm = -INFINITY;
        if (in) {
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t sv[32];
            tmem_ld32(tS + 32 * q, sv);
            tmem_ld_wait();
            reg_fence(sv);
            float mx0 = -INFINITY, mx1 = -INFINITY;
            auto xf = [&](int i) { return 32 * q + i <= lim ? __uint_as_float(sv[i]) : -INFINITY; };
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              mx0 = max3(mx0, xf(i), xf(i + 1));
              mx1 = max3(mx1, xf(i + 2), xf(i + 3));
            }
            pm = max3(pm, mx0, mx1);
          }
          // Written again in block j + 2 at the earliest, after the partner has
          // passed a barrier of block j + 1, i.e. after it has read this value.
          slot[c * 128 + r] = pm;
        }
        if (!named_bar_and(pair_bar, 64, in)) {
          ok = false;
          break;
        }
        const float m_blk = fmaxf(pm, slot[(c ^ 1) * 128 + r]) * sl2;
        float alpha = 1.f;
        if (m_blk > m) {
          alpha = ex2(m - m_blk);  // 0 when m was -inf
          m = m_blk;
        }
        l *= alpha;
        // The second half's S_t(j) was issued after P_t(j-1) V_{j-1}, so its
        // barrier covers both and O_t may be rescaled now.
        if (j > 0) {
#pragma unroll 1
          for (int q = 0; q < DV / 64; ++q) {
            uint32_t ov[32];
            tmem_ld32(tO + 32 * q, ov);
            tmem_ld_wait();
            reg_fence(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(tO + 32 * q, ov);
          }
        }
        pass(std::true_type{});
        tc_fence_before();
        named_bar_and(pair_bar, 64, true);
      }
      tc_fence_after();
      if (c == 0 && lane == 0 && j + 1 < n) mbar_arrive(&s_free[t]);
      l += add;
      tmem_st16(tP, pw[0]);  // over the second half's S, which the pair has read
      tmem_st16(tP + 16, pw[1]);
      if (t == 0 && a.k_lens != nullptr && j == n - 1 && (j + 1) * 128 > sk) {
        // V rows past this sequence's last key (whatever a cache holds there)
        // become zeros before P V reads them: their P is 0, but 0 x inf is
        // not. Both products read V after map 1's warps have arrived below.
        if (!__all_sync(0xffffffffu,
                        wait_bar(&v_full[j % VS], (j / VS) & 1, abort_flag, kRoleSoftmax, j))) {
          ok = false;  // the epilogue's barrier ends every warp
          continue;
        }
        uint8_t* vt = smem + L::OFF_V + (j % VS) * L::VB * L::BLK;
        for (int i = threadIdx.x; i < L::VB * 128 * 8; i += 256) {  // 16-byte chunks, 8 to a row
          const int vr = (i >> 3) & 127;
          if (j * 128 + vr >= sk)
            st_shared_v4(smem_u32(vt + (i >> 10) * L::BLK + vr * 128 + (i & 7) * 16), 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
    }

    // Epilogue: all 16 warps meet with both maps' sums; each warpgroup then
    // writes a quarter of the columns from both accumulators.
    lsum[(t * 2 + c) * 128 + r] = l;
    if (c == 0) msm[t * 128 + r] = m;
    const bool valid = row < a.Sq;
    const bool has = sk > 0 && (!a.causal || row + off >= 0);  // some key is allowed (the same in both maps)
    const float lam = valid && has ? load_lam(a.lam, a.lam_kind, b * a.lam_s[0] + row * a.lam_s[1] + h * a.lam_s[2])
                                   : 0.f;  // asked for here: it arrives while the warps meet
    constexpr int kAllBar = 9;
    bool go = named_bar_and(kAllBar, 512, ok && !*abort_flag);
    const int wg = warp >> 2;
    constexpr int NC = DV / 4;  // columns of one warpgroup
    const int cb = wg * NC;
    if (go && n > 0) {
      go = __all_sync(0xffffffffu, wait_bar(&o_final[0], 0, abort_flag, kRoleSoftmax, n) &&
                                       wait_bar(&o_final[1], 0, abort_flag, kRoleSoftmax, n));
      tc_fence_after();
    }
    if (go) {
      const float l1 = lsum[r] + lsum[128 + r], l2 = lsum[256 + r] + lsum[384 + r];
      const float m1 = msm[r], m2 = msm[128 + r];
      const float inv1 = has ? 1.f / l1 : 0.f, inv2 = has ? 1.f / l2 : 0.f;
      uint32_t o1[NC], o2[NC];
      if (n > 0) {
        const uint32_t t1 = tmem + lane_base + L::OBASE + cb;
        if constexpr (NC == 32) {
          tmem_ld32(t1, o1);
          tmem_ld32(t1 + DV, o2);
        } else {
          tmem_ld16(t1, o1);
          tmem_ld16(t1 + DV, o2);
        }
        tmem_ld_wait();
        reg_fence(o1);
        reg_fence(o2);
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) o1[i] = o2[i] = 0u;
      }
      // A row's quarter goes through shared memory (Q's, read for the last time
      // above; 16-byte chunks swizzled so that neither side meets a bank
      // conflict): straight from the registers a warp's store would touch 32
      // rows' lines at 16 bytes each, from here it writes 8 rows of 64 bytes.
      constexpr int CH = NC / 8, RPI = 32 / CH;  // chunks of a row, rows of one store
      const int wrow = row - lane;               // the warp's first row
      uint8_t* stage = smem + L::OFF_Q + warp * 32 * NC * 2;
      auto slot = [&](int rr, int ch) {
        return reinterpret_cast<uint4*>(stage + rr * NC * 2 + ((ch ^ (rr / (8 / CH) & (CH - 1))) << 4));
      };
      auto store_rows = [&](void* base, const int64_t* st) {
        uint16_t* ob = reinterpret_cast<uint16_t*>(base) + b * st[0] + h * st[2] + cb;
        const int ch = lane % CH;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int rr = i * RPI + lane / CH, gr = wrow + rr;
          const uint4 w = *slot(rr, ch);
          if (gr < a.Sq && cb + 8 * ch < a.dv && checked(b < a.B && h < a.H, 403))
            *reinterpret_cast<uint4*>(ob + gr * st[1] + 8 * ch) = w;
        }
        __syncwarp();
      };
      if (a.o2 != nullptr) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x = 8 * i + 2 * e;
            w[e] = has ? pack2<BF16>(__uint_as_float(o2[x]) * inv2, __uint_as_float(o2[x + 1]) * inv2) : 0u;
          }
          *slot(lane, i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        store_rows(a.o2, a.o2_s);
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = 8 * i + 2 * e;
          const float x0 = __uint_as_float(o1[x]) * inv1 - lam * (__uint_as_float(o2[x]) * inv2);
          const float x1 = __uint_as_float(o1[x + 1]) * inv1 - lam * (__uint_as_float(o2[x + 1]) * inv2);
          w[e] = has ? pack2<BF16>(x0, x1) : 0u;
        }
        *slot(lane, i) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      store_rows(a.o, a.o_s);
      if (valid) {
        if (wg < 2) {  // warpgroup 0 writes map 1's LSE, warpgroup 1 map 2's
          const float lm = wg ? m2 : m1, ll = wg ? l2 : l1;
          a.lse[((static_cast<int64_t>(wg) * a.B + b) * a.H + h) * a.Sq + row] =
              has ? (lm + __log2f(ll)) * 0.69314718055994531f : -INFINITY;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

}  // namespace fa
