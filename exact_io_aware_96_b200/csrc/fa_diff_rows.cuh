// fa_diff_rows.cuh — differential attention forward of few query rows over many
// keys (decoding: one or a few new tokens over a key/value cache).
//
// The same mathematics as fa_diff_fwd.cuh. With R = (H / Hk) * Sq rows per key
// head and R small, the call is bound by reading K_1, K_2 and V once, so the
// kernel is built around that stream. The lengths of the sequences are known on
// the device only, so the work is cut there: all keys of all batch entries, in
// units of 64, form one line that is divided evenly among teams of CTAs, one CTA
// of a team per (key head, 16 rows). A team's stretch of the line covers a run
// of keys of one batch entry, or of a few neighbouring ones ("pieces"); its CTAs
// read neighbouring heads of the same keys, which lie side by side in memory.
// All rows that share a key head form one 16-row operand of m16n8k16 products, so shared heads read their
// keys once. A CTA has four streams of two warps, one warp per map. Each stream
// takes every fourth 16-key tile through a ring of NS stages filled by TMA (a
// lane of its first warp issues the loads; both warps wait on the stage's
// mbarrier and hand it back through another: no producer warp, no block-wide
// barrier in the loop), and each warp keeps its map's running maximum, sum and
// unnormalised O. The streams' results join in shared memory, the pieces' in a
// second small kernel (fa_diff_rows_join), both by the online softmax's
// rescaling. Two CTAs share an SM, so one's start and end overlap the other's
// stream. Calls of many batch entries and heads, or of short caches, need no
// second kernel ("direct"): one CTA takes all keys of its entry and writes the
// result, or a cluster of 2, 4 or 8 does. Each of its CTAs then takes a run of
// units, leaves its piece in its shared memory, and adds up a share of the row
// tile over all of the cluster's pieces.
//
// P is split into two 16-bit terms, p = hi + lo, and multiplied with V twice:
// the tensor cores have time to spare here, and O keeps the fp32 accuracy of P.
//
// Measured (D = 64, DV = 128, bf16): one row of 8 heads over 65,536 keys, 51 us
// and 5.3 TB/s for the main kernel, 82% of the copy rate, 54 us with the join; 32
// sequences of 2,200 to 8,100 keys, 16 query and 4 key heads, 68 us with the join,
// 5.0 TB/s. A grid of fixed runs of keys took 88 us where this one took 79 (the
// lengths leave it uneven), one warp for both maps the same time at 253 registers.
#pragma once

#include "fa_common.cuh"
#include "fa_diff_fwd.cuh"

namespace fa {

struct DiffRowsArgs {
  const uint16_t* q[2];
  int64_t q_s[2][3];
  void* o;
  void* o2;
  float* lse;
  int64_t o_s[3], o2_s[3];
  const void* lam;
  int64_t lam_s[3];
  int lam_kind;
  const int* k_lens;
  int B, H, Hk, Sq, Sk;
  int d, dv;
  float scale_log2;
  int causal;
  int R, n_mt;   // query rows of a key head, ceil(R / 16)
  int teams;     // 0: direct
  int cluster;   // direct: CTAs that share an entry's keys (1, 2, 4 or 8)
  // A piece (batch entry b, team t) has slot b + t: along the line one of the two
  // grows from piece to piece.
  float* part_o;    // [slot][hk, row][2][DV]: a piece's unnormalised O_c
  float2* part_ml;  // [slot][hk, row][2]: its (m, l)
};

// The line of 64-key units. Every lane of a warp calls these together.
__device__ __forceinline__ int64_t rows_units(const DiffRowsArgs& a, int b) {
  return b < a.B ? (diff_keys(a.k_lens, b, a.Sk) + 63) / 64 : 0;
}
__device__ __forceinline__ int64_t rows_warp_sum(int64_t v) {
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
  return v;
}
// Units of the batch entries before `b`.
__device__ __forceinline__ int64_t rows_before(const DiffRowsArgs& a, int b) {
  if (a.k_lens == nullptr) return static_cast<int64_t>(b) * ((a.Sk + 63) / 64);
  int64_t v = 0;
  for (int x = threadIdx.x & 31; x < b; x += 32) v += rows_units(a, x);
  return rows_warp_sum(v);
}
// Teams that get work: each at least two units.
__device__ __forceinline__ int rows_teams(const DiffRowsArgs& a, int64_t total) {
  return static_cast<int>(min(static_cast<int64_t>(a.teams), max(static_cast<int64_t>(1), (total + 1) / 2)));
}
// The batch entry that holds unit `at` of the line, and the units before it.
__device__ __forceinline__ int rows_find(const DiffRowsArgs& a, int64_t at, int64_t& before) {
  before = 0;
  for (int base = 0; base < a.B; base += 32) {
    const int64_t mine = rows_units(a, base + static_cast<int>(threadIdx.x & 31));
    const int64_t all = rows_warp_sum(mine);
    if (at < before + all) {
      for (int x = 0; x < 32; ++x) {  // which of the 32
        const int64_t u = __shfl_sync(0xffffffffu, mine, x);
        if (at < before + u) return base + x;
        before += u;
      }
    }
    before += all;
  }
  return a.B;
}

template <int DV>
struct DiffRowsLayout {
  static constexpr int KT = 16;  // keys of a tile
  static constexpr int NS = 3;   // stages of a warp's ring
  static constexpr int VB = DV / 64;
  static constexpr int TILE = KT * 128 * (2 + VB);  // K_1, K_2, V column blocks
  static constexpr int RING = 4 * NS * TILE;
  // The join's partial results [warp][map][16][DV + 4] reuse the ring.
  static constexpr int OROW = DV + 4;
  static constexpr int JOIN = 4 * 2 * 16 * OROW * 4;
  // A clustered CTA's piece [map][16][DV], behind it.
  static constexpr int OFF_PIECE = JOIN;
  static_assert(OFF_PIECE + 2 * 16 * DV * 4 <= RING, "the piece lies in the ring");
  static constexpr int OFF_ML = RING > JOIN ? RING : JOIN;  // [warp][map][16] (m, l)
  static constexpr int OFF_PML = OFF_ML + 4 * 2 * 16 * 8;  // the piece's [map][16] (m, l)
  static constexpr int OFF_BAR = OFF_PML + 2 * 16 * 8;  // full, empty [stream][stage]
  static constexpr int OFF_MISC = OFF_BAR + 2 * 4 * NS * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static constexpr int SMEM_ALLOC = BYTES + 1024;
};

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The cluster's barrier in two halves, and its shared memory.
__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_at(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// What a finished row writes: O, O_2 and both LSEs from both maps' sums.
// x1, x2: N unnormalised columns from `col` on.
template <int N, bool BF16, typename Args>
__device__ __forceinline__ void diff_row_out(const Args& a, int b, int h, int row, int col, bool has, const float* x1,
                                             const float* x2, float l1, float l2) {
  using namespace sm100;
  const float lam =
      has ? load_lam(a.lam, a.lam_kind, b * a.lam_s[0] + row * a.lam_s[1] + h * a.lam_s[2]) : 0.f;
  const float i1 = has ? 1.f / l1 : 0.f, i2 = has ? 1.f / l2 : 0.f;
  uint32_t* po = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.o) + b * a.o_s[0] + row * a.o_s[1] +
                                             h * a.o_s[2] + col);
  uint32_t* po2 = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.o2) + b * a.o2_s[0] + row * a.o2_s[1] +
                                              h * a.o2_s[2] + col);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const float y0 = has ? x2[e] * i2 : 0.f, y1 = has ? x2[e + 1] * i2 : 0.f;
    const float z0 = has ? x1[e] * i1 : 0.f, z1 = has ? x1[e + 1] * i1 : 0.f;
    if (col + e < a.dv) {
      po[e / 2] = pack2<BF16>(z0 - lam * y0, z1 - lam * y1);
      if (a.o2 != nullptr) po2[e / 2] = pack2<BF16>(y0, y1);
    }
  }
}

template <int DV, bool BF16, bool CLUSTER>
__global__ void __launch_bounds__(256, 2)
    fa_diff_rows_kernel(const __grid_constant__ CUtensorMap tmK1, const __grid_constant__ CUtensorMap tmK2,
                        const __grid_constant__ CUtensorMap tmV, const DiffRowsArgs a) {
  using L = DiffRowsLayout<DV>;
  using namespace sm100;
  constexpr int KT = L::KT, NS = L::NS, NT = DV / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  float2* ml = reinterpret_cast<float2*>(smem + L::OFF_ML);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC);
  const int stream = threadIdx.x >> 6, c = (threadIdx.x >> 5) & 1;  // c: the warp's map
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;  // fragment row group and column pair

  const int T = CLUSTER ? a.cluster : 1, rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int item = CLUSTER ? static_cast<int>(blockIdx.x) / T : static_cast<int>(blockIdx.x);
  const int mt = item % a.n_mt;
  const int hk = item / a.n_mt % a.Hk;
  const int team = item / a.n_mt / a.Hk;  // direct: the batch entry
  const int group = a.H / a.Hk;
  const bool direct = CLUSTER || a.teams == 0;
  // The stretch of the line: units [at, end), `before` the units of entries before b.
  int b = team;
  int64_t at = 0, end = 1, before = 0;
  if (!direct) {
    const int64_t total = rows_before(a, a.B);
    const int teams = rows_teams(a, total);
    at = team < teams ? total * team / teams : 0;
    end = team < teams ? total * (team + 1) / teams : 0;
    if (at < end) b = rows_find(a, at, before);
    if (b >= a.B) at = end;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4 * NS; ++i) {
      mbar_init(&bars[i], 1);
      mbar_init(&bars[4 * NS + i], 2);  // one arrival per map's warp
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  uint64_t* full = bars + stream * NS;
  uint64_t* empty = bars + (4 + stream) * NS;
  uint8_t* ring = smem + stream * NS * L::TILE;
  const float sl2 = a.scale_log2;
  // ldmatrix row addresses: K, matrices = 16-byte chunks 0-3 of 8 keys; V,
  // matrices = (keys 0-7, 8-15) x (chunk, chunk + 1), transposed.
  const int kr = lane & 7, km = lane >> 3;
  const int vr = (km & 1) * 8 + kr, vm = km >> 1;
  int used = 0;  // tiles of this stream in earlier pieces

  while (at < end) {
    const int len = diff_keys(a.k_lens, b, a.Sk);
    const int64_t units = (len + 63) / 64;
    const int lo = CLUSTER  ? static_cast<int>(units * rank / T) * 64
                   : direct ? 0
                            : static_cast<int>(at - before) * 64;
    const int hi = CLUSTER  ? min(len, static_cast<int>(units * (rank + 1) / T) * 64)
                   : direct ? len
                            : static_cast<int>(min(static_cast<int64_t>(len), (end - before) * 64));
    const int tiles = hi > lo ? (hi - lo + KT - 1) / KT : 0;
    const int mine = tiles > stream ? (tiles - stream + 3) / 4 : 0;  // this stream's tiles: stream, stream + 4, ...
    checked(b < a.B && mt * 16 < a.R, 601);
    auto issue = [&](int i) {  // one lane: tile i of this stream into its stage
      const int st = (used + i) % NS, key = lo + (stream + 4 * i) * KT;
      uint8_t* dst = ring + st * L::TILE;
      checked(key < a.Sk, 602);
      mbar_arrive_expect_tx(&full[st], L::TILE);
      tma_load_4d(dst, &tmK1, &full[st], 0, key, hk, b);
      tma_load_4d(dst + KT * 128, &tmK2, &full[st], 0, key, hk, b);
#pragma unroll
      for (int vb = 0; vb < L::VB; ++vb) tma_load_4d(dst + (2 + vb) * KT * 128, &tmV, &full[st], vb * 64, key, hk, b);
    };
    const bool loads = c == 0 && lane == 0;
    bool fed = true;  // false in the loading lane once its wait for a free stage has run out
    int issued = 0;
    if (loads)
      for (; issued < min(NS, mine); ++issued) issue(issued);

    // Row r of the tile: query row i = r % Sq of head hk * group + r / Sq.
    int lim[2];  // last key that rows g and g + 8 see
    uint32_t qf[4][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = mt * 16 + g + 8 * e;
      const int i = r % a.Sq, h = hk * group + r / a.Sq;
      lim[e] = a.causal && r < a.R ? i + len - a.Sq : len - 1;  // rows past R are not written
      const uint16_t* p = (c ? a.q[1] : a.q[0]) + b * a.q_s[c][0] + i * a.q_s[c][1] + h * a.q_s[c][2];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int col = ks * 16 + x * 8 + 2 * tq;
          qf[ks][2 * x + e] = r < a.R && col < a.d ? *reinterpret_cast<const uint32_t*>(p + col) : 0u;
        }
    }
    const int min_lim = __reduce_min_sync(0xffffffffu, min(lim[0], lim[1]));
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g, g + 8
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    for (int i = 0; i < mine; ++i) {
      const int st = (used + i) % NS, key0 = lo + (stream + 4 * i) * KT;
      const uint32_t ph_st = ((used + i) / NS) & 1;
      if (!__all_sync(0xffffffffu, fed && wait_bar_c(&full[st], ph_st, abort_flag, kRoleSoftmax, i))) break;
      uint8_t* tile = ring + st * L::TILE;
      const uint32_t sk = smem_u32(tile) + c * KT * 128, sv = smem_u32(tile) + 2 * KT * 128;
      if (key0 + KT > len) {
        // Rows past the end count nothing, whatever they hold. (Both warps of the
        // stream write the same zeros, each for itself; it is the last tile.)
        for (int x = lane; x < L::VB * KT * 8; x += 32)
          if (key0 + ((x >> 3) & (KT - 1)) >= len) st_shared_v4(sv + x * 16, 0, 0, 0, 0);
        __syncwarp();
      }
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const int row = n * 8 + kr;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t f[4];
          ldsm_x4(f, sk + row * 128 + (((hf * 4 + km) ^ (row & 7)) << 4));
          mma16816<BF16>(s[n], qf[2 * hf], f[0], f[1]);
          mma16816<BF16>(s[n], qf[2 * hf + 1], f[2], f[3]);
        }
      }
      const bool masked = key0 + KT - 1 > min_lim;
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (masked) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (key0 + n * 8 + 2 * tq + x > lim[e]) s[n][2 * e + x] = -INFINITY;
        }
        float mx = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx *= sl2;
        // As in the other forwards, a stale maximum is kept within 2^8.
        const bool raise = mx > m[e] + 8.f;
        if (__any_sync(0xffffffffu, raise)) {
          const float alpha = raise ? ex2(m[e] - mx) : 1.f;
          if (raise) m[e] = mx;
          l[e] *= alpha;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[n][2 * e] *= alpha;
            acc[n][2 * e + 1] *= alpha;
          }
        }
        const float mu = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2(fmaf(s[n][2 * e], sl2, -mu)), p1 = ex2(fmaf(s[n][2 * e + 1], sl2, -mu));
          l[e] += p0 + p1;
          const uint32_t w = pack2<BF16>(p0, p1);
          const float2 r = unpack2<BF16>(w);
          ph[2 * n + e] = w;
          pl[2 * n + e] = pack2<BF16>(p0 - r.x, p1 - r.y);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t f[4];
        ldsm_x4_t(f, sv + (n >> 3) * KT * 128 + vr * 128 + ((((n & 7) + vm) ^ (vr & 7)) << 4));
        mma16816<BF16>(acc[n], ph, f[0], f[1]);
        mma16816<BF16>(acc[n + 1], ph, f[2], f[3]);
        mma16816<BF16>(acc[n], pl, f[0], f[1]);
        mma16816<BF16>(acc[n + 1], pl, f[2], f[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (loads && i + NS < mine) {
        // The other map's warp is at most a tile behind in the same stage.
        // If the wait runs out (the abort flag is then up) the lane does not leave
        // alone: its warp leaves together at the next tile's vote.
        fed = wait_bar_c(&empty[st], ph_st, abort_flag, kRoleLoader, i);
        if (fed) issue(i + NS), ++issued;
      }
    }
    if (loads && *abort_flag)  // let the copies already issued land before the CTA exits
      for (int x = used + max(0, issued - NS); x < used + issued; ++x) drain_wait(&full[x % NS], (x / NS) & 1);
    used += mine;
    __syncwarp();
    __syncthreads();  // every warp has read its last tile: the ring becomes the join's buffer
    if (!CLUSTER && *abort_flag) return;  // a cluster meets below all the same

    float* jo = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[e];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (tq == 0) ml[(stream * 2 + c) * 16 + g + 8 * e] = make_float2(m[e], s);
      float* row = jo + ((stream * 2 + c) * 16 + g + 8 * e) * L::OROW;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float2*>(row + n * 8 + 2 * tq) = make_float2(acc[n][2 * e], acc[n][2 * e + 1]);
    }
    __syncthreads();
    // Rows of the tile x groups of 4 columns over the block's threads.
    for (int x = threadIdx.x; x < 16 * (DV / 4); x += 256) {
      const int tr = x / (DV / 4), col = x % (DV / 4) * 4;
      const int r = mt * 16 + tr;
      if (r >= a.R) break;
      float o[2][4], mm[2], ll[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // both maps
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[(w * 2 + c) * 16 + tr].x);
        mm[c] = top;
        ll[c] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 v = ml[(w * 2 + c) * 16 + tr];
          const float k = v.x == -INFINITY ? (v.y == v.y ? 0.f : v.y) : ex2(v.x - top);  // a NaN sum stays one
          ll[c] += v.y * k;
          const float4 y = *reinterpret_cast<const float4*>(jo + ((w * 2 + c) * 16 + tr) * L::OROW + col);
          o[c][0] = fmaf(y.x, k, o[c][0]);
          o[c][1] = fmaf(y.y, k, o[c][1]);
          o[c][2] = fmaf(y.z, k, o[c][2]);
          o[c][3] = fmaf(y.w, k, o[c][3]);
        }
      }
      const int row = r % a.Sq, h = hk * group + r / a.Sq;
      if constexpr (CLUSTER) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          *reinterpret_cast<float4*>(smem + L::OFF_PIECE + ((c * 16 + tr) * DV + col) * 4) =
              make_float4(o[c][0], o[c][1], o[c][2], o[c][3]);
          if (col == 0) reinterpret_cast<float2*>(smem + L::OFF_PML)[c * 16 + tr] = make_float2(mm[c], ll[c]);
        }
      } else if (direct) {
        const bool has = len > 0 && (!a.causal || row + len - a.Sq >= 0);
        diff_row_out<4, BF16>(a, b, h, row, col, has, o[0], o[1], ll[0], ll[1]);
        if (col == 0)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            a.lse[((static_cast<int64_t>(c) * a.B + b) * a.H + h) * a.Sq + row] =
                has ? (mm[c] + __log2f(ll[c])) * 0.69314718055994531f : -INFINITY;
      } else {
        const int64_t slot = (static_cast<int64_t>(b + team) * a.Hk + hk) * a.R + r;
        checked(slot < static_cast<int64_t>(a.B + a.teams) * a.Hk * a.R, 603);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          *reinterpret_cast<float4*>(a.part_o + (slot * 2 + c) * DV + col) =
              make_float4(o[c][0], o[c][1], o[c][2], o[c][3]);
          if (col == 0) a.part_ml[slot * 2 + c] = make_float2(mm[c], ll[c]);
        }
      }
    }
    if constexpr (CLUSTER) {
      // The cluster's CTAs hold an entry's keys between them: each adds up a
      // share of the row tile over all their pieces, out of shared memory.
      cluster_meet();
      const uint32_t piece = smem_u32(smem + L::OFF_PIECE), pml = smem_u32(smem + L::OFF_PML);
      for (int x = threadIdx.x + 256 * rank; x < 16 * (DV / 4); x += 256 * T) {
        const int tr = x / (DV / 4), col = x % (DV / 4) * 4;
        const int r = mt * 16 + tr;
        if (r >= a.R) break;
        float o[2][4], mm[2], ll[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mm[c] = -INFINITY;
          for (int w = 0; w < T; ++w) mm[c] = fmaxf(mm[c], cluster_ld2(cluster_at(pml + (c * 16 + tr) * 8, w)).x);
          ll[c] = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
          for (int w = 0; w < T; ++w) {
            const float2 v = cluster_ld2(cluster_at(pml + (c * 16 + tr) * 8, w));
            const float k = v.x == -INFINITY ? (v.y == v.y ? 0.f : v.y) : ex2(v.x - mm[c]);
            ll[c] += v.y * k;
            const float4 y = cluster_ld4(cluster_at(piece + ((c * 16 + tr) * DV + col) * 4, w));
            o[c][0] = fmaf(y.x, k, o[c][0]);
            o[c][1] = fmaf(y.y, k, o[c][1]);
            o[c][2] = fmaf(y.z, k, o[c][2]);
            o[c][3] = fmaf(y.w, k, o[c][3]);
          }
        }
        const int row = r % a.Sq, h = hk * group + r / a.Sq;
        const bool has = len > 0 && (!a.causal || row + len - a.Sq >= 0);
        diff_row_out<4, BF16>(a, b, h, row, col, has, o[0], o[1], ll[0], ll[1]);
        if (col == 0)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            a.lse[((static_cast<int64_t>(c) * a.B + b) * a.H + h) * a.Sq + row] =
                has ? (mm[c] + __log2f(ll[c])) * 0.69314718055994531f : -INFINITY;
      }
      cluster_meet();  // no CTA leaves while another reads its piece
    }
    // On to the next batch entry of the stretch.
    at = before + units;
    if (direct || at >= end) break;
    before = at;
    ++b;
    while (b < a.B && rows_units(a, b) == 0) ++b;
    if (b >= a.B) break;
    fence_proxy_async_smem();  // the join's buffer becomes the ring again
    __syncthreads();
  }
}

// Joins the pieces of one row per block. Eight warps take every eighth piece
// each (a lane holds DV / 32 columns of both maps), then meet in shared memory.
template <int DV, bool BF16>
__global__ void __launch_bounds__(256) fa_diff_rows_join(const DiffRowsArgs a) {
  using namespace sm100;
  constexpr int N = DV / 32;
  __shared__ float so[8][2][DV];
  __shared__ float2 sml[8][2];
  const int r = static_cast<int>(blockIdx.x) % a.R;
  const int hk = static_cast<int>(blockIdx.x) / a.R % a.Hk;
  const int b = static_cast<int>(blockIdx.x) / a.R / a.Hk;
  const int row = r % a.Sq, h = hk * (a.H / a.Hk) + r / a.Sq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = diff_keys(a.k_lens, b, a.Sk);
  // The teams that hold this entry's units [u0, u1): team t starts at unit
  // floor(total t / teams), so unit u lies with team ceil((u + 1) teams / total) - 1.
  const int64_t total = rows_before(a, a.B), u0 = rows_before(a, b), u1 = u0 + rows_units(a, b);
  const int teams = rows_teams(a, total);
  int t0 = 0, t1 = -1;
  if (u1 > u0 && total >= u1) {
    t0 = static_cast<int>(((u0 + 1) * teams + total - 1) / total) - 1;
    t1 = min(static_cast<int>((u1 * teams + total - 1) / total) - 1, teams - 1);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are written and visible
  // Team t's piece: slot b + t.
  auto at = [&](int t) { return (static_cast<int64_t>(b + t) * a.Hk + hk) * a.R + r; };
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][N];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < N; ++e) o[c][e] = 0.f;
  // The row's maxima first, so that the pieces' O are added without rescaling.
  for (int t = t0 + lane; t <= t1; t += 32)
#pragma unroll
    for (int c = 0; c < 2; ++c) m[c] = fmaxf(m[c], a.part_ml[at(t) * 2 + c].x);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m[c] = fmaxf(m[c], __shfl_xor_sync(0xffffffffu, m[c], x));
#pragma unroll 4
  for (int t = t0 + warp; t <= t1; t += 8)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float2 v = a.part_ml[at(t) * 2 + c];
      const float k = v.x == -INFINITY ? (v.y == v.y ? 0.f : v.y) : ex2(v.x - m[c]);
      l[c] += v.y * k;
      const float* po = a.part_o + (at(t) * 2 + c) * DV + lane * N;
#pragma unroll
      for (int e = 0; e < N; ++e) o[c][e] = fmaf(po[e], k, o[c][e]);
    }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int e = 0; e < N; ++e) so[warp][c][lane * N + e] = o[c][e];
    if (lane == 0) sml[warp][c] = make_float2(m[c], l[c]);
  }
  __syncthreads();
  if (threadIdx.x >= DV / 2) return;
  const int col = threadIdx.x * 2;
  float x[2][2], lt[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    x[c][0] = x[c][1] = lt[c] = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      x[c][0] += so[w][c][col];
      x[c][1] += so[w][c][col + 1];
      lt[c] += sml[w][c].y;
    }
  }
  const bool has = len > 0 && (!a.causal || row + len - a.Sq >= 0);
  diff_row_out<2, BF16>(a, b, h, row, col, has, x[0], x[1], lt[0], lt[1]);
  if (col == 0)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      a.lse[((static_cast<int64_t>(c) * a.B + b) * a.H + h) * a.Sq + row] =
          has ? (m[c] + __log2f(lt[c])) * 0.69314718055994531f : -INFINITY;
}

}  // namespace fa
