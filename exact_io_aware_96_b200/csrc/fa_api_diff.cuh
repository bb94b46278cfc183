// fa_api_diff.cuh — the C ABI of differential attention and of the rotary
// positions (include/fa.h): argument checks, tensor maps, workspace layout,
// launches. Part of fa_api.cu's translation unit, whose helpers it uses. No
// allocation, no host synchronisation, nothing that throws.
#pragma once

#include "fa_diff_bwd.cuh"
#include "fa_diff_fwd.cuh"
#include "fa_diff_rows.cuh"
#include "fa_rotary.cuh"

namespace {

void set_strides(int64_t (&s)[3], const fa_tensor& t) {
  s[0] = t.stride_b;
  s[1] = t.stride_s;
  s[2] = t.stride_h;
}

// Axes of extent > 1 must be stepped over: a zero stride there (an expanded
// view) is refused, for inputs because a tensor map cannot hold it and for
// outputs because rows would overwrite one another.
int check_axes(const fa_tensor& t, int B, int S, int H) {
  if ((B > 1 && t.stride_b == 0) || (S > 1 && t.stride_s == 0) || (H > 1 && t.stride_h == 0))
    return FA_ERR_INVALID_ARG;
  // A tensor map holds byte strides below 2^40.
  const int64_t lim = int64_t(1) << 39;
  if (t.stride_b >= lim || t.stride_s >= lim || t.stride_h >= lim) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// The stride of an axis of extent 1 is never stepped over and may be anything
// (torch leaves odd ones there): it becomes 0 before the checks.
void one_step(fa_tensor& t, int B, int S, int H) {
  if (B == 1) t.stride_b = 0;
  if (S == 1) t.stride_s = 0;
  if (H == 1) t.stride_h = 0;
}

int check_diff(int B, int H, int Hk, int Sq, int Sk, int D, int Dv, float scale, int causal, int dtype) {
  int st = check_common(B, H, Sq, Sk, D, scale, causal, dtype);
  if (st != FA_OK) return st;
  if (D > 64 || Dv < 8 || Dv > 128 || Dv % 8) return FA_ERR_UNSUPPORTED;
  if (Hk < 1 || H % Hk) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale * 1.4426950408889634f)) return FA_ERR_INVALID_ARG;  // the scale in base 2
  // Row indices of both maps' fp32 dQ accumulators are 32-bit tensor-map
  // coordinates, and grids are 31-bit.
  const int64_t lim = (int64_t(1) << 31) - 1;
  if (2 * int64_t(B) * H * ((int64_t(Sq) + 127) / 128 * 128) > lim) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

int check_lam(const fa_diff_lambda& l, int B, int Sq, int H, int dtype) {
  if (l.ptr == nullptr) return FA_ERR_INVALID_ARG;
  if (l.dtype != FA_LAMBDA_FP32 && l.dtype != dtype) return FA_ERR_UNSUPPORTED;
  if (l.stride_b < 0 || l.stride_s < 0 || l.stride_h < 0) return FA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(l.ptr) & (l.dtype == FA_LAMBDA_FP32 ? 3u : 1u)) return FA_ERR_MISALIGNED;
  if ((l.extent_b != 1 && l.extent_b != B) || (l.extent_s != 1 && l.extent_s != Sq) ||
      (l.extent_h != 1 && l.extent_h != H))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

int lam_kind(const fa_diff_lambda& l) {
  return l.dtype == FA_LAMBDA_FP32 ? fa::kLamF32 : l.dtype == FA_BF16 ? fa::kLamBF16 : fa::kLamF16;
}
void lam_strides(int64_t (&s)[3], const fa_diff_lambda& l) {
  s[0] = l.extent_b == 1 ? 0 : l.stride_b;
  s[1] = l.extent_s == 1 ? 0 : l.stride_s;
  s[2] = l.extent_h == 1 ? 0 : l.stride_h;
}

// Maps of q_1, q_2, k_1, k_2, v (and dO): 128 x 64-column boxes, query boxes of
// `q_rows` rows.
template <typename P>
int diff_maps(const P* p, int q_rows, CUtensorMap (&m)[5]) {
  int st;
  for (int c = 0; c < 2; ++c) {
    if ((st = make_map(&m[c], p->q[c], p->B, p->Sq, p->H, p->D, p->dtype, q_rows)) != FA_OK) return st;
    if ((st = make_map(&m[2 + c], p->k[c], p->B, p->Sk, p->Hk, p->D, p->dtype, 128)) != FA_OK) return st;
  }
  return make_map(&m[4], p->v, p->B, p->Sk, p->Hk, p->Dv, p->dtype, 128);
}

// A programmatic dependent launch: the grid may start while the one before it on
// the stream still runs, and waits on the device (griddepcontrol.wait) for its end.
template <typename... K, typename... T>
int launch_after(void (*kern)(K...), dim3 grid, int threads, int smem, cudaStream_t stream, const T&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int DV, bool BF16>
int launch_diff_fwd(const fa_diff_fwd_params* p, cudaStream_t stream) {
  using L = fa::DiffFwdLayout<DV>;
  static bool done[kMaxDevices] = {};
  auto* kern = &fa::fa_diff_fwd_kernel<DV, BF16>;
  int st = prepare(kern, L::SMEM_ALLOC, done);
  if (st != FA_OK) return st;
  CUtensorMap m[5];
  if ((st = diff_maps(p, 128, m)) != FA_OK) return st;
  fa::DiffFwdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.o = p->o.ptr;
  a.o2 = p->o2.ptr;
  a.lse = p->lse;
  set_strides(a.o_s, p->o);
  set_strides(a.o2_s, p->o2);
  a.lam = p->lambda.ptr;
  lam_strides(a.lam_s, p->lambda);
  a.lam_kind = lam_kind(p->lambda);
  a.k_lens = p->k_lens;
  a.B = p->B, a.H = p->H, a.Hk = p->Hk, a.Sq = p->Sq, a.Sk = p->Sk;
  a.d = p->D, a.dv = p->Dv;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.causal = p->causal;
  a.n_qblocks = (p->Sq + 127) / 128;
  a.by_order = fa::make_div(p->causal ? p->B * p->H : a.n_qblocks);
  a.by_H = fa::make_div(p->H), a.by_group = fa::make_div(p->H / p->Hk);
  const unsigned grid = unsigned(int64_t(a.n_qblocks) * p->B * p->H);
  kern<<<grid, L::kThreads, L::SMEM_ALLOC, stream>>>(m[0], m[1], m[2], m[3], m[4], a);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// The few-row form (fa_diff_rows.cuh): whether a call takes it, and its teams.
// Two CTAs run on an SM. Where a team of one CTA per (key head, row tile) is
// small, as many teams as fit at once share the keys evenly; large teams get a
// few waves, which even out by themselves. "Direct" saves the second kernel and
// the restart between batch entries (about 8 and 4 us), but leaves an entry's
// keys to one CTA, which takes 18 ns a key alone and 28 on a full GPU, or to a
// cluster of 2, 4 or 8, which join their pieces out of each other's shared memory
// (1 us more). It is taken where that is estimated 15% shorter, and for caches of
// two units per stream at most. Measured, us (D = 64, DV = 128), one CTA /
// cluster / teams: 32 entries x 8 heads x 500 keys 16.7 / - / 21.7; 8 x 8 x 1000
// 22.5 / 12.5 / 15.8; 1 x 8 x 1000 22.0 / 8.0 / 8.1 (in one launch instead of
// two); 16 x 2 x 300 10.5 / 7.9 / -; 1 x 8 x 2000 - / - / 9.1.
struct RowsPlan {
  bool rows = false;  // false: the tiled kernel
  int teams = 0;      // 0: direct
  int cluster = 1;    // direct: CTAs that share an entry's keys
  uint64_t off_o = 0, bytes = 0;
};
RowsPlan rows_plan(int B, int H, int Hk, int Sq, int Sk, int Dv) {
  RowsPlan p;
  const int64_t R = int64_t(H / Hk) * Sq;
  if (Sq > 16 || R > 64) return p;
  const int64_t slots = 2 * int64_t(std::max(1, sm_count())), team = int64_t(Hk) * ((R + 15) / 16);
  if (team * B > (int64_t(1) << 31) - 1) return p;
  p.rows = true;
  const int64_t items = team * B;
  const int64_t teams = team * 4 <= slots ? slots / team : (4 * slots + team - 1) / team;
  double direct_us = 0;
  for (int T = 1; T <= 8 && (T == 1 || T * 64 <= Sk); T *= 2) {
    const int64_t ctas = items * T;
    const double full = std::min(1.0, double(ctas) / double(slots)), waves = double((ctas + slots - 1) / slots);
    const double us = waves * ((T == 1 ? 4 : 5) + double(Sk) / T * std::max(0.018, 0.028 * full));
    if (T == 1 || us < 0.95 * direct_us) direct_us = us, p.cluster = T;
  }
  const double teams_us =
      8 + (2 * int64_t(B) > teams ? 4 : 0) + double(items) * Sk * (128 + (Dv <= 64 ? 64 : 128)) * 2 / 5.4e6;
  if (Sk <= 256 || items >= 4 * slots || 1.15 * direct_us < teams_us) return p;
  p.cluster = 1;
  p.teams = int(std::min<int64_t>(teams, (int64_t(B) * ((int64_t(Sk) + 63) / 64) + 1) / 2));
  const uint64_t parts = uint64_t(B + p.teams) * Hk * R * 2;
  p.off_o = round256(parts * sizeof(float2));
  p.bytes = p.off_o + parts * (Dv <= 64 ? 64 : 128) * 4;
  return p;
}

template <int DV, bool BF16>
int launch_diff_rows(const fa_diff_fwd_params* p, const RowsPlan& plan, cudaStream_t stream) {
  using L = fa::DiffRowsLayout<DV>;
  static bool done[kMaxDevices] = {}, done_cluster[kMaxDevices] = {}, done_join[kMaxDevices] = {};
  auto* alone = &fa::fa_diff_rows_kernel<DV, BF16, false>;
  auto* cluster = &fa::fa_diff_rows_kernel<DV, BF16, true>;
  auto* kern = plan.cluster > 1 ? cluster : alone;
  auto* join = &fa::fa_diff_rows_join<DV, BF16>;
  int st = plan.cluster > 1 ? prepare(cluster, L::SMEM_ALLOC, done_cluster) : prepare(alone, L::SMEM_ALLOC, done);
  if (st != FA_OK || (st = prepare(join, 0, done_join)) != FA_OK) return st;
  CUtensorMap mk[2], mv;
  for (int c = 0; c < 2; ++c)
    if ((st = make_map(&mk[c], p->k[c], p->B, p->Sk, p->Hk, p->D, p->dtype, L::KT)) != FA_OK) return st;
  if ((st = make_map(&mv, p->v, p->B, p->Sk, p->Hk, p->Dv, p->dtype, L::KT)) != FA_OK) return st;
  fa::DiffRowsArgs a;
  std::memset(&a, 0, sizeof(a));
  for (int c = 0; c < 2; ++c) {
    a.q[c] = static_cast<const uint16_t*>(p->q[c].ptr);
    set_strides(a.q_s[c], p->q[c]);
  }
  a.o = p->o.ptr;
  a.o2 = p->o2.ptr;
  a.lse = p->lse;
  set_strides(a.o_s, p->o);
  set_strides(a.o2_s, p->o2);
  a.lam = p->lambda.ptr;
  lam_strides(a.lam_s, p->lambda);
  a.lam_kind = lam_kind(p->lambda);
  a.k_lens = p->k_lens;
  a.B = p->B, a.H = p->H, a.Hk = p->Hk, a.Sq = p->Sq, a.Sk = p->Sk;
  a.d = p->D;
  a.dv = p->Dv;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.causal = p->causal;
  a.R = p->H / p->Hk * p->Sq;
  a.n_mt = (a.R + 15) / 16;
  a.teams = plan.teams;
  a.cluster = plan.cluster;
  if (plan.teams > 0) {
    if (p->workspace == nullptr || p->workspace_bytes < plan.bytes) return FA_ERR_WORKSPACE;
    a.part_ml = static_cast<float2*>(p->workspace);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(p->workspace) + plan.off_o);
  }
  const unsigned grid = unsigned(int64_t(plan.teams > 0 ? plan.teams : p->B) * p->Hk * a.n_mt * plan.cluster);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = plan.cluster, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = L::SMEM_ALLOC;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = plan.cluster > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, mk[0], mk[1], mv, a) != cudaSuccess) return FA_ERR_CUDA;
  if (plan.teams > 0) {
    return launch_after(join, dim3(unsigned(int64_t(p->B) * p->Hk * a.R)), 256, 0, stream, a);
  }
  return FA_OK;
}

// Parts that the backward's (head, query block) lists are cut into: the number
// up to 16 with the shortest estimated time. Lists count 128 x 128 blocks, at
// about 3.5 us each on one SM; a CTA costs about one block more; the SMs take
// the lists longest first, so the grid ends no earlier than its longest list
// or the average; joining P > 1 parts writes and reads P fp32 copies of dK and
// dV (4 TB/s assumed). Measured (B = 2, 12 query and 4 key heads, 2000 keys,
// causal): 200 us with 1 part, 144 with the 2 chosen.
int diff_bwd_parts(int B, int H, int Hk, int Sq, int Sk, int Dv, int causal) {
  const int sms = sm_count();
  if (sms <= 0) return 1;
  const int64_t group = H / Hk, nq = (int64_t(Sq) + 127) / 128, nk = (int64_t(Sk) + 127) / 128;
  double work = 0;
  for (int64_t k = 0; k < nk; ++k) work += double(std::max<int64_t>(0, nq - fa::bwd_first_qblock(int(k), Sq, Sk, causal)));
  const double lists = double(B) * Hk * nk, longest = double(nq * group);
  work *= double(group) * B * Hk;
  const double copy_us = double(B) * Hk * nk * 128 * (128 + (Dv <= 64 ? 64 : 128)) * 4 * 2 / 4e6;
  int best = 1;
  double best_us = 0;
  for (int P = 1; P <= 16 && (P == 1 || longest / P >= 2); ++P) {
    const double us = 3.5 * std::max(longest / P + 1, (work + lists * P) / sms) + (P > 1 ? 3 + P * copy_us : 0);
    if (P == 1 || us < 0.95 * best_us) best = P, best_us = us;
  }
  return lists * best < double((int64_t(1) << 31) - 1) ? best : 1;
}

// Workspace of the backward: dQ accumulators (or, deterministic, the slots),
// the row terms, -Delta_2 per row, dlambda's partial sums, the parts' dK and dV;
// 256-byte aligned.
struct DiffBwdWs {
  uint64_t off_vec, off_drow, off_part, off_dkv, bytes;
  int parts;
};
constexpr int kLamParts = 1024;
DiffBwdWs diff_bwd_ws(int B, int H, int Hk, int Sq, int Sk, int Dv, int causal, int deterministic) {
  const uint64_t nq = (uint64_t(Sq) + 127) / 128, nk = (uint64_t(Sk) + 127) / 128;
  const uint64_t rows = uint64_t(B) * H * nq * 128;
  DiffBwdWs w;
  w.parts = diff_bwd_parts(B, H, Hk, Sq, Sk, Dv, causal);
  w.off_vec = deterministic ? uint64_t(B) * H * nq * nk * 2 * 128 * 64 * 4 : rows * 2 * 64 * 4;
  w.off_drow = w.off_vec + rows * 5 * 4;
  w.off_part = round256(w.off_drow + uint64_t(B) * H * Sq * 4);
  w.off_dkv = w.off_part + uint64_t(kLamParts) * 4;
  w.bytes = w.off_dkv;
  if (w.parts > 1) w.bytes += uint64_t(w.parts) * B * Hk * nk * 128 * (128 + (Dv <= 64 ? 64 : 128)) * 4;
  return w;
}

int launch_lam(const fa_diff_bwd_params* p, const float* drow, float* part, cudaStream_t stream) {
  fa::LamSumArgs a;
  std::memset(&a, 0, sizeof(a));
  a.drow = drow;
  a.part = part;
  a.dlam = p->dlambda;
  a.dlam_kind = lam_kind(p->lambda);
  a.B = p->B, a.H = p->H, a.Sq = p->Sq;
  const fa_diff_lambda& l = p->lambda;
  a.by_s = fa::make_div(l.extent_s), a.by_h = fa::make_div(l.extent_h);
  a.by_ns = fa::make_div(l.extent_s == 1 ? p->Sq : 1), a.by_nh = fa::make_div(l.extent_h == 1 ? p->H : 1);
  a.n_out = int64_t(l.extent_b) * l.extent_s * l.extent_h;
  a.count = int64_t(a.B) * a.H * a.Sq / a.n_out;
  if (a.count <= 32)
    return launch_after(&fa::fa_diff_lam_few, dim3(unsigned((a.n_out + 255) / 256)), 256, 0, stream, a);
  // Sums of up to 8192 terms take one block, in less than a second launch would
  // add; longer ones are cut into runs of 2048 or more, at most kLamParts in
  // all, and joined by a second kernel. (On top of the rest of the backward, 8
  // heads x 4096 rows: 2.1 us; with two kernels and 64-bit divisions 6.6.)
  a.parts = a.count <= 8192 ? 1 : int(std::max<int64_t>(1, std::min<int64_t>(kLamParts / a.n_out, a.count / 2048)));
  const int st =
      launch_after(&fa::fa_diff_lam_part, dim3(unsigned(a.n_out * a.parts)), fa::kLamThreads, 0, stream, a);
  if (st != FA_OK || a.parts == 1) return st;
  return launch_after(&fa::fa_diff_lam_sum, dim3(unsigned(a.n_out)), 256, 0, stream, a);
}

template <int DV, bool BF16>
int launch_diff_bwd(const fa_diff_bwd_params* p, cudaStream_t stream) {
  using L = fa::DiffBwdLayout<DV>;
  static bool done[kMaxDevices] = {}, done_pre[kMaxDevices] = {}, done_dq[kMaxDevices] = {};
  static bool done_det[kMaxDevices] = {}, done_dkv[kMaxDevices] = {};
  auto* kern = &fa::fa_diff_bwd_main<DV, BF16>;
  int st = prepare(kern, L::SMEM_ALLOC, done);
  if (st != FA_OK) return st;
  if ((st = prepare(&fa::fa_diff_pre<DV, BF16>, 0, done_pre)) != FA_OK) return st;
  if ((st = prepare(&fa::fa_diff_dq<BF16, false>, 0, done_dq)) != FA_OK) return st;
  if ((st = prepare(&fa::fa_diff_dq<BF16, true>, 0, done_det)) != FA_OK) return st;
  if ((st = prepare(&fa::fa_diff_dkv<DV, BF16>, 0, done_dkv)) != FA_OK) return st;
  CUtensorMap m[5], mdo;
  if ((st = diff_maps(p, 64, m)) != FA_OK) return st;
  if ((st = make_map(&mdo, p->dO, p->B, p->Sq, p->H, p->Dv, p->dtype, 64)) != FA_OK) return st;
  fa::DiffBwdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.o = p->o.ptr, a.o2 = p->o2.ptr, a.dO = p->dO.ptr;
  a.lse = p->lse;
  a.lam = p->lambda.ptr;
  lam_strides(a.lam_s, p->lambda);
  a.lam_kind = lam_kind(p->lambda);
  set_strides(a.o_s, p->o);
  set_strides(a.o2_s, p->o2);
  set_strides(a.do_s, p->dO);
  for (int c = 0; c < 2; ++c) {
    a.dq[c] = p->dq[c].ptr;
    a.dk[c] = p->dk[c].ptr;
    set_strides(a.dq_s[c], p->dq[c]);
    set_strides(a.dk_s[c], p->dk[c]);
  }
  a.dv = p->dv.ptr;
  set_strides(a.dv_s, p->dv);
  a.B = p->B, a.H = p->H, a.Hk = p->Hk, a.Sq = p->Sq, a.Sk = p->Sk;
  a.Sq_pad = (p->Sq + 127) / 128 * 128;
  a.nqb = (p->Sq + 127) / 128;
  a.nkb = (p->Sk + 127) / 128;
  a.d = p->D;
  a.dv_cols = p->Dv;
  a.scale = p->scale;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.causal = p->causal;
  const DiffBwdWs w = diff_bwd_ws(p->B, p->H, p->Hk, p->Sq, p->Sk, p->Dv, p->causal, p->deterministic);
  char* ws = static_cast<char*>(p->workspace);
  a.dq_acc = reinterpret_cast<float*>(ws);
  a.dq_part = p->deterministic ? reinterpret_cast<float*>(ws) : nullptr;
  a.vec = reinterpret_cast<float*>(ws + w.off_vec);
  a.drow = reinterpret_cast<float*>(ws + w.off_drow);
  const fa_diff_lambda& lam = p->lambda;
  if (lam.extent_b == p->B && lam.extent_s == p->Sq && lam.extent_h == p->H) a.dlam = p->dlambda;
  a.parts = w.parts;
  a.group = p->H / p->Hk;
  a.by_H = fa::make_div(p->H), a.by_Hk = fa::make_div(p->Hk), a.by_parts = fa::make_div(w.parts);
  a.by_Sq = fa::make_div(p->Sq), a.by_Sq_pad = fa::make_div(a.Sq_pad), a.by_Sk = fa::make_div(p->Sk);
  a.by_order = fa::make_div(p->causal ? p->B * p->Hk : a.nkb);
  a.dkv_part = w.parts > 1 ? reinterpret_cast<float*>(ws + w.off_dkv) : nullptr;
  const int64_t rows = int64_t(p->B) * p->H * a.Sq_pad;
  fa::fa_diff_pre<DV, BF16><<<unsigned(rows * (DV / 8) / 256), 256, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  CUtensorMap mdq = m[0];  // not read in deterministic mode
  if (!p->deterministic && (st = make_dq_map(&mdq, a.dq_acc, 2 * rows, 64)) != FA_OK) return st;
  const unsigned grid = unsigned(int64_t(a.nkb) * p->B * p->Hk * a.parts);
  if ((st = launch_after(kern, dim3(grid), L::kThreads, L::SMEM_ALLOC, stream, m[0], m[1], m[2], m[3], m[4], mdo, mdq, a)) != FA_OK) return st;
  if (a.parts > 1) {
    const int64_t threads = int64_t(p->B) * p->Hk * p->Sk * ((128 + DV) / 8);
    if ((st = launch_after(&fa::fa_diff_dkv<DV, BF16>, dim3(unsigned((threads + 255) / 256)), 256, 0, stream, a)) != FA_OK)
      return st;
  }
  const dim3 dq_grid(unsigned((int64_t(p->B) * p->H * p->Sq * 8 + 255) / 256), 2);
  st = launch_after(p->deterministic ? &fa::fa_diff_dq<BF16, true> : &fa::fa_diff_dq<BF16, false>, dq_grid, 256, 0, stream, a);
  if (st != FA_OK) return st;
  return a.dlam != nullptr ? FA_OK : launch_lam(p, a.drow, reinterpret_cast<float*>(ws + w.off_part), stream);
}

template <bool BF16>
int launch_rotary(const fa_rotary_params* p, cudaStream_t stream) {
  fa::RotArgs a;
  std::memset(&a, 0, sizeof(a));
  const fa_tensor* in[2] = {&p->q, &p->k};
  const fa_tensor* out[2] = {&p->q_out, &p->k_out};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = static_cast<const uint16_t*>(in[i]->ptr);
    a.y[i] = static_cast<uint16_t*>(out[i]->ptr);
    set_strides(a.xs[i], *in[i]);
    set_strides(a.ys[i], *out[i]);
  }
  a.heads[0] = p->H;
  a.heads[1] = p->Hk;
  a.pos = p->positions;
  a.pos_s[0] = p->pos_stride_axis, a.pos_s[1] = p->pos_stride_b, a.pos_s[2] = p->pos_stride_s;
  a.pos64 = p->pos_int64;
  a.inv_freq = p->inv_freq;
  a.freq64 = p->inv_freq_fp64;
  a.axes = p->axes;
  for (int i = 0; i < p->axes; ++i) a.R += p->sections[i], a.end[i] = a.R;
  a.B = p->B, a.S = p->S, a.D = p->D;
  a.sign = p->inverse ? -1.f : 1.f;
  // Work items: pairs in groups of VEC, the largest power of two up to 8 that
  // divides R, so that both halves of a group are aligned (interleaved: 8
  // columns, four pairs); then the copied columns.
  const int vec = p->interleaved || a.R % 8 == 0 ? 8 : a.R % 4 == 0 ? 4 : a.R % 2 == 0 ? 2 : 1;
  a.n_rot = p->interleaved ? (2 * a.R + 7) / 8 : a.R / vec;
  a.n_item = p->interleaved ? a.D / 8 : a.n_rot + (a.D - 2 * a.R) / vec;
  const int64_t per_tok = int64_t(p->H + p->Hk) * a.n_item;
  a.per_tok = int(per_tok);
  // Tokens per block: up to 2048 items, of which four per thread have their loads go out
  // before the angles are computed, while the grid still covers the SMs; the
  // sines and cosines stay within 16 KB.
  const int64_t total = int64_t(p->B) * p->S;
  int64_t tokens = std::max<int64_t>(1, 2048 / per_tok);
  tokens = std::min<int64_t>(tokens, std::max<int64_t>(1, 2048 / a.R));
  tokens = std::min<int64_t>(tokens, std::max<int64_t>(1, total / 592));
  // (Divisions by reciprocals: items * per_tok below 2^32; see div_by.)
  tokens = std::min<int64_t>({tokens, fa::kRotMaxTokens, std::max<int64_t>(1, 0xffffffffll / (per_tok * per_tok))});
  a.tokens = int(tokens);
  auto inverse = [](int64_t d) { return d == 1 ? 0u : uint32_t((uint64_t(1) << 32) / uint64_t(d) + 1); };
  a.inv_item = inverse(a.n_item);
  a.inv_tok = tokens == 1 ? 1u : inverse(per_tok);  // 1 gives 0 for every item
  const unsigned grid = unsigned((total + tokens - 1) / tokens);
  const int smem = int(tokens) * a.R * int(sizeof(float2));
  auto go = [&](auto* kern) {
    kern<<<grid, 256, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  };
  if (p->interleaved) return go(&fa::fa_rotary_kernel<BF16, true, 8>);
  if (vec == 8) return go(&fa::fa_rotary_kernel<BF16, false, 8>);
  if (vec == 4) return go(&fa::fa_rotary_kernel<BF16, false, 4>);
  if (vec == 2) return go(&fa::fa_rotary_kernel<BF16, false, 2>);
  return go(&fa::fa_rotary_kernel<BF16, false, 1>);
}

}  // namespace

extern "C" {

size_t fa_diff_fwd_workspace_size(int B, int H, int Hk, int Sq, int Sk, int D, int Dv, int causal) {
  if (check_diff(B, H, Hk, Sq, Sk, D, Dv, 1.f, causal, FA_BF16) != FA_OK) return 0;
  return size_t(rows_plan(B, H, Hk, Sq, Sk, Dv).bytes);
}

int fa_diff_fwd(const fa_diff_fwd_params* given, fa_stream_t stream) {
  if (given == nullptr) return FA_ERR_INVALID_ARG;
  fa_diff_fwd_params args = *given;
  const fa_diff_fwd_params* p = &args;
  fa_tensor* qs[4] = {&args.q[0], &args.q[1], &args.o, &args.o2};
  for (fa_tensor* t : qs) one_step(*t, p->B, p->Sq, p->H);
  fa_tensor* ks[3] = {&args.k[0], &args.k[1], &args.v};
  for (fa_tensor* t : ks) one_step(*t, p->B, p->Sk, p->Hk);
  int st = check_diff(p->B, p->H, p->Hk, p->Sq, p->Sk, p->D, p->Dv, p->scale, p->causal, p->dtype);
  if (st != FA_OK) return st;
  for (const fa_tensor* t : qs) {
    if (t == &p->o2 && t->ptr == nullptr) continue;
    if ((st = check_view(*t)) != FA_OK || (st = check_axes(*t, p->B, p->Sq, p->H)) != FA_OK) return st;
  }
  for (const fa_tensor* t : ks)
    if ((st = check_view(*t)) != FA_OK || (st = check_axes(*t, p->B, p->Sk, p->Hk)) != FA_OK) return st;
  if ((st = check_lam(p->lambda, p->B, p->Sq, p->H, p->dtype)) != FA_OK) return st;
  if (p->lse == nullptr) return FA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p->lse) & 3u) return FA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(p->k_lens) & 3u) return FA_ERR_MISALIGNED;
  if (p->workspace != nullptr && (reinterpret_cast<uintptr_t>(p->workspace) & 255u)) return FA_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RowsPlan plan = rows_plan(p->B, p->H, p->Hk, p->Sq, p->Sk, p->Dv);
  if (plan.rows) {
    if (p->Dv <= 64)
      return p->dtype == FA_BF16 ? launch_diff_rows<64, true>(p, plan, s) : launch_diff_rows<64, false>(p, plan, s);
    return p->dtype == FA_BF16 ? launch_diff_rows<128, true>(p, plan, s) : launch_diff_rows<128, false>(p, plan, s);
  }
  if (p->Dv <= 64) return p->dtype == FA_BF16 ? launch_diff_fwd<64, true>(p, s) : launch_diff_fwd<64, false>(p, s);
  return p->dtype == FA_BF16 ? launch_diff_fwd<128, true>(p, s) : launch_diff_fwd<128, false>(p, s);
}

size_t fa_diff_bwd_workspace_size(int B, int H, int Hk, int Sq, int Sk, int D, int Dv, int causal, int deterministic) {
  if (deterministic != 0 && deterministic != 1) return 0;
  if (check_diff(B, H, Hk, Sq, Sk, D, Dv, 1.f, causal, FA_BF16) != FA_OK) return 0;
  const uint64_t bytes = diff_bwd_ws(B, H, Hk, Sq, Sk, Dv, causal, deterministic).bytes;
  return bytes > (uint64_t(1) << 50) ? 0 : size_t(bytes);
}

int fa_diff_bwd(const fa_diff_bwd_params* given, fa_stream_t stream) {
  if (given == nullptr) return FA_ERR_INVALID_ARG;
  fa_diff_bwd_params args = *given;
  const fa_diff_bwd_params* p = &args;
  fa_tensor* qs[7] = {&args.q[0], &args.q[1], &args.o, &args.o2, &args.dO, &args.dq[0], &args.dq[1]};
  for (fa_tensor* t : qs) one_step(*t, p->B, p->Sq, p->H);
  fa_tensor* ks[6] = {&args.k[0], &args.k[1], &args.v, &args.dk[0], &args.dk[1], &args.dv};
  for (fa_tensor* t : ks) one_step(*t, p->B, p->Sk, p->Hk);
  int st = check_diff(p->B, p->H, p->Hk, p->Sq, p->Sk, p->D, p->Dv, p->scale, p->causal, p->dtype);
  if (st != FA_OK) return st;
  for (const fa_tensor* t : qs)
    if ((st = check_view(*t)) != FA_OK || (st = check_axes(*t, p->B, p->Sq, p->H)) != FA_OK) return st;
  for (const fa_tensor* t : ks)
    if ((st = check_view(*t)) != FA_OK || (st = check_axes(*t, p->B, p->Sk, p->Hk)) != FA_OK) return st;
  if ((st = check_lam(p->lambda, p->B, p->Sq, p->H, p->dtype)) != FA_OK) return st;
  if (p->dlambda == nullptr || p->lse == nullptr) return FA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p->dlambda) & (p->lambda.dtype == FA_LAMBDA_FP32 ? 3u : 1u)) return FA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(p->lse) & 3u) return FA_ERR_MISALIGNED;
  if (p->deterministic != 0 && p->deterministic != 1) return FA_ERR_INVALID_ARG;
  const size_t need = fa_diff_bwd_workspace_size(p->B, p->H, p->Hk, p->Sq, p->Sk, p->D, p->Dv, p->causal, p->deterministic);
  if (p->workspace == nullptr || p->workspace_bytes < need || need == 0) return FA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(p->workspace) & 255u) return FA_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->Dv <= 64) return p->dtype == FA_BF16 ? launch_diff_bwd<64, true>(p, s) : launch_diff_bwd<64, false>(p, s);
  return p->dtype == FA_BF16 ? launch_diff_bwd<128, true>(p, s) : launch_diff_bwd<128, false>(p, s);
}

int fa_rotary(const fa_rotary_params* given, fa_stream_t stream) {
  if (given == nullptr) return FA_ERR_INVALID_ARG;
  fa_rotary_params args = *given;
  const fa_rotary_params* p = &args;
  one_step(args.q, p->B, p->S, p->H);
  one_step(args.q_out, p->B, p->S, p->H);
  one_step(args.k, p->B, p->S, p->Hk);
  one_step(args.k_out, p->B, p->S, p->Hk);
  if (p->B < 1 || p->S < 1 || p->H < 1 || p->Hk < 0) return FA_ERR_INVALID_ARG;
  if (p->dtype != FA_FP16 && p->dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (p->D < 8 || p->D > 256 || p->D % 8) return FA_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t(1) << 31) - 1;
  if (int64_t(p->B) * p->S > lim || int64_t(p->H) + p->Hk > 4095) return FA_ERR_INVALID_ARG;
  if (p->axes < 1 || p->axes > FA_ROTARY_MAX_AXES) return FA_ERR_INVALID_ARG;
  int64_t pairs = 0;
  for (int i = 0; i < p->axes; ++i) {
    if (p->sections[i] < 0) return FA_ERR_INVALID_ARG;
    pairs += p->sections[i];
  }
  if (pairs < 1 || 2 * pairs > p->D) return FA_ERR_INVALID_ARG;
  if ((p->interleaved | 1) != 1 || (p->inverse | 1) != 1 || (p->pos_int64 | 1) != 1 || (p->inv_freq_fp64 | 1) != 1)
    return FA_ERR_INVALID_ARG;
  const fa_tensor* t[4] = {&p->q, &p->q_out, &p->k, &p->k_out};
  for (int i = 0; i < (p->Hk > 0 ? 4 : 2); ++i) {
    int st = check_view(*t[i]);
    if (st != FA_OK) return st;
    if ((i & 1) && (st = check_axes(*t[i], p->B, p->S, i < 2 ? p->H : p->Hk)) != FA_OK) return st;
  }
  if (p->positions == nullptr || p->inv_freq == nullptr) return FA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p->positions) & (p->pos_int64 ? 7u : 3u)) return FA_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(p->inv_freq) & (p->inv_freq_fp64 ? 7u : 3u)) return FA_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return p->dtype == FA_BF16 ? launch_rotary<true>(p, s) : launch_rotary<false>(p, s);
}

}  // extern "C"
