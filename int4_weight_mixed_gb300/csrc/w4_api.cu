// w4_api.cu — the C ABI of libw4 (declared in include/w4.h): argument
// validation, the schedule table and default heuristic, workspace planning,
// tensor-map creation and kernel launch.  No allocation happens here: the
// caller owns every buffer.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdlib>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>
#include <string>

#include "../../include/w4.h"
#include "w4_internal.h"

namespace w4 {
namespace {

thread_local std::string g_last_error;

w4_status fail(w4_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

w4_status cuda_fail(cudaError_t e, const char* what) {
  return fail(W4_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Schedules ("Machete Readme", "Code Generation": a set of schedule configs
// with a default heuristic and an optional explicit choice).
const Schedule kSchedules[] = {
    {"simt", kEngineSimt, 0, kDataParallel, 1},       {"tc16_sk", kEngineTc, 16, kStreamK, 1},
    {"tc32_sk", kEngineTc, 32, kStreamK, 1},          {"tc64_sk", kEngineTc, 64, kStreamK, 1},
    {"tc128_sk", kEngineTc, 128, kStreamK, 1},        {"tc128_dp", kEngineTc, 128, kDataParallel, 1},
    {"tc256_sk", kEngineTc, 256, kStreamK, 1},        {"tc256_dp", kEngineTc, 256, kDataParallel, 1},
    {"dk8_sk", kEngineDk, 8, kStreamK, 1},            {"dk16_sk", kEngineDk, 16, kStreamK, 1},
    {"tc128x2_sk", kEngineTc, 128, kStreamK, 2},      {"tc128x2_dp", kEngineTc, 128, kDataParallel, 2},
    {"tc128x2_kp", kEngineTc, 128, kSplitK, 2},
    {"ds8_sk", kEngineDs, 8, kStreamK, 1},            {"ds16_sk", kEngineDs, 16, kStreamK, 1},
    {"tc256_kp", kEngineTc, 256, kSplitK, 1},
    {"ds32_sk", kEngineDs, 32, kStreamK, 1},
    {"gv8_cl", kEngineGv, 8, kSplitK, 1},             {"gv16_cl", kEngineGv, 16, kSplitK, 1},
    {"gv32_cl", kEngineGv, 32, kSplitK, 1},
    // two CTAs of a cluster share each MMA (cta_group::2): 256 weight columns
    // x 256 activation rows per tile, 128 activation rows per CTA
    {"tc256p_sk", kEngineTc, 256, kStreamK, 1, 1},    {"tc256p_dp", kEngineTc, 256, kDataParallel, 1, 1},
    // the same with 128 activation rows (64 per CTA): the accumulator is half
    // as wide, so the W4A8 int32 running sum stays in tensor memory beside it
    {"tc128p_sk", kEngineTc, 128, kStreamK, 1, 1},
};
constexpr int kNumSchedules = sizeof(kSchedules) / sizeof(kSchedules[0]);

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 152;  // GB300
  }
  return n;
}

int mode_of(int a_type) {
  return a_type == W4_F16    ? kW4A16_F16
         : a_type == W4_BF16 ? kW4A16_BF16
         : a_type == W4_E4M3 ? kW4A8F8
                             : kW4A8;
}
bool valid_a_type(int a_type) {
  return a_type == W4_F16 || a_type == W4_BF16 || a_type == W4_S8 || a_type == W4_E4M3;
}

TcPlan make_plan(int si, int mode, int64_t M, int64_t N, int64_t K, int64_t gs);
DkPlan make_dk_plan(int si, int mode, int64_t M, int64_t N, int64_t K, size_t* ws_partials,
                    size_t* ws_total);
constexpr size_t kMaxDynSmem = 227 * 1024;  // dynamic shared memory a CTA may opt into

// Whether schedule `si` can run this (already validated) problem shape.
bool schedule_fits(int si, int mode, int64_t M, int64_t N, int64_t K, int64_t gs, bool has_sg) {
  const Schedule& sc = kSchedules[si];
  if (sc.engine == kEngineSimt) return true;
  // fp8 activations: the clustered skinny-M and the tensor-core schedules
  if (mode == kW4A8F8 && sc.engine != kEngineGv && sc.engine != kEngineTc) return false;
  if (sc.engine == kEngineDk) {  // M rows in 8-row tiles; a 128-wide K block in one group
    if (M > sc.bm || (gs != K && gs % 128 != 0)) return false;
    size_t wp, wt;  // and the staged activations of a unit fit in shared memory
    return make_dk_plan(si, mode, M, N, K, &wp, &wt).smem_bytes <= kMaxDynSmem;
  }
  if (sc.engine == kEngineDs || sc.engine == kEngineGv)  // also bulk copies of 16-byte-multiple scale rows
    return M <= sc.bm && (gs == K || gs % 128 == 0) && N % 8 == 0 &&
           !(mode == kW4A8 && has_sg && N % 16 != 0);
  if (N % 8 != 0) return false;                      // 16-byte scale rows
  if (mode == kW4A8 && has_sg && N % 16 != 0) return false;
  // tensor memory must hold the accumulators (and the W4A8 int32 copies)
  // beside at least one stage of converted weights
  return make_plan(si, mode, M, N, K, gs).tstages >= 1;
}

// Build the launch plan of a tc schedule.
TcPlan make_plan_uncached(int si, int mode, int64_t M, int64_t N, int64_t K, int64_t gs) {
  const Schedule& sc = kSchedules[si];
  TcPlan p{};
  p.mode = mode;
  p.bm = sc.bm;
  p.nt = sc.nt;
  p.pair = sc.pair;
  const int ncta = p.pair ? 2 : 1;
  const int bmc = p.bm / ncta;  // activation rows in each CTA's shared memory
  // K block: 64 16-bit values (4 KB of nibbles per tile), or 128 E4M3 values
  // (8 KB) for fp8 activations
  const int bk = mode == kW4A8F8 ? 128 : kStageK;
  const int wblk = mode == kW4A8F8 ? 8192 : 4096;
  // K depth of a pipeline stage: skinny tiles need >= 8 KB of nibbles per
  // stage to hide the per-stage cost of the producer; wide tiles are
  // compute-bound and take shallower stages so that several fit in shared
  // memory.
  int nsub = p.bm <= 64 ? 4 : (p.bm <= 128 ? 2 : 1);
  nsub = nsub / p.nt > 0 ? nsub / p.nt : 1;
  const int64_t G = K / gs;
  auto group_ok = [&](int ns) {  // a stage covers whole groups or lies inside one
    return G <= 1 || (ns * kStageK) % gs == 0 || gs % (ns * kStageK) == 0;
  };
  while (nsub > 1 && !group_ok(nsub)) nsub /= 2;
  // The converter groups need at least kConvGroups stages in shared memory
  // (the order of their barrier waits relies on it): shallower stages when
  // the deep ones do not fit that many times.
  while (nsub > 1 && tc_max_stages(bmc, nsub, p.nt, wblk) < kConvGroups) {
    nsub /= 2;
    while (nsub > 1 && !group_ok(nsub)) nsub /= 2;
  }
  p.nsub = nsub;
  p.gps = (G > 1 && gs < nsub * kStageK) ? static_cast<int>(nsub * kStageK / gs) : 1;
  p.stages = tc_max_stages(bmc, nsub, p.nt, wblk);
  p.smem_bytes = tc_smem_bytes(bmc, nsub, p.nt, p.stages, wblk);
  p.m_tiles = static_cast<int>((M + p.bm - 1) / p.bm);
  p.n128 = static_cast<int>((N + kTileN - 1) / kTileN);
  p.n_tiles = (p.n128 + p.nt * ncta - 1) / (p.nt * ncta);
  p.tiles = p.m_tiles * p.n_tiles;
  p.k64 = static_cast<int>(K / bk);
  p.kb_total = (p.k64 + nsub - 1) / nsub;
  // W4A8 exactness: |a| <= 128 and |v*sg| <= 128 (group) or |v| <= 8
  // (per-channel) keep every fp32 partial sum of a chunk within 2^24.
  p.chunk_stages = static_cast<int>(((gs < K) ? 1024 : 16384) / (kStageK * nsub));
  // units of work distribution: CTAs, or the two-CTA clusters that can be
  // resident at once
  int sms = sm_count();
  if (p.pair) {
    // queried once per mode (a pair plan's shared memory depends on the mode
    // only); without a device, one pair per two SMs
    static std::mutex mu;
    static int cache[4];  // resident clusters + 1 (0: not yet queried)
    std::lock_guard<std::mutex> lock(mu);
    if (cache[mode] == 0) {
      const int c = tc_pair_clusters(mode, p.smem_bytes);
      cache[mode] = (c > 0 ? c : sms / 2) + 1;
    }
    sms = cache[mode] - 1;
  }
  p.decomp = sc.decomp;
  if (p.tiles * static_cast<size_t>(kConvWarps) * 4 * ncta > kCounterBytes)
    p.decomp = kDataParallel;
  p.ws_counters = kWsHeader;
  p.ws_partials = p.ws_counters + kCounterBytes;
  p.ksplit = 1;
  p.max_segs = 1;
  size_t part = 0;
  const size_t slot_bytes = static_cast<size_t>(p.nt) * kTileN * p.bm * 4;
  if (p.decomp == kDataParallel) {
    p.grid = (p.tiles < sms ? p.tiles : sms) * ncta;
  } else if (p.decomp == kSplitK) {
    // K splits: W4A8 splits at least until no unit is longer than one exact
    // chunk; then the split count minimizes waves x stages per unit, with a
    // charge for writing the partial sums when there is more than one split.
    int ks_min = 1;
    if (mode == kW4A8) ks_min = (p.kb_total + p.chunk_stages - 1) / p.chunk_stages;
    double best = 1e30;
    int best_ks = ks_min;
    for (int ks = ks_min; ks <= 16 && ks <= p.kb_total; ++ks) {
      const int64_t units = static_cast<int64_t>(p.tiles) * ks;
      const int64_t waves = (units + sms - 1) / sms;
      const int kbu = (p.kb_total + ks - 1) / ks;
      // a partial-sum slot costs about as much as a dozen stages to write
      const double cost = static_cast<double>(waves) * (kbu + 8 + (ks > 1 ? 12 : 0));
      if (cost < best) {
        best = cost;
        best_ks = ks;
      }
    }
    p.ksplit = best_ks;
    const int64_t units = static_cast<int64_t>(p.tiles) * p.ksplit;
    p.grid = static_cast<int>(units < sms ? units : sms) * ncta;
    if (p.ksplit > 1) part = static_cast<size_t>(p.tiles) * p.ksplit * slot_bytes * ncta;
  } else {
    const int64_t T = static_cast<int64_t>(p.tiles) * p.kb_total;
    int64_t g = T / 2;  // at least 2 stages per CTA (pair)
    if (g > sms) g = sms;
    if (g < 1) g = 1;
    p.grid = static_cast<int>(g) * ncta;
    int ms = 1;
    for (int64_t c = 0; c < g; ++c) {
      int64_t b = c * T / g, e = (c + 1) * T / g;
      if (e <= b) continue;
      int segs = static_cast<int>((e - 1) / p.kb_total - b / p.kb_total + 1);
      if (segs > ms) ms = segs;
    }
    p.max_segs = ms;
    part = static_cast<size_t>(p.grid) * p.max_segs * slot_bytes;  // one slot set per CTA
  }
  // Tensor memory: accumulators (NT x BM columns), the W4A8 int32 copies
  // when a unit can span several exact chunks, then the converted-weight
  // stages (NT x nsub x 32 columns each).
  bool long_units = p.kb_total > p.chunk_stages;
  if (p.decomp == kSplitK) long_units = (p.kb_total + p.ksplit - 1) / p.ksplit > p.chunk_stages;
  const int dcols = p.nt * p.bm;
  // W4A8 units longer than one exact chunk keep an int32 running sum: in
  // tensor memory beside the accumulators when that leaves two or more
  // converted-weight stages, else in a per-CTA global scratch (its owner
  // thread writes and reads it back, one element per accumulator cell).
  const bool need_i = mode == kW4A8 && long_units;
  const bool tmem_i = need_i && 512 - 2 * dcols >= 2 * p.nt * nsub * 32;
  p.icol = tmem_i ? dcols : 0;
  p.gicopy = need_i && !tmem_i ? 1 : 0;
  const int used = (p.icol ? 2 * dcols : dcols);
  p.acol = (used + 31) / 32 * 32;
  int ts = p.acol >= 512 ? 0 : (512 - p.acol) / (p.nt * nsub * 32);
  if (p.ksplit > 16) ts = 0;  // too many partial sums to be worth it: not offered
  if (ts > kMaxTmemStages) ts = kMaxTmemStages;
  if (ts > p.stages - 1) ts = p.stages - 1;
  if (p.stages < kConvGroups) ts = 0;  // not offered (see above)
  p.tstages = ts;
  p.ws_act = align256(p.ws_partials + part);
  size_t act = mode == kW4A8 ? static_cast<size_t>(M) * K * 2 : 0;
  p.ws_icopy = align256(p.ws_act + act);
  const size_t icopy = p.gicopy ? static_cast<size_t>(p.grid) * dcols * kTileN * 4 : 0;
  p.ws_total = align256(p.ws_icopy + icopy);
  return p;
}

// The plan of a tc schedule, remembered per shape and device: a call plans
// its schedule several times (fit, workspace, launch), each a few
// microseconds of host time.
TcPlan make_plan(int si, int mode, int64_t M, int64_t N, int64_t K, int64_t gs) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const auto key = std::make_tuple(si, mode, M, N, K, gs, dev);
  static std::mutex mu;
  static std::map<decltype(key), TcPlan> cache;
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) return it->second;
  }
  const TcPlan p = make_plan_uncached(si, mode, M, N, K, gs);
  std::lock_guard<std::mutex> lock(mu);
  if (cache.size() >= 4096) cache.clear();
  cache.emplace(key, p);
  return p;
}

size_t simt_ws_bytes() { return kWsHeader; }
// Plan of the skinny-M (mma.sync) schedule: 128-column tiles x K splits,
// two CTAs per SM; the split count minimizes waves x blocks per unit with a
// small penalty per split (partials and the reduction).
DkPlan make_dk_plan(int si, int mode, int64_t M, int64_t N, int64_t K, size_t* ws_partials,
                    size_t* ws_total) {
  DkPlan p{};
  p.mode = mode;
  p.nj = kSchedules[si].bm / 8;
  p.n_tiles = static_cast<int>((N + kTileN - 1) / kTileN);
  p.kblocks = static_cast<int>((K + 127) / 128);
  const int slots = 2 * sm_count();
  double best = 1e30;
  int best_s = 1;
  for (int ks = 1; ks <= 64 && ks <= p.kblocks; ++ks) {
    // a K split counts its contributors in one counter per weight tile
    if (ks > 1 && static_cast<size_t>(p.n_tiles) * 4 > kCounterBytes) break;
    const int kbu = (p.kblocks + ks - 1) / ks;
    if (dk_smem_bytes(p.nj, kbu) > 100 * 1024) continue;
    const int64_t units = static_cast<int64_t>(p.n_tiles) * ks;
    const int64_t waves = (units + slots - 1) / slots;
    // a wave costs its K blocks plus a fixed prologue / epilogue (~6 blocks)
    const double cost = static_cast<double>(waves) * (kbu + 6) * (1.0 + 0.01 * ks);
    if (cost < best) {
      best = cost;
      best_s = ks;
    }
  }
  p.ksplit = best_s;
  p.kbu_max = (p.kblocks + p.ksplit - 1) / p.ksplit;
  p.grid = p.n_tiles * p.ksplit;
  p.smem_bytes = dk_smem_bytes(p.nj, p.kbu_max);
  (void)M;
  const size_t part = p.ksplit > 1 ? static_cast<size_t>(p.ksplit) * p.n_tiles * 8 * p.nj *
                                         kTileN * 4
                                   : 0;
  *ws_partials = kWsHeader + kCounterBytes;
  *ws_total = align256(*ws_partials + part);
  return p;
}

// Plan of the streamed skinny-M schedule: two or three persistent CTAs per SM over a
// stream-K split of the (128-column tile, 128-K block) iterations.
DsPlan make_ds_plan_uncached(int si, int mode, int64_t M, int64_t N, int64_t K) {
  DsPlan p{};
  p.mode = mode;
  p.nj = kSchedules[si].bm / 8;
  p.n_tiles = static_cast<int>((N + kTileN - 1) / kTileN);
  p.kblocks = static_cast<int>((K + 127) / 128);
  // two K blocks (16 KB of nibbles) per stage: each stage costs its producer
  // thread a fixed few hundred nanoseconds, so stages must not be smaller
  p.sb = 2;  // must match the kernel's stage depth
  p.stages = 16;
  while (p.stages > 2 &&
         ds_smem_bytes(p.sb, p.nj, static_cast<int>(M), p.stages) > ds_smem_budget(p.nj))
    --p.stages;
  p.smem_bytes = ds_smem_bytes(p.sb, p.nj, static_cast<int>(M), p.stages);
  const int64_t T = static_cast<int64_t>(p.n_tiles) * p.kblocks;
  // every CTA streams at least eight blocks (four stages): a CTA has a fixed
  // start-up cost, and a tile split over many CTAs a long reduction
  int64_t g = ds_ctas_per_sm(p.nj) * static_cast<int64_t>(sm_count());
  if (g > (T + 7) / 8) g = (T + 7) / 8;
  if (g < 1) g = 1;
  p.grid = static_cast<int>(g);
  int ms = 1;
  for (int64_t c = 0; c < g; ++c) {
    const int64_t b = c * T / g, e = (c + 1) * T / g;
    if (e <= b) continue;
    const int segs = static_cast<int>((e - 1) / p.kblocks - b / p.kblocks + 1);
    if (segs > ms) ms = segs;
  }
  p.max_segs = ms;
  p.ws_partials = kWsHeader + kCounterBytes;
  const size_t part = static_cast<size_t>(p.grid) * p.max_segs * 8 * p.nj * kTileN * 4;
  p.ws_prep = align256(p.ws_partials + part);
  p.ws_total = align256(p.ws_prep + ds_prep_bytes(p.nj, static_cast<int>(M), p.kblocks));
  return p;
}

// The plan of a streamed schedule, remembered per shape and device as the tc
// plans are.
DsPlan make_ds_plan(int si, int mode, int64_t M, int64_t N, int64_t K) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const auto key = std::make_tuple(si, mode, M, N, K, dev);
  static std::mutex mu;
  static std::map<decltype(key), DsPlan> cache;
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) return it->second;
  }
  const DsPlan p = make_ds_plan_uncached(si, mode, M, N, K);
  std::lock_guard<std::mutex> lock(mu);
  if (cache.size() >= 4096) cache.clear();
  cache.emplace(key, p);
  return p;
}

// Plan of the clustered skinny-M schedule: the cluster size C (CTAs per
// 128-column tile, each streaming an equal share of the tile's K blocks) is
// the smallest that minimizes the K blocks of the busiest CTA while every
// cluster of the grid is resident at once.
GvPlan make_gv_plan(int si, int mode, int64_t M, int64_t N, int64_t K) {
  GvPlan p{};
  p.mode = mode;
  p.nj = kSchedules[si].bm / 8;
  p.n_tiles = static_cast<int>((N + kTileN - 1) / kTileN);
  p.kblocks = static_cast<int>((K + 127) / 128);
  p.stages = p.nj == 1 ? 4 : 3;
  p.smem_bytes = gv_smem_bytes(p.nj, mode, p.stages);
  // resident clusters per cluster size, from the occupancy calculator when a
  // device is present (cached per mode, row tiles and size), else from the
  // design's CTAs per SM
  static std::mutex mu;
  static int cache[4][3][17];  // resident clusters + 1 (0: not yet queried)
  const int mi = mode, ni = p.nj == 1 ? 0 : p.nj == 2 ? 1 : 2;
  const int per_sm = gv_ctas_per_sm(p.nj);
  const int sms = sm_count();
  int best_c = 1, best_nkb = p.kblocks;
  for (int C = 1; C <= 16 && C <= p.kblocks; ++C) {
    int clusters;
    {
      std::lock_guard<std::mutex> lock(mu);
      if (cache[mi][ni][C] == 0) {
        const int q = gv_max_clusters(mode, p.nj, C, p.smem_bytes);
        cache[mi][ni][C] = (q >= 0 ? q : sms * per_sm / C) + 1;
      }
      clusters = cache[mi][ni][C] - 1;
    }
    if (static_cast<int64_t>(p.n_tiles) > clusters) continue;  // more than one wave
    const int nkb = (p.kblocks + C - 1) / C;
    if (nkb < best_nkb) {
      best_nkb = nkb;
      best_c = C;
    }
  }
  p.cluster = best_c;
  p.grid = p.n_tiles * p.cluster;
  (void)M;
  return p;
}

// Per-shape overrides of the default heuristic ("Machete Readme", "Code
// Generation": a default heuristic with per-shape exceptions; the vLLM
// "rdna_hybrid_w4a16" page keeps a table of them, _GFX1X_PREFILL_OVERRIDES).
// Built-in entries come from A/B timings of the candidate schedules on
// GB300 (graphs of 16 back-to-back launches over rotated weight copies, more
// than 2x L2 between two reads of a copy); entries installed at run time
// (w4_override_schedule; w4_override_epilogue_schedule for products with an
// epilogue of their own, whose fastest schedule may be another) are consulted
// first.  M in [m_lo, m_hi]; group_size as resolved (K for one group per
// column).
struct Override {
  int mode;
  int64_t m_lo, m_hi, N, K, gs;
  int schedule;
  bool epilogue;  // of products with an epilogue (the built-in entries: of both)
};
const char* const kBuiltinOverrideNames[] = {"tc256p_dp", "tc256p_dp"};
const Override kBuiltinOverrides[] = {
    // W4A16 bf16, Llama-3-70B MLP down projection (N=8192, K=28672), M=4096:
    // tc256p_dp 1252 us, tc256p_sk 1349, tc256_sk 1598
    {kW4A16_BF16, 4096, 8192, 8192, 28672, 128, -1, false},
    // W4A16 bf16, Llama-3-70B MLP gate/up (N=57344, K=8192), M=4096:
    // tc256p_dp 2585 us, tc256p_sk 2594, tc256_sk 3341
    {kW4A16_BF16, 4096, 8192, 57344, 8192, 128, -1, false},
};
constexpr int kMaxOverrides = 256;
std::mutex g_ov_mutex;
Override g_overrides[kMaxOverrides];
int g_num_overrides = 0;

int schedule_index(const char* name) {
  for (int i = 0; i < kNumSchedules; ++i)
    if (strcmp(kSchedules[i].name, name) == 0) return i;
  return -1;
}

bool override_matches(const Override& o, int mode, int64_t M, int64_t N, int64_t K, int64_t gs) {
  return o.mode == mode && M >= o.m_lo && M <= o.m_hi && N == o.N && K == o.K && gs == o.gs;
}

// The schedule an override names for this problem, or -1.
int override_for(int mode, int64_t M, int64_t N, int64_t K, int64_t gs, bool epilogue) {
  {
    std::lock_guard<std::mutex> lock(g_ov_mutex);
    for (int i = g_num_overrides - 1; i >= 0; --i)  // the latest installed wins
      if (g_overrides[i].epilogue == epilogue && override_matches(g_overrides[i], mode, M, N, K, gs))
        return g_overrides[i].schedule;
  }
  for (size_t i = 0; i < sizeof(kBuiltinOverrides) / sizeof(kBuiltinOverrides[0]); ++i)
    if (override_matches(kBuiltinOverrides[i], mode, M, N, K, gs))
      return schedule_index(kBuiltinOverrideNames[i]);
  return -1;
}

// The heuristic's choice, whatever the overrides say.
int rule_schedule(int mode, int64_t M, int64_t N, int64_t K, int64_t gs, bool has_sg) {
  // skinny M (up to 32 rows with the clustered or streamed schedule, 16 with
  // the register-fed one where neither can run: N not a multiple of 8):
  // warp-level MMAs on dequantized weights
  // The clustered schedule (one launch) wins while its fixed costs dominate:
  // up to 16 rows on at most 16 MiB of packed weights; the streamed one
  // (stream-K with its own reduction launch) keeps more bytes in flight per
  // SM on larger weights.
  const bool small_w = K * N / 2 <= (int64_t{16} << 20);
  for (int eng : {kEngineGv, kEngineDs, kEngineDk})
    for (int si = 1; si < kNumSchedules; ++si)
      if (kSchedules[si].engine == eng &&
          !(eng == kEngineGv && (kSchedules[si].bm > 16 || (!small_w && mode != kW4A8F8))) &&
          schedule_fits(si, mode, M, N, K, gs, has_sg))
        return si;
  int bm = 16;
  while (bm < M && bm < 256) bm *= 2;
  // stream-K balances fewer than four waves of wide tiles; data-parallel beyond
  const int64_t tiles = ((M + bm - 1) / bm) * ((N + kTileN - 1) / kTileN);
  const bool dp = tiles >= 4 * static_cast<int64_t>(sm_count()) && bm >= 128;
  // 256-row tiles on CTA pairs (W4A8 N=8192 K=21760 M=1024: 241 us against
  // 406 for 128-row single-CTA tiles; fp8 M=1024 153 against 221 for
  // single-CTA 256-row tiles; W4A16 prefill 20-23% faster), and 128-row W4A8
  // tiles (M=128: 66.2 against 67.6 us)
  const bool pair = bm == 256 || (bm == 128 && mode == kW4A8);
  for (int pass = 0; pass < 2; ++pass)
    for (int si = 1; si < kNumSchedules; ++si) {
      const Schedule& sc = kSchedules[si];
      if (sc.engine == kEngineTc && sc.bm == bm && (sc.pair != 0) == pair &&
          (pass == 1 || (sc.decomp == kDataParallel) == dp) &&
          schedule_fits(si, mode, M, N, K, gs, has_sg))
        return si;
    }
  for (int si = 1; si < kNumSchedules; ++si)
    if (kSchedules[si].engine == kEngineTc && kSchedules[si].bm == bm &&
        schedule_fits(si, mode, M, N, K, gs, has_sg))
      return si;
  return 0;
}

int default_schedule_impl(int mode, int64_t M, int64_t N, int64_t K, int64_t gs, bool has_sg) {
  const int ov = override_for(mode, M, N, K, gs, false);
  if (ov >= 0 && schedule_fits(ov, mode, M, N, K, gs, has_sg)) return ov;
  return rule_schedule(mode, M, N, K, gs, has_sg);
}

// ---------------------------------------------------------------------------
// The schedule of a product with an epilogue of its own, beyond 16 rows: the
// one whose plan has the least estimated time.  (Up to 16 rows the rule above
// is within 1.0-1.7% of the fastest.  The plain product keeps that rule at every
// size, and with it the order of its sums; an epilogue's schedules, sums and
// plans are otherwise the plain product's.)
//
// A tensor-core plan takes a fixed time, one time per pipeline stage of its
// busiest CTA, one per tile that CTA drains, and what its split tiles cost:
// where their last contributor adds the others' partial sums, a time per slot
// (and drains that take longer with taller tiles); where tc_reduce_kernel adds
// them, its launch, a time per slot and one per megabyte of partial sums.
// W4A8 also takes the pass that stages its activations.  (W4A16 up to 32 rows:
// among the decode schedules, see keeps_weights.)  The constants
// (microseconds) are fitted to timings of every schedule at 7000 shapes (bf16
// g128 and per-channel, int8 per-channel and g128, E4M3; M 17..4096, N
// 256..57344, K 512..28672).  On 1750 other shapes of more than 16 rows, drawn
// over the logarithm of each size, the pick is within 2.1-2.6% of the fastest
// schedule in the geometric mean of each type (at most 1.41 times), where the
// rule above is 13-23% off.
enum CostClass { kCost16 = 0, kCostS8 = 1, kCostS8G = 2, kCostF8 = 3 };
struct TcCost {
  double fixed;
  double stage[7];  // tiles of 16, 32, 64, 128, 256 rows, pairs of 128, 256
  double drain_row, staging;
};
constexpr TcCost kTcCost[4] = {
    {2.35, {1.12, 1.07, 1.08, 0.654, 0.469, 0.562, 0.306}, 0.0293, 0.0},
    {3.08, {1.14, 1.12, 1.11, 0.639, 0.429, 0.579, 0.313}, 0.0395, 5.4e-7},
    {2.47, {1.57, 1.55, 1.59, 0.942, 0.713, 0.905, 0.608}, 0.0283, 5.4e-7},
    {2.42, {1.56, 1.54, 0.842, 0.883, 0.699, 0.752, 0.407}, 0.0297, 0.0}};
constexpr double kTcDrain = 1.16, kTcSlot = 3.16, kTcSlotRow = 0.0091;
constexpr double kTcSplitDrain = 2.74, kTcReduce = 1.81, kTcReduceSlot = 0.153, kTcReduceMB = 0.397;
// streamed at 32 rows: fixed, per 128-K block of the busiest CTA, per slot, and
// per 128 columns for the reduction (without which M=32 N=8192 K=21760 int8 was
// taken for 47.1 us against 46.9 on tc32_sk: 43 and 52 measured)
constexpr double kDs32Cost[3][4] = {{4.80, 0.561, 0.150, 0.0317},
                                    {5.05, 0.491, 0.173, 0.0326},
                                    {4.84, 0.717, 0.172, 0.0323}};
// clustered at 32 rows: fixed, per 128-K block of the busiest CTA, per CTA,
// per block of the average SM
constexpr double kGv32Cost[4][4] = {{3.58, 0.775, 0.0095, 0.565},
                                    {3.71, 0.593, 0.0089, 0.567},
                                    {3.55, 0.798, 0.0091, 0.586},
                                    {3.74, 0.512, 0.0085, 0.430}};

double estimated_us(int si, int mode, int64_t M, int64_t N, int64_t K, int64_t gs) {
  const Schedule& sc = kSchedules[si];
  const int cls = mode == kW4A8 ? (gs < K ? kCostS8G : kCostS8) : mode == kW4A8F8 ? kCostF8 : kCost16;
  if (sc.engine == kEngineGv) {
    const GvPlan p = make_gv_plan(si, mode, M, N, K);
    if (p.grid > sm_count() * gv_ctas_per_sm(p.nj)) return 1e30;  // more than one wave
    const int per = (p.kblocks + p.cluster - 1) / p.cluster;
    const double* g = kGv32Cost[cls];
    return g[0] + g[1] * per + g[2] * p.grid + g[3] * per * p.grid / sm_count();
  }
  if (sc.engine == kEngineDs) {
    const DsPlan p = make_ds_plan(si, mode, M, N, K);
    const int64_t T = static_cast<int64_t>(p.n_tiles) * p.kblocks, per = (T + p.grid - 1) / p.grid;
    const int64_t least = std::max<int64_t>(T / p.grid, 1);
    const double* d = kDs32Cost[cls];
    return d[0] + d[1] * per + d[2] * ((p.kblocks + least - 1) / least) + d[3] * p.n_tiles;
  }
  const TcPlan p = make_plan(si, mode, M, N, K, gs);
  const TcCost& c = kTcCost[cls];
  const int units = p.grid / (p.pair ? 2 : 1);
  const int row = p.pair ? (p.bm == 128 ? 5 : 6)
                         : p.bm == 16 ? 0 : p.bm == 32 ? 1 : p.bm == 64 ? 2 : p.bm == 128 ? 3 : 4;
  double us = c.fixed + c.staging * static_cast<double>(M) * K;
  const double drain = kTcDrain + c.drain_row * p.bm;
  if (p.decomp == kDataParallel) {
    const int drains = (p.tiles + units - 1) / units;
    return us + drains * (p.kb_total * c.stage[row] + drain);
  }
  const int64_t T = static_cast<int64_t>(p.tiles) * p.kb_total, it = (T + units - 1) / units;
  const double drains = static_cast<double>(it) / p.kb_total + 1;
  const int64_t slots = it < p.kb_total ? (p.kb_total + it - 1) / it
                                        : T % units != 0 || it % p.kb_total != 0;
  us += it * c.stage[row];
  if (!tc_reduces(p)) return us + drains * drain + slots * (kTcSlot + kTcSlotRow * p.bm);
  const double mb = (p.tiles + units) * (p.bm * kTileN * 4e-6) * (p.pair ? 2 : 1);
  return us + drains * kTcSplitDrain + kTcReduce + (slots + 1) * kTcReduceSlot + mb * kTcReduceMB;
}

// aligned: whether the arrays are as the tensor-core schedules' epilogue wants
// them (epilogue_aligned); the decode schedules' takes them by element.
int epilogue_schedule_impl(int mode, int64_t M, int64_t N, int64_t K, int64_t gs, bool has_sg,
                           bool aligned) {
  const auto runs = [&](int si) {
    return (aligned || kSchedules[si].engine != kEngineTc) &&
           schedule_fits(si, mode, M, N, K, gs, has_sg);
  };
  const int ov = override_for(mode, M, N, K, gs, true);
  if (ov >= 0 && runs(ov)) return ov;
  const int plain = rule_schedule(mode, M, N, K, gs, has_sg);
  if ((M <= 16 && runs(plain)) || kSchedules[plain].engine == kEngineSimt) return plain;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const auto key = std::make_tuple(mode, M, N, K, gs, has_sg, aligned, dev);
  static std::mutex mu;
  static std::map<decltype(key), int> cache;
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) return it->second;
  }
  // W4A16: the decode schedules scale sums in fp32, the tensor-core ones round
  // each dequantized weight to 16 bits (bf16 24 x 57344 x 8192: relative error
  // 0.0017 and 0.0022).  Where the plain product does not round them, a residual
  // or an activation does not make it do so, although that is faster on large
  // weights (that shape 140 us on ds32_sk, 115 on tc32_sk; 19 x 14576 x 19584 83
  // and 71; 32 x 23904 x 20608 per channel 112 and 115; 18 x 18256 x 896 14 and
  // 18): a caller who wants it says so (schedule, or an override).
  const bool keeps_weights = mode != kW4A8 && mode != kW4A8F8 && kSchedules[plain].engine != kEngineTc;
  int best = runs(plain) ? plain : 0;
  double best_us = HUGE_VAL;  // (above the estimate of a schedule that is a last resort)
  for (int si = 1; si < kNumSchedules; ++si) {
    const Schedule& sc = kSchedules[si];
    // one weight tile a CTA, stream-K or data-parallel; or 32-row decode
    const bool takes = sc.engine == kEngineTc
                           ? sc.nt == 1 && sc.decomp != kSplitK
                           : sc.bm == 32 && (sc.engine == kEngineGv || sc.engine == kEngineDs);
    if (!takes || !runs(si)) continue;
    if (keeps_weights && sc.engine == kEngineTc) continue;
    const double us = estimated_us(si, mode, M, N, K, gs);
    if (us < best_us) {
      best_us = us;
      best = si;
    }
  }
  std::lock_guard<std::mutex> lock(mu);
  if (cache.size() >= 4096) cache.clear();
  cache.emplace(key, best);
  return best;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether [p, p + np) and [q, q + nq) share a byte; null arrays share none.
bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a && b && a < b + nq && b < a + np;
}
// The same for two arrays that may also be one and the same.
bool overlap_but_same(const void* p, size_t np, const void* q, size_t nq) {
  return p != q && overlap(p, np, q, nq);
}

struct Problem {
  int mode;
  int64_t M, N, K, gs;
  bool has_sg;
};

w4_status validate(const void* a, int a_type, int64_t M, int64_t K, const void* b_packed,
                   int wtype, int64_t N, const void* b_scales, int scale_type,
                   const void* b_zeros, int64_t group_size, const float* s_tok,
                   const float* s_ch, void* out, int out_type, Problem& pr) {
  if (M < 0 || N < 0 || K < 0) return fail(W4_ERR_INVALID_ARGUMENT, "negative size");
  if (!valid_a_type(a_type))
    return fail(W4_ERR_INVALID_ARGUMENT, "a_type must be W4_F16, W4_BF16, W4_S8 or W4_E4M3");
  if (wtype < W4_UINT4B8 || wtype > W4_INT4) return fail(W4_ERR_INVALID_ARGUMENT, "bad wtype");
  if (K % 8 != 0) return fail(W4_ERR_INVALID_ARGUMENT, "K must be a multiple of 8");
  const int64_t gs = (group_size == -1) ? K : group_size;
  if (K > 0 && (gs <= 0 || K % gs != 0))
    return fail(W4_ERR_INVALID_ARGUMENT, "group_size must be -1 or a positive divisor of K");
  pr.mode = mode_of(a_type);
  pr.M = M;
  pr.N = N;
  pr.K = K;
  pr.gs = gs;
  pr.has_sg = b_scales != nullptr;
  if (M == 0 || N == 0) return W4_OK;
  if (!out) return fail(W4_ERR_INVALID_ARGUMENT, "out is null");
  if (pr.mode == kW4A8F8) {
    // W4A8 with E4M3 activations: symmetric weights, one scale per column
    if (wtype == W4_UINT4)
      return fail(W4_ERR_UNSUPPORTED, "W4A8 supports symmetric weights only (int4 / uint4b8)");
    if (b_zeros) return fail(W4_ERR_UNSUPPORTED, "W4A8 takes no zero-points");
    if (b_scales || gs != K)
      return fail(W4_ERR_UNSUPPORTED, "fp8 activations: per-channel weights only");
    if (out_type != W4_F16) return fail(W4_ERR_UNSUPPORTED, "fp8 activations: fp16 output only");
    if (!s_tok || !s_ch)
      return fail(W4_ERR_INVALID_ARGUMENT, "W4A8 fp16 out needs token and channel scales");
    if (K > 0 && (!a || !b_packed))
      return fail(W4_ERR_INVALID_ARGUMENT, "a and b_packed are required");
  } else if (pr.mode != kW4A8) {
    if (out_type != a_type)
      return fail(W4_ERR_INVALID_ARGUMENT, "W4A16: out_type must equal a_type");
    if (K > 0 && (!a || !b_packed || !b_scales))
      return fail(W4_ERR_INVALID_ARGUMENT, "W4A16: a, b_packed and b_scales are required");
    if (scale_type != a_type)
      return fail(W4_ERR_INVALID_ARGUMENT, "W4A16: scale_type must equal a_type");
    if (s_tok || s_ch)
      return fail(W4_ERR_INVALID_ARGUMENT, "W4A16 takes no token or channel scales");
  } else {
    if (wtype == W4_UINT4)
      return fail(W4_ERR_UNSUPPORTED, "W4A8 supports symmetric weights only (int4 / uint4b8)");
    if (b_zeros) return fail(W4_ERR_UNSUPPORTED, "W4A8 takes no zero-points");
    if (out_type == W4_F16) {
      if (!s_tok || !s_ch)
        return fail(W4_ERR_INVALID_ARGUMENT, "W4A8 fp16 out needs token and channel scales");
    } else if (out_type == W4_S32) {
      if (s_tok || s_ch)
        return fail(W4_ERR_INVALID_ARGUMENT, "W4A8 int32 out takes no float scales");
    } else {
      return fail(W4_ERR_UNSUPPORTED, "W4A8 output must be W4_F16 or W4_S32");
    }
    if (b_scales && scale_type != W4_S8)
      return fail(W4_ERR_INVALID_ARGUMENT, "W4A8 group scales must be int8 (W4_S8)");
    if (!b_scales && gs != K)
      return fail(W4_ERR_INVALID_ARGUMENT, "W4A8 per-group needs int8 group scales");
    if (K > 0 && (!a || !b_packed))
      return fail(W4_ERR_INVALID_ARGUMENT, "a and b_packed are required");
  }
  // every kernel reads or writes each array at least element by element;
  // the prepacked weights as 32-bit words
  const uintptr_t asz = (a_type == W4_S8 || a_type == W4_E4M3) ? 1 : 2;
  const uintptr_t osz = (pr.mode == kW4A8 && out_type == W4_S32) ? 4 : 2;
  const uintptr_t ssz = pr.mode == kW4A8 ? 1 : 2;
  if (!aligned_to(a, asz) || !aligned_to(out, osz) || !aligned_to(b_packed, 4) ||
      !aligned_to(b_scales, ssz) || !aligned_to(b_zeros, 2) || !aligned_to(s_tok, 4) ||
      !aligned_to(s_ch, 4))
    return fail(W4_ERR_INVALID_ARGUMENT,
                "a pointer is not aligned to its element size (b_packed: 4 bytes)");
  if (K % kStageK != 0) return fail(W4_ERR_UNSUPPORTED, "K must be a multiple of 64");
  if (pr.mode == kW4A8F8 && K % 128 != 0)
    return fail(W4_ERR_UNSUPPORTED, "fp8 activations: K must be a multiple of 128");
  if (K > 0 && gs % kStageK != 0)
    return fail(W4_ERR_UNSUPPORTED, "group_size must be a multiple of 64 (or K)");
  return W4_OK;
}

size_t ws_needed(int si, const Problem& pr) {
  if (kSchedules[si].engine == kEngineSimt) return simt_ws_bytes();
  if (kSchedules[si].engine == kEngineDk) {
    size_t wp, wt;
    make_dk_plan(si, pr.mode, pr.M, pr.N, pr.K, &wp, &wt);
    return wt;
  }
  if (kSchedules[si].engine == kEngineDs) return make_ds_plan(si, pr.mode, pr.M, pr.N, pr.K).ws_total;
  if (kSchedules[si].engine == kEngineGv) return kWsHeader;  // the status word only
  return make_plan(si, pr.mode, pr.M, pr.N, pr.K, pr.gs).ws_total;
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" {

int w4_layout_version(void) { return kLayoutVersion; }

size_t w4_prepacked_size(int64_t K, int64_t N) {
  if (K <= 0 || N <= 0 || K % kStageK != 0) return 0;
  return static_cast<size_t>((N + kTileN - 1) / kTileN * kTileN) * static_cast<size_t>(K / 2);
}

w4_status w4_prepack_B(const int32_t* w_q, int wtype, int in_layout, int64_t K, int64_t N,
                       void* b_packed, void* stream) {
  if (!w_q || !b_packed) return fail(W4_ERR_INVALID_ARGUMENT, "null pointer");
  if (wtype < W4_UINT4B8 || wtype > W4_INT4) return fail(W4_ERR_INVALID_ARGUMENT, "bad wtype");
  if (in_layout < W4_LAYOUT_KN_SEQ || in_layout > W4_LAYOUT_NK_EXLLAMA)
    return fail(W4_ERR_INVALID_ARGUMENT, "bad layout");
  if (K <= 0 || N <= 0 || K % 8 != 0)
    return fail(W4_ERR_INVALID_ARGUMENT, "K and N must be positive, K a multiple of 8");
  if (K % kStageK != 0) return fail(W4_ERR_UNSUPPORTED, "K must be a multiple of 64");
  if (!aligned_to(w_q, 4) || !aligned_to(b_packed, 4))
    return fail(W4_ERR_INVALID_ARGUMENT, "w_q and b_packed must be 4-byte aligned");
  cudaError_t e = launch_prepack(w_q, wtype, in_layout, K, N, static_cast<uint8_t*>(b_packed),
                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "prepack launch");
}

w4_status w4_unprepack_B(const void* b_packed, int wtype, int out_layout, int64_t K, int64_t N,
                         int32_t* w_q, void* stream) {
  if (!w_q || !b_packed) return fail(W4_ERR_INVALID_ARGUMENT, "null pointer");
  if (wtype < W4_UINT4B8 || wtype > W4_INT4) return fail(W4_ERR_INVALID_ARGUMENT, "bad wtype");
  if (out_layout < W4_LAYOUT_KN_SEQ || out_layout > W4_LAYOUT_NK_EXLLAMA)
    return fail(W4_ERR_INVALID_ARGUMENT, "bad layout");
  if (K <= 0 || N <= 0 || K % 8 != 0)
    return fail(W4_ERR_INVALID_ARGUMENT, "K and N must be positive, K a multiple of 8");
  if (K % kStageK != 0) return fail(W4_ERR_UNSUPPORTED, "K must be a multiple of 64");
  if (!aligned_to(w_q, 4) || !aligned_to(b_packed, 4))
    return fail(W4_ERR_INVALID_ARGUMENT, "w_q and b_packed must be 4-byte aligned");
  cudaError_t e = launch_unprepack(static_cast<const uint8_t*>(b_packed), wtype, out_layout, K,
                                   N, w_q, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "unprepack launch");
}

int w4_num_schedules(void) { return kNumSchedules; }

const char* w4_schedule_name(int schedule) {
  if (schedule < 0 || schedule >= kNumSchedules) return nullptr;
  return kSchedules[schedule].name;
}

}  // extern "C"

namespace {
int default_of(int64_t M, int64_t N, int64_t K, int a_type, int64_t group_size, bool epilogue) {
  if (M <= 0 || N <= 0 || K <= 0 || K % kStageK != 0) return -1;
  if (!valid_a_type(a_type)) return -1;
  if (a_type == W4_E4M3 && K % 128 != 0) return -1;
  const int64_t gs = group_size == -1 ? K : group_size;
  return epilogue ? epilogue_schedule_impl(mode_of(a_type), M, N, K, gs, gs != K, true)
                  : default_schedule_impl(mode_of(a_type), M, N, K, gs, gs != K);
}

w4_status install_override(int a_type, int64_t m_lo, int64_t m_hi, int64_t N, int64_t K,
                           int64_t group_size, int schedule, bool epilogue) {
  if (!valid_a_type(a_type))
    return fail(W4_ERR_INVALID_ARGUMENT, "a_type must be W4_F16, W4_BF16, W4_S8 or W4_E4M3");
  if (m_lo < 1 || m_hi < m_lo || N < 1 || K < 1 || K % kStageK != 0)
    return fail(W4_ERR_INVALID_ARGUMENT, "bad M range or shape");
  const int64_t gs = group_size == -1 ? K : group_size;
  if (gs <= 0 || K % gs != 0) return fail(W4_ERR_INVALID_ARGUMENT, "bad group_size");
  if (schedule >= kNumSchedules)
    return fail(W4_ERR_INVALID_ARGUMENT, "bad schedule index");
  const int mode = mode_of(a_type);
  std::lock_guard<std::mutex> lock(g_ov_mutex);
  // drop earlier entries for exactly this range, then add (schedule >= 0)
  int n = 0;
  for (int i = 0; i < g_num_overrides; ++i) {
    const Override& o = g_overrides[i];
    if (!(o.mode == mode && o.m_lo == m_lo && o.m_hi == m_hi && o.N == N && o.K == K &&
          o.gs == gs && o.epilogue == epilogue))
      g_overrides[n++] = o;
  }
  g_num_overrides = n;
  if (schedule < 0) return W4_OK;
  if (g_num_overrides == kMaxOverrides) return fail(W4_ERR_UNSUPPORTED, "override table full");
  g_overrides[g_num_overrides++] = Override{mode, m_lo, m_hi, N, K, gs, schedule, epilogue};
  return W4_OK;
}
}  // namespace

extern "C" {

int w4_default_schedule(int64_t M, int64_t N, int64_t K, int a_type, int64_t group_size) {
  return default_of(M, N, K, a_type, group_size, false);
}

int w4_default_epilogue_schedule(int64_t M, int64_t N, int64_t K, int a_type, int64_t group_size) {
  return default_of(M, N, K, a_type, group_size, true);
}

w4_status w4_override_schedule(int a_type, int64_t m_lo, int64_t m_hi, int64_t N, int64_t K,
                               int64_t group_size, int schedule) {
  return install_override(a_type, m_lo, m_hi, N, K, group_size, schedule, false);
}

w4_status w4_override_epilogue_schedule(int a_type, int64_t m_lo, int64_t m_hi, int64_t N,
                                        int64_t K, int64_t group_size, int schedule) {
  return install_override(a_type, m_lo, m_hi, N, K, group_size, schedule, true);
}

size_t w4_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int a_type, int64_t group_size) {
  Problem pr{};
  pr.mode = mode_of(a_type);
  pr.M = M < 0 ? 0 : M;
  pr.N = N < 0 ? 0 : N;
  pr.K = K < 0 ? 0 : K;
  pr.gs = group_size == -1 ? pr.K : group_size;
  pr.has_sg = pr.gs != pr.K;
  size_t need = kWsHeader;
  if (pr.M == 0 || pr.N == 0 || pr.K == 0 || pr.K % kStageK != 0) return need;
  // Remembered per shape and device (planning every schedule costs tens of
  // microseconds of host time, and callers ask once per call).
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const auto key = std::make_tuple(pr.M, pr.N, pr.K, pr.gs, pr.mode, dev);
  static std::mutex mu;
  static std::map<decltype(key), size_t> cache;
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) return it->second;
  }
  for (int si = 0; si < kNumSchedules; ++si) {
    if (!schedule_fits(si, pr.mode, pr.M, pr.N, pr.K, pr.gs, pr.has_sg)) continue;
    size_t b = ws_needed(si, pr);
    if (b > need) need = b;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (cache.size() >= 4096) cache.clear();
  cache.emplace(key, need);
  return need;
}

}  // extern "C"

namespace {
// What follows the product (w4_gemm_epilogue): nothing, or an activation, a
// gate and a residual.
struct Epilogue {
  int act = W4_ACT_NONE;
  int gated = 0;
  const void* residual = nullptr;
  bool any() const { return act != W4_ACT_NONE || gated || residual; }
};

w4_status check_epilogue(const Epilogue& ep, int64_t M, int64_t N, const void* out,
                         int out_type) {
  if (ep.act < W4_ACT_NONE || ep.act > W4_ACT_GELU_TANH)
    return fail(W4_ERR_INVALID_ARGUMENT, "bad act");
  if (!ep.any()) return W4_OK;
  if (out_type == W4_S32)
    return fail(W4_ERR_INVALID_ARGUMENT, "the raw int32 output takes no epilogue");
  if (ep.gated && N % 2 != 0)
    return fail(W4_ERR_INVALID_ARGUMENT, "a gated product needs an even N");
  if (!aligned_to(ep.residual, 2))
    return fail(W4_ERR_INVALID_ARGUMENT, "residual is not aligned to its element size");
  const size_t bytes = static_cast<size_t>(M) * (ep.gated ? N / 2 : N) * 2;
  if (overlap_but_same(ep.residual, bytes, out, bytes))
    return fail(W4_ERR_INVALID_ARGUMENT, "residual overlaps out without being out");
  return W4_OK;
}

// Held from a call's first launch to its last.  What a launch leaves in the
// workspace for the call's next one (partial sums, staged activations, codes)
// would be overwritten if another host thread's call with the same workspace
// enqueued a launch between them.  One of a few locks by the workspace's
// address: calls with different workspaces seldom wait for each other.
std::mutex& enqueue_mutex(const void* workspace) {
  static std::mutex mu[64];
  const uintptr_t p = reinterpret_cast<uintptr_t>(workspace);
  return mu[(p >> 8 ^ p >> 14 ^ p >> 21) % 64];
}

// The tensor-core schedules' epilogue reads and writes 16 bytes at a time.
bool epilogue_aligned(const Epilogue& ep, const void* out, const void* bias,
                      const float* ch_scales) {
  return !ep.any() ||
         (aligned16(out) && aligned16(ep.residual) && aligned16(bias) && aligned16(ch_scales));
}

// The caller holds the workspace's enqueue_mutex.
// prestaged: W4A8 on the tensor-core schedule with its bf16 activation copy
// already in the workspace (the dynamic-quantization entry point writes it)
w4_status gemm_impl(const void* a, int a_type, int64_t M, int64_t K, const void* b_packed,
                    int wtype, int64_t N, const void* b_scales, int scale_type,
                    const void* b_zeros, int64_t group_size, const float* a_token_scales,
                    const float* ch_scales, const void* bias, const Epilogue& ep, void* out,
                    int out_type, void* workspace, size_t workspace_bytes, void* stream,
                    int schedule, bool prestaged = false) {
  Problem pr{};
  w4_status st = validate(a, a_type, M, K, b_packed, wtype, N, b_scales, scale_type, b_zeros,
                          group_size, a_token_scales, ch_scales, out, out_type, pr);
  if (st != W4_OK) return st;
  if (bias) {
    if (pr.mode == kW4A8 && out_type == W4_S32)
      return fail(W4_ERR_INVALID_ARGUMENT, "the raw int32 output takes no bias");
    if (!aligned_to(bias, 2))
      return fail(W4_ERR_INVALID_ARGUMENT, "bias is not aligned to its element size");
  }
  st = check_epilogue(ep, M, N, out, out_type);
  if (st != W4_OK) return st;
  if (schedule >= kNumSchedules) return fail(W4_ERR_INVALID_ARGUMENT, "bad schedule index");
  if (M == 0 || N == 0) return W4_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0 && ep.any()) {  // the epilogue of a product of zeros
    EpArgs ea{};
    ea.s_tok = a_token_scales;
    ea.s_ch = ch_scales;
    ea.out = out;
    ea.bias = bias;
    ea.M = M;
    ea.N = N;
    ea.residual = ep.residual;
    ea.act = ep.act;
    ea.gated = ep.gated;
    cudaError_t e = launch_epilogue_rows(pr.mode, ea, s);
    return e == cudaSuccess ? W4_OK : cuda_fail(e, "epilogue launch");
  }
  if (K == 0 && !bias) {
    const size_t esz = (pr.mode == kW4A8 && out_type == W4_S32) ? 4 : 2;
    cudaError_t e = cudaMemsetAsync(out, 0, static_cast<size_t>(M) * N * esz, s);
    return e == cudaSuccess ? W4_OK : cuda_fail(e, "memset");
  }
  if (K == 0) {  // every output is its column's bias
    cudaError_t e = launch_bias_rows(pr.mode, M, N, bias, a_token_scales != nullptr, out, s);
    return e == cudaSuccess ? W4_OK : cuda_fail(e, "bias launch");
  }
  int si = schedule;
  const bool forced = schedule >= 0;
  if (!forced)
    si = ep.any() ? epilogue_schedule_impl(pr.mode, M, N, K, pr.gs, pr.has_sg,
                                           epilogue_aligned(ep, out, bias, ch_scales))
                  : default_schedule_impl(pr.mode, M, N, K, pr.gs, pr.has_sg);
  if (!schedule_fits(si, pr.mode, M, N, K, pr.gs, pr.has_sg))
    return fail(W4_ERR_UNSUPPORTED, "schedule %s cannot run this shape", kSchedules[si].name);
  const bool ptrs_ok = aligned16(a) && aligned16(b_packed) && aligned16(b_scales) &&
                       aligned16(b_zeros);
  if (kSchedules[si].engine != kEngineSimt && !ptrs_ok) {
    if (forced)
      return fail(W4_ERR_UNSUPPORTED, "tensor-core schedules need 16-byte aligned inputs");
    si = 0;
  }
  if (kSchedules[si].engine == kEngineTc && !epilogue_aligned(ep, out, bias, ch_scales))
    return fail(W4_ERR_UNSUPPORTED,  // (a given schedule: the rule picks another)
                "the tensor-core schedules' epilogue needs 16-byte aligned out, residual, bias "
                "and channel scales");
  if (!workspace) return fail(W4_ERR_WORKSPACE, "workspace is null");
  if (!aligned16(workspace)) return fail(W4_ERR_WORKSPACE, "workspace is not 16-byte aligned");
  const size_t need = ws_needed(si, pr);
  if (workspace_bytes < need)
    return fail(W4_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", workspace_bytes, need);

  TcArgs args{};
  args.b_packed = static_cast<const uint8_t*>(b_packed);
  args.scales = b_scales;
  args.zeros = b_zeros;
  args.s_tok = a_token_scales;
  args.s_ch = ch_scales;
  args.out = out;
  args.bias = bias;
  args.out_s32 = (pr.mode == kW4A8 && out_type == W4_S32) ? 1 : 0;
  args.wbias = (wtype == W4_UINT4) ? 0 : 8;
  args.M = M;
  args.N = N;
  args.K = K;
  args.group_size = pr.gs;
  args.status = static_cast<int*>(workspace);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  // runs a launcher on the arguments of the kernels with or without an
  // epilogue of their own
  auto with_epilogue = [&](auto&& launch) -> cudaError_t {
    if (!ep.any()) return launch(args);
    EpArgs ea{};
    static_cast<TcArgs&>(ea) = args;
    ea.residual = ep.residual;
    ea.act = ep.act;
    ea.gated = ep.gated;
    return launch(ea);
  };

  if (kSchedules[si].engine == kEngineSimt) {
    cudaError_t e =
        with_epilogue([&](const auto& x) { return launch_simt(pr.mode, a, x, s); });
    return e == cudaSuccess ? W4_OK : cuda_fail(e, "simt launch");
  }
  if (kSchedules[si].engine == kEngineDk) {
    size_t wp, wt;
    DkPlan dp = make_dk_plan(si, pr.mode, M, N, K, &wp, &wt);
    args.counters = reinterpret_cast<int*>(ws + kWsHeader);
    args.partials = ws + wp;
    static const bool debug = getenv("W4_DEBUG") != nullptr;
    if (debug)
      fprintf(stderr, "w4: %s M=%lld N=%lld K=%lld nj=%d tiles=%d kblocks=%d ksplit=%d grid=%d smem=%zu\n",
              kSchedules[si].name, (long long)M, (long long)N, (long long)K, dp.nj, dp.n_tiles,
              dp.kblocks, dp.ksplit, dp.grid, dp.smem_bytes);
    cudaError_t e =
        with_epilogue([&](const auto& x) { return launch_dk(dp, a, x, s); });
    return e == cudaSuccess ? W4_OK : cuda_fail(e, "dk launch");
  }
  if (kSchedules[si].engine == kEngineDs) {
    DsPlan dp = make_ds_plan(si, pr.mode, M, N, K);
    args.counters = reinterpret_cast<int*>(ws + kWsHeader);
    args.partials = ws + dp.ws_partials;
    static const bool debug = getenv("W4_DEBUG") != nullptr;
    if (debug)
      fprintf(stderr,
              "w4: %s M=%lld N=%lld K=%lld nj=%d tiles=%d kblocks=%d sb=%d stages=%d grid=%d "
              "segs=%d smem=%zu\n",
              kSchedules[si].name, (long long)M, (long long)N, (long long)K, dp.nj, dp.n_tiles,
              dp.kblocks, dp.sb, dp.stages, dp.grid, dp.max_segs, dp.smem_bytes);
    cudaError_t e =
        with_epilogue([&](const auto& x) { return launch_ds(dp, a, x, ws + dp.ws_prep, s); });
    return e == cudaSuccess ? W4_OK : cuda_fail(e, "ds launch");
  }

  if (kSchedules[si].engine == kEngineGv) {
    GvPlan gp = make_gv_plan(si, pr.mode, M, N, K);
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    CUtensorMap amap;
    CUresult r;
    const cuuint32_t rows = static_cast<cuuint32_t>(8 * gp.nj);
    if (pr.mode == kW4A8 || pr.mode == kW4A8F8) {
      // int8 / E4M3 [M][K]: one box of 128 K x all rows per K block
      const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(M)};
      const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
      const cuuint32_t box[2] = {128, rows};
      const cuuint32_t estr[2] = {1, 1};
      r = enc(&amap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {
      // 16-bit [M][K] as (k % 64, m, k / 64): one box {64, rows, 2} per K block
      const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kStageK), static_cast<cuuint64_t>(M),
                                  static_cast<cuuint64_t>(K / kStageK)};
      const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K) * 2, 128};
      const cuuint32_t box[3] = {static_cast<cuuint32_t>(kStageK), rows, 2};
      const cuuint32_t estr[3] = {1, 1, 1};
      r = enc(&amap,
              pr.mode == kW4A16_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              3, const_cast<void*>(a), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    if (r != CUDA_SUCCESS)
      return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled (activations) failed (%d)", (int)r);
    static const bool debug = getenv("W4_DEBUG") != nullptr;
    if (debug)
      fprintf(stderr, "w4: %s M=%lld N=%lld K=%lld nj=%d tiles=%d kblocks=%d cluster=%d "
                      "stages=%d grid=%d smem=%zu\n",
              kSchedules[si].name, (long long)M, (long long)N, (long long)K, gp.nj, gp.n_tiles,
              gp.kblocks, gp.cluster, gp.stages, gp.grid, gp.smem_bytes);
    cudaError_t e =
        with_epilogue([&](const auto& x) { return launch_gv(gp, amap, x, s); });
    return e == cudaSuccess ? W4_OK : cuda_fail(e, "gv launch");
  }

  TcPlan plan = make_plan(si, pr.mode, M, N, K, pr.gs);
  args.counters = reinterpret_cast<int*>(ws + plan.ws_counters);
  args.partials = ws + plan.ws_partials;
  args.icopy = reinterpret_cast<int32_t*>(ws + plan.ws_icopy);
  // W4A8 runs on the bf16 copy of its int8 activations in the workspace
  // (staged below, once every tensor map is encoded: an error before that
  // point leaves nothing enqueued)
  const void* act = pr.mode == kW4A8 ? static_cast<const void*>(ws + plan.ws_act) : a;
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  CUtensorMap amap, smap, zmap;
  memset(&smap, 0, sizeof(smap));
  memset(&zmap, 0, sizeof(zmap));
  const CUtensorMapDataType t16 =
      pr.mode == kW4A16_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (pr.mode == kW4A8F8) {
    // E4M3 [M][K]: one 2-D box of 128 K x BM rows per K block (128-byte rows)
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(plan.bm / (plan.pair ? 2 : 1))};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(&amap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(act), dims,
                     strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
      return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled (activations) failed (%d)", (int)r);
    plan.a3d = 0;
  } else {
    // Preferred: one 3-D box {64, BM, nsub} per stage over the view
    // (k % 64, m, k / 64); strides K*2 and 128 bytes.  Fallback: 2-D boxes.
    const cuuint64_t dims3[3] = {static_cast<cuuint64_t>(kStageK), static_cast<cuuint64_t>(M),
                                 static_cast<cuuint64_t>(K / kStageK)};
    const cuuint64_t strides3[2] = {static_cast<cuuint64_t>(K) * 2, 128};
    const cuuint32_t box3[3] = {static_cast<cuuint32_t>(kStageK),
                                static_cast<cuuint32_t>(plan.bm / (plan.pair ? 2 : 1)),
                                static_cast<cuuint32_t>(plan.nsub)};
    const cuuint32_t estr3[3] = {1, 1, 1};
    CUresult r = enc(&amap, t16, 3, const_cast<void*>(act), dims3, strides3, box3, estr3,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    plan.a3d = r == CUDA_SUCCESS ? 1 : 0;
    if (!plan.a3d) {
      const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(M)};
      const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K) * 2};
      const cuuint32_t box[2] = {static_cast<cuuint32_t>(kStageK),
                                 static_cast<cuuint32_t>(plan.bm / (plan.pair ? 2 : 1))};
      const cuuint32_t estr[2] = {1, 1};
      r = enc(&amap, t16, 2, const_cast<void*>(act), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS)
        return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled (activations) failed (%d)", (int)r);
    }
  }
  // [G][N] scale / zero-point rows: one box of 128 columns x gps groups per stage
  auto row_map = [&](CUtensorMap* m, const void* ptr, CUtensorMapDataType dt, int esz,
                     const char* what) -> w4_status {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(K / pr.gs)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * esz};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kTileN), static_cast<cuuint32_t>(plan.gps)};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(m, dt, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled (%s) failed (%d)", what, (int)r);
    return W4_OK;
  };
  if (b_scales) {
    w4_status st2 = pr.mode == kW4A8
                        ? row_map(&smap, b_scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, "group scales")
                        : row_map(&smap, b_scales, t16, 2, "scales");
    if (st2 != W4_OK) return st2;
  }
  if (b_zeros) {
    w4_status st2 = row_map(&zmap, b_zeros, t16, 2, "zero-points");
    if (st2 != W4_OK) return st2;
  }
  static const bool debug = getenv("W4_DEBUG") != nullptr;
  if (debug)
    fprintf(stderr,
            "w4: %s M=%lld N=%lld K=%lld bm=%d nt=%d nsub=%d stages=%d tstages=%d icol=%d gi=%d "
            "acol=%d gps=%d a3d=%d mma2=%d tiles=%d kb=%d grid=%d decomp=%d ksplit=%d segs=%d "
            "smem=%zu\n",
            kSchedules[si].name, (long long)M, (long long)N, (long long)K, plan.bm, plan.nt,
            plan.nsub, plan.stages, plan.tstages, plan.icol, plan.gicopy, plan.acol, plan.gps, plan.a3d,
            tc_mma2(plan) ? 1 : 0, plan.tiles, plan.kb_total, plan.grid, plan.decomp, plan.ksplit,
            plan.max_segs, plan.smem_bytes);
  if (pr.mode == kW4A8 && !prestaged) {
    cudaError_t e = launch_a8_to_bf16(static_cast<const int8_t*>(a), M * K, ws + plan.ws_act, s);
    if (e != cudaSuccess) return cuda_fail(e, "int8->bf16 launch");
  }
  cudaError_t e =
      with_epilogue([&](const auto& x) { return launch_tc(plan, amap, smap, zmap, x, s); });
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "tc launch");
}

// Workspace of the dynamic-quantization call: the W4A8 GEMM's own, then the
// codes [M][K] and the token scales [M].
struct DynLayout {
  int si;           // schedule of the W4A8 GEMM
  bool prestage;    // tensor-core int8: the quantizer writes the bf16 copy
  size_t gemm_ws, codes, stok, total;
};
DynLayout dyn_layout(int act_type, int64_t M, int64_t N, int64_t K, int64_t gs, bool epilogue,
                     bool aligned) {
  DynLayout d{};
  Problem pr{};
  pr.mode = mode_of(act_type);
  pr.M = M;
  pr.N = N;
  pr.K = K;
  pr.gs = gs;
  pr.has_sg = gs != K;
  d.si = epilogue ? epilogue_schedule_impl(pr.mode, M, N, K, gs, pr.has_sg, aligned)
                  : default_schedule_impl(pr.mode, M, N, K, gs, pr.has_sg);
  d.prestage = pr.mode == kW4A8 && kSchedules[d.si].engine == kEngineTc && K % 8 == 0 &&
               K <= 32768;
  // the GEMM part always spans the status word and the split-K counters
  // (which every call expects to find zero), whatever its schedule needs
  d.gemm_ws = align256(std::max(ws_needed(d.si, pr), kWsHeader + kCounterBytes));
  d.codes = d.gemm_ws;
  d.stok = align256(d.codes + static_cast<size_t>(M) * K);
  d.total = align256(d.stok + static_cast<size_t>(M) * 4);
  return d;
}

// ------------------------------------------------- the key-value cache's calls
constexpr int64_t kMaxPositions = int64_t{1} << 30;  // of a sequence: int32 with room

// Checks what all four calls share and fills in their views.
w4_status cache_views(const w4_kv_cache* cache, const w4_kv_batch* batch, int type, int64_t rows,
                      CacheView& c, BatchView& b) {
  if (!cache || !batch) return fail(W4_ERR_INVALID_ARGUMENT, "cache and batch are required");
  if (type != W4_F16 && type != W4_BF16)
    return fail(W4_ERR_INVALID_ARGUMENT, "type must be W4_F16 or W4_BF16");
  if (cache->type != W4_S8 && cache->type != W4_E4M3)
    return fail(W4_ERR_INVALID_ARGUMENT, "the cache's type must be W4_S8 or W4_E4M3");
  if (rows < 0 || batch->sequences < 0 || batch->table_width < 0 || cache->pages < 0 ||
      cache->heads <= 0 || cache->page_size <= 0 || cache->head_dim <= 0)
    return fail(W4_ERR_INVALID_ARGUMENT, "negative size, or no heads, slots or dimensions");
  if (cache->page_size < 16 || (cache->page_size & (cache->page_size - 1)) != 0)
    return fail(W4_ERR_UNSUPPORTED, "page_size must be a power of two, 16 at least");
  if (cache->head_dim % 16 != 0 || cache->head_dim > 256)
    return fail(W4_ERR_UNSUPPORTED, "head_dim must be a multiple of 16 up to 256");
  if (cache->heads > 65535 || cache->pages > 0x7fffffff || batch->sequences > 0x7ffffffe ||
      rows > 0x7fffffff)
    return fail(W4_ERR_UNSUPPORTED, "pages, sequences or rows above 2^31 - 1, or heads above 65535");
  if (batch->table_width > kMaxPositions / cache->page_size)
    return fail(W4_ERR_UNSUPPORTED, "more than 2^30 positions a sequence");
  if (rows > 0 && batch->sequences > 0) {
    if (!batch->starts || !batch->lens || (batch->table_width > 0 && !batch->table))
      return fail(W4_ERR_INVALID_ARGUMENT, "starts, lens and table are required");
    if (cache->pages > 0 && (!cache->k || !cache->v || !cache->k_scales || !cache->v_scales))
      return fail(W4_ERR_INVALID_ARGUMENT, "a null array of the cache");
  }
  if (!aligned_to(batch->table, 4) || !aligned_to(batch->starts, 4) || !aligned_to(batch->lens, 4))
    return fail(W4_ERR_INVALID_ARGUMENT, "starts, lens and table must be 4-byte aligned");
  if (!aligned16(cache->k) || !aligned16(cache->v) || !aligned16(cache->k_scales) ||
      !aligned16(cache->v_scales))
    return fail(W4_ERR_INVALID_ARGUMENT, "the cache's arrays must be 16-byte aligned");
  c.k = static_cast<uint8_t*>(cache->k);
  c.v = static_cast<uint8_t*>(cache->v);
  c.k_scales = cache->k_scales;
  c.v_scales = cache->v_scales;
  c.pages = cache->pages;
  c.heads = cache->heads;
  c.page_shift = 0;
  while ((1 << c.page_shift) < cache->page_size) ++c.page_shift;
  c.dim = cache->head_dim;
  c.e4m3 = cache->type == W4_E4M3;
  b.table = batch->table;
  b.width = batch->table_width;
  b.starts = batch->starts;
  b.lens = batch->lens;
  b.sequences = static_cast<int>(batch->sequences);
  b.rows = static_cast<int>(rows);
  return W4_OK;
}

// Whether an output shares a byte with one of the cache's arrays.
bool overlaps_cache(const w4_kv_cache* c, const void* out, size_t bytes) {
  const size_t slots = static_cast<size_t>(c->pages) * c->heads * c->page_size;
  return overlap(out, bytes, c->k, slots * c->head_dim) || overlap(out, bytes, c->v, slots * c->head_dim) ||
         overlap(out, bytes, c->k_scales, slots * 4) || overlap(out, bytes, c->v_scales, slots * 4);
}

// Which kernel attends, and (tensor cores) whether the visible keys and values are
// unpacked to 16 bits first, each tile of 128 keys once (tiles_each: tiles of a
// sequence and key head), instead of by every unit of 256 rows that visits it.
enum AttnEngine { kAttnSimt, kAttnDec, kAttnTc };
struct AttnPlan {
  AttnEngine engine;
  int64_t tiles_each;
  size_t partials, tiles;  // bytes
};
constexpr int64_t kMaxTileBytes = int64_t{256} << 20;
// most: the plan that needs the most workspace, whatever the window.
AttnPlan attn_plan(const w4_kv_cache* cache, const w4_kv_batch* batch, int64_t rows, int heads,
                   int window, int sinks, bool most = false) {
  AttnPlan p{kAttnSimt, 0, 0, 0};
  const int dim = cache->head_dim;
  // (with no page there is no key, and the others load some key's row)
  if ((dim != 64 && dim != 128) || cache->pages == 0 || cache->heads <= 0) return p;
  const int sms = sm_count();
  p.partials = std::max(attn_dec_partials(sms, dim), attn_tc_partials(sms, dim));
  // The kernel with the less estimated time, from the longest a sequence can be (its
  // line of the table; its window): the decode kernel reads a key head's codes for
  // every 16 of its rows, at about 4.5 GB/ms; the tensor cores' has 35 us before and
  // after, and an SM takes a tile of 128 keys by 256 rows in about 3.7 us (64
  // dimensions: 2.2), half of it by 128.  (One tree of 64 drafts, 32 heads over 8, 2112
  // keys: 32 us and 54; 32 trees of up to 48, 64 heads, 4096 keys: 680 and 282.)
  const int64_t lines = batch->sequences * cache->heads;
  const int64_t flat = rows * heads;
  if (lines > 0) {
    const double each_rows = std::ceil(static_cast<double>(flat) / lines);
    double keys = static_cast<double>(batch->table_width) * cache->page_size;
    if (window > 0) keys = std::min(keys, static_cast<double>(window) + sinks + each_rows);
    const double dec = 8 + lines * std::ceil(each_rows / 16) * keys * (2 * dim) / 4.5e6;
    const double tc = 35 + lines * std::ceil(each_rows / 128) / 2 * std::ceil(keys / 128) *
                              (dim == 128 ? 3.7 : 2.2) / sms;
    if (each_rows <= 16 || (!most && dec <= tc)) {
      p.engine = kAttnDec;
      return p;
    }
  }
  p.engine = kAttnTc;
  const int64_t each = (batch->table_width * cache->page_size + 127) / 128;
  if (flat >= 3 * 256 * lines && each > 0 && lines > 0 &&
      each <= kMaxTileBytes / attn_tc_tile_bytes(dim) / lines) {
    p.tiles_each = each;
    p.tiles = static_cast<size_t>(each * lines * attn_tc_tile_bytes(dim));
  }
  return p;
}

w4_status attention(const w4_kv_cache* cache, const w4_kv_batch* batch, const void* q,
                    const uint8_t* mask, int64_t mask_width, int type, int64_t rows, int heads,
                    int64_t q_stride, float scale, int window, int sinks, void* out,
                    void* workspace, size_t workspace_bytes, void* stream) {
  AttnArgs a{};
  w4_status st = cache_views(cache, batch, type, rows, a.c, a.b);
  if (st != W4_OK) return st;
  if (heads <= 0 || heads % cache->heads != 0)
    return fail(W4_ERR_INVALID_ARGUMENT, "heads must be a multiple of the cache's");
  if (!std::isfinite(scale)) return fail(W4_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (sinks < 0) return fail(W4_ERR_INVALID_ARGUMENT, "sinks must not be negative");
  const int64_t dense = static_cast<int64_t>(heads) * cache->head_dim;
  if (q_stride < dense && rows > 1)
    return fail(W4_ERR_INVALID_ARGUMENT, "q_stride is below heads * head_dim");
  if (heads > 65535) return fail(W4_ERR_UNSUPPORTED, "more than 65535 heads");
  if (rows * static_cast<int64_t>(heads) > (int64_t{1} << 30))
    return fail(W4_ERR_UNSUPPORTED, "more than 2^30 rows times heads");
  if (rows == 0 || batch->sequences == 0) return W4_OK;
  if (!q || !out) return fail(W4_ERR_INVALID_ARGUMENT, "q and out are required");
  if (!aligned_to(q, 2) || !aligned_to(out, 2))
    return fail(W4_ERR_INVALID_ARGUMENT, "q or out is not aligned to its element size");
  if (overlap(out, static_cast<size_t>(rows) * dense * 2, q,
              (static_cast<size_t>(rows - 1) * q_stride + dense) * 2))
    return fail(W4_ERR_INVALID_ARGUMENT, "out overlaps q");
  if (overlaps_cache(cache, out, static_cast<size_t>(rows) * dense * 2))
    return fail(W4_ERR_INVALID_ARGUMENT, "out overlaps the cache");
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.bf16 = type == W4_BF16;
  a.heads = heads;
  a.scale = scale;
  a.window = window > 0 && window < kMaxPositions ? window : 0;
  a.sinks = sinks;
  a.mask = mask;
  a.mask_width = mask_width;
  const AttnPlan plan = attn_plan(cache, batch, rows, heads, a.window, a.sinks);
  // (without room for unpacked tiles every unit converts those that it visits)
  const size_t need = kWsHeader + kCounterBytes + align256(plan.partials);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(W4_ERR_WORKSPACE, "workspace of %zu bytes, 16-byte aligned, is required", need);
  char* const ws = static_cast<char*>(workspace);
  a.status = reinterpret_cast<int*>(ws);
  a.counters = reinterpret_cast<int*>(ws + kWsHeader);
  a.partials = reinterpret_cast<float*>(ws + kWsHeader + kCounterBytes);
  if (plan.tiles_each > 0 && workspace_bytes - need >= plan.tiles) {
    a.tiles = reinterpret_cast<uint8_t*>(ws + kWsHeader + kCounterBytes + align256(plan.partials));
    a.tiles_each = plan.tiles_each;
  }
  std::lock_guard<std::mutex> lock(enqueue_mutex(workspace));
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = plan.engine == kAttnSimt  ? launch_attn_simt(a, cs)
                        : plan.engine == kAttnDec ? launch_attn_dec(a, sm_count(), cs)
                                                  : launch_attn_tc(a, sm_count(), cs);
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "attention launch");
}

}  // namespace

extern "C" {

size_t w4_gemm_dynamic_workspace_size(int64_t M, int64_t N, int64_t K, int act_type,
                                      int64_t group_size) {
  if (M <= 0 || N <= 0 || K <= 0 || K % kStageK != 0) return kWsHeader;
  if (act_type != W4_S8 && act_type != W4_E4M3) return kWsHeader;
  const int64_t gs = group_size == -1 ? K : group_size;
  if (gs <= 0 || K % gs != 0) return kWsHeader;
  if (act_type == W4_E4M3 && K % 128 != 0) return kWsHeader;
  // the largest over the schedules the call may take (the default one),
  // with room for any schedule an override may name
  const DynLayout d = dyn_layout(act_type, M, N, K, gs, false, true);
  const size_t any = w4_gemm_workspace_size(M, N, K, act_type, group_size);
  const size_t extra = d.total - d.gemm_ws;
  return (any > d.gemm_ws ? align256(any) : d.gemm_ws) + extra;
}

}  // extern "C"

namespace {
w4_status dynamic_impl(const void* a, int a_type, int64_t M, int64_t K, const void* b_packed,
                          int wtype, int64_t N, const void* b_scales, int scale_type,
                          int64_t group_size, const float* ch_scales, int act_type,
                          const void* bias, const Epilogue& ep, void* out,
                          float* token_scales_out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (M < 0 || N < 0 || K < 0) return fail(W4_ERR_INVALID_ARGUMENT, "negative size");
  if (a_type != W4_F16 && a_type != W4_BF16)
    return fail(W4_ERR_INVALID_ARGUMENT, "a_type must be W4_F16 or W4_BF16");
  if (act_type != W4_S8 && act_type != W4_E4M3)
    return fail(W4_ERR_INVALID_ARGUMENT, "act_type must be W4_S8 or W4_E4M3");
  if (M == 0 || N == 0) return W4_OK;
  if (K > 0 && !a) return fail(W4_ERR_INVALID_ARGUMENT, "a is null");
  if (!aligned_to(a, 2) || !aligned_to(token_scales_out, 4))
    return fail(W4_ERR_INVALID_ARGUMENT, "a pointer is not aligned to its element size");
  if (K % 8 != 0) return fail(W4_ERR_INVALID_ARGUMENT, "K must be a multiple of 8");
  const int64_t gs = group_size == -1 ? K : group_size;
  if (K > 0 && (gs <= 0 || K % gs != 0))
    return fail(W4_ERR_INVALID_ARGUMENT, "group_size must be -1 or a positive divisor of K");
  if (K == 0 || K % kStageK != 0 || (act_type == W4_E4M3 && K % 128 != 0))
    return fail(W4_ERR_UNSUPPORTED, "K must be a positive multiple of 64 (128 for fp8)");
  if (!workspace || !aligned16(workspace)) return fail(W4_ERR_WORKSPACE, "workspace is null or not 16-byte aligned");
  const DynLayout d = dyn_layout(act_type, M, N, K, gs, ep.any(),
                                 epilogue_aligned(ep, out, bias, ch_scales));
  if (workspace_bytes < d.total)
    return fail(W4_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", workspace_bytes, d.total);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* stok = token_scales_out ? token_scales_out : reinterpret_cast<float*>(ws + d.stok);
  void* codes = ws + d.codes;
  // Check the GEMM's arguments before anything is enqueued (the codes and
  // scales it will read are in the workspace).
  {
    Problem pr{};
    w4_status st = validate(codes, act_type, M, K, b_packed, wtype, N, b_scales, scale_type,
                            nullptr, group_size, stok, ch_scales, out, W4_F16, pr);
    if (st != W4_OK) return st;
    if (bias && !aligned_to(bias, 2))
      return fail(W4_ERR_INVALID_ARGUMENT, "bias is not aligned to its element size");
    st = check_epilogue(ep, M, N, out, W4_F16);
    if (st != W4_OK) return st;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> together(enqueue_mutex(workspace));
  void* qdst = codes;
  int qout = act_type == W4_E4M3 ? 2 : 0;
  // the bf16 form is written from rows held in registers (16-byte loads)
  const bool prestage = d.prestage && aligned16(a);
  if (prestage) {
    const TcPlan plan = make_plan(d.si, kW4A8, M, N, K, gs);
    qdst = ws + plan.ws_act;
    qout = 1;
  }
  cudaError_t e = launch_quant_per_token(a_type == W4_BF16, a, M, K, qdst, stok, qout, s);
  if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
  return gemm_impl(codes, act_type, M, K, b_packed, wtype, N, b_scales, scale_type, nullptr,
                   group_size, stok, ch_scales, bias, ep, out, W4_F16, workspace, d.gemm_ws, stream,
                   prestage ? d.si : -1, prestage);
}
}  // namespace

extern "C" {

w4_status w4_gemm_dynamic(const void* a, int a_type, int64_t M, int64_t K, const void* b_packed,
                          int wtype, int64_t N, const void* b_scales, int scale_type,
                          int64_t group_size, const float* ch_scales, int act_type,
                          const void* bias, void* out, float* token_scales_out,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return dynamic_impl(a, a_type, M, K, b_packed, wtype, N, b_scales, scale_type, group_size,
                      ch_scales, act_type, bias, Epilogue{}, out, token_scales_out, workspace,
                      workspace_bytes, stream);
}

w4_status w4_gemm_dynamic_epilogue(const void* a, int a_type, int64_t M, int64_t K,
                                   const void* b_packed, int wtype, int64_t N,
                                   const void* b_scales, int scale_type, int64_t group_size,
                                   const float* ch_scales, int act_type, const void* bias,
                                   int act, int gated, const void* residual, void* out,
                                   float* token_scales_out, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  return dynamic_impl(a, a_type, M, K, b_packed, wtype, N, b_scales, scale_type, group_size,
                      ch_scales, act_type, bias, Epilogue{act, gated != 0 ? 1 : 0, residual}, out,
                      token_scales_out, workspace, workspace_bytes, stream);
}

w4_status w4_gemm_ex(const void* a, int a_type, int64_t M, int64_t K, const void* b_packed,
                     int wtype, int64_t N, const void* b_scales, int scale_type,
                     const void* b_zeros, int64_t group_size, const float* a_token_scales,
                     const float* ch_scales, void* out, int out_type, void* workspace,
                     size_t workspace_bytes, void* stream, int schedule) {
  std::lock_guard<std::mutex> together(enqueue_mutex(workspace));
  return gemm_impl(a, a_type, M, K, b_packed, wtype, N, b_scales, scale_type, b_zeros,
                   group_size, a_token_scales, ch_scales, nullptr, Epilogue{}, out, out_type,
                   workspace, workspace_bytes, stream, schedule);
}

w4_status w4_gemm_bias(const void* a, int a_type, int64_t M, int64_t K, const void* b_packed,
                       int wtype, int64_t N, const void* b_scales, int scale_type,
                       const void* b_zeros, int64_t group_size, const float* a_token_scales,
                       const float* ch_scales, const void* bias, void* out, int out_type,
                       void* workspace, size_t workspace_bytes, void* stream, int schedule) {
  std::lock_guard<std::mutex> together(enqueue_mutex(workspace));
  return gemm_impl(a, a_type, M, K, b_packed, wtype, N, b_scales, scale_type, b_zeros,
                   group_size, a_token_scales, ch_scales, bias, Epilogue{}, out, out_type,
                   workspace, workspace_bytes, stream, schedule);
}

w4_status w4_gemm_epilogue(const void* a, int a_type, int64_t M, int64_t K, const void* b_packed,
                           int wtype, int64_t N, const void* b_scales, int scale_type,
                           const void* b_zeros, int64_t group_size, const float* a_token_scales,
                           const float* ch_scales, const void* bias, int act, int gated,
                           const void* residual, void* out, int out_type, void* workspace,
                           size_t workspace_bytes, void* stream, int schedule) {
  std::lock_guard<std::mutex> together(enqueue_mutex(workspace));
  return gemm_impl(a, a_type, M, K, b_packed, wtype, N, b_scales, scale_type, b_zeros,
                   group_size, a_token_scales, ch_scales, bias,
                   Epilogue{act, gated != 0 ? 1 : 0, residual}, out, out_type, workspace,
                   workspace_bytes, stream, schedule);
}

w4_status w4_gemm(const void* a, int a_type, int64_t M, int64_t K, const void* b_packed,
                  int wtype, int64_t N, const void* b_scales, int scale_type,
                  const void* b_zeros, int64_t group_size, const float* a_token_scales,
                  const float* ch_scales, void* out, int out_type, void* workspace,
                  size_t workspace_bytes, void* stream) {
  return w4_gemm_ex(a, a_type, M, K, b_packed, wtype, N, b_scales, scale_type, b_zeros,
                    group_size, a_token_scales, ch_scales, out, out_type, workspace,
                    workspace_bytes, stream, -1);
}

w4_status w4_quantize_per_token(const void* a, int a_type, int64_t M, int64_t K, int8_t* a_q,
                                float* s_tok, void* stream) {
  if (M < 0 || K < 0) return fail(W4_ERR_INVALID_ARGUMENT, "negative size");
  if (a_type != W4_F16 && a_type != W4_BF16)
    return fail(W4_ERR_INVALID_ARGUMENT, "a_type must be W4_F16 or W4_BF16");
  if (M == 0) return W4_OK;
  if (!s_tok || (K > 0 && (!a || !a_q))) return fail(W4_ERR_INVALID_ARGUMENT, "null pointer");
  if (!aligned_to(a, 2) || !aligned_to(s_tok, 4))
    return fail(W4_ERR_INVALID_ARGUMENT, "a and s_tok must be aligned to their element size");
  if (M > 0x7fffffff) return fail(W4_ERR_UNSUPPORTED, "M above 2^31 - 1");
  cudaError_t e = launch_quant_per_token(a_type == W4_BF16, a, M, K, a_q, s_tok, 0,
                                         static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "quantize launch");
}

w4_status w4_quantize_per_token_fp8(const void* a, int a_type, int64_t M, int64_t K,
                                    uint8_t* a_q, float* s_tok, void* stream) {
  if (M < 0 || K < 0) return fail(W4_ERR_INVALID_ARGUMENT, "negative size");
  if (a_type != W4_F16 && a_type != W4_BF16)
    return fail(W4_ERR_INVALID_ARGUMENT, "a_type must be W4_F16 or W4_BF16");
  if (M == 0) return W4_OK;
  if (!s_tok || (K > 0 && (!a || !a_q))) return fail(W4_ERR_INVALID_ARGUMENT, "null pointer");
  if (!aligned_to(a, 2) || !aligned_to(s_tok, 4))
    return fail(W4_ERR_INVALID_ARGUMENT, "a and s_tok must be aligned to their element size");
  if (M > 0x7fffffff) return fail(W4_ERR_UNSUPPORTED, "M above 2^31 - 1");
  cudaError_t e = launch_quant_per_token(a_type == W4_BF16, a, M, K, a_q, s_tok, 2,
                                         static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "quantize launch");
}

w4_status w4_rmsnorm(const void* x, int x_type, int64_t M, int64_t K, const void* residual,
                     const void* weight, float eps, void* residual_out, void* y, int y_type,
                     float* y_scales, void* stream) {
  if (M < 0 || K < 0) return fail(W4_ERR_INVALID_ARGUMENT, "negative size");
  if (x_type != W4_F16 && x_type != W4_BF16)
    return fail(W4_ERR_INVALID_ARGUMENT, "x_type must be W4_F16 or W4_BF16");
  const bool q8 = y_type == W4_S8 || y_type == W4_E4M3;
  if (!q8 && y_type != x_type)
    return fail(W4_ERR_INVALID_ARGUMENT, "y_type must be x_type, W4_S8 or W4_E4M3");
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return fail(W4_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
  if (residual_out && !residual)
    return fail(W4_ERR_INVALID_ARGUMENT, "residual_out without a residual");
  if (y_scales && !q8) return fail(W4_ERR_INVALID_ARGUMENT, "a 16-bit output takes no scales");
  if (M == 0) return W4_OK;
  if (q8 && !y_scales) return fail(W4_ERR_INVALID_ARGUMENT, "an 8-bit output needs y_scales");
  if (K > 0 && (!x || !y)) return fail(W4_ERR_INVALID_ARGUMENT, "null pointer");
  if (!aligned_to(x, 2) || !aligned_to(residual, 2) || !aligned_to(weight, 2) ||
      !aligned_to(residual_out, 2) || !aligned_to(y, q8 ? 1 : 2) || !aligned_to(y_scales, 4))
    return fail(W4_ERR_INVALID_ARGUMENT, "a pointer is not aligned to its element size");
  if (M > 0x7fffffff) return fail(W4_ERR_UNSUPPORTED, "M above 2^31 - 1");
  if (K > 0x7fffffff) return fail(W4_ERR_UNSUPPORTED, "K above 2^31 - 1");
  // an output may take the place of x or residual, element for element
  const size_t e16 = static_cast<size_t>(M) * K * 2, ey = q8 ? e16 / 2 : e16;
  const size_t es = q8 ? static_cast<size_t>(M) * 4 : 0, ew = weight ? K * 2 : 0;
  const bool bad =
      overlap_but_same(residual_out, e16, x, e16) ||
      overlap_but_same(residual_out, e16, residual, e16) ||
      (q8 ? overlap(y, ey, x, e16) || overlap(y, ey, residual, e16)
          : overlap_but_same(y, ey, x, e16) || overlap_but_same(y, ey, residual, e16)) ||
      overlap(residual_out, e16, y, ey) || overlap(residual_out, e16, weight, ew) ||
      overlap(y, ey, weight, ew) || overlap(y_scales, es, x, e16) ||
      overlap(y_scales, es, residual, e16) || overlap(y_scales, es, weight, ew) ||
      overlap(y_scales, es, y, ey) || overlap(y_scales, es, residual_out, e16);
  if (bad) return fail(W4_ERR_INVALID_ARGUMENT, "an output overlaps another array");
  NormArgs a{};
  a.bf16 = x_type == W4_BF16;
  a.out = y_type == W4_S8 ? kNormS8 : y_type == W4_E4M3 ? kNormE4M3 : kNorm16;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.h_out = residual_out;
  a.y = y;
  a.scales = y_scales;
  a.M = M;
  a.K = K;
  a.eps = eps;
  cudaError_t e = launch_norm(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "norm launch");
}

w4_status w4_cache_write(const w4_kv_cache* cache, const w4_kv_batch* batch, const void* k,
                         const void* v, int type, int64_t rows, int64_t k_stride,
                         int64_t v_stride, void* stream) {
  CacheWriteArgs a{};
  w4_status st = cache_views(cache, batch, type, rows, a.c, a.b);
  if (st != W4_OK) return st;
  const int64_t dense = static_cast<int64_t>(cache->heads) * cache->head_dim;
  if ((k_stride < dense || v_stride < dense) && rows > 1)
    return fail(W4_ERR_INVALID_ARGUMENT, "a row stride is below heads * head_dim");
  if (rows == 0 || batch->sequences == 0) return W4_OK;
  if (!k || !v) return fail(W4_ERR_INVALID_ARGUMENT, "k and v are required");
  if (!aligned_to(k, 2) || !aligned_to(v, 2))
    return fail(W4_ERR_INVALID_ARGUMENT, "k or v is not aligned to its element size");
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.bf16 = type == W4_BF16;
  const cudaError_t e = launch_cache_write(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "cache write launch");
}

w4_status w4_cache_read(const w4_kv_cache* cache, const w4_kv_batch* batch, void* k, void* v,
                        int type, int64_t rows, void* stream) {
  CacheReadArgs a{};
  w4_status st = cache_views(cache, batch, type, rows, a.c, a.b);
  if (st != W4_OK) return st;
  if (rows == 0 || batch->sequences == 0) return W4_OK;
  if (!k || !v) return fail(W4_ERR_INVALID_ARGUMENT, "k and v are required");
  if (!aligned_to(k, 2) || !aligned_to(v, 2))
    return fail(W4_ERR_INVALID_ARGUMENT, "k or v is not aligned to its element size");
  const size_t bytes = static_cast<size_t>(rows) * cache->heads * cache->head_dim * 2;
  if (overlap(k, bytes, v, bytes) || overlaps_cache(cache, k, bytes) || overlaps_cache(cache, v, bytes))
    return fail(W4_ERR_INVALID_ARGUMENT, "an output overlaps the other or the cache");
  a.k = k;
  a.v = v;
  a.bf16 = type == W4_BF16;
  const cudaError_t e = launch_cache_read(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "cache read launch");
}

size_t w4_attention_workspace_size(const w4_kv_cache* cache, const w4_kv_batch* batch,
                                   int64_t rows, int heads) {
  if (!cache || !batch) return kWsHeader + kCounterBytes;
  const AttnPlan p = attn_plan(cache, batch, rows, heads, 0, 0, true);
  return kWsHeader + kCounterBytes + align256(p.partials) + p.tiles;
}

w4_status w4_cache_attention(const w4_kv_cache* cache, const w4_kv_batch* batch, const void* q,
                             int type, int64_t rows, int heads, int64_t q_stride, float scale,
                             int window, int sinks, void* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return attention(cache, batch, q, nullptr, 0, type, rows, heads, q_stride, scale, window, sinks,
                   out, workspace, workspace_bytes, stream);
}

w4_status w4_tree_attention(const w4_kv_cache* cache, const w4_kv_batch* batch, const void* q,
                            const uint8_t* mask, int64_t mask_width, int type, int64_t rows,
                            int heads, int64_t q_stride, float scale, int window, int sinks,
                            void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (mask_width < 0) return fail(W4_ERR_INVALID_ARGUMENT, "negative mask_width");
  if (!mask && rows > 0) return fail(W4_ERR_INVALID_ARGUMENT, "mask is required");
  return attention(cache, batch, q, mask, mask_width, type, rows, heads, q_stride, scale, window,
                   sinks, out, workspace, workspace_bytes, stream);
}

w4_status w4_check_status(void* workspace, size_t workspace_bytes, void* stream) {
  if (!workspace || workspace_bytes < kWsHeader)
    return fail(W4_ERR_WORKSPACE, "workspace is null or smaller than its header");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  int word = 0;
  e = cudaMemcpy(&word, workspace, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  if (word == 0) return W4_OK;
  size_t clear = workspace_bytes < kWsHeader + kCounterBytes ? workspace_bytes
                                                            : kWsHeader + kCounterBytes;
  e = cudaMemset(workspace, 0, clear);
  if (e != cudaSuccess) return cuda_fail(e, "status reset");
  return fail(W4_ERR_TIMEOUT, "a device-side wait timed out");
}

const char* w4_status_string(int status) {
  switch (status) {
    case W4_OK: return "W4_OK";
    case W4_ERR_INVALID_ARGUMENT: return "W4_ERR_INVALID_ARGUMENT";
    case W4_ERR_UNSUPPORTED: return "W4_ERR_UNSUPPORTED";
    case W4_ERR_WORKSPACE: return "W4_ERR_WORKSPACE";
    case W4_ERR_CUDA: return "W4_ERR_CUDA";
    case W4_ERR_TIMEOUT: return "W4_ERR_TIMEOUT";
    default: return "W4_ERR_UNKNOWN";
  }
}

const char* w4_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
