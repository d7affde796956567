// rel_attn_sink.cu -- host side of the sliding-window attention with sinks
// (rel_attn_sink_decode, rel_attn_sink_prefill and their E4M3 forms):
// argument checks, the split heuristic and the launches.
#include <algorithm>
#include <cstring>

#include "rel_attn_sink_step.cuh"
#include "rel_attn_sink_tiles.h"

namespace relattn {
namespace sink {
namespace {

template <class K, typename F>
int launch_step(F* kernel, const Params& prm, const rel_attn_shape* s, int dev, bool (&set)[kMaxDev], cudaStream_t st) {
  if (!allow_shared(kernel, K::kAlloc, dev, set)) return REL_ATTN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(prm.num_splits, s->num_kv_heads, s->batch);
  cfg.blockDim = dim3(K::kThreads);
  cfg.dynamicSmemBytes = K::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)prm.num_splits, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = prm.num_splits > 1 && prm.num_splits <= kMaxCluster ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, prm) != cudaSuccess) {
    cudaGetLastError();
    return REL_ATTN_ERR_CUDA;
  }
  return REL_ATTN_OK;
}

template <bool F8, bool PARTS>
int launch_one(const Params& prm, const rel_attn_shape* s, int dev, cudaStream_t st) {
  static bool set[kMaxDev];
  return launch_step<StepConfig<F8>>(sink_step_kernel<F8, PARTS>, prm, s, dev, set, st);
}

int launch_codes(const Params& prm, const rel_attn_shape* s, int dev, cudaStream_t st) {
  static bool set[kMaxDev];
  return launch_step<CodesConfig>(sink_codes_kernel, prm, s, dev, set, st);
}

// Pages that one sequence's step can see, at most.
long long pages_bound(const rel_attn_shape* s, int window, int sinks, int tokens) {
  const long long cap = (long long)s->max_pages_per_seq * kKeys;
  const long long len = s->max_seq_len > 0 ? std::min<long long>(s->max_seq_len, cap) : cap;
  return std::min((len + kKeys - 1) / kKeys,
                  ((long long)sinks + kKeys - 1) / kKeys + ((long long)window + tokens - 2) / kKeys + 2);
}

// Splits of the step and codes kernels: their blocks fill the GPU once, up to 8
// to a sequence and KV head where a few pages to a block are enough.  (2 tokens
// over 512 keys, one sequence: whole 23 us, in 8 9; 32 sequences of 4 tokens
// whole 28, in 2 35.)
int splits_steps(const rel_attn_shape* s, int window, int sinks, int sm_count) {
  const long long units = (long long)s->batch * s->num_kv_heads;
  const long long pages = pages_bound(s, window, sinks, s->q_tokens);
  long long n = std::max(1LL, 2LL * sm_count / units);       // (two blocks to an SM)
  if (n > kMaxCluster && pages <= 4 * kMaxCluster) n = kMaxCluster;
  return (int)std::max(1LL, std::min({n, pages, 256LL}));
}

// Splits of the tile kernel: the fewest page times of the busiest SM, a tile's
// beginning and end counted as kTileCost pages and the combine kernel as
// kCombineCost.  8 tokens, chosen against every other count of splits: over codes
// and 1,024 keys 2 sequences with 64/8 heads in 8 15.0 us (whole 25.1, in 6 14.7),
// 16 with 32/8 heads whole 30.0 (in 2 48.0); over bf16 one with 48/8 heads and
// 32K keys in 18 39.5 (whole 464, in 16 41.4), 16 over 1,024 keys whole 22.6 (in 2
// 41.2), 8 in 2 24.4 (whole 20.9: the rule's worst case).
int splits_tiles(const rel_attn_shape* s, int window, int sinks, int sm_count) {
  constexpr double kTileCost = 6, kCombineCost = 4;
  const int G = s->num_q_heads / s->num_kv_heads, per = 128 / G;
  const long long tiles = (long long)s->batch * s->num_kv_heads * ((s->q_tokens + per - 1) / per);
  const double pages = (double)pages_bound(s, window, sinks, std::min(s->q_tokens, per));
  int best = 1;
  double least = 0;
  for (int n = 1; n <= 256 && n <= pages && (n == 1 || tiles * n <= 2LL * sm_count); ++n) {
    const double cost = (double)((tiles * n + sm_count - 1) / sm_count) * (pages / n + kTileCost) + (n > 1 ? kCombineCost : 0);
    if (n == 1 || cost < least) {
      best = n;
      least = cost;
    }
  }
  return best;
}

// Several tokens go to the tile kernel.  Over codes those of up to 16 rows to a
// KV head have a kernel of their own: (64 query heads, 8 KV heads) 16 sequences
// of 2 tokens over 1,024 keys 26.1 us, as tiles 27.6; (32, 8) 32 sequences of 4
// tokens over 512 keys 27.2 against 36.3.  With more rows tiles win: (32, 8) 16
// sequences of 8 tokens over 1,024 keys 30 against 61.
// (A page of those two kernels holds 64 or 72 relative rows: a table whose
// indices lie further apart goes to the tiles as well.)
bool tiled(const rel_attn_shape* s, bool e4m3, bool prefill) {
  if (prefill || (s->q_tokens > 1 && !(e4m3 && s->q_tokens * (s->num_q_heads / s->num_kv_heads) <= 16))) return true;
  return host::page_bucket_span(s, s->q_tokens) > (s->q_tokens == 1 ? 64 : 72);
}

int choose_splits(const rel_attn_shape* s, int window, int sinks, int sm_count, bool tiles) {
  return tiles ? splits_tiles(s, window, sinks, sm_count) : splits_steps(s, window, sinks, sm_count);
}

bool off(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0; }

int check_shape(const rel_attn_shape* s, int window, int sinks, bool prefill) {
  if (!s || window < 1 || sinks < 0) return REL_ATTN_ERR_INVALID_ARG;
  rel_attn_shape step = *s;
  if (prefill) {
    if (s->q_tokens < 1 || s->q_tokens > (1 << 20)) return REL_ATTN_ERR_INVALID_ARG;
    step.q_tokens = 1;                  // (the rest of the shape is checked as a step's)
  }
  return host::validate(&step);
}

// One token, or a few over codes.
int run_step(const rel_attn_shape* s, const Params& prm, bool e4m3, int dev, cudaStream_t st) {
  if (prm.T == 1)
    return (e4m3 ? prm.out_fp32 ? launch_one<true, true> : launch_one<true, false>
                 : prm.out_fp32 ? launch_one<false, true> : launch_one<false, false>)(prm, s, dev, st);
  return launch_codes(prm, s, dev, st);
}

// What both kinds of parameters have.
template <class P>
void fill(P& prm, const rel_attn_shape* s, const int32_t* block_table, const int32_t* seq_lens, int window, int sinks,
          void* out, float* lse, void* workspace, int splits) {
  memset(&prm, 0, sizeof(prm));
  const size_t rows = (size_t)s->batch * s->q_tokens * s->num_q_heads;
  host::workspace_parts(workspace, splits, rows, &prm.status, &prm.ws_lse, &prm.ws_o);
  host::buckets(s, &prm.bt);
  prm.block_table = block_table;
  prm.seq_lens = seq_lens;
  prm.out = out;
  prm.lse = lse;
  prm.timeout_ns = host::wait_limit_ns();
  prm.Hq = s->num_q_heads;
  prm.rows_total = (int)rows;
  prm.num_pages = s->num_pages;
  prm.max_pages = s->max_pages_per_seq;
  const int capacity = s->max_pages_per_seq * kKeys;  // (further ones are the same, without their overflows)
  prm.window = std::min(window, capacity);
  prm.sinks = std::min(sinks, capacity);
  prm.out_fp32 = s->out_fp32;
}

int run(const rel_attn_shape* s, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
        const float* v_scale, bool e4m3, bool prefill, const int32_t* block_table, const int32_t* seq_lens,
        const void* rel_table, int window, int sinks, int num_splits, void* out, float* lse, void* workspace,
        size_t bytes, void* stream) {
  // ---- arguments (no CUDA call before this block passes)
  int rc = check_shape(s, window, sinks, prefill);
  if (rc != REL_ATTN_OK) return rc;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !rel_table || !out || !workspace ||
      (e4m3 && (!k_scale || !v_scale || off(k_scale, 4) || off(v_scale, 4))))
    return REL_ATTN_ERR_INVALID_ARG;
  if (off(q, 16) || off(k_cache, 16) || off(v_cache, 16) || off(rel_table, 16) || off(out, 16) ||
      off(workspace, 256) || off(block_table, 4) || off(seq_lens, 4) || (lse && off(lse, 4)))
    return REL_ATTN_ERR_INVALID_ARG;
  if (num_splits > 256) return REL_ATTN_ERR_INVALID_ARG;
  if (bytes < kWorkspaceHeader) return REL_ATTN_ERR_WORKSPACE_TOO_SMALL;
  int dev, sms;
  rc = host::current_device(&dev, &sms);
  if (rc != REL_ATTN_OK) return rc;
  const bool tiles = tiled(s, e4m3, prefill);
  int splits = num_splits > 0 ? num_splits : choose_splits(s, window, sinks, sms, tiles);
  const bool merged = splits == 1 || (!tiles && splits <= kMaxCluster);        // in the same launch
  if (!merged && bytes < host::workspace_bytes(s, splits)) {
    if (!prefill) return REL_ATTN_ERR_WORKSPACE_TOO_SMALL;
    splits = 1;                         // (a prefill splits where it is given the room)
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tiles) {
    TileParams prm;
    fill(prm, s, block_table, seq_lens, window, sinks, out, lse, workspace, splits);
    if (!host::pool_map(&prm.tmap_k, k_cache, s, false, e4m3) || !host::pool_map(&prm.tmap_v, v_cache, s, true, e4m3))
      return REL_ATTN_ERR_CUDA;
    prm.rel = reinterpret_cast<const __nv_bfloat16*>(rel_table);
    prm.k_scale = k_scale;
    prm.v_scale = v_scale;
    prm.B = s->batch;
    prm.C = s->q_tokens;
    prm.Hkv = s->num_kv_heads;
    prm.NB = s->num_buckets;
    prm.splits = splits;
    const bool few = prm.window - 1 > prm.bt.ex;    // pages of the window lie in the log buckets
    rc = (e4m3 ? few ? run_tiles<true, true> : run_tiles<true, false>
               : few ? run_tiles<false, true> : run_tiles<false, false>)(s, q, rel_table, prm, sms, dev, st);
  } else {
    Params prm;
    fill(prm, s, block_table, seq_lens, window, sinks, out, lse, workspace, splits);
    if (!host::pool_map(&prm.tmap_k, k_cache, s, false, e4m3) || !host::pool_map(&prm.tmap_v, v_cache, s, true, e4m3) ||
        !host::rel_map(&prm.tmap_r, rel_table, s, s->q_tokens == 1 ? 64 : 72))
      return REL_ATTN_ERR_CUDA;
    prm.q = reinterpret_cast<const __nv_bfloat16*>(q);
    prm.k_scale = k_scale;
    prm.v_scale = v_scale;
    prm.T = s->q_tokens;
    prm.G = s->num_q_heads / s->num_kv_heads;
    prm.num_splits = splits;
    rc = run_step(s, prm, e4m3, dev, st);
  }
  if (rc != REL_ATTN_OK || splits == 1 || (!tiles && splits <= kMaxCluster)) return rc;
  return host::combine(s, splits, out, lse, workspace, st);
}

size_t workspace_bytes(const rel_attn_shape* s, int window, int sinks, int splits, bool e4m3, bool prefill) {
  if (check_shape(s, window, sinks, prefill) != REL_ATTN_OK || splits > 256) return 0;
  const bool tiles = tiled(s, e4m3, prefill);
  if (splits <= 0) {
    int dev, sms;
    if (host::current_device(&dev, &sms) != REL_ATTN_OK) sms = 148;
    splits = choose_splits(s, window, sinks, sms, tiles);
  }
  return splits == 1 || (!tiles && splits <= kMaxCluster) ? kWorkspaceHeader : host::workspace_bytes(s, splits);
}

}  // namespace
}  // namespace sink
}  // namespace relattn

using namespace relattn;

extern "C" size_t rel_attn_sink_workspace_bytes(const rel_attn_shape* shape, int window, int num_sinks, int num_splits) {
  // (of the two caches the one that needs more)
  return std::max(sink::workspace_bytes(shape, window, num_sinks, num_splits, false, false),
                  sink::workspace_bytes(shape, window, num_sinks, num_splits, true, false));
}

extern "C" size_t rel_attn_sink_prefill_workspace_bytes(const rel_attn_shape* shape, int window, int num_sinks) {
  return sink::workspace_bytes(shape, window, num_sinks, 0, false, true);
}

extern "C" int rel_attn_sink_decode(const rel_attn_shape* shape, const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_table, const int32_t* seq_lens, const void* rel_table,
                                    int window, int num_sinks, int num_splits, void* out, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return sink::run(shape, q, k_cache, v_cache, nullptr, nullptr, false, false, block_table, seq_lens, rel_table, window,
                   num_sinks, num_splits, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int rel_attn_sink_decode_e4m3(const rel_attn_shape* shape, const void* q, const void* k_cache,
                                         const void* v_cache, const float* k_scale, const float* v_scale,
                                         const int32_t* block_table, const int32_t* seq_lens, const void* rel_table,
                                         int window, int num_sinks, int num_splits, void* out, float* lse,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  return sink::run(shape, q, k_cache, v_cache, k_scale, v_scale, true, false, block_table, seq_lens, rel_table, window,
                   num_sinks, num_splits, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int rel_attn_sink_prefill(const rel_attn_shape* shape, const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* block_table, const int32_t* seq_lens, const void* rel_table,
                                     int window, int num_sinks, void* out, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  return sink::run(shape, q, k_cache, v_cache, nullptr, nullptr, false, true, block_table, seq_lens, rel_table, window,
                   num_sinks, 0, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int rel_attn_sink_prefill_e4m3(const rel_attn_shape* shape, const void* q, const void* k_cache,
                                          const void* v_cache, const float* k_scale, const float* v_scale,
                                          const int32_t* block_table, const int32_t* seq_lens, const void* rel_table,
                                          int window, int num_sinks, void* out, float* lse, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  return sink::run(shape, q, k_cache, v_cache, k_scale, v_scale, true, true, block_table, seq_lens, rel_table, window,
                   num_sinks, 0, out, lse, workspace, workspace_bytes, stream);
}
