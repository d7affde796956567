// rel_attn_sink_step.cuh -- the attention of rel_attn_sink_common.cuh for one
// token over either cache (step kernel) and for a few tokens over an E4M3 cache
// (codes kernel).
//
// One CTA walks a range of the pages that hold a visible key (the sinks'
// pages, then the window's) for one sequence and KV head; a page is a tile of
// 64 keys.  One warp copies the page's K, V and relative rows to shared memory
// (TMA, 128-byte swizzle), the others compute on warp-level matrix
// instructions.  A step of one token has 4 to 8 rows to a KV head and is bound
// by memory or, for one window of a thousand keys, by latency: what counts is
// that nothing is staged, converted or exchanged between warps inside the
// loop, and that enough pages are under way.  Each warp keeps its own online
// softmax.
//
// The relative term.  Row u of a page's relative chunk, reversed, belongs to
// distance p_0 + T - 1 - j_0 - u, so that key jj of token t needs row
// jj + (T - 1 - t).  The chunk holds each bucket once; a row's address is
// formed per lane where the matrix instruction's operand is loaded, which is
// the gather.  With one token the product lands on the logits' own
// accumulators; with several it goes through a warp's own strip of shared
// memory and comes back shifted by T - 1 - t columns.
//
// The parts of a cluster's CTAs (up to 8 splits) are merged through
// distributed shared memory in the same launch; more splits go through the
// workspace and the combine kernel.
#pragma once

#include "rel_attn_sink_common.cuh"

namespace relattn {
namespace sink {

constexpr int kMaxCluster = 8;
// log2: a logit may be this far above the reference before that follows; and where
// the reference is put below a maximum that it follows to.  f16 weights reach
// 2^15 and keep their 22 bits in two parts down to 2^-4 (with the reference at the
// maximum itself a weight of 2^-7 would keep 17: its second part would be subnormal).
template <bool F8> constexpr float kBelow = F8 ? 7.f : 0.f;
template <bool F8> constexpr float kRescaleAt = 8.f + kBelow<F8>;

struct Params {
  CUtensorMap tmap_k, tmap_v, tmap_r;
  const __nv_bfloat16* q;
  const int* block_table;
  const int* seq_lens;
  const float* k_scale;
  const float* v_scale;
  void* out;
  float* lse;
  float* ws_lse;
  float* ws_o;
  unsigned* status;
  unsigned long long timeout_ns;
  int T, G, Hq;
  int rows_total, num_pages, max_pages, window, sinks, num_splits, out_fp32;
  BucketTable bt;
};

// Shared memory behind the stages, alike in both kernels: offsets from kTail.
template <int STAGES, int FULL, int MERGE_ROWS>
struct Tail {
  static constexpr int oEdges = 0;
  static constexpr int oMl = oEdges + 516 * 4;             // float2 {reference, sum} of each part's row
  static constexpr int oInfo = oMl + MERGE_ROWS * 8;       // int4 {first key, first bucket, bad, -} of a stage
  static constexpr int oBar = oInfo + STAGES * 16;
  static constexpr int oFlags = oBar + (FULL + STAGES) * 8;
  static constexpr int kBytes = oFlags + 16;
};

// One token: G rows of one KV head are the 8 columns of the products, keys and
// head dims their rows.  Four warps to a page, 16 keys each, and two pages at a
// time; two CTAs to an SM.
template <bool F8>
struct StepConfig {
  static constexpr int kKeyWarps = 4, kStreams = 2, kWarps = kKeyWarps * kStreams;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kKvBytes = kKeys * kDim * (F8 ? 1 : 2), kRelHalf = 64 * 128;
  static constexpr int kStageBytes = 2 * kKvBytes + 2 * kRelHalf;
  static constexpr int kStages = F8 ? 3 : 2;
  // barriers of arrived pages: a ring of both the stages and the streams, so that
  // a barrier has one stream's pages alone.  (With one to a stage, three stages
  // and two streams, a stream that was ahead by a page took the other one's phase
  // before last for its own, and read a page that was still arriving.)
  static constexpr int kFull = F8 ? 6 : 2;
  static_assert(kFull % kStages == 0 && kFull % kStreams == 0, "one stream to a barrier");
  static constexpr int kRowStride = 132;                   // floats of a merged row: 4 banks on per row
  static constexpr int kTail = kStages * kStageBytes;
  using T = Tail<kStages, kFull, kWarps * 8>;
  static constexpr int kAlloc = kTail + T::kBytes + 1024;
  static_assert(kWarps * 8 * kRowStride * 4 <= kTail, "the warps' outputs reuse the stages");
  static_assert(2 * (kAlloc + 1024) <= 233472, "two CTAs to an SM");
};

// A few tokens over codes: up to 16 rows, a quarter of a page's keys to a warp.
struct CodesConfig {
  static constexpr int kWarps = 4;                         // share a page's keys
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kWarpKeys = kKeys / kWarps;
  static constexpr int kChunk = 72;                        // relative rows of a page
  static constexpr int kKvBytes = kKeys * kDim;
  static constexpr int kRelHalf = kChunk * 128;
  static constexpr int kStageBytes = 2 * kKvBytes + 2 * kRelHalf;
  static constexpr int kStages = 3, kFull = kStages;       // (all warps take every page)
  static constexpr int kXStride = kWarpKeys + 8;           // floats of a row of a warp's strip
  static constexpr int oX = kStages * kStageBytes;
  static constexpr int kTail = oX + kWarps * 16 * kXStride * 4;
  using T = Tail<kStages, kFull, kWarps * 16>;
  static constexpr int kAlloc = kTail + T::kBytes + 1024;
  static_assert(kWarps * 16 * kDim * 4 <= kStages * kStageBytes, "the warps' outputs reuse the stages");
};

// ------------------------------------------------------------------ pieces
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// a b^T
template <bool HALF>
__device__ __forceinline__ void mma_from_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (HALF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
template <bool HALF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (HALF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the 8x8 matrix of 16-bit values that a warp holds, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
  return fmaxf(v, __shfl_xor_sync(~0u, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(~0u, v, 1);
  return v + __shfl_xor_sync(~0u, v, 2);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_remote2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_remote4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// One finished row: 4 of its 128 outputs per lane, natural-log lse.
__device__ __forceinline__ void store_row(const Params& p, size_t row, int lane, float4 o, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;      // no visible key: zeros and -inf
  o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
  if (p.out_fp32) {
    reinterpret_cast<float4*>(p.out)[row * (kDim / 4) + lane] = o;
  } else {
    reinterpret_cast<uint2*>(p.out)[row * (kDim / 4) + lane] =
        make_uint2(pack<false>(o.x, o.y), pack<false>(o.z, o.w));
  }
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// ------------------------------------------------------ shared by the kernels
// What a CTA works on.
struct Job {
  int b, h, split, v0, v1, p_last;
  bool bad;                                         // length out of range
  Walk walk;
  __device__ __forceinline__ Job(const Params& p)
      : b(blockIdx.z), h(blockIdx.y), split(blockIdx.x), walk(1, 1, 1, 0) {
    const int L = __ldg(p.seq_lens + b);
    bad = L != 0 && (L < p.T || L > p.max_pages * kKeys);
    const bool none = L == 0 || bad;                // (0: a free slot of the batch: zeros and -inf)
    walk = Walk(none ? p.T : L, p.T, p.window, p.sinks);
    const int nv = none ? 0 : walk.nv;
    v0 = (int)((long long)nv * split / p.num_splits);
    v1 = (int)((long long)nv * (split + 1) / p.num_splits);
    p_last = walk.p0 + p.T - 1;
  }
  // no row of the page masks any of its keys
  __device__ __forceinline__ bool whole(const Params& p, int j0) const {
    return j0 + kKeys - 1 <= walk.p0 && (j0 > p_last - p.window || j0 + kKeys <= p.sinks);
  }
  // some row sees position j
  __device__ __forceinline__ bool seen(const Params& p, int j) const {
    return j <= p_last && (walk.p0 - j < p.window || j < p.sinks);
  }
};

// Barriers, flags and the edge table; then everything that a kernel before
// this one wrote may be read.
template <class K>
__device__ __forceinline__ void begin(const Params& p, uint8_t* tail, int warps_of_a_stage) {
  const uint32_t full = ptx::smem_addr(tail) + K::T::oBar, empty = full + 8 * K::kFull;
  volatile int* const flags = reinterpret_cast<volatile int*>(tail + K::T::oFlags);   // abort, bad page, drain
  if (threadIdx.x == 0) {
    for (int s = 0; s < K::kFull; ++s) ptx::mbar_init(full + 8 * s, 1);
    for (int s = 0; s < K::kStages; ++s) ptx::mbar_init(empty + 8 * s, warps_of_a_stage);
    flags[0] = flags[1] = flags[2] = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tmap_k);
    ptx::prefetch_tmap(&p.tmap_v);
    ptx::prefetch_tmap(&p.tmap_r);
  }
  if (p.bt.nl > 1)
    for (int i = threadIdx.x; i <= p.bt.nl; i += K::kThreads) reinterpret_cast<int*>(tail + K::T::oEdges)[i] = p.bt.edges[i];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_primary();
  __syncthreads();
}

// The copying warp: every page of the job through the stages.
template <class K, bool F8>
__device__ __forceinline__ void copy_pages(const Params& p, const Job& job, uint32_t stages, uint8_t* tail) {
  const uint32_t full = ptx::smem_addr(tail) + K::T::oBar, empty = full + 8 * K::kFull;
  volatile int* const flags = reinterpret_cast<volatile int*>(tail + K::T::oFlags);
  int4* const info = reinterpret_cast<int4*>(tail + K::T::oInfo);
  const int* const edges = reinterpret_cast<const int*>(tail + K::T::oEdges);
  const int lane = threadIdx.x & 31;
  int entry = 0, issued = 0;
  for (int v = job.v0; v < job.v1; ++v) {
    const int it = v - job.v0, s = it % K::kStages;
    if ((it & 31) == 0 && v + lane < job.v1)
      entry = __ldg(p.block_table + (size_t)job.b * p.max_pages + job.walk.logical(v + lane));
    const int page = __shfl_sync(~0u, entry, it & 31);
    // (one vote: no lane leaves the loop alone where a wait runs out)
    if (it >= K::kStages &&
        !__all_sync(~0u, ptx::mbar_wait(empty + 8 * s, ((it / K::kStages) - 1) & 1, flags, p.timeout_ns)))
      break;
    if (lane == 0) {
      const int j0 = job.walk.logical(v) * kKeys;
      const int base = bucket_of(max(0, job.walk.p0 - j0 - (kKeys - 1)), p.bt, edges);
      const bool bad = page < 0 || page >= p.num_pages;
      info[s] = make_int4(j0, base, bad, 0);
      if (bad) {
        flags[1] = 1;
        ptx::mbar_arrive(full + 8 * (it % K::kFull));
      } else {
        const uint32_t st = stages + s * K::kStageBytes, bar = full + 8 * (it % K::kFull);
        const int y = (page * (int)gridDim.y + job.h) * kKeys;
        const uint64_t once = ptx::l2_policy_evict_first();
        ptx::mbar_arrive_expect_tx(bar, K::kStageBytes);
        ptx::tma_load_2d(st, &p.tmap_k, bar, 0, y, once);
        if (!F8) ptx::tma_load_2d(st + K::kKvBytes / 2, &p.tmap_k, bar, 64, y, once);
        ptx::tma_load_3d(st + 2 * K::kKvBytes, &p.tmap_r, bar, 0, base, job.h);
        ptx::tma_load_3d(st + 2 * K::kKvBytes + K::kRelHalf, &p.tmap_r, bar, 64, base, job.h);
        ptx::tma_load_2d(st + K::kKvBytes, &p.tmap_v, bar, 0, y, once);
        if (!F8) ptx::tma_load_2d(st + K::kKvBytes + K::kKvBytes / 2, &p.tmap_v, bar, 64, y, once);
      }
    }
    issued = it + 1;
    __syncwarp();
  }
  // the copies in flight land before the block ends or reuses the stages,
  // whatever became of the warps that were to read them
  for (int it = max(0, issued - K::kStages); it < issued; ++it)
    ptx::mbar_wait(full + 8 * (it % K::kFull), (it / K::kFull) & 1, flags + 2, kDrainNs);
  __syncwarp();
}

// The parts of PARTS groups of warps (rows of STRIDE floats, `per` rows to a
// part) to the CTA's rows, and on: to the output, to the workspace, or through
// the cluster.  All threads of all the job's CTAs call it.
template <class K, bool F8, int PARTS, int STRIDE>
__device__ __forceinline__ void finish(const Params& p, const Job& job, float* part, uint8_t* tail, int per) {
  float2* const ml = reinterpret_cast<float2*>(tail + K::T::oMl);
  volatile int* const flags = reinterpret_cast<volatile int*>(tail + K::T::oFlags);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = K::kThreads / 32;
  const int R = p.G * p.T;
  const bool poison = job.bad || flags[0] || flags[1];
  if (poison && tid == 0)
    atomicOr(p.status, (flags[0] ? kStatusBitTimeout : 0u) | (job.bad || flags[1] ? kStatusBitBadSeq : 0u));
  const float vs = F8 ? __ldg(p.v_scale + job.h) : 1.f;
  const float qnan = __int_as_float(0x7fc00000);
  const bool clustered = p.num_splits > 1 && p.num_splits <= kMaxCluster;
  for (int r = warp; r < R; r += warps) {
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < PARTS; ++g) m = fmaxf(m, ml[g * per + r].x);
#pragma unroll
    for (int g = 0; g < PARTS; ++g) {
      const float2 s = ml[g * per + r];
      const float w = s.x == -INFINITY ? 0.f : exp2_fast(s.x - m);
      const float4 y = reinterpret_cast<const float4*>(part + (size_t)(g * per + r) * STRIDE)[lane];
      l += s.x == -INFINITY ? s.y : s.y * w;        // (a NaN sum stays)
      a.x = fmaf(w, y.x, a.x); a.y = fmaf(w, y.y, a.y); a.z = fmaf(w, y.z, a.z); a.w = fmaf(w, y.w, a.w);
    }
    if (poison) { l = qnan; m = 0.f; a = make_float4(qnan, qnan, qnan, qnan); }
    a.x *= vs; a.y *= vs; a.z *= vs; a.w *= vs;
    const int t = r / p.G;
    const size_t row = ((size_t)job.b * p.T + t) * p.Hq + job.h * p.G + (r - t * p.G);
    if (clustered) {
      __syncwarp();
      reinterpret_cast<float4*>(part + (size_t)r * STRIDE)[lane] = a;
      if (lane == 0) ml[r] = make_float2(m, l);
    } else if (p.num_splits == 1) {
      store_row(p, row, lane, a, m, l);
    } else {
      const size_t at = (size_t)job.split * p.rows_total + row;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      reinterpret_cast<float4*>(p.ws_o + at * kDim)[lane] = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      if (lane == 0) p.ws_lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
  if (!clustered) return;
  cluster_sync();
  const uint32_t ml_at = ptx::smem_addr(ml), part_at = ptx::smem_addr(part);
  for (int r = job.split + p.num_splits * warp; r < R; r += p.num_splits * warps) {
    float2 s[kMaxCluster];
    float4 y[kMaxCluster];
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < kMaxCluster; ++q) {
      s[q] = make_float2(-INFINITY, 0.f);
      if (q < p.num_splits) {
        s[q] = ld_remote2(remote(ml_at + r * 8, q));
        y[q] = ld_remote4(remote(part_at + (r * STRIDE + lane * 4) * 4, q));
      }
    }
#pragma unroll
    for (int q = 0; q < kMaxCluster; ++q) m = fmaxf(m, s[q].x);
#pragma unroll
    for (int q = 0; q < kMaxCluster; ++q)
      if (q < p.num_splits) {
        const float w = s[q].x == -INFINITY ? 0.f : exp2_fast(s[q].x - m);
        l += s[q].x == -INFINITY ? s[q].y : s[q].y * w;
        a.x = fmaf(w, y[q].x, a.x); a.y = fmaf(w, y[q].y, a.y); a.z = fmaf(w, y[q].z, a.z); a.w = fmaf(w, y[q].w, a.w);
      }
    const int t = r / p.G;
    store_row(p, ((size_t)job.b * p.T + t) * p.Hq + job.h * p.G + (r - t * p.G), lane, a, m, l);
  }
  cluster_sync();                                   // nobody leaves while its memory is read
}

// 8 of a query row's dims per 32-bit word pair as f16 times a power of two that
// brings the row's largest value to [2^7, 2^8): exact but for values 2^-22
// times smaller.  `big`: the row's largest magnitude.
__device__ __forceinline__ int f16_exponent(float big) {
  return big > 0.f && big < INFINITY ? min(max(7 - ilogbf(big), -120), 100) : 0;
}

// ------------------------------------------------------------- one token
// Products with keys (or head dims) as rows and the G heads as 8 columns:
//   S^T [16 keys x 8] += K . q^T, then += R . q^T;  O^T [128 x 8] += V^T . P^T
// Half the instructions and accumulators of 16-row tiles that are half empty.
//
// What bounds it: the long window, memory (4 sequences x 32,768 keys, 64/8 heads,
// fp32 outputs: 90 us, 542 MB at 6.0 TB/s, 92 % of a plain copy); a batch over codes, the
// latency of a page's chain (load, product, exponential, product) in two blocks
// of 9 warps to an SM (32 sequences x 1,024 keys + 64 sinks: 19.7 us, 74 MB at
// 3.8 TB/s); one sequence, launch and merge (1,024 keys: 6.5 us).  Measured on
// the way: heads as rows, one page at a time, 49 us for the batch and 104 for
// the long window; a warp number that the compiler does not know to be the
// warp's, 21.7 and 93; PARTS as a branch in one kernel, 20.1 for the batch.
//
// Weights are rounded once (bf16 over a bf16 cache, f16 over codes) where the
// output is bf16 and rounded as coarsely itself; all their parts cost one sequence
// 7.2 us against 6.4, the batch over codes 21.6 against 19.6, the long window 90
// against 85.
// PARTS (fp32 outputs): weights in all their parts, and a page's products summed
// by themselves before they are added (the matrix instructions cut off what their
// accumulator cannot hold: the long window 1.7e-6 off, relative, against 4.8e-7).
template <bool F8, bool PARTS>
__global__ void __launch_bounds__(StepConfig<F8>::kThreads, 2) sink_step_kernel(const __grid_constant__ Params p) {
  using K = StepConfig<F8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* const tail = smem + K::kTail;
  const uint32_t sbase = ptx::smem_addr(smem);
  begin<K>(p, tail, K::kKeyWarps);
  const Job job(p);
  const uint32_t full = ptx::smem_addr(tail) + K::T::oBar, empty = full + 8 * K::kFull;
  volatile int* const flags = reinterpret_cast<volatile int*>(tail + K::T::oFlags);
  const int4* const info = reinterpret_cast<const int4*>(tail + K::T::oInfo);
  const int* const edges = reinterpret_cast<const int*>(tail + K::T::oEdges);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, c = lane & 3;   // (known to be the warp's)
  float o[8][4];
  float m_ref[2] = {-INFINITY, -INFINITY}, l_sum[2] = {0.f, 0.f};   // of heads 2 c and 2 c + 1
  if (warp == K::kWarps) {
    copy_pages<K, F8>(p, job, sbase, tail);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const int head = lane >> 2;
    const bool real = head < p.G;
    const uint32_t* const src = reinterpret_cast<const uint32_t*>(p.q + ((size_t)job.b * p.Hq + job.h * p.G + (real ? head : 0)) * kDim);
    uint32_t qb[8][2];                              // bf16, for the bf16 keys and the relative rows
    uint32_t qh[F8 ? 8 : 1][2];                     // f16 times a power of two, for the codes
    const float scale_log2 = 1.4426950408889634f * 0.08838834764831845f;
    float mul[2] = {scale_log2, scale_log2};        // logit multipliers of the keys' product
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      qb[s][0] = real ? __ldg(src + 8 * s + c) : 0;
      qb[s][1] = real ? __ldg(src + 8 * s + 4 + c) : 0;
    }
    if constexpr (F8) {
      // the codes' operand order: k index 2c + i is dim 4c + i, 8 + 2c + i is
      // 4c + 2 + i (one 32-bit word of four codes feeds both halves)
      float big = 0.f;
      uint2 w[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        w[s] = real ? __ldg(reinterpret_cast<const uint2*>(src) + 4 * s + c) : make_uint2(0, 0);
        const float2 x = unpack<false>(w[s].x), y = unpack<false>(w[s].y);
        big = fmaxf(big, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
      }
      const int qe = f16_exponent(quad_max(big));
      const float up = ldexpf(1.f, qe);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float2 x = unpack<false>(w[s].x), y = unpack<false>(w[s].y);
        qh[s][0] = pack<true>(x.x * up, x.y * up);
        qh[s][1] = pack<true>(y.x * up, y.y * up);
      }
      const float back = scale_log2 * __ldg(p.k_scale + job.h) * ldexpf(1.f, -qe);
      mul[0] = __shfl_sync(~0u, back, 8 * c);
      mul[1] = __shfl_sync(~0u, back, 8 * c + 4);
    }
    // where the output is fp32 P has as many parts as 22 bits and more take:
    // two of f16, three of bf16
    const int jw = (warp & (K::kKeyWarps - 1)) * 16, pos = job.p_last;
    const int half_row = lane & 15, half_col = lane >> 4, swz = lane & 7;

    for (int v = job.v0 + warp / K::kKeyWarps; v < job.v1; v += K::kStreams) {
      const int it = v - job.v0, s = it % K::kStages;
      if (!__all_sync(~0u, ptx::mbar_wait(full + 8 * (it % K::kFull), (it / K::kFull) & 1, flags, p.timeout_ns))) break;
      const int4 inf = info[s];
      const int j0 = inf.x;
      if (!inf.z) {
        const uint32_t ks = sbase + s * K::kStageBytes, vs = ks + K::kKvBytes, rs = vs + K::kKvBytes;
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, x[4] = {0.f, 0.f, 0.f, 0.f};
        // ---- relative rows (each key's row by its own address: the gather)
        {
          const int rr = min(max(bucket_of(max(0, pos - j0 - jw - half_row), p.bt, edges) - inf.y, 0), 63);
          const uint32_t ra = rs + rr * 128;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t f[4];
            ldsm4(f, ra + (i >> 2) * K::kRelHalf + (((2 * (i & 3) + half_col) ^ (rr & 7)) << 4));
            mma<false>(F8 ? x : acc, f, qb[i][0], qb[i][1]);
          }
        }
        // ---- keys
        const uint32_t ka = ks + (jw + half_row) * 128;
        if constexpr (F8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
            ldsm4(f, ka + (((2 * i + half_col) ^ swz) << 4));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t a[4] = {widen(f[2 * u]), widen(f[2 * u + 1]), widen(f[2 * u] >> 16), widen(f[2 * u + 1] >> 16)};
              mma<true>(acc, a, qh[2 * i + u][0], qh[2 * i + u][1]);
            }
          }
        } else {
          float acc2[4] = {0.f, 0.f, 0.f, 0.f};     // (a second chain of products)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t f[4];
            ldsm4(f, ka + (i >> 2) * (K::kKvBytes / 2) + (((2 * (i & 3) + half_col) ^ swz) << 4));
            mma<false>(acc2, f, qb[i][0], qb[i][1]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += acc2[e];
        }
        // ---- logits (log2 domain), masks; the reference follows where a logit
        // exceeds it by far (f16 weights stay finite)
        const bool whole = job.whole(p, j0);
        const int ja = j0 + jw + (lane >> 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[e] = F8 ? fmaf(acc[e], mul[e & 1], x[e] * scale_log2) : acc[e] * scale_log2;
          if (!whole && !job.seen(p, ja + 8 * (e >> 1))) acc[e] = -INFINITY;
        }
        float mx[2] = {fmaxf(acc[0], acc[2]), fmaxf(acc[1], acc[3])};
        if (__any_sync(~0u, mx[0] > m_ref[0] + kRescaleAt<F8> || mx[1] > m_ref[1] + kRescaleAt<F8>)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(~0u, mx[e], d));
            const float m = mx[e] > m_ref[e] + kRescaleAt<F8> ? mx[e] - kBelow<F8> : m_ref[e];
            const float a = m == m_ref[e] ? 1.f : exp2_fast(m_ref[e] - m);
            m_ref[e] = m;
            l_sum[e] *= a;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[i][e] *= a;
              o[i][2 + e] *= a;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[e] = exp2_fast(acc[e] - (m_ref[e & 1] == -INFINITY ? 0.f : m_ref[e & 1]));
          l_sum[e & 1] += acc[e];
        }
        uint32_t hi[2], lo[2], lo2[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          hi[u] = pack<F8>(acc[2 * u], acc[2 * u + 1]);
          if (PARTS) {
            const float2 r = unpack<F8>(hi[u]);
            lo[u] = pack<F8>(acc[2 * u] - r.x, acc[2 * u + 1] - r.y);
            const float2 q = unpack<F8>(lo[u]);
            lo2[u] = F8 ? 0 : transposed(pack<F8>(acc[2 * u] - r.x - q.x, acc[2 * u + 1] - r.y - q.y));
            lo[u] = transposed(lo[u]);
          }
          hi[u] = transposed(hi[u]);
        }
        // ---- values: rows that no token sees count as zeros (0 * NaN must not happen)
        uint32_t keep[2] = {~0u, ~0u};
        if (!whole) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (!job.seen(p, j0 + jw + 2 * c + (u & 1) + 8 * (u >> 1))) keep[u >> 1] &= (u & 1) ? 0x0000ffffu : 0xffff0000u;
        }
        if constexpr (F8) {
          const uint32_t va = vs + (jw + half_row) * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
            ldsm4t(f, va + (((2 * i + half_col) ^ swz) << 4));
#pragma unroll
            for (int u = 0; u < 2; ++u) {           // 16 dims: even ones are rows 0-7, odd ones rows 8-15
              const uint32_t f0 = f[2 * u] & keep[0], f1 = f[2 * u + 1] & keep[1];
              const uint32_t a[4] = {widen(__byte_perm(f0, 0, 0x4420)), widen(__byte_perm(f0, 0, 0x4431)),
                                     widen(__byte_perm(f1, 0, 0x4420)), widen(__byte_perm(f1, 0, 0x4431))};
              if (PARTS) {
                float sum[4];
                mma_from_zero<true>(sum, a, hi[0], hi[1]);
                mma<true>(sum, a, lo[0], lo[1]);
                for (int e = 0; e < 4; ++e) o[2 * i + u][e] += sum[e];
              } else {
                mma<true>(o[2 * i + u], a, hi[0], hi[1]);
              }
            }
          }
        } else {
          const uint32_t va = vs + (jw + swz + 8 * half_col) * 128;
          const int chunk = (lane >> 3) & 1;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t f[4];
            ldsm4t(f, va + (i >> 2) * (K::kKvBytes / 2) + (((2 * (i & 3) + chunk) ^ swz) << 4));
            f[0] &= keep[0]; f[1] &= keep[0]; f[2] &= keep[1]; f[3] &= keep[1];
            if (PARTS) {
              float sum[4];
              mma_from_zero<false>(sum, f, hi[0], hi[1]);
              mma<false>(sum, f, lo[0], lo[1]);
              mma<false>(sum, f, lo2[0], lo2[1]);
              for (int e = 0; e < 4; ++e) o[i][e] += sum[e];
            } else {
              mma<false>(o[i], f, hi[0], hi[1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty + 8 * s);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l_sum[e] += __shfl_xor_sync(~0u, l_sum[e], d);
  }
  __syncthreads();                                  // over the stages: every copy has been waited for
  float* const part = reinterpret_cast<float*>(smem);
  if (warp < K::kWarps) {
    if (lane < 4) {
      float2* const ml = reinterpret_cast<float2*>(tail + K::T::oMl) + warp * 8 + 2 * c;
      ml[0] = make_float2(m_ref[0], l_sum[0]);
      ml[1] = make_float2(m_ref[1], l_sum[1]);
    }
    float* const dst = part + (size_t)(warp * 8 + 2 * c) * K::kRowStride + (F8 ? 2 : 1) * (lane >> 2);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(e & 1) * K::kRowStride + 16 * i + (F8 ? 1 : 8) * (e >> 1)] = o[i][e];
  }
  __syncthreads();
  finish<K, F8, K::kWarps, K::kRowStride>(p, job, part, tail, 8);
}

// ------------------------------------------------- a few tokens over codes
// Rows (tokens x heads, up to 16) as rows, keys and dims as columns; four warps,
// a quarter of a page's keys each.  The relative product goes through a strip of
// shared memory of the warp's own, where each token's row is shifted.  Bound by
// the latency of that chain: 16 sequences of 2 tokens over 1,024 keys (64/8
// heads) 26 us, 32 of 4 tokens over 512 keys (32/8) 27 us, each of 34 MB that a
// plain copy would take 5.7 us for.  (More rows: tiles.)  Weights are one f16
// part where the output is bf16: 2^-11 of them beside the output's own 2^-8.
__global__ void __launch_bounds__(CodesConfig::kThreads, 2) sink_codes_kernel(const __grid_constant__ Params p) {
  using K = CodesConfig;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* const tail = smem + K::kTail;
  const uint32_t sbase = ptx::smem_addr(smem);
  begin<K>(p, tail, K::kWarps);
  const Job job(p);
  const uint32_t full = ptx::smem_addr(tail) + K::T::oBar, empty = full + 8 * K::kFull;
  volatile int* const flags = reinterpret_cast<volatile int*>(tail + K::T::oFlags);
  const int4* const info = reinterpret_cast<const int4*>(tail + K::T::oInfo);
  const int* const edges = reinterpret_cast<const int*>(tail + K::T::oEdges);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int R = p.G * p.T;
  // rows of this thread: r0 and r0 + 8
  const int c = lane & 3, r0 = lane >> 2;
  float o[16][4];
  float m_ref[2] = {-INFINITY, -INFINITY}, l_sum[2] = {0.f, 0.f};
  if (warp == K::kWarps) {
    copy_pages<K, true>(p, job, sbase, tail);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    uint32_t qa[8][4];                             // bf16 rows, for the relative rows
    uint32_t qh[8][4];                             // f16 rows times a power of two, for the codes
    int pos[2];
    float mul[2];                                  // logit multiplier of the keys' product, log2 domain
    const float scale_log2 = 1.4426950408889634f * 0.08838834764831845f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + 8 * e, t = r < R ? r / p.G : 0;
      pos[e] = job.walk.p0 + t;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.q + (((size_t)job.b * p.T + t) * p.Hq + job.h * p.G + (r < R ? r - t * p.G : 0)) * kDim);
      float big = 0.f;
      uint2 w[8];                                  // (operand order of the codes as in the step kernel)
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        qa[s][e] = r < R ? __ldg(src + 8 * s + c) : 0;
        qa[s][2 + e] = r < R ? __ldg(src + 8 * s + 4 + c) : 0;
        w[s] = r < R ? __ldg(reinterpret_cast<const uint2*>(src) + 4 * s + c) : make_uint2(0, 0);
        const float2 x = unpack<false>(w[s].x), y = unpack<false>(w[s].y);
        big = fmaxf(big, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
      }
      const int qe = f16_exponent(quad_max(big));
      const float up = ldexpf(1.f, qe);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float2 x = unpack<false>(w[s].x), y = unpack<false>(w[s].y);
        qh[s][e] = pack<true>(x.x * up, x.y * up);
        qh[s][2 + e] = pack<true>(y.x * up, y.y * up);
      }
      mul[e] = scale_log2 * __ldg(p.k_scale + job.h) * ldexpf(1.f, -qe);
    }
    const bool both_parts = p.out_fp32;            // P in two parts (hi + lo) where the output is fp32
    const int jw = warp * K::kWarpKeys;           // this warp's keys within a page
    const uint32_t row7 = lane & 7;
    float* const xs = reinterpret_cast<float*>(smem + K::oX) + warp * 16 * K::kXStride;

    for (int v = job.v0; v < job.v1; ++v) {
      const int it = v - job.v0, s = it % K::kStages;
      if (!__all_sync(~0u, ptx::mbar_wait(full + 8 * (it % K::kFull), (it / K::kFull) & 1, flags, p.timeout_ns))) break;
      const int4 inf = info[s];
      const int j0 = inf.x;
      if (!inf.z) {
        const uint32_t ks = sbase + s * K::kStageBytes, vs = ks + K::kKvBytes, rs = vs + K::kKvBytes;
        constexpr int NT = K::kWarpKeys / 8;        // 8-key tiles of this warp
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;

        // ---- relative rows (operand row address per lane: the gather), shifted
        // by each token's columns on their way through the strip
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NT + 1; ++n) {
          float xa[4] = {0.f, 0.f, 0.f, 0.f};
          const int u = jw + n * 8 + row7;
          const int rr = min(max(bucket_of(max(0, job.p_last - j0 - u), p.bt, edges) - inf.y, 0), K::kChunk - 1);
          const uint32_t ra = rs + rr * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
            ldsm4(f, ra + (i >> 1) * K::kRelHalf + (((4 * (i & 1) + (lane >> 3)) ^ (rr & 7)) << 4));
            mma<false>(xa, qa[2 * i], f[0], f[1]);
            mma<false>(xa, qa[2 * i + 1], f[2], f[3]);
          }
          float* d = xs + (lane >> 2) * K::kXStride + n * 8 + 2 * c;
          *reinterpret_cast<float2*>(d) = make_float2(xa[0], xa[1]);
          *reinterpret_cast<float2*>(d + 8 * K::kXStride) = make_float2(xa[2], xa[3]);
        }
        __syncwarp();

        // ---- keys
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t ka = ks + (jw + n * 8 + row7) * 128;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t f[4];
            ldsm4(f, ka + (((4 * i + (lane >> 3)) ^ row7) << 4));
#pragma unroll
            for (int u = 0; u < 4; ++u) mma<true>(acc[n], qh[4 * i + u], widen(f[u]), widen(f[u] >> 16));
          }
        }

        // ---- logits (log2 domain), masks, running maximum and sum
        const bool whole = job.whole(p, j0);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = xs[((lane >> 2) + 8 * (e >> 1)) * K::kXStride + n * 8 + 2 * c + (e & 1) + job.p_last - pos[e >> 1]];
            float z = fmaf(acc[n][e], mul[e >> 1], x * scale_log2);
            if (!whole) {
              const int j = j0 + jw + n * 8 + 2 * c + (e & 1), d = pos[e >> 1] - j;
              z = d >= 0 && (d < p.window || j < p.sinks) ? z : -INFINITY;
            }
            acc[n][e] = z;
            mx[e >> 1] = fmaxf(mx[e >> 1], z);
          }
        mx[0] = quad_max(mx[0]);
        mx[1] = quad_max(mx[1]);
        if (__any_sync(~0u, mx[0] > m_ref[0] + kRescaleAt<true> || mx[1] > m_ref[1] + kRescaleAt<true>)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float m = mx[e] > m_ref[e] + kRescaleAt<true> ? mx[e] - kBelow<true> : m_ref[e];
            const float a = m == m_ref[e] ? 1.f : exp2_fast(m_ref[e] - m);
            m_ref[e] = m;
            l_sum[e] *= a;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              o[i][2 * e] *= a;
              o[i][2 * e + 1] *= a;
            }
          }
        }
        const float mu[2] = {m_ref[0] == -INFINITY ? 0.f : m_ref[0], m_ref[1] == -INFINITY ? 0.f : m_ref[1]};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[n][e] = exp2_fast(acc[n][e] - mu[e >> 1]);
            l_sum[e >> 1] += acc[n][e];
          }

        // ---- values: rows that no token sees count as zeros (0 * NaN must not happen)
#pragma unroll
        for (int k = 0; k < K::kWarpKeys / 16; ++k) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float a0 = acc[2 * k + (u >> 1)][2 * (u & 1)], a1 = acc[2 * k + (u >> 1)][2 * (u & 1) + 1];
            hi[u] = pack<true>(a0, a1);
            const float2 r = unpack<true>(hi[u]);
            lo[u] = pack<true>(a0 - r.x, a1 - r.y);
          }
          uint32_t keep[2] = {~0u, ~0u};
          if (!whole) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (!job.seen(p, j0 + jw + k * 16 + 2 * c + (u & 1) + 8 * (u >> 1)))
                keep[u >> 1] &= (u & 1) ? 0x0000ffffu : 0xffff0000u;
          }
          const uint32_t va = vs + (jw + k * 16 + (lane & 15)) * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
            ldsm4t(f, va + (((2 * i + (lane >> 4)) ^ row7) << 4));
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t f0 = f[2 * w] & keep[0], f1 = f[2 * w + 1] & keep[1];
#pragma unroll
              for (int odd = 0; odd < 2; ++odd) {
                const uint32_t b0 = widen(__byte_perm(f0, 0, odd ? 0x4431 : 0x4420));
                const uint32_t b1 = widen(__byte_perm(f1, 0, odd ? 0x4431 : 0x4420));
                if (both_parts) {
                  float sum[4];
                  mma_from_zero<true>(sum, hi, b0, b1);
                  mma<true>(sum, lo, b0, b1);
                  for (int e = 0; e < 4; ++e) o[4 * i + 2 * w + odd][e] += sum[e];
                } else {
                  mma<true>(o[4 * i + 2 * w + odd], hi, b0, b1);
                }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty + 8 * s);
    }
    l_sum[0] = quad_sum(l_sum[0]);
    l_sum[1] = quad_sum(l_sum[1]);
  }
  __syncthreads();                                  // over the stages: every copy has been waited for
  float* const part = reinterpret_cast<float*>(smem);               // [warp][16][128]
  if (warp < K::kWarps) {
    if (c == 0) {
      float2* const ml = reinterpret_cast<float2*>(tail + K::T::oMl) + warp * 16 + r0;
      ml[0] = make_float2(m_ref[0], l_sum[0]);
      ml[8] = make_float2(m_ref[1], l_sum[1]);
    }
    float* dst = part + (size_t)(warp * 16 + r0) * kDim;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dst[8 * (e >> 1) * kDim + 16 * (i >> 1) + 2 * (2 * c + (e & 1)) + (i & 1)] = o[i][e];
  }
  __syncthreads();
  finish<K, true, K::kWarps, kDim>(p, job, part, tail, 16);
}

}  // namespace sink
}  // namespace relattn
