// rel_attn_sink_tiles.cuh -- the attention of rel_attn_sink_common.cuh for many
// query tokens per sequence, on the tensor cores (tcgen05).
//
// A tile of queries is 128 / G tokens x G heads of one KV head: the 128 rows
// (lanes) of the accumulators.  Keys come in pages of 64.  Per page one
// product [S | X] = Q . [K; R]^T gives the 64 logits and, beside them, the
// relative terms of all distances that the tile's tokens have to the page:
// column c of X belongs to distance p_0 - j_0 - 63 + c.  K's rows and the
// relative rows lie behind one another in shared memory, so that it is one
// operand of 64 + kRel rows and Q is read once for both.
//
// Over an E4M3 cache four warps widen a page's codes to bf16 (exactly) where the
// products read them, in the place of the third group; k_scale goes into the
// logits' sum with X, v_scale into the outputs' division.
//
// Where a page's distances lie in the log buckets there are few of those (one
// to five in the standard table): then the relative rows are the buckets', X
// has a column for each, and a row picks by comparing keys with the buckets'
// first distances.
//
// The shear.  Key jj of token t takes column 63 + t - jj.  A warp's 32 rows
// hold at most 8 neighbouring tokens; the first one's t goes into the tensor
// memory address of the load, what is left (0..7) is a shift by register
// renaming and two or three steps of selects: no shared memory, and about as
// many instructions as the exponentials.
//
// The softmax weights are written back to tensor memory (bf16; three parts where
// the output is fp32) as the A operand of O += P . V.  (One part, 2^-8 of a
// weight, where the output is rounded as coarsely itself: with three 8K tokens
// take 663 us against 341, verify steps 36.5 against 22.8.)  [S | X] and P have two
// buffers; pages go round three groups of 128 threads (one thread a row), as
// [S | X] is free again when a group has read it to registers.
//
// The reference of a row's exponentials is the maximum of the first page that
// it sees anything of (the tile's first or second page, as a tile is shorter
// than a page) and stays: weights are bf16, whose exponents reach 2^127, and
// sums are fp32, so that a later weight may be far above the first page's: a
// row's may sum to 2^40 (of which 2^80 are left for the values).  Nothing is
// handed from page to page, no maximum is sought on the pages behind, and O is
// never rescaled.  A row that did go further shows in its sum; its tile is gone
// over again at the end of the round, once for the maxima, once with them as
// references.
//
// A step of few tokens is a tile with few rows in use; where the tiles are
// fewer than the SMs their pages are split, and the parts go to the combine
// kernel.  One block per SM goes through query tiles in turn; loads run ahead
// over the tiles' borders.
#pragma once

#include <algorithm>
#include <type_traits>

#include "rel_attn_sink_tiles.h"

namespace relattn {
namespace sink {

// 2^40: what a row's weights may sum to (28 nats above the first page's maximum).
// |O| <= sum * max|v|, so that values up to 2^80 leave it finite.  (At 2^64 those
// above 2^63 could come out as infinities.)
constexpr float kReach = 1099511627776.f;
constexpr int kRound = 64;                          // tiles a block does between two looks at what went further

template <int G, bool KV8, bool THREE>
struct TileConfig {
  static constexpr int kTokens = 128 / G;           // of a query tile
  static constexpr int kRel = G == 8 ? 80 : 96;     // distances of a page: 64 + kTokens - 1, in sixteens
  static constexpr int kN = kKeys + kRel;
  static constexpr int kFew = 16;                   // buckets of a page by buckets
  static constexpr int kHalf = kN * 128;            // 64 dims of [K; R]
  static constexpr int kKrBytes = 2 * kHalf, kVBytes = kKeys * kDim * 2, kQHalf = 128 * 128;
  static constexpr int kKrStages = 3 - KV8 - THREE, kVStages = 3 - THREE, kCodeStages = 2;
  static constexpr int kGroups = KV8 ? 2 : 3;       // of softmax threads, 128 each
  // barriers of a page's [S | X] and of its product with V: a ring of both the
  // buffers and the groups, so that one group alone waits on a barrier, phase
  // after phase
  static constexpr int kRing = 2 * kGroups;
  static constexpr int kThreads = 512;              // copies (Q, K and R; V) and the two products: a warp each
  static constexpr int oKr = 2 * kQHalf;
  static constexpr int oV = oKr + kKrStages * kKrBytes;
  static constexpr int oCodes = oV + kVStages * kVBytes;
  static constexpr int kCodeBytes = KV8 ? 2 * kKeys * kDim : 0;   // K's, then V's
  // (three parts) after so many pages O is added to sums in shared memory, float4
  // [32 dims / 4][128 rows]
  static constexpr int kSegment = KV8 ? 4 : 3;
  static constexpr int oAcc = oCodes + kCodeStages * kCodeBytes;
  static constexpr int oEdges = oAcc + (THREE ? 128 * kDim * 4 : 0);
  static constexpr int oFirst = oEdges + 516 * 4;   // float [2 tiles][2 pages][128]: first pages' maxima
  static constexpr int oSum = oFirst + 2048;        // float [2 tiles][groups][128]: sums
  static constexpr int oMax = oSum + 1024 * kGroups;  // the same: maxima
  static constexpr int oMark = oMax + 1024 * kGroups;         // int [kRound]: tiles to go over again
  static constexpr int oInfo = oMark + kRound * 4;    // int2 [8]: of a page, {first bucket or -1, buckets}
  static constexpr int oBar = oInfo + 64;
  static constexpr int kBars = 2 + 2 * kKrStages + 2 * kVStages + 2 * kRing + 4 + 4 + 2 * kCodeStages + kKrStages;
  static constexpr int oFlags = oBar + kBars * 8;
  static constexpr int kAlloc = oFlags + 64 + 1024;
  static_assert(kAlloc <= 232448, "shared memory of a block");
  // tensor memory columns
  static constexpr int kColP = 320, kColO = 384;
  static_assert(2 * kN <= kColP, "two [S | X] buffers");
};

// ------------------------------------------------------------------ pieces
// (as ptx::tma_load_2d without a cache hint: neighbouring tiles read the same pages)
__device__ __forceinline__ void tma_load_2d_kept(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// D += A (tensor memory) . B (shared memory)
__device__ __forceinline__ void umma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t a, float& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(reinterpret_cast<uint32_t&>(v)) : "r"(a));
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Two fp32 operations in one instruction, and the largest of three.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// One lane of a converged warp: what only one thread may issue is issued
// under this predicate, with operands the whole warp agrees on.
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// all of a block, from either side of a branch
__device__ __forceinline__ void block_sync() { asm volatile("barrier.cta.sync 0;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16_async(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies16_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// bits 0 .. n - 1
__device__ __forceinline__ unsigned long long keys_below(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// One query tile and split: its tokens, and the pages of the split that they
// see (page(i) for i < n).
template <int G>
struct QueryTile {
  int b, h, t0, tokens, length, p0, split, v0, n;
  bool idle, bad;
  Walk walk;
  __device__ __forceinline__ QueryTile(const TileParams& p, int tile) : walk(1, 1, 1, 0) {
    constexpr int TQ = 128 / G;
    split = 0;
    if (p.splits > 1) {
      split = tile % p.splits;
      tile /= p.splits;
    }
    const int qt = tile % p.q_tiles, bh = tile / p.q_tiles;
    h = bh % p.Hkv;
    b = bh / p.Hkv;
    t0 = qt * TQ;
    tokens = min(TQ, p.C - t0);
    const int L = __ldg(p.seq_lens + b);
    length = L;
    idle = L == 0;
    bad = !idle && (L < p.C || L > p.max_pages * kKeys);
    n = p0 = v0 = 0;
    if (!idle && !bad) {
      walk = Walk(L - (p.C - t0 - tokens), tokens, p.window, p.sinks);
      p0 = walk.p0;
      n = walk.nv;
      if (p.splits > 1) {
        v0 = (int)((long long)walk.nv * split / p.splits);
        n = (int)((long long)walk.nv * (split + 1) / p.splits) - v0;
      }
    }
  }
  __device__ __forceinline__ int page(int i) const { return walk.logical(v0 + i); }
};

// What a block goes through: the tiles of a round, or (again) the marked ones
// of them, each twice.
struct Schedule {
  int first, step, count;                           // tile of turn j: first + j * step ...
  const int* marks;                                 // ... or, where given, of the (j / 2)th mark that is set
  __device__ __forceinline__ int tile(int j) const {
    if (!marks) return first + j * step;
    int at = 0;
    for (int seen = marks[0]; seen <= j / 2; seen += marks[at]) ++at;
    return first + at * step;
  }
};

// The pages of a schedule's tiles in order.  g and used count on from schedule
// to schedule: pages, and tiles with pages, before this one.
template <int G>
struct PageCursor {
  const TileParams& p;
  const Schedule& sched;
  int j, used, i, n, g;
  int next_j, next_n;                               // the next tile with pages, looked up while this one's go on (next_j < 0: not yet)
  __device__ __forceinline__ PageCursor(const TileParams& prm, const Schedule& s, int g0, int used0)
      : p(prm), sched(s), used(used0), i(0), g(g0) {
    look(0);
    j = next_j;
    n = next_n;
    next_j = -1;
  }
  __device__ __forceinline__ void look(int from) {
    for (next_j = from; next_j < sched.count; ++next_j) {
      next_n = QueryTile<G>(p, sched.tile(next_j)).n;
      if (next_n > 0) return;
    }
  }
  __device__ __forceinline__ bool valid() const { return j < sched.count; }
  __device__ __forceinline__ void next() {
    ++g;
    if (next_j < 0) look(j + 1);
    if (++i < n) return;
    i = 0;
    ++used;
    j = next_j;
    n = next_n;
    next_j = -1;
  }
};

// ptx::mbar_wait without a call (the register split below leaves no room for
// the calling convention).
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned long long limit) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (ptx::global_timer_ns() - t0 > limit) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
// Both phases complete (all lanes agree); false where a wait ran out.
__device__ __forceinline__ bool wait_both(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, volatile int* abort_flag,
                                          unsigned long long limit) {
  const bool ra = ptx::mbar_try_wait(a, pa), rb = ptx::mbar_try_wait(b, pb);
  if (__all_sync(~0u, ra && rb)) return true;
  return __all_sync(~0u, wait_for(a, pa, abort_flag, limit) && wait_for(b, pb, abort_flag, limit));
}

// 16 codes as 16 bf16 values, exactly (NaN stays NaN).
__device__ __forceinline__ void widen16(const uint4& codes, uint4 (&v)[2]) {
  const uint32_t in[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack<true>(widen(in[i >> 1] >> (16 * (i & 1))));
    out[i] = pack<false>(f.x, f.y);
  }
  v[0] = make_uint4(out[0], out[1], out[2], out[3]);
  v[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// The four widening warps: each page's codes to where the products read them.
// Two threads to a key, 64 dims each.
template <class K, int G>
__device__ __forceinline__ void widen_pages(const TileParams& p, const Schedule& sched, int& g, bool& dead, uint8_t* smem,
                                            uint32_t k_wide, uint32_t kr_empty, uint32_t v_full, uint32_t v_empty,
                                            uint32_t code_full, uint32_t code_empty, volatile int* flags) {
  const int th = threadIdx.x & 127, key = th >> 1, half = th & 1;
  for (int j = 0; j < sched.count; ++j) {
    const int n = QueryTile<G>(p, sched.tile(j)).n;
#pragma unroll 1
    for (int i = 0; i < n; ++i, ++g) {
      const int cs = g % K::kCodeStages;
      const uint8_t* const codes = smem + K::oCodes + cs * K::kCodeBytes + key * 128;
      dead = dead || !wait_for(code_full + 8 * cs, (g / K::kCodeStages) & 1, flags, p.timeout_ns);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int stages = kv ? K::kVStages : K::kKrStages, s = g % stages;
        dead = dead || !wait_for((kv ? v_empty : kr_empty) + 8 * s, ((g / stages) & 1) ^ 1, flags, p.timeout_ns);
        if (dead) continue;
        uint8_t* const to = smem + (kv ? K::oV + s * K::kVBytes + half * (K::kVBytes / 2) : K::oKr + s * K::kKrBytes + half * K::kHalf) + key * 128;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 v[2];
          widen16(*reinterpret_cast<const uint4*>(codes + kv * (K::kCodeBytes / 2) + (((4 * half + q) ^ (key & 7)) << 4)), v);
          *reinterpret_cast<uint4*>(to + (((2 * q) ^ (key & 7)) << 4)) = v[0];
          *reinterpret_cast<uint4*>(to + (((2 * q + 1) ^ (key & 7)) << 4)) = v[1];
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive((kv ? v_full : k_wide) + 8 * s);
      }
      if (!dead) ptx::mbar_arrive(code_empty + 8 * cs);
    }
  }
}

// ------------------------------------------------------------------ kernel
// WIDE: fp32 is stored; THREE: weights in three parts; FEW: pages of few buckets
// are taken by buckets.  (A kernel of its own: with both ways in one, 8K tokens
// over a window that has none took 25 % more; without it, four verify steps over
// 32K keys took 337 us against 147.)
//
// What bounds it.  Per page and SM the products compute 896 clocks (128 x 160 x
// 128 and 128 x 128 x 64), shared memory moves 146 KB, 1,140 clocks, and a page
// goes by in 1,120; a tile's beginning and end cost 4 to 6 pages more, where its
// first page's maxima, its outputs and the next tile's first loads follow one
// another.  8,192 tokens, 48/8 heads, window 1,024, 4 sinks: 340 us, 855 TFLOP/s;
// 2 x 509 tokens, 64/16 heads, window 512: 45.5 us; 16 verify steps of 8 tokens,
// window 1,024: 22.8 us (73 MB, 128 tiles of 18 pages on 148 SMs: the latency of
// a tile).  Measured on the way, 8,192 tokens: in chunks of a few tokens on
// warp-level matrix instructions 2,322 us; keys, values and the two products from
// two warps 634, from four 414; masks by bits and wide gathers 379 from 405; warp
// numbers that the compiler does not know to be the warp's 372 against 341.
template <int G, bool WIDE, bool THREE, bool FEW, bool KV8>
__global__ void __launch_bounds__(512, 1) sink_tiles_kernel(const __grid_constant__ TileParams p) {
  using K = TileConfig<G, KV8, THREE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = ptx::smem_addr(smem);
  int* const edges = reinterpret_cast<int*>(smem + K::oEdges);
  int* const marks = reinterpret_cast<int*>(smem + K::oMark);
  volatile int* const info = reinterpret_cast<volatile int*>(smem + K::oInfo);
  // flags: abort, drain, tensor memory base, -, then (from 8) the last bad
  // tile + 1 of each eighth tile
  volatile int* const flags = reinterpret_cast<volatile int*>(smem + K::oFlags);
  const uint32_t q_full = sbase + K::oBar, q_empty = q_full + 8, kr_full = q_empty + 8, kr_empty = kr_full + 8 * K::kKrStages,
                 v_full = kr_empty + 8 * K::kKrStages, v_empty = v_full + 8 * K::kVStages, sx_ready = v_empty + 8 * K::kVStages,
                 sx_free = sx_ready + 8 * K::kRing, p_ready = sx_free + 16, pv_done = p_ready + 16, o_free = pv_done + 8 * K::kRing, drained = o_free + 8,
                 first_max = drained + 8,           // two: of the tile's first and of its second page
                 code_full = first_max + 16, code_empty = code_full + 8 * K::kCodeStages,
                 k_wide = code_empty + 8 * K::kCodeStages;   // K's part of a [K; R] that is widened
  const int tid = threadIdx.x, lane = tid & 31;
  // (from one lane: the compiler then knows that the roles' branches, and what the
  // issuing warps work with there, are the warp's: 8K tokens 370 us without, 336 with)
  const int warp = __shfl_sync(~0u, tid >> 5, 0);
  const int tiles = p.B * p.Hkv * p.q_tiles * p.splits;
  const unsigned long long limit = p.timeout_ns;

  if (tid == 0) {
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int s = 0; s < K::kKrStages; ++s) { ptx::mbar_init(kr_full + 8 * s, 1); ptx::mbar_init(kr_empty + 8 * s, 1); }
    for (int s = 0; s < K::kVStages; ++s) { ptx::mbar_init(v_full + 8 * s, KV8 ? 128 : 1); ptx::mbar_init(v_empty + 8 * s, 1); }
    for (int s = 0; s < K::kCodeStages; ++s) { ptx::mbar_init(code_full + 8 * s, 1); ptx::mbar_init(code_empty + 8 * s, 128); }
    for (int s = 0; s < K::kKrStages; ++s) ptx::mbar_init(k_wide + 8 * s, 128);
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(sx_free + 8 * s, 128);
      ptx::mbar_init(p_ready + 8 * s, 128);
      ptx::mbar_init(first_max + 8 * s, 128);
    }
    for (int s = 0; s < K::kRing; ++s) { ptx::mbar_init(sx_ready + 8 * s, 1); ptx::mbar_init(pv_done + 8 * s, 1); }
    ptx::mbar_init(o_free, 256);                   // (two of the groups read O)
    ptx::mbar_init(drained, 2);
    for (int i = 0; i < 16; ++i) flags[i] = 0;
    for (int i = 0; i < 16; ++i) info[i] = -1;     // (a page whose wait ran out may be looked at before it is written)
    ptx::fence_mbar_init();
  }
  if (tid < kRound) marks[tid] = 0;
  if (warp == 0) {
    ptx::tmem_alloc(sbase + K::oFlags + 8, 512);
    ptx::tmem_relinquish();
  }
  if (p.bt.nl > 1)
    for (int i = tid; i <= p.bt.nl; i += K::kThreads) edges[i] = p.bt.edges[i];
  ptx::tc_fence_before();
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_primary();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = (uint32_t)flags[2];
  int g = 0, used = 0, used2 = 0;                   // pages, tiles with pages, tiles with two or more: gone through
  // registers where they are needed: 128 x 104 + 384 x 136 = 512 x 128
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    int sent = 0;                                     // Q's copies
    int segment = 0;                                  // of O's pages (three parts)
    bool dead = false;                                // this role gave up a wait
    for (int first = blockIdx.x; first < tiles; first += kRound * gridDim.x) {
      const int round = min(kRound, (tiles - first + (int)gridDim.x - 1) / (int)gridDim.x);
      Schedule sched = {first, (int)gridDim.x, round, nullptr};
#pragma unroll 1
      for (int again = 0; again < 2; ++again) {
        if (warp == 0) {
          // ---- copies of Q and [K; R].  (V from a warp of its own: one for both
          // made the next keys wait for a product that was itself waiting for
          // them.  The warp sets the pace where its loop is long: what a page
          // needs is worked out for 32 pages at once, one to a lane.)
          constexpr int kStages = K::kKrStages;
          int issued = g, s = g % kStages;
          uint32_t before = ((g / kStages) & 1) ^ 1;
          const int g0 = g;
          for (int j = 0; j < sched.count; ++j) {
            const QueryTile<G> t(p, sched.tile(j));
            if (t.n == 0) continue;
            const int* const entries = p.block_table + (size_t)t.b * p.max_pages;
            const uint4* const table = reinterpret_cast<const uint4*>(p.rel + (size_t)t.h * p.NB * kDim) + (lane & 15);
            const int p_last = t.p0 + t.tokens - 1;
            // Q, once the products of the tile before have read theirs (the block's
            // first one before its pages)
            auto send_q = [&] {
              dead = dead || !__all_sync(~0u, wait_for(q_empty, (used & 1) ^ 1, flags, limit));
              if (!dead && elected()) {
                ptx::mbar_arrive_expect_tx(q_full, 2 * K::kTokens * G * 128);
                ptx::tma_load_3d(sbase, &p.tmap_q, q_full, 0, t.h * G, t.b * p.C + t.t0);
                ptx::tma_load_3d(sbase + K::kQHalf, &p.tmap_q, q_full, 64, t.h * G, t.b * p.C + t.t0);
              }
              __syncwarp();
              if (!dead) sent = used + 1;
            };
            if (used == 0) send_q();
            for (int i0 = 0; i0 < t.n; i0 += 32) {
              // of this lane's page: first key, nearest distance, row in the pool
              int my_j0 = 0, my_y = -1;
              if (i0 + lane < t.n) {
                const int page = __ldg(entries + t.page(i0 + lane));
                my_j0 = t.page(i0 + lane) * kKeys;
                if (page >= 0 && page < p.num_pages) my_y = (page * p.Hkv + t.h) * kKeys;
              }
              // relative rows: where bucket(d) = d for every visible distance they
              // are taken as they lie; else by buckets, where these are few; else a
              // row for each distance of the columns [c0, c1) (of a page of sinks
              // alone not all)
              const unsigned lie = __ballot_sync(~0u, (my_j0 < p.sinks ? p_last - my_j0 : min(p_last - my_j0, p.window - 1)) <= p.bt.ex);
              const int m = min(32, t.n - i0);
              for (int i = 0; i < m; ++i) {
                const int y = __shfl_sync(~0u, my_y, i), j0 = __shfl_sync(~0u, my_j0, i), near = t.p0 - j0 - (kKeys - 1);
                const uint32_t bar = kr_full + 8 * s, st = sbase + K::oKr + s * K::kKrBytes;
                const bool as_they_lie = (lie >> i) & 1;
                int b0 = -1, nb = 0, c0 = 0;
                if (!as_they_lie) {
                  c0 = j0 <= t.p0 - p.window - (kKeys - 1) ? max(0, kKeys - (p.sinks - j0)) : 0;
                  b0 = bucket_of(max(0, near + c0), p.bt, edges);
                  nb = bucket_of(max(0, near + kKeys + t.tokens - 2), p.bt, edges) - b0 + 1;
                  if (!FEW || nb > K::kFew) b0 = -1;
                }
                // (one vote: no lane goes on alone where a wait runs out; nothing is issued after that)
                dead = dead || !__all_sync(~0u, wait_for(kr_empty + 8 * s, before, flags, limit));
                if (!dead) {
                  if (y < 0) {
                    if (lane == 0) {
                      if (FEW) info[2 * ((g + i0 + i) & 7)] = -1;
                      flags[8 + (used & 7)] = used + 1;
                      ptx::mbar_arrive(bar);
                    }
                  } else {
                    const bool by_distance = !as_they_lie && b0 < 0;
                    if (by_distance) {
                      // a half-warp to a row, 16 lanes x 16 bytes; all rows under way at once
                      const uint32_t rows = st + kKeys * 128 + ((lane >> 3) & 1) * K::kHalf;
                      const int side = lane >> 4, c1 = kKeys + t.tokens - 1;
                      for (int c = c0; c < c1; c += 32) {
                        const int mine = bucket_of(max(0, near + min(c + lane, c1 - 1)), p.bt, edges);
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                          const int at_c = c + 2 * u + side, bucket = __shfl_sync(~0u, mine, 2 * u + side);
                          if (at_c < c1) copy16_async(rows + at_c * 128 + (((lane & 7) ^ (at_c & 7)) << 4), table + (size_t)bucket * (kDim / 8));
                        }
                      }
                      copies16_wait();
                      ptx::fence_proxy_async_smem();
                      __syncwarp();
                    }
                    if (elected()) {
                      if (FEW) {
                        info[2 * ((g + i0 + i) & 7)] = b0;
                        info[2 * ((g + i0 + i) & 7) + 1] = nb;
                      }
                      const int bytes = (KV8 ? 0 : kKeys * kDim * 2) + (by_distance ? 0 : b0 >= 0 ? 2 * K::kFew * 128 : 2 * K::kRel * 128);
                      if (bytes) ptx::mbar_arrive_expect_tx(bar, bytes); else ptx::mbar_arrive(bar);
                      if (!KV8) {                     // (else the widening warps write them)
                        tma_load_2d_kept(st, &p.tmap_k, bar, 0, y);
                        tma_load_2d_kept(st + K::kHalf, &p.tmap_k, bar, 64, y);
                      }
                      if (!by_distance) {
                        const CUtensorMap* const rel = b0 >= 0 ? &p.tmap_few : &p.tmap_r;
                        const int first_row = b0 >= 0 ? b0 : near;
                        ptx::tma_load_3d(st + kKeys * 128, rel, bar, 0, first_row, t.h);
                        ptx::tma_load_3d(st + K::kHalf + kKeys * 128, rel, bar, 64, first_row, t.h);
                      }
                    }
                  }
                  __syncwarp();
                  issued = g + i0 + i + 1;
                }
                if (i0 + i == 0 && used > 0) send_q();
                if (++s == kStages) s = 0, before ^= 1;
              }
            }
            g += t.n;
            ++used;
          }
          // the copies in flight land before the round or the block ends
          for (int q = max(g0, issued - kStages); q < issued; ++q)
            wait_for(kr_full + 8 * (q % kStages), (q / kStages) & 1, flags + 1, kDrainNs);
          if (sent > 0) wait_for(q_full, (sent - 1) & 1, flags + 1, kDrainNs);
          __syncwarp();
        } else if (warp == 3) {
          // ---- copies of V, or of K's and V's codes
          constexpr int kStages = KV8 ? K::kCodeStages : K::kVStages;
          const uint32_t full = KV8 ? code_full : v_full, empty = KV8 ? code_empty : v_empty;
          int issued = g, s = g % kStages;
          uint32_t before = ((g / kStages) & 1) ^ 1;
          const int g0 = g;
          for (int j = 0; j < sched.count; ++j) {
            const QueryTile<G> t(p, sched.tile(j));
            const int* const entries = p.block_table + (size_t)t.b * p.max_pages;
            for (int i0 = 0; i0 < t.n; i0 += 32) {
              const int mine = i0 + lane < t.n ? __ldg(entries + t.page(i0 + lane)) : -1;
              const int my_y = mine >= 0 && mine < p.num_pages ? (mine * p.Hkv + t.h) * kKeys : -1;
              const int m = min(32, t.n - i0);
              for (int i = 0; i < m; ++i) {
                const int y = __shfl_sync(~0u, my_y, i);
                const uint32_t bar = full + 8 * s, st = sbase + (KV8 ? K::oCodes + s * K::kCodeBytes : K::oV + s * K::kVBytes);
                dead = dead || !__all_sync(~0u, wait_for(empty + 8 * s, before, flags, limit));
                if (!dead) {
                  if (elected()) {
                    if (y < 0) {
                      ptx::mbar_arrive(bar);
                    } else if (KV8) {
                      ptx::mbar_arrive_expect_tx(bar, K::kCodeBytes);
                      tma_load_2d_kept(st, &p.tmap_k, bar, 0, y);
                      tma_load_2d_kept(st + K::kCodeBytes / 2, &p.tmap_v, bar, 0, y);
                    } else {
                      ptx::mbar_arrive_expect_tx(bar, K::kVBytes);
                      tma_load_2d_kept(st, &p.tmap_v, bar, 0, y);
                      tma_load_2d_kept(st + K::kVBytes / 2, &p.tmap_v, bar, 64, y);
                    }
                  }
                  __syncwarp();
                  issued = g + i0 + i + 1;
                }
                if (++s == kStages) s = 0, before ^= 1;
              }
            }
            g += t.n;
          }
          for (int q = max(g0, issued - kStages); q < issued; ++q)
            wait_for(full + 8 * (q % kStages), (q / kStages) & 1, flags + 1, kDrainNs);
          __syncwarp();
        } else if (warp == 1) {
          // ---- [S | X] = Q . [K; R]^T
          constexpr uint32_t kIdesc = ptx::idesc_bf16(128, K::kN, false, false), kIdescFew = ptx::idesc_bf16(128, kKeys + K::kFew, false, false);
          const uint64_t qd = ptx::sdesc_sw128(sbase, 16, 1024), krd = ptx::sdesc_sw128(sbase + K::oKr, 16, 1024);
          PageCursor<G> at(p, sched, g, used);
          for (int s = g % K::kKrStages, turn = g / K::kKrStages; at.valid(); at.next()) {
            const int buf = at.g & 1;
            const uint32_t before = ((at.g >> 1) & 1) ^ 1;
            if (!dead) dead = !wait_both(kr_full + 8 * s, turn & 1, sx_free + 8 * buf, before, flags, limit);
            if (KV8 && !dead) dead = !__all_sync(~0u, wait_for(k_wide + 8 * s, turn & 1, flags, limit));
            if (!dead && at.i == 0) dead = !__all_sync(~0u, wait_for(q_full, at.used & 1, flags, limit));
            // (P's other parts lie in S's columns: the product that reads them comes first)
            if (THREE && !dead && at.g >= 2)
              dead = !__all_sync(~0u, wait_for(pv_done + 8 * ((at.g - 2) % K::kRing), ((at.g - 2) / K::kRing) & 1, flags, limit));
            ptx::tc_fence_after();
            if (!dead && elected()) {
              const uint64_t b = krd + (uint64_t)((s * K::kKrBytes) >> 4);
              const uint32_t idesc = FEW && info[2 * (at.g & 7)] >= 0 ? kIdescFew : kIdesc;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                ptx::umma_bf16(tmem + buf * K::kN, qd + (uint64_t)(((k >> 2) * K::kQHalf + (k & 3) * 32) >> 4),
                               b + (uint64_t)(((k >> 2) * K::kHalf + (k & 3) * 32) >> 4), idesc, k > 0);
              ptx::umma_commit(sx_ready + 8 * (at.g % K::kRing));
              ptx::umma_commit(kr_empty + 8 * s);
              if (at.i == at.n - 1) ptx::umma_commit(q_empty);
            }
            __syncwarp();
            if (++s == K::kKrStages) s = 0, ++turn;
          }
          g = at.g;
          used = at.used;
        } else if (warp == 2) {
          // ---- O += P . V.  (One thread for both products took 2,450 clocks a
          // page, three times what they compute for.)
          constexpr uint32_t kIdesc = ptx::idesc_bf16(128, kDim, false, true);
          const uint64_t vd = ptx::sdesc_sw128(sbase + K::oV, K::kVBytes / 2, 1024);   // rows are keys: dims-major
          PageCursor<G> at(p, sched, g, used);
          for (int s = g % K::kVStages, turn = g / K::kVStages; at.valid(); at.next()) {
            const int buf = at.g & 1;
            const int past = THREE ? at.i % K::kSegment : at.i;         // pages that O holds
            if (THREE) segment += past == 0;
            const int turn_of_o = THREE ? segment - 1 : at.used;
            if (!dead && past == 0) dead = !__all_sync(~0u, wait_for(o_free, (turn_of_o & 1) ^ 1, flags, limit));
            if (!dead) dead = !wait_both(v_full + 8 * s, turn & 1, p_ready + 8 * buf, (at.g >> 1) & 1, flags, limit);
            ptx::tc_fence_after();
            if (!dead && elected()) {
              const uint64_t b = vd + (uint64_t)((s * K::kVBytes) >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_bf16_ts(tmem + K::kColO, tmem + K::kColP + buf * 32 + k * 8, b + (uint64_t)((k * 2048) >> 4), kIdesc,
                             past > 0 || k > 0);
              if (THREE) {
#pragma unroll
                for (int k = 0; k < 8; ++k)           // the second and third parts, where S was
                  umma_bf16_ts(tmem + K::kColO, tmem + buf * K::kN + k * 8, b + (uint64_t)(((k & 3) * 2048) >> 4),
                               kIdesc, 1);
              }
              ptx::umma_commit(pv_done + 8 * (at.g % K::kRing));
              ptx::umma_commit(v_empty + 8 * s);
            }
            __syncwarp();
            if (++s == K::kVStages) s = 0, ++turn;
          }
          g = at.g;
          used = at.used;
        }
        block_sync();
        if (again) break;
        int more = 0;
        for (int j = 0; j < round; ++j) more += marks[j];
        if (more == 0) break;
        sched.count = 2 * more;
        sched.marks = marks;
      }
      if (tid < kRound) marks[tid] = 0;
      block_sync();
    }
    if (warp == 1 || warp == 2) {                     // every product is done before its memory is given back
      if (elected()) ptx::umma_commit(drained);
      wait_for(drained, 0, flags + 1, kDrainNs);
    }
    ptx::tc_fence_before();
    block_sync();
    if (warp == 0) ptx::tmem_dealloc(tmem, 512);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    float m_forced = 0.f;
    bool dead = false;                                // (of a widening thread)
    for (int first = blockIdx.x; first < tiles; first += kRound * gridDim.x) {
      const int round = min(kRound, (tiles - first + (int)gridDim.x - 1) / (int)gridDim.x);
      Schedule sched = {first, (int)gridDim.x, round, nullptr};
#pragma unroll 1
      for (int again = 0; again < 2; ++again) {
        if (KV8 && warp >= 12) {
          widen_pages<K, G>(p, sched, g, dead, smem, k_wide, kr_empty, v_full, v_empty, code_full, code_empty, flags);
        } else {
          // ---- softmax: thread = row of the tile, pages in turn
          const int grp = (warp - 4) >> 2, sub = warp & 3, r = sub * 32 + lane;
          const int tw = (sub * 32) / G, tok = r / G, rho = tok - tw;
          const uint32_t lanes = (uint32_t)(sub * 32) << 16;
          const float scale_log2 = 1.4426950408889634f * 0.08838834764831845f;
          for (int j = 0; j < sched.count; ++j) {
            const QueryTile<G> t(p, sched.tile(j));
            const float ks = KV8 ? __ldg(p.k_scale + t.h) : 1.f;
            float* const first_at = reinterpret_cast<float*>(smem + K::oFirst) + (used & 1) * 256 + r;
            const int pt = t.p0 + tok, p_last = t.p0 + t.tokens - 1, n = t.n;
            const bool forced = again && (j & 1);
            float m = forced ? m_forced : -INFINITY, mx_all = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            const int first_i = (grp + K::kGroups - g % K::kGroups) % K::kGroups;
            const int seg_part = K::kGroups == 2 ? grp : first_i - 1;     // of O's dims, at a segment's end
#pragma unroll 1
            for (int i = first_i; i < n; i += K::kGroups) {
              const int gi = g + i, buf = gi & 1, j0 = t.page(i) * kKeys;
              const uint32_t s_at = tmem + lanes + buf * K::kN, x_at = s_at + kKeys + tw;
              wait_for(sx_ready + 8 * (gi % K::kRing), (gi / K::kRing) & 1, flags, limit);
              __syncwarp();
              ptx::tc_fence_after();
              float2 z[32];                           // keys 2 c and 2 c + 1
              // (one answer for the warp and in range, even where a wait ran out)
              const int b0 = FEW ? __shfl_sync(~0u, info[2 * (gi & 7)], 0) : -1, nb = FEW ? __shfl_sync(~0u, min(info[2 * (gi & 7) + 1], K::kFew), 0) : 0;
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                // keys 16 u .. 16 u + 15: x[i] is the relative term of key 16 u + 15 - i
                float x[24], s[16];
                ptx::tmem_ld16(s_at + 16 * u, s);
                if (!FEW || b0 < 0) {
                  // columns 48 - 16 u + rho + 0 .. 15
                  ptx::tmem_ld16(x_at + 48 - 16 * u, x);
                  ptx::tmem_ld8(x_at + 64 - 16 * u, x + 16);
                  ptx::tmem_wait_ld();
                  if constexpr (G != 8) {
#pragma unroll
                    for (int c = 0; c < 20; ++c) x[c] = (rho & 4) ? x[c + 4] : x[c];
                  }
#pragma unroll
                  for (int c = 0; c < 18; ++c) x[c] = (rho & 2) ? x[c + 2] : x[c];
#pragma unroll
                  for (int c = 0; c < 16; ++c) x[c] = (rho & 1) ? x[c + 1] : x[c];
                } else {
#pragma unroll 1
                  for (int k = 0; k < nb; ++k) {
                    float xk;
                    tmem_ld1(s_at + kKeys + k, xk);
                    ptx::tmem_wait_ld();
                    // the bucket's distances start at its edge: keys up to there
                    const int e = b0 + k, i = k == 0 ? 0 : 16 * u + 15 - (pt - j0 - (e <= p.bt.ex ? e : edges[e - p.bt.ex]));
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = c >= i ? xk : x[c];
                  }
                }
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  z[8 * u + c] = KV8 ? fma2(make_float2(s[2 * c], s[2 * c + 1]), make_float2(ks, ks), make_float2(x[15 - 2 * c], x[14 - 2 * c]))
                                     : add2(make_float2(s[2 * c], s[2 * c + 1]), make_float2(x[15 - 2 * c], x[14 - 2 * c]));
              }
              ptx::tc_fence_before();
              ptx::mbar_arrive(sx_free + 8 * buf);
              const bool whole = j0 + kKeys - 1 <= t.p0 && (j0 > p_last - p.window || j0 + kKeys <= p.sinks);
              if (!whole) {
                const unsigned long long seen =
                    keys_below(pt + 1 - j0) & (~keys_below(pt - p.window + 1 - j0) | keys_below(p.sinks - j0));
                const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  const uint32_t bits = (c < 16 ? lo : hi) >> ((2 * c) & 31);
                  z[c].x = (bits & 1) ? z[c].x : -INFINITY;
                  z[c].y = (bits & 2) ? z[c].y : -INFINITY;
                }
              }
              // ---- the reference: of the first page, else of the second
              if (i <= 3 || again) {
                float mx = fmaxf(z[0].x, z[0].y);
#pragma unroll
                for (int c = 1; c < 32; ++c) mx = max3(mx, z[c].x, z[c].y);
                mx *= scale_log2;
                mx_all = fmaxf(mx_all, mx);
                if (i <= 1) {
                  first_at[i * 128] = mx;
                  ptx::mbar_arrive(first_max + 8 * i);
                }
                if (i == 1 || i == 2) wait_for(first_max, used & 1, flags, limit);
                if (i == 2 || i == 3) wait_for(first_max + 8, used2 & 1, flags, limit);
                if (i <= 3 && !forced) {
                  m = first_at[0];
                  if (i >= 1 && m == -INFINITY) m = first_at[128];
                }
              }
              const float mu = m == -INFINITY ? 0.f : m;
              const float2 scale2 = make_float2(scale_log2, scale_log2), mu2 = make_float2(-mu, -mu);
              // ---- P's place is free once the product two pages before has read it
              if (gi >= 2) wait_for(pv_done + 8 * ((gi - 2) % K::kRing), ((gi - 2) / K::kRing) & 1, flags, limit);
              __syncwarp();
              ptx::tc_fence_after();
              float2 page2 = make_float2(0.f, 0.f);   // (fp32 outputs: the page's own sum first)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t w[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  float2& e = z[16 * u + c];
                  e = fma2(e, scale2, mu2);
                  e = make_float2(exp2_fast(e.x), exp2_fast(e.y));
                  (THREE ? page2 : l2) = add2(THREE ? page2 : l2, e);
                  w[c] = pack<false>(e.x, e.y);
                }
                tmem_st16(tmem + lanes + K::kColP + buf * 32 + 16 * u, w);
                if (THREE) {
#pragma unroll
                  for (int part = 0; part < 2; ++part) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                      const float2 v = unpack<false>(w[c]);
                      float2& e = z[16 * u + c];
                      e = make_float2(e.x - v.x, e.y - v.y);
                      w[c] = pack<false>(e.x, e.y);
                    }
                    tmem_st16(s_at + 32 * part + 16 * u, w);
                  }
                }
              }
              if (THREE) l2 = add2(l2, page2);
              tmem_wait_st();
              const int oldest = t.length - p.C - p.window + 1;      // first position in any token's window
              if (j0 + kKeys > t.length || (j0 < oldest && j0 + kKeys > p.sinks)) {
                // value rows that no token of the step sees become zeros (0 * NaN must not happen)
                const int vs = gi % K::kVStages, c = r & 63, key = j0 + c;
                wait_for(v_full + 8 * vs, (gi / K::kVStages) & 1, flags, limit);
                if (key >= t.length || (key < oldest && key >= p.sinks)) {
                  uint4* row = reinterpret_cast<uint4*>(smem + K::oV + vs * K::kVBytes + (r >> 6) * (K::kVBytes / 2) + c * 128);
#pragma unroll
                  for (int e = 0; e < 8; ++e) row[e] = make_uint4(0, 0, 0, 0);
                }
                ptx::fence_proxy_async_smem();
              }
              ptx::tc_fence_before();
              ptx::mbar_arrive(p_ready + 8 * buf);
              if constexpr (THREE) {
                // the end of a segment that is not the tile's last: O to the sums, by the
                // groups that do not have the next one's first page.  (The tensor cores cut
                // off what an accumulator cannot hold, at every instruction: over 18 pages
                // of 12 instructions fp32 outputs were 3.7e-6 off.)
                const int last = i - i % K::kSegment + K::kSegment - 1;
                if (seg_part >= 0 && i + K::kGroups > last && last + 1 < n) {
                  wait_for(pv_done + 8 * ((g + last) % K::kRing), ((g + last) / K::kRing) & 1, flags, limit);
                  __syncwarp();
                  ptx::tc_fence_after();
                  float o[64];
                  tmem_ld32(tmem + lanes + K::kColO + 64 * seg_part, o);
                  tmem_ld32(tmem + lanes + K::kColO + 64 * seg_part + 32, o + 32);
                  ptx::tmem_wait_ld();
                  float4* const acc = reinterpret_cast<float4*>(smem + K::oAcc) + seg_part * 16 * 128 + r;
#pragma unroll
                  for (int c = 0; c < 16; ++c) {
                    float4 v = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                    if (last >= K::kSegment) {
                      const float4 x = acc[c * 128];
                      v = make_float4(x.x + v.x, x.y + v.y, x.z + v.z, x.w + v.w);
                    }
                    acc[c * 128] = v;
                  }
                  ptx::tc_fence_before();
                  ptx::mbar_arrive(o_free);
                }
              }
            }
            g += n;
            // ---- the tile's outputs, 64 dims to a group: of three the two that do
            // not have the next tile's first page
            const int part = K::kGroups == 2 ? grp : (grp + K::kGroups - g % K::kGroups) % K::kGroups - 1;
            float total = 0.f;
            float o[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) o[c] = 0.f;
            bool bad = t.bad;
            if (n > 0) {
              float* const sum = reinterpret_cast<float*>(smem + K::oSum) + (used & 1) * (128 * K::kGroups) + r;
              float* const top = reinterpret_cast<float*>(smem + K::oMax) + (used & 1) * (128 * K::kGroups) + r;
              sum[grp * 128] = l2.x + l2.y;
              top[grp * 128] = mx_all;
              bar_sync(1, 128 * K::kGroups);
              total = sum[0] + sum[128] + (K::kGroups == 3 ? sum[256] : 0.f);
              if (!forced) {
                m = first_at[0];
                if (n > 1 && m == -INFINITY) m = first_at[128];
                m_forced = max3(top[0], top[128], K::kGroups == 3 ? top[256] : -INFINITY);
                // (a weight above kReach makes the sum so)
                if (!again && total > kReach && r < K::kTokens * G && tok < t.tokens) marks[j] = 1;
              }
              if (part >= 0) {
                const int last = g - 1;
                wait_for(pv_done + 8 * (last % K::kRing), (last / K::kRing) & 1, flags, limit);
                __syncwarp();
                ptx::tc_fence_after();
                tmem_ld32(tmem + lanes + K::kColO + 64 * part, o);
                tmem_ld32(tmem + lanes + K::kColO + 64 * part + 32, o + 32);
                ptx::tmem_wait_ld();
                if (THREE && n > K::kSegment) {
                  const float4* const acc = reinterpret_cast<const float4*>(smem + K::oAcc) + part * 16 * 128 + r;
#pragma unroll
                  for (int c = 0; c < 16; ++c) {
                    const float4 x = acc[c * 128];
                    o[4 * c] += x.x, o[4 * c + 1] += x.y, o[4 * c + 2] += x.z, o[4 * c + 3] += x.w;
                  }
                }
                ptx::tc_fence_before();
                ptx::mbar_arrive(o_free);
              }
              bad = flags[8 + (used & 7)] == used + 1;
              used2 += n > 1;
              ++used;
            }
            if (part < 0) continue;
            const bool poison = bad || flags[0];
            if (poison && lane == 0)
              atomicOr(p.status, (flags[0] ? kStatusBitTimeout : 0u) | (bad ? kStatusBitBadSeq : 0u));
            const float inv = poison ? __int_as_float(0x7fc00000) : total == 0.f ? 0.f : (KV8 ? __ldg(p.v_scale + t.h) : 1.f) / total;
            const bool parts = WIDE && p.splits > 1;  // normalised fp32 parts and their lse
            float* const lse = parts ? p.ws_lse + (size_t)t.split * p.rows_total : p.lse;
            const size_t row0 = ((size_t)t.b * p.C + t.t0) * p.Hq + t.h * G;
            const int live = t.tokens * G;
            if (lse && part == 0 && r < live)
              lse[row0 + (size_t)tok * p.Hq + (r - tok * G)] =
                  poison ? inv : total == 0.f ? -INFINITY : (m + log2f(total)) * 0.6931471805599453f;
            // four lanes exchange their rows' 16-byte pieces, so that a store
            // writes 64 bytes of a row (not 16 bytes of 32 rows)
            {
              constexpr int kPieces = WIDE ? 16 : 8;  // of 16 bytes: 64 dims
              uint4* const out = parts ? reinterpret_cast<uint4*>(p.ws_o + (size_t)t.split * p.rows_total * kDim)
                                       : reinterpret_cast<uint4*>(p.out);
#pragma unroll
              for (int q = 0; q < kPieces / 4; ++q) {
                uint32_t w[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                  for (int u = 0; u < 4; ++u) {
                    if constexpr (WIDE) w[e][u] = __float_as_uint(o[16 * q + 4 * e + u] * inv);
                    else w[e][u] = pack<false>(o[32 * q + 8 * e + 2 * u] * inv, o[32 * q + 8 * e + 2 * u + 1] * inv);
                  }
#pragma unroll
                for (int bit = 1; bit <= 2; bit <<= 1)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (!(e & bit))
#pragma unroll
                      for (int u = 0; u < 4; ++u) {
                        const bool up = lane & bit;
                        const uint32_t give = up ? w[e][u] : w[e | bit][u];
                        const uint32_t got = __shfl_xor_sync(~0u, give, bit);
                        if (up) w[e][u] = got; else w[e | bit][u] = got;
                      }
#pragma unroll
                for (int e = 0; e < 4; ++e) {         // now piece (lane & 3) of the quad's row e
                  const int row = (r & ~3) + e, tk = row / G;
                  if (row < live)
                    out[(row0 + (size_t)tk * p.Hq + (row - tk * G)) * (2 * kPieces) + part * kPieces + 4 * q + (lane & 3)] =
                        make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
                }
              }
            }
          }
        }
        block_sync();
        if (again) break;
        int more = 0;
        for (int j = 0; j < round; ++j) more += marks[j];
        if (more == 0) break;
        sched.count = 2 * more;
        sched.marks = marks;
      }
      if (tid < kRound) marks[tid] = 0;
      block_sync();
    }
    ptx::tc_fence_before();
    block_sync();
  }
}

// ------------------------------------------------------------------ launch
template <int G, bool WIDE, bool THREE, bool FEW, bool KV8>
int launch_tiles(TileParams& prm, const rel_attn_shape* s, const void* q, const void* rel_table, int sms, int dev,
                   cudaStream_t st) {
  using K = TileConfig<G, KV8, THREE>;
  static bool set[kMaxDev];
  auto* kernel = sink_tiles_kernel<G, WIDE, THREE, FEW, KV8>;
  if (!allow_shared(kernel, K::kAlloc, dev, set)) return REL_ATTN_ERR_CUDA;
  prm.q_tiles = (s->q_tokens + K::kTokens - 1) / K::kTokens;
  const long long tiles = (long long)s->batch * s->num_kv_heads * prm.q_tiles * prm.splits;
  if (tiles >= (1ll << 31) - sms) return REL_ATTN_ERR_INVALID_ARG;
  if (!host::query_map(&prm.tmap_q, q, s, K::kTokens) || !host::rel_map(&prm.tmap_r, rel_table, s, K::kRel) ||
      !host::rel_map(&prm.tmap_few, rel_table, s, K::kFew))
    return REL_ATTN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(tiles, sms));
  cfg.blockDim = dim3(K::kThreads);
  cfg.dynamicSmemBytes = K::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, prm) != cudaSuccess) {
    cudaGetLastError();
    return REL_ATTN_ERR_CUDA;
  }
  return REL_ATTN_OK;
}

template <bool KV8, bool FEW>
int run_tiles(const rel_attn_shape* s, const void* q, const void* rel_table, TileParams& prm, int sms, int dev, cudaStream_t st) {
  auto launch = [&](auto group) {
    constexpr int G = decltype(group)::value;
    return (s->out_fp32 ? launch_tiles<G, true, true, FEW, KV8> : prm.splits > 1 ? launch_tiles<G, true, false, FEW, KV8>
                                                                : launch_tiles<G, false, false, FEW, KV8>)(prm, s, q, rel_table, sms, dev, st);
  };
  switch (s->num_q_heads / s->num_kv_heads) {
    case 4: return launch(std::integral_constant<int, 4>{});
    case 6: return launch(std::integral_constant<int, 6>{});
    case 8: return launch(std::integral_constant<int, 8>{});
    default: return REL_ATTN_ERR_INVALID_ARG;
  }
}

}  // namespace sink
}  // namespace relattn
