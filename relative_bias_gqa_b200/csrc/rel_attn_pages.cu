// rel_attn_pages.cu -- the bookkeeping of the paged cache on the device:
// rel_attn_pages_resize (pages given to new positions and taken back from
// positions nothing can see any more), rel_attn_pages_fork (a sequence
// continued in another row) and rel_attn_pages_compact (live pages moved to
// the front of the pool).
//
// The state is the block table, the lengths and a reference count per page
// (the block-table entries that hold it; 0: free).  There is no free list: a
// call takes the lowest free pages, found by a scan over the counts, so that
// equal states give equal results whatever came before.
//
// What bounds it.  The integers of a large server (a few MB at most) lie in
// L2; a step is a chain of dependent phases (give back, count, pick, write),
// and their barriers and memory latencies are its time.  So a plan is one
// launch.  A small one is a single block, whose phases are parted by the
// block's own barrier; a large one is a block per SM, started together
// (cooperative launch) with a barrier of theirs in the workspace.  (A cluster
// of 8 blocks for every size took 13 us on a batch of 8 and 39 us on a server
// of 512 rows: its barrier costs the small one more than its work, and 8 SMs
// read 2 MB of counts too slowly.)  Page contents are then copied by a second
// kernel over the whole GPU, which starts early (PDL) and moves them at the
// rate of a plain copy.
#include <algorithm>
#include <type_traits>

#include "rel_attn_host.h"
#include "sm100_ptx.cuh"

namespace relattn {
namespace pages {

constexpr int kKeys = 64;                 // positions of a page
constexpr int kSoloThreads = 1024, kTeamThreads = 512;
// Plans up to these sizes are one block's.  One block / a block per SM, us: resize
// of 16 rows 5.8 / 10.1, 64 rows 6.9 / 10.3, 256 rows 12.0 / 11.8 (lengths to 2,000);
// 64 rows to 60,000 12.1 / 11.7, 512 rows to 2,000 20.6 / 12.4; fork of 8 rows to
// 60,000 14.3 / 17.7, 32 to 2,000 11.7 / 17.3, 128 to 2,000 20.6 / 19.0; compact of
// 2,311 pages 7.3 / 10.3, 9,728 15.1 / 15.0.  The rule goes by what a book may hold,
// not by what a call changes: at both limits one block is the slower one (resize of
// 256 rows to 16,000, 30,558 pages, 19.6 / 12.0; compact of 25,901 pages 31.9 / 26.5).
constexpr int kSoloPages = 32768, kSoloRows = 256;
constexpr int kMaxCtas = 256;
constexpr unsigned long long kBroken = 1ull << 63;   // among the arrivals: a wait at the barrier ran out
constexpr int kMaxPools = 512;
constexpr int kCopyThreads = 256;
constexpr int kChunk = kCopyThreads * 16 * 4;   // bytes a copying CTA moves at a time
// Entries of a task, in flight together: 8 to a lane where one block has all the
// tasks (its 32 warps go through them in turn: 16 branches of rows of up to 1,563
// entries 18.2 us, with 64 to a task 20.7), 2 where a block per SM has its share
// (a warp's scattered atomics are what the others wait for: a server of 512 rows
// 17.3 us, with 128 to a task 18.6).  (These with a copy of the state before each
// call: 1.4 us of the one, 4.3 of the other.)
constexpr int kSoloBlock = 256, kTeamBlock = 64;
constexpr int kTasks = 1024;              // tasks a block holds at a time

struct Book {
  int* table;
  int* lens;
  int* refs;
  int rows, width, num_pages;
};

// Workspace.  In the header, behind the status word: the team's barrier, its
// errors, the number of page copies.  Behind it: the blocks' counts, the pages
// to copy of each task of a fork and the rank of the first of them, the free
// (or destination) pages, the pages to copy, the new name of each page, -1 of a
// free one (a fork: a mark per row).
struct Work {
  unsigned* status;
  unsigned long long* arrived;
  unsigned* errors;
  int* copies;
  int* cta_count;
  int* task_count;
  int* task_first;
  int* dst;
  int* src;
  int* name;
  unsigned long long wait_ns;                // of a wait for the team
};

size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

size_t task_bytes(int rows, int width) { return align16((size_t)rows * ((width + kTeamBlock - 1) / kTeamBlock) * 4); }
size_t name_bytes(int rows, int num_pages) { return align16((size_t)std::max(rows, num_pages) * 4); }

size_t work_bytes(int rows, int width, int num_pages) {
  return kWorkspaceHeader + kMaxCtas * 4 + 2 * task_bytes(rows, width) + 2 * align16((size_t)num_pages * 4) +
         name_bytes(rows, num_pages);
}

Work work_parts(void* ws, const rel_attn_pages* g) {
  Work w;
  uint8_t* p = reinterpret_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    int* at = reinterpret_cast<int*>(p);
    p += bytes;
    return at;
  };
  w.status = reinterpret_cast<unsigned*>(take(kWorkspaceHeader));
  w.arrived = reinterpret_cast<unsigned long long*>(w.status + 32);   // (a 128-byte line of its own: it is polled)
  w.errors = w.status + 17;
  w.copies = reinterpret_cast<int*>(w.status + 18);
  w.cta_count = take(kMaxCtas * 4);
  w.task_count = take(task_bytes(g->num_seqs, g->max_pages_per_seq));
  w.task_first = take(task_bytes(g->num_seqs, g->max_pages_per_seq));
  w.dst = take(align16((size_t)g->num_pages * 4));
  w.src = take(align16((size_t)g->num_pages * 4));
  w.name = take(name_bytes(g->num_seqs, g->num_pages));
  w.wait_ns = host::wait_limit_ns();
  return w;
}

// ------------------------------------------------------------------ pieces
// The threads that carry out a plan: one block (SOLO) or a block per SM.
template <bool SOLO>
struct Team {
  // sums over rows: a small plan's stay below 2^31 (at most kSoloRows rows of
  // 2^25 entries, in blocks, and new pages counted to one more than the pool has)
  using Sum = std::conditional_t<SOLO, int, long long>;
  static constexpr int kThreads = SOLO ? kSoloThreads : kTeamThreads;
  static constexpr int kWarps = kThreads / 32;
  static constexpr int kBlock = SOLO ? kSoloBlock : kTeamBlock;
  const Work& w;
  bool ok;                                   // no wait has run out
  bool met;                                  // has come to the barrier before
  unsigned long long goal;                   // (thread 0) arrivals at the last turn, or found at the start
  __device__ __forceinline__ explicit Team(const Work& work) : w(work), ok(true), met(false), goal(0) {
    if (!SOLO && threadIdx.x == 0)
      asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(goal) : "l"(w.arrived) : "memory");
  }
  __device__ __forceinline__ int rank() const { return SOLO ? 0 : blockIdx.x; }
  __device__ __forceinline__ int ctas() const { return SOLO ? 1 : gridDim.x; }
  __device__ __forceinline__ int warp() const { return threadIdx.x >> 5; }
  // All of the team; what was written before is read after it (through L2).
  // Where a wait runs out the barrier is broken until the workspace is
  // initialised anew: every block that comes to it or waits there goes on with
  // ok false, and what others were to write is read only under ok.
  __device__ __forceinline__ void sync() {
    if constexpr (SOLO) {
      __syncthreads();
    } else {
      __syncthreads();
      if (!ok) return;
      bool here = true;
      if (threadIdx.x == 0) {
        auto arrivals = [&] {
          unsigned long long v;
          asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(w.arrived) : "memory");
          return v;
        };
        // (a launch finds whole turns: what is past them has arrived at its first one)
        if (!met) goal -= goal % gridDim.x;
        met = true;
        goal += gridDim.x;
        asm volatile("red.release.gpu.global.add.u64 [%0], %1;" ::"l"(w.arrived), "l"(1ull) : "memory");
        const unsigned long long t0 = ptx::global_timer_ns();
        unsigned long long v;
        for (unsigned n = 1; (v = arrivals()) < goal && !(v & kBroken); ++n) {
          if (n % 64 == 0 && ptx::global_timer_ns() - t0 > w.wait_ns) {   // (reading the timer takes longer than a poll)
            atomicOr(w.arrived, kBroken);
            v = kBroken;
            break;
          }
        }
        here = !(v & kBroken);
        if (!here) atomicOr(w.status, kStatusBitTimeout);
      }
      ok = __syncthreads_and(here) && ok;
    }
  }
};
// Data that other blocks of the team write: through L2.
__device__ __forceinline__ int load(const int* p) { return __ldcg(p); }

__device__ __forceinline__ int ceil_pages(int positions) { return (int)(((unsigned)positions + kKeys - 1) / kKeys); }

// Exclusive prefixes of each thread's two values over the block, and the
// block's sums.
// (32 bits where the sums fit: a shuffle moves one word)
template <typename I>
struct Two {
  I a, b;
};
template <int kThreads, typename I>
__device__ __forceinline__ Two<I> block_prefix(Two<I> v, Two<I>* sum, Two<I>* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](Two<I> x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const I a = __shfl_up_sync(~0u, x.a, d), b = __shfl_up_sync(~0u, x.b, d);
      if (lane >= d) x.a += a, x.b += b;
    }
    return x;
  };
  const Two<I> x = scan(v);
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  const Two<I> w = scan(lane < kThreads / 32 ? scratch[lane] : Two<I>{0, 0});
  *sum = {__shfl_sync(~0u, w.a, 31), __shfl_sync(~0u, w.b, 31)};
  const I a = __shfl_sync(~0u, w.a, (warp + 31) & 31), b = __shfl_sync(~0u, w.b, (warp + 31) & 31);
  __syncthreads();
  return {(warp ? a : 0) + x.a - v.a, (warp ? b : 0) + x.b - v.b};
}

// The stretch of the reference counts that a warp of the team owns.
struct Stretch {
  int first, last;
  template <bool SOLO>
  __device__ __forceinline__ Stretch(const Team<SOLO>& team, int num_pages) {
    const int warps = team.ctas() * Team<SOLO>::kWarps;
    const int len = ((num_pages + warps - 1) / warps + 31) / 32 * 32;
    const long long f = (long long)(team.rank() * Team<SOLO>::kWarps + team.warp()) * len;
    first = (int)min(f, (long long)num_pages);
    last = (int)min(f + len, (long long)num_pages);
  }
};

// Calls f(page, in range and matching, rank within the stretch) for each of
// the warp's pages, in order; returns the number that match.
template <typename Match, typename F>
__device__ __forceinline__ int for_matching(const int* refs, const Stretch& s, Match match, F f) {
  const int lane = threadIdx.x & 31;
  // loads in flight per lane (more makes code that a plan, run once per launch,
  // waits longer to fetch)
  constexpr int kAhead = 8;
  int rank = 0;
  for (int p = s.first; p < s.last; p += 32 * kAhead) {
    int v[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) v[q] = p + 32 * q + lane < s.last ? load(refs + p + 32 * q + lane) : -1;
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (p + 32 * q >= s.last) break;
      const bool in = p + 32 * q + lane < s.last, hit = in && match(v[q]);
      const unsigned mask = __ballot_sync(~0u, hit);
      f(p + 32 * q + lane, in, hit, rank + __popc(mask & ((1u << lane) - 1)));
      rank += __popc(mask);
    }
  }
  return rank;
}

// Of each warp's count `n`: the sum of the team's warps before it, and of all.
// (One synchronisation; `scratch`: an int per warp and two.)
template <bool SOLO>
__device__ __forceinline__ int before_warp(Team<SOLO>& team, int n, int* total, int* scratch) {
  constexpr int W = Team<SOLO>::kWarps;
  const int lane = threadIdx.x & 31, warp = team.warp();
  if (lane == 0) scratch[warp] = n;
  __syncthreads();
  const int mine = lane < W ? scratch[lane] : 0;
  int before = __reduce_add_sync(~0u, lane < warp ? mine : 0);
  const int block = __reduce_add_sync(~0u, mine);
  *total = block;
  if constexpr (!SOLO) {
    if (threadIdx.x == 0) team.w.cta_count[team.rank()] = block;
    team.sync();
    int all = 0, below = 0;
    for (int q = lane; q < team.ctas(); q += 32) {
      const int c = load(team.w.cta_count + q);
      all += c;
      below += q < team.rank() ? c : 0;
    }
    *total = __reduce_add_sync(~0u, all);
    before += __reduce_add_sync(~0u, below);
  }
  return before;
}

// The free pages of [first, last), at most 1,024 of them, as bits: lane l has
// those of 32 pages from first + 32 l.
__device__ __forceinline__ unsigned free_bits(const int* refs, int first, int last) {
  const int lane = threadIdx.x & 31;
  unsigned mine = 0;
#pragma unroll 1
  for (int p = first; p < last; p += 256) {
    int v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = p + 32 * q + lane < last ? load(refs + p + 32 * q + lane) : -1;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const unsigned mask = __ballot_sync(~0u, v[q] == 0);
      if (lane == (p - first) / 32 + q) mine = mask;
    }
  }
  return mine;
}

// The `need` lowest free pages into w.dst, in rising order; false (and no
// list) if there are fewer, or where a wait ran out.  All of the team calls it.
template <bool SOLO>
__device__ __forceinline__ bool pick_free(Team<SOLO>& team, const Book& bk, const Work& w, long long need, int* scratch) {
  if (need == 0) return true;
  const Stretch s(team, bk.num_pages);
  const int lane = threadIdx.x & 31;
  unsigned bits = 0;
  int n = 0, total;
  for (int p = s.first; p < s.last; p += 1024) {
    bits = free_bits(bk.refs, p, min(p + 1024, s.last));
    n += __reduce_add_sync(~0u, __popc(bits));
  }
  int rank = before_warp(team, n, &total, scratch);
  if (!team.ok || need > total) return false;
  for (int p = s.first; p < s.last && rank < need; p += 1024) {
    if (s.last - s.first > 1024) bits = free_bits(bk.refs, p, min(p + 1024, s.last));   // (else still at hand)
    int before = __popc(bits);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(~0u, before, d);
      if (lane >= d) before += x;
    }
    int at = rank + before - __popc(bits);
    for (unsigned m = bits; m && at < need; m &= m - 1) w.dst[at++] = p + 32 * lane + __ffs(m) - 1;
    rank += __shfl_sync(~0u, before, 31);
  }
  team.sync();
  return team.ok;
}

// Errors that any thread of the team met, as status bits for all of them.
// w.errors is zero before a plan and after it.
template <bool SOLO>
__device__ __forceinline__ unsigned team_errors(Team<SOLO>& team, unsigned mine) {
  if constexpr (SOLO) {
    return __syncthreads_or(mine != 0) ? kStatusBitBadSeq : 0u;
  } else {
    const unsigned any = __reduce_or_sync(~0u, mine);
    if (any && (threadIdx.x & 31) == 0) atomicOr(team.w.errors, any);
    team.sync();
    return load(reinterpret_cast<const int*>(team.w.errors)) | (team.ok ? 0u : kStatusBitTimeout);
  }
}

// A stretch of up to Team::kBlock entries of one row; `at`: what belongs to its
// first entry (a rank among the new pages), or -1 where pages are given back.
// (A fork's: `at` its destination, `from` the first entry that is copied.)
struct Task {
  int row, first, last, at, from;
};

// Tasks are numbered in row order; every ctas-th falls to this block, so that
// all warps share the long rows.  put(id, count, task): keeps those of the tasks
// id, id + 1, ... (task(k) for k < count) that are this block's and this round's.
struct TaskList {
  Task* tasks;
  int rank, ctas;
  long long base;                            // first id of this round
  __device__ __forceinline__ long long per_round() const { return (long long)kTasks * ctas; }
  template <typename F>
  __device__ __forceinline__ void put(long long id, int count, F task) const {
    long long k = max(base - id, 0ll);
    if (k >= count || id + k - base >= per_round()) return;
    const unsigned at = (unsigned)(id + k - base), past = at % (unsigned)ctas;
    const int on = (int)(rank >= (int)past ? rank - past : rank + ctas - past);   // to this block's next one
    unsigned slot = (at + on) / (unsigned)ctas;
#pragma unroll 1
    for (k += on; k < count && slot < kTasks; k += ctas, ++slot) tasks[slot] = task((int)k);
  }
  // number of this block's tasks of the round, of `total` in all
  __device__ __forceinline__ int count(long long total) const {
    const long long n = min(total - base, per_round()) - rank;
    return n <= 0 ? 0 : (int)((n + ctas - 1) / ctas);
  }
};

template <int kBlock>
__device__ __forceinline__ int blocks(int first, int last) { return last > first ? (last - first + kBlock - 1) / kBlock : 0; }

// f(entry) for the entries of a lane: the values first, so that their loads are
// in flight together.
template <int kBlock, typename V, typename F>
__device__ __forceinline__ void for_entries(const Task& t, V value, F f) {
  const int lane = threadIdx.x & 31;
  int v[kBlock / 32];
#pragma unroll
  for (int q = 0; q < kBlock / 32; ++q)
    if (t.first + 32 * q + lane < t.last) v[q] = value(t.first + 32 * q + lane);
#pragma unroll
  for (int q = 0; q < kBlock / 32; ++q)
    if (t.first + 32 * q + lane < t.last) f(t.first + 32 * q + lane, v[q]);
}

// ------------------------------------------------------------------ resize
// Entries [sinks_end, keep_from) left the window, [end_new, end_old) lie past
// the new length: both are given back; [end_old, end_new) get pages.
struct Change {
  int sinks_end, keep_from, end_old, end_new;
  __device__ __forceinline__ Change(int L, int N, int window, int sinks) {
    end_old = ceil_pages(L);
    end_new = ceil_pages(N);
    const int oldest = window > 0 ? min(L, N) - max(window - 1, 3) : 0;   // first position still needed
    keep_from = oldest > 0 ? oldest / kKeys : 0;
    sinks_end = ceil_pages(sinks);
  }
};

struct Plan {
  long long need, tasks, given;              // new pages, all tasks, those that give back
};

// Bound by the latencies of its phases: 8 rows 6 us (rows, give back, count,
// pick, write: each a trip to L2); 512 rows over 484K pages 13 us, of which the
// barriers are three times 1.8.  With a window a call goes over all entries between
// the sinks and the window's start, given back long ago or not, as the state does
// not say from where on: rows of 128K positions, window 1,024, one position more to
// each, 8 rows 9.7 us, 64 rows (one block, 126,000 entries) 36, 512 rows of up to
// that length (a block per SM) 14.
template <bool SOLO>
__global__ void __launch_bounds__(Team<SOLO>::kThreads)
resize_kernel(const Book bk, const Work w, const int* new_lens, int window, int sinks) {
  constexpr int kThreads = Team<SOLO>::kThreads, kBlock = Team<SOLO>::kBlock;
  __shared__ Task tasks[kTasks];
  using Sum = typename Team<SOLO>::Sum;
  __shared__ Two<Sum> scratch[32];
  __shared__ int counts[34];
  Team<SOLO> team(w);
  TaskList list = {tasks, team.rank(), team.ctas(), 0};
  ptx::pdl_launch_dependents();
  // ---- tasks of the rows and the places of their new pages, in row order;
  // every block goes over all rows, so that no exchange is needed
  bool bad_len = false;
  auto plan_round = [&](long long base) {
    list.base = base;
    Plan plan = {0, 0, 0};
    for (int b0 = 0; b0 < bk.rows; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      int L = 0, N = 0;
      if (b < bk.rows) {
        L = load(bk.lens + b);
        N = __ldg(new_lens + b);
        if ((unsigned)L > (unsigned)bk.width * kKeys || (unsigned)N > (unsigned)bk.width * kKeys) {
          bad_len = true;
          L = N = 0;
        }
      }
      const Change c(L, N, window, sinks);
      const int out = blocks<kBlock>(c.sinks_end, c.keep_from), cut = blocks<kBlock>(c.end_new, c.end_old);
      const int fresh = max(0, c.end_new - c.end_old), in = blocks<kBlock>(c.end_old, c.end_new);
      Two<Sum> sum;
      const Two<Sum> at = block_prefix<kThreads, Sum>({out + cut + in, min(fresh, bk.num_pages + 1)}, &sum, scratch);
      const long long id = plan.tasks + at.a;
      const long long page = plan.need + at.b;
      plan.tasks += sum.a;
      plan.need += sum.b;
      plan.given += out + cut;               // (of this thread's rows: summed by the vote below)
      list.put(id, out, [&](int k) {
        return Task{b, c.sinks_end + k * kBlock, min(c.sinks_end + (k + 1) * kBlock, c.keep_from), -1, 0};
      });
      list.put(id + out, cut, [&](int k) {
        return Task{b, c.end_new + k * kBlock, min(c.end_new + (k + 1) * kBlock, c.end_old), -1, 0};
      });
      list.put(id + out + cut, in, [&](int k) {
        return Task{b, c.end_old + k * kBlock, min(c.end_old + (k + 1) * kBlock, c.end_new),
                    (int)min(page + (long long)k * kBlock, (long long)bk.num_pages), 0};
      });
    }
    return plan;
  };
  const Plan plan = plan_round(0);
  const bool any_given = __syncthreads_or(plan.given > 0);
  const bool any_bad = __syncthreads_or(bad_len);
  const bool rounds = plan.tasks > list.per_round();
  auto for_tasks = [&](auto f) {
    for (long long base = 0; base < plan.tasks; base += list.per_round()) {
      if (rounds) {                          // more than the list holds: round by round
        __syncthreads();
        plan_round(base);
        __syncthreads();
      }
      const int n = list.count(plan.tasks);
      for (int k = team.warp(); k < n; k += Team<SOLO>::kWarps) f(list.tasks[k]);
    }
  };
  // ---- give back
  unsigned bad = 0;
  auto give = [&](int delta) {
    for_tasks([&](const Task& t) {
      if (t.at >= 0) return;
      const int* row = bk.table + (size_t)t.row * bk.width;
      int had[kBlock / 32];                  // (the atomics' answers together as well)
      for_entries<kBlock>(t, [&](int i) { return load(row + i); }, [&](int i, int page) {
        int& h = had[(i - t.first) / 32];
        h = page < 0 ? 1 : page < bk.num_pages ? atomicAdd(bk.refs + page, delta) : 0;
      });
      if (delta < 0)
        for_entries<kBlock>(t, [](int) { return 0; }, [&](int i, int) {
          if (had[(i - t.first) / 32] <= 0) bad = kStatusBitBadSeq;
        });
    });
  };
  if (any_bad) bad = kStatusBitBadSeq;
  if (!any_bad) {
    if (any_given) {
      give(-1);
      bad = team_errors(team, bad);
    }
    if (!bad && !pick_free(team, bk, w, plan.need, counts)) bad = team.ok ? kStatusBitNoPages : kStatusBitTimeout;
    if (bad && any_given) {                  // as it was before the call
      const unsigned why = bad;
      team.sync();
      if (team.rank() == 0 && threadIdx.x == 0) *w.errors = 0;
      give(+1);
      bad = why;
    }
  }
  if (bad) {
    if (team.rank() == 0 && threadIdx.x == 0) atomicOr(w.status, bad);
    return;
  }
  // ---- the rows.  (Where nothing was exchanged, every block must still have
  // read the lengths.)
  if (!any_given && plan.need == 0) team.sync();
  for_tasks([&](const Task& t) {
    int* row = bk.table + (size_t)t.row * bk.width;
    for_entries<kBlock>(t, [&](int i) { return t.at < 0 ? -1 : load(w.dst + t.at + i - t.first); }, [&](int i, int page) {
      row[i] = page;
      if (page >= 0) bk.refs[page] = 1;
    });
  });
  if (rounds) team.sync();                   // (the rounds read the lengths again)
  if (!team.ok) return;
  for (int b = team.rank() * kThreads + threadIdx.x; b < bk.rows; b += team.ctas() * kThreads) bk.lens[b] = __ldg(new_lens + b);
}

// -------------------------------------------------------------------- fork
// The sources' entries are gone over twice (to count the copies and check, and to
// write the new rows); in one block that is 4 rounds of its 32 warps for 16 rows
// of up to 1,563 entries: 13.5 us, and 3 us for the copies of their last pages.
template <bool SOLO>
__global__ void __launch_bounds__(Team<SOLO>::kThreads)
fork_kernel(const Book bk, const Work w, const int* src_rows, const int* dst_rows, int forks, int all) {
  constexpr int kThreads = Team<SOLO>::kThreads, kBlock = Team<SOLO>::kBlock;
  __shared__ Task tasks[kTasks];
  using Sum = typename Team<SOLO>::Sum;
  __shared__ Two<Sum> scratch[32];
  __shared__ int counts[34];
  Team<SOLO> team(w);
  TaskList list = {tasks, team.rank(), team.ctas(), 0};
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, first = team.rank() * kThreads + threadIdx.x, step = team.ctas() * kThreads;
  if (first == 0) *w.copies = 0;
  // a mark per row: of a destination 0 (against two forks into one), of another source -1
  __shared__ int near_marks[SOLO ? kSoloRows : 1];
  int* const marks = SOLO ? near_marks : w.name;
  for (int k = first; k < forks; k += step) {
    const int d = __ldg(dst_rows + k), s = __ldg(src_rows + k);
    if ((unsigned)d < (unsigned)bk.rows) marks[d] = -1;
    if ((unsigned)s < (unsigned)bk.rows) marks[s] = -1;
  }
  team.sync();
  unsigned bad = 0;
  for (int k = first; k < forks; k += step) {
    const int d = __ldg(dst_rows + k);
    if ((unsigned)d >= (unsigned)bk.rows || atomicAdd(marks + d, 1) != -1) bad = kStatusBitBadSeq;
  }
  // ---- tasks: the entries of the sources, by fork and block (every CTA goes
  // over all forks)
  auto plan_round = [&](long long base) {
    list.base = base;
    long long total = 0;
    for (int k0 = 0; k0 < forks; k0 += kThreads) {
      const int k = k0 + threadIdx.x;
      int end = 0, s = 0, d = 0, from = 0;       // (a copied entry: the page at and behind the last full one; all: every one)
      if (k < forks) {
        d = __ldg(dst_rows + k);
        s = __ldg(src_rows + k);
        if ((unsigned)s >= (unsigned)bk.rows || (unsigned)d >= (unsigned)bk.rows) {
          bad = kStatusBitBadSeq;
        } else {
          const int L = load(bk.lens + s);
          if ((unsigned)L > (unsigned)bk.width * kKeys || load(bk.lens + d) != 0) bad = kStatusBitBadSeq;
          else end = ceil_pages(L), from = all ? 0 : L / kKeys;
        }
      }
      Two<Sum> sum;
      const long long id = total + block_prefix<kThreads, Sum>({blocks<kBlock>(0, end), 0}, &sum, scratch).a;
      total += sum.a;
      list.put(id, blocks<kBlock>(0, end), [&](int i) { return Task{s, i * kBlock, min((i + 1) * kBlock, end), d, from}; });
    }
    return total;
  };
  const long long total = plan_round(0);
  __syncthreads();
  const bool rounds = total > list.per_round();
  auto for_tasks = [&](auto f) {
    for (long long base = 0; base < total; base += list.per_round()) {
      if (rounds) {
        __syncthreads();
        plan_round(base);
        __syncthreads();
      }
      const int n = list.count(total);
      for (int k = team.warp(); k < n; k += Team<SOLO>::kWarps) f(list.tasks[k], base + (long long)k * team.ctas() + team.rank());
    }
  };
  // ---- pages to copy of each task
  for_tasks([&](const Task& t, long long id) {
    const int* const row = bk.table + (size_t)t.row * bk.width;
    int v[kBlock / 32], n = 0;
#pragma unroll
    for (int q = 0; q < kBlock / 32; ++q) v[q] = t.first + 32 * q + lane < t.last ? load(row + t.first + 32 * q + lane) : -1;
#pragma unroll
    for (int q = 0; q < kBlock / 32; ++q) {
      n += v[q] >= 0 && t.first + 32 * q + lane >= t.from;
      v[q] = v[q] < 0 ? 1 : v[q] < bk.num_pages ? load(bk.refs + v[q]) : 0;
    }
#pragma unroll
    for (int q = 0; q < kBlock / 32; ++q)
      if (v[q] <= 0) bad = kStatusBitBadSeq;
    n = __reduce_add_sync(~0u, n);
    if (lane == 0) w.task_count[id] = n;
  });
  bad = team_errors(team, bad);
  // ---- first new page of each task
  long long need = 0;
  if (!bad) {
    for (long long i0 = 0; i0 < total; i0 += kThreads) {
      const long long i = i0 + threadIdx.x;
      Two<Sum> sum;
      const long long at = need + block_prefix<kThreads, Sum>({i < total ? load(w.task_count + i) : 0, 0}, &sum, scratch).a;
      if (i < total && i % team.ctas() == team.rank()) w.task_first[i] = (int)min(at, (long long)bk.num_pages);
      need += sum.a;
    }
    __syncthreads();                         // (a task's rank is read in the block that wrote it)
    if (!pick_free(team, bk, w, need, counts)) bad = team.ok ? kStatusBitNoPages : kStatusBitTimeout;
  }
  if (bad) {
    team.sync();
    if (first == 0) {
      *w.errors = 0;
      atomicOr(w.status, bad);
    }
    return;
  }
  // ---- the new rows
  for_tasks([&](const Task& t, long long id) {
    const int* const from_row = bk.table + (size_t)t.row * bk.width;
    int* const row = bk.table + (size_t)t.at * bk.width;
    int at = load(w.task_first + id);
    int v[kBlock / 32];
#pragma unroll
    for (int q = 0; q < kBlock / 32; ++q)
      v[q] = t.first + 32 * q + lane < t.last ? load(from_row + t.first + 32 * q + lane) : -1;
#pragma unroll
    for (int q = 0; q < kBlock / 32; ++q) {
      const int i = t.first + 32 * q + lane, page = v[q];
      const bool copied = page >= 0 && i >= t.from;
      const unsigned mask = __ballot_sync(~0u, copied);
      int now = page < 0 ? -1 : page;
      if (copied) {
        const int to = at + __popc(mask & ((1u << lane) - 1));
        now = load(w.dst + to);
        w.src[to] = page;
        bk.refs[now] = 1;
      } else if (page >= 0) {
        atomicAdd(bk.refs + page, 1);
      }
      if (i < t.last) row[i] = now;
      at += __popc(mask);
    }
  });
  team.sync();                               // (every block has read the lengths)
  if (!team.ok) return;
  // (a source that is a destination as well was free: its length, which another
  // thread may have written by now, is not read)
  for (int k = first; k < forks; k += step) {
    const int s = __ldg(src_rows + k), mark = SOLO ? near_marks[s] : load(w.name + s);
    bk.lens[__ldg(dst_rows + k)] = mark == -1 ? load(bk.lens + s) : 0;
  }
  if (first == 0) *w.copies = (int)need;
}

// ----------------------------------------------------------------- compact
// With n live pages: the live page of rank r (counted from page 0) that lies
// at n or behind goes to the hole of rank r - (n - holes), where the holes are
// the free pages below n, and there are as many of the one as of the other.
// Two passes over the counts with a barrier between: 5 us for a pool of a few
// hundred pages, with the copies.
template <bool SOLO>
__global__ void __launch_bounds__(Team<SOLO>::kThreads) compact_kernel(const Book bk, const Work w, int* num_live) {
  __shared__ int counts[34];
  Team<SOLO> team(w);
  ptx::pdl_launch_dependents();
  const int first = team.rank() * Team<SOLO>::kThreads + threadIdx.x, step = team.ctas() * Team<SOLO>::kThreads;
  const Stretch s(team, bk.num_pages);
  auto is_live = [](int refs) { return refs > 0; };
  const int c = for_matching(bk.refs, s, is_live, [](int, bool, bool, int) {});
  int n;
  const int before = before_warp(team, c, &n, counts);
  if (!team.ok) return;
  // w.src takes the live pages at n and behind by rank from the end (they are
  // as many as the holes, but how many is not known yet), w.dst the holes; a
  // live page keeps its name until it moves, a free one has none
  for_matching(bk.refs, s, is_live, [&](int page, bool in, bool hit, int rank) {
    rank += before;
    if (in && page >= n) {
      if (hit) w.src[n - 1 - rank] = page;
    } else if (in && !hit) {
      w.dst[page - rank] = page;
    }
    if (in) w.name[page] = hit ? page : -1;
    if (in && page == n) *w.copies = n - rank;   // holes = live pages at n and behind
  });
  if (first == 0) {
    if (n == bk.num_pages) *w.copies = 0;
    *num_live = n;
  }
  team.sync();
  if (!team.ok) return;
  // (hole k takes the live page of rank n - holes + k, which is entry holes - 1 - k)
  const int holes = load(w.copies);
  for (int k = first; k < holes; k += step) {
    const int from = load(w.src + holes - 1 - k), to = load(w.dst + k);
    w.name[from] = to;
    bk.refs[to] = load(bk.refs + from);
    bk.refs[from] = 0;
  }
}

// -------------------------------------------------------------- page copies
// (few pools in a small struct: it travels with every launch)
template <int N>
struct Pools {
  int count;
  unsigned chunks;                          // chunks of a page over all pools
  unsigned first[N];                        // a pool's first one
  unsigned long long bytes[N];              // of a page
  uint8_t* data[N];
};

// Copies w.copies pages (w.src to w.dst, no page on both sides) in every
// pool (16 KB to a block at a time, 64 bytes in flight to a thread: 1.11 GB read
// and written in 179 us, 6.2 TB/s); with `rename`, also gives the block table's
// entries their new names, and reports those that name no live page.
template <int N>
__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(const __grid_constant__ Pools<N> pools, const Book bk, const Work w, const int* num_live, int rename) {
  // (a compaction lists its sources from the last)
  ptx::pdl_wait_primary();
  if (*w.status & kStatusBitTimeout) return;      // (the plan is not whole)
  const int copies = *w.copies;
  if (rename) {
    // (where no page moves too: every entry is looked at, whether it names a live page)
    const int n = *num_live;
    bool bad = false;
    for (int b = blockIdx.x; b < bk.rows; b += gridDim.x) {
      const int L = bk.lens[b];
      if ((unsigned)L > (unsigned)bk.width * kKeys) {
        bad = true;
        continue;
      }
      for (int i = threadIdx.x; i < ceil_pages(L); i += kCopyThreads) {
        int* e = bk.table + (size_t)b * bk.width + i;
        const int page = *e;
        if (page < 0) continue;
        const int name = page < bk.num_pages ? w.name[page] : -1;
        if (name < 0) bad = true;
        else if (page >= n) *e = name;
      }
    }
    if (bad) atomicOr(w.status, kStatusBitBadSeq);
  }
  const unsigned long long units = (unsigned long long)copies * pools.chunks;
  for (unsigned long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int k = (int)(u / pools.chunks);
    const unsigned c = (unsigned)(u - (unsigned long long)k * pools.chunks);
    int lo = 0, hi = pools.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pools.first[mid] <= c) lo = mid; else hi = mid - 1;
    }
    const unsigned long long bytes = pools.bytes[lo], off = (unsigned long long)(c - pools.first[lo]) * kChunk;
    const uint4* from = reinterpret_cast<const uint4*>(pools.data[lo] + (size_t)w.src[rename ? copies - 1 - k : k] * bytes + off);
    uint4* to = reinterpret_cast<uint4*>(pools.data[lo] + (size_t)w.dst[k] * bytes + off);
    const int n = (int)(min((unsigned long long)kChunk, bytes - off) / 16);
    uint4 v[kChunk / 16 / kCopyThreads];
#pragma unroll
    for (int q = 0; q < kChunk / 16 / kCopyThreads; ++q)
      if (q * kCopyThreads + (int)threadIdx.x < n) v[q] = __ldcs(from + q * kCopyThreads + threadIdx.x);
#pragma unroll
    for (int q = 0; q < kChunk / 16 / kCopyThreads; ++q)
      if (q * kCopyThreads + (int)threadIdx.x < n) __stcs(to + q * kCopyThreads + threadIdx.x, v[q]);
  }
}

// -------------------------------------------------------------------- host
namespace {

bool off(const void* p, uintptr_t a) { return !p || (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// (rows and pages up to 2^30: the loops over them step past the last by less than that)
bool sizes_fit(const rel_attn_pages* p) {
  return p && p->num_seqs >= 1 && p->num_seqs <= (1 << 30) && p->max_pages_per_seq >= 1 && p->num_pages >= 1 &&
         p->num_pages <= (1 << 30) && (long long)p->max_pages_per_seq * kKeys < (1ll << 31);
}

int check(const rel_attn_pages* p, const void* workspace, size_t bytes) {
  if (!sizes_fit(p)) return REL_ATTN_ERR_INVALID_ARG;
  if (off(p->block_table, 4) || off(p->seq_lens, 4) || off(p->page_refs, 4) || off(workspace, 256))
    return REL_ATTN_ERR_INVALID_ARG;
  return bytes < work_bytes(p->num_seqs, p->max_pages_per_seq, p->num_pages) ? REL_ATTN_ERR_WORKSPACE_TOO_SMALL : REL_ATTN_OK;
}

int check_pools(const rel_attn_pool* pools, int count) {
  if (count < 0 || count > kMaxPools || (count > 0 && !pools)) return REL_ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (off(pools[i].data, 16) || pools[i].page_bytes == 0 || pools[i].page_bytes % 16 ||
        pools[i].page_bytes > (1ull << 32))
      return REL_ATTN_ERR_INVALID_ARG;
  return REL_ATTN_OK;
}

Book book(const rel_attn_pages* p) {
  return {p->block_table, p->seq_lens, p->page_refs, p->num_seqs, p->max_pages_per_seq, p->num_pages};
}

// One block where the plan is small, else a block per SM, started together.
template <typename... A, typename... B>
int launch_plan(void (*solo)(A...), void (*team)(A...), const rel_attn_pages* p, int sms, cudaStream_t st, B... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  const bool small = p->num_pages <= kSoloPages && p->num_seqs <= kSoloRows;
  cfg.gridDim = dim3(small ? 1 : std::min(sms, kMaxCtas));
  cfg.blockDim = dim3(small ? kSoloThreads : kTeamThreads);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = small ? 0 : 1;
  if (cudaLaunchKernelEx(&cfg, small ? solo : team, A(args)...) != cudaSuccess) {
    cudaGetLastError();
    return REL_ATTN_ERR_CUDA;
  }
  return REL_ATTN_OK;
}

template <int N>
int launch_copies(const rel_attn_pool* pools, int count, const Book& bk, const Work& w, const int* num_live, int rename,
                  int sms, cudaStream_t st) {
  Pools<N> pl;
  pl.count = count;
  pl.chunks = 0;
  for (int i = 0; i < count; ++i) {
    pl.first[i] = pl.chunks;
    pl.bytes[i] = pools[i].page_bytes;
    pl.data[i] = reinterpret_cast<uint8_t*>(pools[i].data);
    pl.chunks += (unsigned)((pools[i].page_bytes + kChunk - 1) / kChunk);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms * 8);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, copy_kernel<N>, pl, bk, w, num_live, rename) != cudaSuccess) {
    cudaGetLastError();
    return REL_ATTN_ERR_CUDA;
  }
  return REL_ATTN_OK;
}

int copy_pages(const rel_attn_pool* pools, int count, const Book& bk, const Work& w, const int* num_live, int rename,
               int sms, cudaStream_t st) {
  return (count <= 8 ? launch_copies<8> : launch_copies<kMaxPools>)(pools, count, bk, w, num_live, rename, sms, st);
}

}  // namespace
}  // namespace pages
}  // namespace relattn

using namespace relattn;

extern "C" size_t rel_attn_pages_workspace_bytes(const rel_attn_pages* p) {
  if (!pages::sizes_fit(p)) return 0;
  return pages::work_bytes(p->num_seqs, p->max_pages_per_seq, p->num_pages);
}

extern "C" int rel_attn_pages_resize(const rel_attn_pages* p, const int32_t* new_lens, int window, int num_sinks,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  int rc = pages::check(p, workspace, workspace_bytes);
  if (rc != REL_ATTN_OK) return rc;
  if (pages::off(new_lens, 4) || num_sinks < 0) return REL_ATTN_ERR_INVALID_ARG;
  int dev, sms;
  rc = host::current_device(&dev, &sms);
  if (rc != REL_ATTN_OK) return rc;
  return pages::launch_plan(pages::resize_kernel<true>, pages::resize_kernel<false>, p, sms,
                            reinterpret_cast<cudaStream_t>(stream), pages::book(p), pages::work_parts(workspace, p),
                            new_lens, window, num_sinks);
}

extern "C" int rel_attn_pages_fork(const rel_attn_pages* p, const int32_t* src_rows, const int32_t* dst_rows,
                                   int num_forks, int copy_all, const rel_attn_pool* pools, int num_pools,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  int rc = pages::check(p, workspace, workspace_bytes);
  if (rc != REL_ATTN_OK) return rc;
  if (pages::off(src_rows, 4) || pages::off(dst_rows, 4) || num_forks < 1 || num_forks > p->num_seqs ||
      (copy_all != 0 && copy_all != 1))
    return REL_ATTN_ERR_INVALID_ARG;
  rc = pages::check_pools(pools, num_pools);
  if (rc != REL_ATTN_OK) return rc;
  int dev, sms;
  rc = host::current_device(&dev, &sms);
  if (rc != REL_ATTN_OK) return rc;
  const pages::Book bk = pages::book(p);
  const pages::Work w = pages::work_parts(workspace, p);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = pages::launch_plan(pages::fork_kernel<true>, pages::fork_kernel<false>, p, sms, st, bk, w, src_rows, dst_rows,
                          num_forks, copy_all);
  if (rc != REL_ATTN_OK || num_pools == 0) return rc;
  return pages::copy_pages(pools, num_pools, bk, w, nullptr, 0, sms, st);
}

extern "C" int rel_attn_pages_compact(const rel_attn_pages* p, const rel_attn_pool* pools, int num_pools,
                                      int32_t* num_live, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = pages::check(p, workspace, workspace_bytes);
  if (rc != REL_ATTN_OK) return rc;
  if (pages::off(num_live, 4)) return REL_ATTN_ERR_INVALID_ARG;
  rc = pages::check_pools(pools, num_pools);
  if (rc != REL_ATTN_OK) return rc;
  int dev, sms;
  rc = host::current_device(&dev, &sms);
  if (rc != REL_ATTN_OK) return rc;
  const pages::Book bk = pages::book(p);
  const pages::Work w = pages::work_parts(workspace, p);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = pages::launch_plan(pages::compact_kernel<true>, pages::compact_kernel<false>, p, sms, st, bk, w, num_live);
  if (rc != REL_ATTN_OK) return rc;
  return pages::copy_pages(pools, num_pools, bk, w, num_live, 1, sms, st);
}
