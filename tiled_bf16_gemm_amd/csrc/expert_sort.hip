// Slots sorted by expert: offsets of the groups, the slot of every row and the row of every slot.
//
//   offsets[e] = number of slots with an id in 0..e-1
//   place[s]   = offsets[id_s] + number of slots before s with the same id      (-1: an id outside 0..E-1)
//   source[place[s]] = s, and -1 from offsets[E] on
//
// A counting sort.  A workgroup takes its slots in order, a wave 64 of them at a time: the lanes that
// share an id are found with one ballot per bit of the ids, a slot's rank among them is the number of
// such lanes before it, and the wave's own counters in LDS carry the ranks from one 64 to the next.
// Ranks need no atomics, so the order (and with it every output) is fixed.
//
// Up to kSmallSlots slots one workgroup does everything in one launch.  Above that the slots are cut
// into parts: one launch counts every part's ids into a table in the workspace, and in a second one
// each workgroup adds up the table's columns (all parts: the offsets; the parts before its own: where
// its rows start) and places its part.  Up to a few hundred experts a third launch for the sums would
// cost more than the table's reads, which come from the caches (131072 slots over 256 experts: 64 KB a
// workgroup).  They grow with parts² · experts, though: with the two waves that a workgroup has for
// thousands of experts they are what 2^20 slots over 4096 take 629 µs for (256 parts, 4 MiB each; over
// 1024 experts 54 µs, over 256 25).
//
// Bound by dependent steps, not by bytes: 64 slots over 64 experts 2.2 µs; 131072 slots over 256 experts (1.6 MB)
// 2.8 µs for the counts and 8.3 for the rest, of which the launches are about 3 each.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert.hpp"
#include "ragged.hpp"

namespace tbg {

namespace {

constexpr int kMostWaves = 16;
constexpr int kWaveCounters = 8192;  // 16-bit counters of all waves, an id's side by side: up to 512 ids have 16
                                     // waves, 4096 two
constexpr int kMostGroups = 4096;
constexpr int kAhead = 16;  // values of the table that a thread asks for before it ranks its slots

// Lanes whose slot has this lane's id (among the lanes with `held`; e is below 2^bits).
__device__ __forceinline__ uint64_t peers(int e, bool held, int bits) {
  uint64_t m = __ballot(held);
  for (int b = 0; b < bits; ++b) {
    const bool one = (e >> b) & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

__device__ __forceinline__ int lanes_before(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Exclusive prefix sum over the E values of `v` in LDS, in place; v[E] becomes their sum.  `part` holds a
// value per wave.  Ends with a barrier.
__device__ __forceinline__ void scan_groups(int* v, int* part, int E) {
  const int per = (E + blockDim.x - 1) / blockDim.x, lo = min((int)threadIdx.x * per, E), hi = min(lo + per, E);
  int sum = 0;
  for (int e = lo; e < hi; ++e) sum += v[e];
  const int upto = wave_prefix_sum(sum);
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 63) part[wave] = upto;
  __syncthreads();
  int at = upto - sum;
  for (int w = 0; w < wave; ++w) at += part[w];
  for (int e = lo; e < hi; ++e) {
    const int n = v[e];
    v[e] = at;
    at += n;
  }
  if (threadIdx.x == blockDim.x - 1) {
    int all = 0;
    for (int w = 0; w < waves; ++w) all += part[w];
    v[E] = all;
  }
  __syncthreads();
}

// One step of a workgroup: blockDim.x·I slots from `first` on, wave w the w-th 64·I of them.
template <int I>
struct Step {
  int id[I], rank[I];  // id -1: none; rank among the wave's slots of the same id
};

template <int I>
__device__ __forceinline__ void load_ids(Step<I>& s, const SortParams& p, int64_t first, int64_t end) {
  const int64_t at = first + (threadIdx.x >> 6) * (64 * I) + (threadIdx.x & 63);
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int id = at + 64 * i < end ? p.experts[at + 64 * i] : -1;
    s.id[i] = (uint32_t)id < (uint32_t)p.groups ? id : -1;
  }
}

// Ranks, and the wave's counters (zero before; id e's at mine[e * waves]) with its slots of every id.
template <int I>
__device__ __forceinline__ void rank_ids(Step<I>& s, uint16_t* mine, int waves, int bits) {
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const bool held = s.id[i] >= 0;
    const uint64_t m = peers(s.id[i], held, bits);
    uint16_t* const count = mine + (held ? s.id[i] * waves : 0);
    const int before = held ? *count : 0;
    const int rank = lanes_before(m), all = __popcll(m);
    s.rank[i] = before + rank;
    // the reads of this 64 come before the writes, those before the next 64's reads: one wave's LDS
    // accesses complete in order, and the fences keep the compiler's order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (held && rank == all - 1) *count = (uint16_t)(before + all);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// The waves' counters become the counts of the waves before; sums[e] gets the step's count.  (An id's counters lie
// side by side, two to a dword: with a wave's side by side this took a dependent read and write for every wave.)
__device__ __forceinline__ void sum_waves(uint16_t* counters, int* sums, int E) {
  const int waves = blockDim.x >> 6;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    if (waves == 1) {
      sums[e] = counters[e];
      counters[e] = 0;
      continue;
    }
    uint32_t* const pairs = (uint32_t*)(counters + e * waves);
    uint32_t v[kMostWaves / 2];
#pragma unroll
    for (int w = 0; w < kMostWaves / 2; ++w) v[w] = 2 * w < waves ? pairs[w] : 0;
    uint32_t run = 0;
#pragma unroll
    for (int w = 0; w < kMostWaves / 2; ++w) {
      const uint32_t lo = v[w] & 0xFFFFu, hi = v[w] >> 16;
      if (2 * w < waves) pairs[w] = run | (run + lo) << 16;
      run += lo + hi;
    }
    sums[e] = (int)run;
  }
}

// The step's rows, base[e] being the first of id e.
template <int I>
__device__ __forceinline__ void store_step(const Step<I>& s, const SortParams& p, int64_t first, int64_t end,
                                           const uint16_t* mine, int waves, const int* base) {
  const int64_t at = first + (threadIdx.x >> 6) * (64 * I) + (threadIdx.x & 63);
#pragma unroll
  for (int i = 0; i < I; ++i) {
    if (at + 64 * i >= end) break;
    int row = -1;
    if (s.id[i] >= 0) {
      row = base[s.id[i]] + mine[s.id[i] * waves] + s.rank[i];
      p.source[row] = (int)(at + 64 * i);
    }
    p.place[at + 64 * i] = row;
  }
}

__device__ __forceinline__ void clear_counters(uint16_t* counters, int E) {
  const int n = (blockDim.x >> 6) * E;
  for (int i = threadIdx.x; i < (n + 1) / 2; i += blockDim.x) ((uint32_t*)counters)[i] = 0;
}

template <int I>
__global__ void __launch_bounds__(64 * kMostWaves) sort_small_kernel(SortParams p) {
  __shared__ __attribute__((aligned(4))) uint16_t counters[kWaveCounters + 2];
  __shared__ int base[kMostGroups + 1];
  __shared__ int part[kMostWaves];
  const int E = p.groups;
  const int waves = blockDim.x >> 6;
  uint16_t* mine = counters + (threadIdx.x >> 6);
  Step<I> s;
  load_ids(s, p, 0, p.slots);
  clear_counters(counters, E);
  __syncthreads();
  rank_ids(s, mine, waves, p.bits);
  __syncthreads();
  sum_waves(counters, base, E);
  __syncthreads();
  scan_groups(base, part, E);
  for (int e = threadIdx.x; e <= E; e += blockDim.x) p.offsets[e] = base[e];
  store_step(s, p, 0, p.slots, mine, waves, base);
  for (int r = base[E] + threadIdx.x; r < p.slots; r += blockDim.x) p.source[r] = -1;
}

// Counts of every id in part blockIdx.x.
__global__ void __launch_bounds__(1024) sort_count_kernel(SortParams p) {
  __shared__ int count[kMostGroups];
  const int E = p.groups;
  for (int e = threadIdx.x; e < E; e += blockDim.x) count[e] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * p.part, end = min(lo + p.part, (int64_t)p.slots);
  for (int64_t s = lo + threadIdx.x; s < end; s += blockDim.x) {
    const int id = p.experts[s];
    if ((uint32_t)id < (uint32_t)E) atomicAdd(&count[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) p.table[(int64_t)blockIdx.x * E + e] = count[e];
}

template <int I>
__global__ void __launch_bounds__(64 * kMostWaves) sort_place_kernel(SortParams p) {
  __shared__ __attribute__((aligned(4))) uint16_t counters[kWaveCounters + 2];
  __shared__ int base[kMostGroups + 1];
  __shared__ int before[kMostGroups];
  __shared__ int part[kMostWaves];
  const int E = p.groups, me = blockIdx.x, parts = gridDim.x;
  const int waves = blockDim.x >> 6;
  uint16_t* mine = counters + (threadIdx.x >> 6);
  const int64_t lo = (int64_t)me * p.part, end = min(lo + p.part, (int64_t)p.slots);
  const int step = blockDim.x * I;
  Step<I> s;
  load_ids(s, p, lo, end);  // on the way while the table is read
  clear_counters(counters, E);
  for (int e = threadIdx.x; e < E; e += blockDim.x) base[e] = before[e] = 0;
  __syncthreads();
  // Consecutive threads take consecutive ids; the threads beyond E take other parts.  The first kAhead values of a
  // thread are on the way while the slots are ranked.
  const int lanes = E < (int)blockDim.x ? E : (int)blockDim.x, rows = E ? blockDim.x / lanes : 0;
  const int row = E ? threadIdx.x / lanes : 0, e0 = E ? threadIdx.x % lanes : 0;
  int ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int b = row + i * rows;
    ahead[i] = e0 < E && row < rows && b < parts ? p.table[(int64_t)b * E + e0] : 0;
  }
  rank_ids(s, mine, waves, p.bits);
  if (e0 < E && row < rows) {
    int all = 0, first = 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      all += ahead[i];
      first += row + i * rows < me ? ahead[i] : 0;
    }
    for (int e = e0, from = row + kAhead * rows; e < E; e += lanes, from = row) {
#pragma unroll 8
      for (int b = from; b < parts; b += rows) {
        const int n = p.table[(int64_t)b * E + e];
        all += n;
        first += b < me ? n : 0;
      }
      atomicAdd(&base[e], all);
      atomicAdd(&before[e], first);
      all = first = 0;
    }
  }
  __syncthreads();
  scan_groups(base, part, E);
  if (me == 0)
    for (int e = threadIdx.x; e <= E; e += blockDim.x) p.offsets[e] = base[e];
  const int filled = base[E];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) base[e] += before[e];
  for (int64_t first = lo; first < end; first += step) {
    if (first > lo) {
      for (int e = threadIdx.x; e < E; e += blockDim.x) base[e] += before[e];
      clear_counters(counters, E);
      load_ids(s, p, first, end);
    }
    if (first > lo) {
      __syncthreads();
      rank_ids(s, mine, waves, p.bits);
    }
    __syncthreads();
    sum_waves(counters, before, E);
    __syncthreads();
    store_step(s, p, first, end, mine, waves, base);
    if (first + step < end) __syncthreads();
  }
  for (int64_t r = filled + lo + threadIdx.x; r < p.slots && r < filled + end; r += blockDim.x) p.source[r] = -1;
}

int waves_for(int groups) {
  int w = kMostWaves;  // a power of two: an id's counters are whole dwords, or one
  while (w > 1 && w * groups > kWaveCounters) w /= 2;
  return w;
}

}  // namespace

hipError_t launch_expert_sort(SortParams p, const SortPlan& plan, hipStream_t stream) {
  p.bits = 0;
  while ((1 << p.bits) < p.groups) ++p.bits;
  p.part = plan.part;
  const int most = 64 * waves_for(p.groups);
  if (plan.small) {
    const int want = p.slots > p.groups ? p.slots : p.groups;
    int threads = 64;
    while (threads < want && threads < most) threads *= 2;
    if (p.slots <= threads) hipLaunchKernelGGL((sort_small_kernel<1>), dim3(1), dim3(threads), 0, stream, p);
    else hipLaunchKernelGGL((sort_small_kernel<4>), dim3(1), dim3(threads), 0, stream, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(sort_count_kernel, dim3(plan.parts), dim3(1024), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((sort_place_kernel<2>), dim3(plan.parts), dim3(most), 0, stream, p);
  return hipGetLastError();
}

}  // namespace tbg
