// Token embedding, out[t] = scale table[ids[t]], and its gradient: the dense
// table gradient with one fixed-order fp32 sum per row.
//
// The gradient sorts the tokens by id (stable, so a row's sum runs in token
// order), then adds the sorted rows in chunks of equal length, so that a
// token that makes up a large share of the batch costs no more than any
// other; a row that spans chunks leaves fp32 partials that a last kernel adds
// in chunk order.  No atomics on floating-point values: bit-reproducible.
#include "common.cuh"
#include "ptx.cuh"
#include "step.h"

namespace moe {
namespace {

constexpr int kFwdThreads = 256;
constexpr int kFwdVecs = 4;       // vectors of 8 per thread
constexpr int kSortThreads = 512;  // of a sorting CTA; as many again clear its rows
constexpr int kSortEach = 32;        // consecutive tokens per thread, one bit of a mask each
constexpr int kSortStep = 8;         // of them at a time
constexpr int kSortBatch = kSortThreads * kSortEach;  // tokens collected and placed at a time
constexpr int kSortMaxIds = 8192;    // ids per sorting CTA
constexpr int kSortPlaces = 8192;    // places of the placing warps: warps x ids, at least one warp
constexpr int kChunkMax = 32;     // sorted rows per CTA of the sum
constexpr int kAhead = 8;         // rows a thread has in flight
constexpr int kSumThreads = 128;  // vectors of 8 columns per CTA of the sum
constexpr int kFullCtas = 152;    // CTAs of the sum that leave no SM idle
constexpr int kJoinGroups = 4;    // parts of a row's partials that a CTA of the join adds at once

// Vector i of [T, nv]: token i / nv, four vectors per thread in flight.  Bound by
// memory: T = 8192, d = 2048: 9.2 us for 67 MB (part of it from L2).  The launch covers at most 2^31 vectors,
// so the index arithmetic is 32-bit; out and ids point at its first token.
__global__ void __launch_bounds__(kFwdThreads)
    embedding_kernel(const uint4* table, const int32_t* ids, unsigned total, unsigned nv, int V, float scale,
                     uint4* out, int* status) {
  dependency_wait();
  const unsigned base = blockIdx.x * (kFwdThreads * kFwdVecs) + threadIdx.x;
  uint4 v[kFwdVecs];
#pragma unroll
  for (int j = 0; j < kFwdVecs; ++j) {
    const unsigned i = base + j * kFwdThreads;
    v[j] = make_uint4(0, 0, 0, 0);
    if (i >= total) continue;
    const unsigned t = i / nv;
    const int id = __ldg(ids + t);
    if (id >= V) {
      record_status(status, MOE_ERR_DEVICE_BOUNDS);
    } else if (id >= 0) {
      v[j] = __ldg(table + (long long)id * nv + (i - t * nv));
    }
  }
#pragma unroll
  for (int j = 0; j < kFwdVecs; ++j) {
    const unsigned i = base + j * kFwdThreads;
    if (i >= total) continue;
    float f[8];
    unpack8(v[j], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale;
    out[i] = pack8(f);
  }
}

// Layout of the gradient's workspace.
struct SortWs {
  int32_t* order;  // [T] tokens by id, stable
  int32_t* sid;    // [T] their ids
  int32_t* n;      // [1] tokens with an id in [0, V)
  float* part;     // [chunks][2][d]: partial of the chunk's first row if it began
                   // earlier (0), of its last row if it goes on (1)
};
// Rows per chunk: 32, or 8 while chunks of 32 leave SMs without a CTA (a chunk's
// rows are added one after another: the call for 58 tokens of 320 channels takes
// 9.5 us with 8, 12.3 with 32; 8 up to two CTAs per SM instead: T = 9000, d =
// 1024, 23.8 us against 21.4).
int chunk_of(int T, int nv) {
  const long long ctas = (long long)((T + kChunkMax - 1) / kChunkMax) * ((nv + kSumThreads - 1) / kSumThreads);
  return ctas < kFullCtas ? 8 : kChunkMax;
}
int chunks_of(int T, int nv) { return (T + chunk_of(T, nv) - 1) / chunk_of(T, nv); }
SortWs carve(void* ws, int T) {
  char* w = static_cast<char*>(ws);
  SortWs s;
  s.order = reinterpret_cast<int32_t*>(w);
  w += up256((size_t)T * 4);
  s.sid = reinterpret_cast<int32_t*>(w);
  w += up256((size_t)T * 4);
  s.n = reinterpret_cast<int32_t*>(w);
  w += 256;
  s.part = reinterpret_cast<float*>(w);
  return s;
}

// The sorting threads of a CTA wait for each other.
__device__ __forceinline__ void sort_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSortThreads) : "memory"); }

// Exclusive sum of v over the sorting threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += u;
  }
  sort_sync();  // the previous call's sums have been read
  if (lane == 31) warp_sums[w] = incl;
  sort_sync();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kSortThreads / 32; ++i) {
    const int u = warp_sums[i];
    if (i < w) before += u;
    all += u;
  }
  *total = all;
  return before + incl - v;
}

// A thread's 32 consecutive tokens of a batch, a few at a time: calls f(j, id)
// for each, with id -1 past the end (16-byte loads where `ids` allows them).
// Eight at a time keep the kernel within 32 registers and its code short: T =
// 7312, d = 128: the call 18.9 us, 19.8 with all 32 at once.
template <typename F>
__device__ __forceinline__ void each_token(const int32_t* ids, int t, int T, bool aligned, F f) {
#pragma unroll 1
  for (int j0 = 0; j0 < kSortEach; j0 += kSortStep) {
    int id[kSortStep];
    if (aligned && t + j0 + kSortStep <= T) {
      const int4* v = reinterpret_cast<const int4*>(ids + t + j0);
#pragma unroll
      for (int j = 0; j < kSortStep; j += 4) {
        const int4 k = __ldg(v + j / 4);
        id[j] = k.x, id[j + 1] = k.y, id[j + 2] = k.z, id[j + 3] = k.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kSortStep; ++j) id[j] = t + j0 + j < T ? __ldg(ids + t + j0 + j) : -1;
    }
#pragma unroll
    for (int j = 0; j < kSortStep; ++j) f(j0 + j, id[j]);
  }
}

// Each CTA sorts the tokens of its own range of ids [v0, v1): it reads all T
// ids (a few tens of KB, from L2), counts the valid ones below its range (its
// base in the order) and those of each of its ids, then collects its tokens
// in token order and places them.  The CTA's upper threads clear the range's
// rows of the gradient meanwhile: that write is most of the traffic and needs
// nothing of the sort (the rows with tokens are written again by the sum).
// T = 8192, V = 50304, d = 2048: 36 us, of which the clearing of 206 MB takes 32
// and hides the sort (16 us alone).  Clearing only the rows without a token, half
// here and half beside the sum, was slower (55 to 62 us for the whole against 50, then).
// Every CTA reads all ids, twice beyond one batch of 16384: past some 100 K tokens
// that is the call (d = 64: 131072 tokens 0.19 ms, a million 1.5 ms).
__global__ void __launch_bounds__(2 * kSortThreads)
    embedding_sort_kernel(const int32_t* ids, int T, int V, int per, int warps, int nv, SortWs S, uint4* dtable,
                          int zero, int* status) {
  extern __shared__ int sm[];
  int* next = sm;                // [per] next place of each id
  int* place = sm + per;         // [warps][per]
  uint16_t* pos = reinterpret_cast<uint16_t*>(place + warps * per);  // [kSortBatch] token of the batch
  uint16_t* pid = pos + kSortBatch;                                  // [kSortBatch] id of the range
  __shared__ int warp_sums[kSortThreads / 32];
  __shared__ int base_s, any_bad;
  dependency_wait();
  const int v0 = blockIdx.x * per, n_ids = min(per, V - v0);
  if (threadIdx.x >= kSortThreads) {
    if (!zero) return;
    uint4* rows = dtable + (long long)v0 * nv;
    const int n = n_ids * nv;
    for (int i = threadIdx.x - kSortThreads; i < n; i += kSortThreads) rows[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const bool aligned = (reinterpret_cast<uintptr_t>(ids) & 15u) == 0;
  for (int i = tid; i < per; i += kSortThreads) next[i] = 0;
  if (tid == 0) base_s = any_bad = 0;
  sort_sync();
  int below = 0;
  bool bad = false;
  unsigned mask = 0;  // this thread's tokens of the range, in the last batch
  for (int t0 = 0; t0 < T; t0 += kSortBatch) {
    mask = 0;
    each_token(ids, t0 + kSortEach * tid, T, aligned, [&](int j, int id) {
      below += id >= 0 && id < v0;
      bad |= id >= V;
      const unsigned k = (unsigned)id - (unsigned)v0;
      if (k < (unsigned)n_ids) {
        atomicAdd(&next[k], 1);
        mask |= 1u << j;
      }
    });
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) below += __shfl_xor_sync(0xffffffffu, below, s);
  if (lane == 0 && below) atomicAdd(&base_s, below);
  if (bad) any_bad = 1;
  sort_sync();
  if (blockIdx.x == 0 && tid == 0 && any_bad) record_status(status, MOE_ERR_DEVICE_BOUNDS);
  // counts -> first places
  int run = base_s;
  for (int i0 = 0; i0 < per; i0 += kSortThreads) {
    const int i = i0 + tid;
    const int c = i < per ? next[i] : 0;
    int total;
    const int at = run + block_scan(c, warp_sums, &total);
    if (i < per) next[i] = at;
    run += total;
  }
  if (tid == 0 && v0 + n_ids == V) *S.n = run;
  if (run == base_s) return;  // no token of the batch is in this range
  for (int t0 = 0; t0 < T; t0 += kSortBatch) {
    const int t = t0 + kSortEach * tid;
    if (T > kSortBatch) {  // more than one batch: the masks again
      mask = 0;
      each_token(ids, t, T, aligned, [&](int j, int id) {
        if ((unsigned)id - (unsigned)v0 < (unsigned)n_ids) mask |= 1u << j;
      });
    }
    // the batch's tokens of this range, in token order
    for (int i = tid; i < warps * per; i += kSortThreads) place[i] = 0;
    int held;
    int at = block_scan(__popc(mask), warp_sums, &held);
    for (unsigned m = mask; m; m &= m - 1u, ++at) {
      const int j = __ffs(m) - 1;
      pos[at] = (uint16_t)(kSortEach * tid + j);
      pid[at] = (uint16_t)(__ldg(ids + t + j) - v0);
    }
    sort_sync();
    if (held == 0) continue;
    // Place them, stable: each placing warp takes a run of the list, counts its
    // run's ids, starts after the runs before it, and places its run in order,
    // 32 tokens at a time (equal ids of one step take consecutive places).  One
    // warp alone took 25 us for the 3900 tokens that the most frequent ids of a
    // Zipf-like batch of 8192 bring to one CTA.
    const int r0 = held * w / warps, r1 = held * (w + 1) / warps;
    int* mine = place + w * per;
    if (w < warps)
      for (int i = r0 + lane; i < r1; i += 32) atomicAdd(&mine[pid[i]], 1);
    sort_sync();
    for (int i = tid; i < n_ids; i += kSortThreads) {
      int to = next[i];
      for (int u = 0; u < warps; ++u) {
        const int c = place[u * per + i];
        place[u * per + i] = to;
        to += c;
      }
      next[i] = to;
    }
    sort_sync();
    if (w < warps) {
      for (int i0 = r0; i0 < r1; i0 += 32) {
        const int i = i0 + lane;
        const int id = i < r1 ? pid[i] : -1 - lane;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        if (i < r1) {
          const int to = mine[id] + __popc(same & ((1u << lane) - 1u));
          S.order[to] = t0 + pos[i];
          S.sid[to] = v0 + id;
        }
        __syncwarp();
        if (i < r1 && lane == 31 - __clz(same)) mine[id] += __popc(same);
        __syncwarp();
      }
    }
    sort_sync();
  }
}

__device__ __forceinline__ void put_row(uint4* dtable, long long at, const float (&acc)[8], float scale, bool add) {
  float f[8];
  if (add) unpack8(dtable[at], f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = add ? fmaf(scale, acc[e], f[e]) : scale * acc[e];
  dtable[at] = pack8(f);
}

// Sorted rows [chunk c, + chunk) of one slab of columns.  Each thread copies its
// own 16 bytes of the next kAhead rows into shared memory and adds them as they
// land; the loop's code stays short (rows in registers need it once for each).
// Bound by the latency of a few dependent loads.  The whole call, T = 8192, d =
// 2048: 48.8 us; 16 rows ahead 49.2; 8 / 16 / 32 rows in registers 50.6 / 53.2 /
// 54.9.  T = 16384, d = 4096: 169.4; 170.2; 168.7 / 172 / 179.
__global__ void __launch_bounds__(kSumThreads)
    embedding_sum_kernel(const uint4* dout, int T, int nv, int chunk, SortWs S, float scale, int add,
                         uint4* dtable) {
  __shared__ uint4 ring[kAhead][kSumThreads];  // each thread its own column: no barrier
  __shared__ int tok[kChunkMax], id[kChunkMax + 2];
  static_assert(kChunkMax + 2 <= kSumThreads, "one thread per position");
  dependency_wait();
  const int i0 = blockIdx.x * chunk, i = threadIdx.x;
  // the count and the chunk's positions are read at once (entries past the
  // count hold nothing and are not used); id[] has the neighbours on both sides
  const int n = *S.n, at = i0 + i - 1;
  const bool in = i < chunk + 2 && at >= 0 && at < T;
  const int my_id = in ? S.sid[at] : -1, my_tok = in ? S.order[at] : 0;
  const int m = min(chunk, n - i0);
  if (m <= 0) return;
  if (i < m + 2) id[i] = at < n ? my_id : -1;
  if (i >= 1 && i <= m) tok[i - 1] = my_tok;
  __syncthreads();
  const int v = blockIdx.y * kSumThreads + threadIdx.x;
  if (v >= nv) return;
  float* part = S.part + (long long)blockIdx.x * 2 * nv * 8;
  const uint4* src = dout + v;
  const uint32_t slot0 = ptx::smem_u32(&ring[0][threadIdx.x]);
  // row j into its slot, whose last row this thread has read; an empty group past
  // the end
  auto fetch = [&](int j) {
    if (j < m)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot0 + (j % kAhead) * (kSumThreads * 16)),
                   "l"(src + (long long)tok[j] * nv)
                   : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int j = 0; j < kAhead; ++j) fetch(j);
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  bool began_before = id[0] == id[1];
#pragma unroll 1
  for (int b = 0; b < m; ++b) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    float f[8];
    unpack8(ring[b % kAhead][threadIdx.x], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += f[e];
    fetch(b + kAhead);
    const bool goes_on = id[b + 2] == id[b + 1];
    if (goes_on && b + 1 < m) continue;
    if (began_before || goes_on) {
      float4* p = reinterpret_cast<float4*>(part + (began_before ? 0 : nv * 8)) + 2 * v;
      p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
      put_row(dtable, (long long)id[b + 1] * nv + v, acc, scale, add);
    }
    began_before = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  }
}

// Rows that span chunks: the CTA of the chunk where a row begins adds the
// partials of the chunks it covers, a quarter of them per group of threads in
// chunk order, then the quarters in order.  4 us for the hot rows of a Zipf-like
// batch of 8192 (700 tokens of one id: 22 chunks); with the loop over the chunks
// unrolled by 8 instead of 2, for more loads in flight, 2 us more.
__global__ void __launch_bounds__(kSumThreads* kJoinGroups)
    embedding_join_kernel(int T, int nv, int chunk, SortWs S, float scale, int add, uint4* dtable) {
  __shared__ float4 quarter[kJoinGroups - 1][2][kSumThreads];
  dependency_wait();
  // the count and the ids around the chunk's end and start at once (entries
  // past the count hold nothing and are not used)
  const int c = blockIdx.x, last = (c + 1) * chunk - 1;
  if (last + 1 >= T) return;
  const int n = *S.n, id = S.sid[last], next = S.sid[last + 1], before = c > 0 ? S.sid[c * chunk - 1] : -1;
  if (last + 1 >= n || next != id) return;  // no row crosses this boundary
  if (c > 0 && before == id) return;        // it began in an earlier chunk
  // the chunks it covers: those whose first row is its own, counted a CTA's
  // width at a time
  int covers = 1;
  for (int j0 = c + 1;; j0 += kSumThreads * kJoinGroups) {
    const long long at = (long long)(j0 + threadIdx.x) * chunk;
    const int more = __syncthreads_count(at < n && S.sid[at] == id);
    covers += more;
    if (more < kSumThreads * kJoinGroups) break;
  }
  const int g = threadIdx.x / kSumThreads, lt = threadIdx.x % kSumThreads, v = blockIdx.y * kSumThreads + lt;
  const int j0 = covers * g / kJoinGroups, j1 = covers * (g + 1) / kJoinGroups;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  if (v < nv) {
#pragma unroll 2
    for (int j = j0; j < j1; ++j) {
      const float4* p = reinterpret_cast<const float4*>(S.part + ((long long)(c + j) * 2 + (j == 0)) * nv * 8) + 2 * v;
      const float4 a = __ldg(p), b = __ldg(p + 1);
      acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
      acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
    }
  }
  if (g > 0) {
    quarter[g - 1][0][lt] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    quarter[g - 1][1][lt] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  __syncthreads();
  if (g > 0 || v >= nv) return;
#pragma unroll
  for (int q = 0; q < kJoinGroups - 1; ++q) {
    const float4 a = quarter[q][0][lt], b = quarter[q][1][lt];
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
    acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
  }
  put_row(dtable, (long long)id * nv + v, acc, scale, add);
}

}  // namespace

size_t embedding_ws_bytes(int T, int d) {
  return 2 * up256((size_t)T * 4) + 256 + up256((size_t)chunks_of(T, d / 8) * 2 * d * 4);
}

// Chunks of 8 need more partials than the chunks of 32 that follow them: the
// most is at the longest batch that still has them (d = 2048: 2400 tokens 4.9
// MB, 2401 tokens 1.3 MB).
size_t embedding_ws_bytes_up_to(int T, int d) {
  const int nv = d / 8;
  const int short_ones = (kFullCtas - 1) / ((nv + kSumThreads - 1) / kSumThreads) * kChunkMax;  // chunk_of: 8 up to here
  const int last = T < short_ones ? T : short_ones;
  int chunks = chunks_of(T, nv);
  if (last > 0 && chunks_of(last, nv) > chunks) chunks = chunks_of(last, nv);
  return 2 * up256((size_t)T * 4) + 256 + up256((size_t)chunks * 2 * d * 4);
}

cudaError_t launch_embedding(const void* table, const int32_t* ids, int T, int V, int d, float scale, void* out,
                             int* status, cudaStream_t s) {
  const unsigned nv = d / 8;
  const long long per_launch = (1LL << 30) / nv;  // tokens
  for (long long t0 = 0; t0 < T; t0 += per_launch) {
    const long long n = T - t0 < per_launch ? T - t0 : per_launch;
    const unsigned total = (unsigned)(n * nv);
    timing_mark(s, "embedding");
    cudaError_t e = launch_pdl(embedding_kernel, dim3((total + kFwdThreads * kFwdVecs - 1) / (kFwdThreads * kFwdVecs)),
                               dim3(kFwdThreads), 0, s, static_cast<const uint4*>(table), ids + t0, total, nv, V,
                               scale, static_cast<uint4*>(out) + t0 * nv, status);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_embedding_bwd(const void* dout, const int32_t* ids, int T, int V, int d, float scale,
                                 bool accumulate, void* dtable, void* ws, int* status, cudaStream_t s) {
  const SortWs S = carve(ws, T);
  const int nv = d / 8, sms = device_sm_count();
  int ctas = 2 * sms;
  if (ctas > V) ctas = V;
  int per = (V + ctas - 1) / ctas;
  if (per > kSortMaxIds) per = kSortMaxIds;
  ctas = (V + per - 1) / per;
  int warps = kSortPlaces / per;
  if (warps > kSortThreads / 32) warps = kSortThreads / 32;
  const size_t smem = (size_t)(per + warps * per) * 4 + kSortBatch * 2 * sizeof(uint16_t);
  static std::atomic<unsigned long long> devices{0};
  cudaError_t e = allow_smem(embedding_sort_kernel, devices, (kSortMaxIds + kSortPlaces) * 4 + kSortBatch * 2 * (int)sizeof(uint16_t));
  if (e != cudaSuccess) return e;
  uint4* out = static_cast<uint4*>(dtable);
  timing_mark(s, "embedding_sort");
  e = launch_pdl(embedding_sort_kernel, dim3(ctas), dim3(2 * kSortThreads), smem, s, ids, T, V, per, warps, nv, S,
                 out, accumulate ? 0 : 1, status);
  if (e != cudaSuccess) return e;
  const int chunk = chunk_of(T, nv);
  const dim3 grid(chunks_of(T, nv), (nv + kSumThreads - 1) / kSumThreads);
  timing_mark(s, "embedding_sum");
  e = launch_pdl(embedding_sum_kernel, grid, dim3(kSumThreads), 0, s, static_cast<const uint4*>(dout), T, nv, chunk, S, scale,
                 accumulate ? 1 : 0, out);
  if (e != cudaSuccess) return e;
  if (T <= chunk) return cudaSuccess;
  timing_mark(s, "embedding_join");
  return launch_pdl(embedding_join_kernel, grid, dim3(kSumThreads * kJoinGroups), 0, s, T, nv, chunk, S, scale, accumulate ? 1 : 0, out);
}

}  // namespace moe
