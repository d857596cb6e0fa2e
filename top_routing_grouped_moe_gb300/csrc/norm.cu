// Residual update of a block with the norms on both sides of it:
//   n  = o rstd_post w_post   (or o),   rstd_post = 1 / sqrt(mean(o^2) + eps)
//   r' = r + alpha gate n
//   x  = r' rstd_pre w_pre,             rstd_pre  = 1 / sqrt(mean(r'^2) + eps)
// and its backward.  Every value is fp32 from the load to the one rounding at
// the store; a row stays in registers between its two reductions, so each
// tensor is read once and written once.
#include "common.cuh"
#include "ptx.cuh"
#include "step.h"

namespace moe {
namespace {

// A row of d values is nv = d / 8 vectors of 8; the row's threads (NT) hold
// vectors tid, tid + NT, ... (VPT of them).

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// Sum over the row's threads, the same value (and bits) in all of them.  One
// warp per row: shuffles.  A CTA per row: the warps' sums meet in `slots`.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* slots) {
  v = warp_sum(v);
  if (WARP_ROW) return v;
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  return warp_sum(lane < nw ? slots[lane] : 0.0f);
}

template <bool F32>
struct RowIo {  // residual stream in bf16 (plain loads: a gradient or the stream may be updated in place)
  __device__ static void load(const void* p, long long vec, float (&f)[8]) {
    unpack8(reinterpret_cast<const uint4*>(p)[vec], f);
  }
  __device__ static void store(void* p, long long vec, const float (&f)[8]) {
    reinterpret_cast<uint4*>(p)[vec] = pack8(f);
  }
};
template <>
struct RowIo<true> {  // ... in fp32
  __device__ static void load(const void* p, long long vec, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[2 * vec];
    const float4 b = reinterpret_cast<const float4*>(p)[2 * vec + 1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ static void store(void* p, long long vec, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[2 * vec] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[2 * vec + 1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
using Bf16Io = RowIo<false>;

// Forward.  Bound by HBM: r and o in, r' and x out, and a CTA per row (a warp
// for d <= 512, eight rows per CTA) has all of it in flight at once; with 256 to
// 1024 threads per row and 32 registers the SM is full of rows at different
// stages.  T = 8192, d = 4096, fp32 stream: 62 us, 6.5 TB/s (0.96 of the copy
// rate); a single token is a launch.
template <int VPT, bool RF32, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 256 : 1024) residual_norm_kernel(const NormArgs A) {
  __shared__ float slots[2][32];
  dependency_wait();
  const int nt = WARP_ROW ? 32 : blockDim.x;
  const int tid = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
  const long long t = WARP_ROW ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP_ROW && t >= A.T) return;
  const int nv = A.d >> 3;
  const long long row = t * nv;
  const float inv_d = 1.0f / (float)A.d;

  float r[VPT][8];
  float o[VPT][8];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + j * nt;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[j][e] = o[j][e] = 0.0f;
    if (v >= nv) continue;
    if (A.o) Bf16Io::load(A.o, row + v, o[j]);
    if (A.r) RowIo<RF32>::load(A.r, row + v, r[j]);
  }
  float scale = A.alpha;
  if (A.gate_kind == MOE_GATE_TOKEN) scale *= __ldg(A.gate + t);
  if (A.o) {
    if (A.w_post) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(o[j][e], o[j][e], ss);
      const float rstd = __frsqrt_rn(row_sum<WARP_ROW>(ss, slots[0]) * inv_d + A.eps);
      if (A.rstd_post && tid == 0) A.rstd_post[t] = rstd;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * nt;
        if (v >= nv) continue;
        float w[8];
        Bf16Io::load(A.w_post, v, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[j][e] *= rstd * w[e];
      }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = tid + j * nt;
      if (A.gate_kind == MOE_GATE_CHANNEL && v < nv) {
        float g[8];
        RowIo<true>::load(A.gate, v, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[j][e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] = fmaf(scale, o[j][e], r[j][e]);
    }
  }
  if (A.r_out) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (tid + j * nt < nv) RowIo<RF32>::store(A.r_out, row + tid + j * nt, r[j]);
  }
  if (!A.x) return;
  ss = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(r[j][e], r[j][e], ss);
  const float rstd = __frsqrt_rn(row_sum<WARP_ROW>(ss, slots[1]) * inv_d + A.eps);
  if (A.rstd_pre && tid == 0) A.rstd_pre[t] = rstd;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + j * nt;
    if (v >= nv) continue;
    float w[8];
    Bf16Io::load(A.w_pre, v, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= r[j][e] * rstd;
    Bf16Io::store(A.x, row + v, w);
  }
}

// Two fp32 values in a register pair, for the packed fp32 instructions: the
// backward is bound by instruction issue before it is by HBM when each value
// takes its own.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 both(float v) { return pack2(v, v); }
__device__ __forceinline__ float2 split2(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(F2 v) {
  const float2 f = split2(v);
  return f.x + f.y;
}

template <bool F32>
__device__ __forceinline__ void load2(const void* p, long long vec, F2 (&f)[4]) {
  float v[8];
  RowIo<F32>::load(p, vec, v);
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = pack2(v[2 * e], v[2 * e + 1]);
}
template <bool F32>
__device__ __forceinline__ void store2(void* p, long long vec, const F2 (&f)[4]) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 u = split2(f[e]);
    v[2 * e] = u.x;
    v[2 * e + 1] = u.y;
  }
  RowIo<F32>::store(p, vec, v);
}

// Backward.  With x^ = r' rstd_pre and o^ = o rstd_post:
//   G  = dr_out + rstd_pre (dx w_pre - x^ mean(dx w_pre x^))      -> dr
//   dn = alpha gate G;  dgate = alpha G n (summed over the row or the tokens)
//   do = rstd_post (dn w_post - o^ mean(dn w_post o^))            (or dn)
//   dw_pre = sum_t dx x^;  dw_post = sum_t dn o^
// What the kernel computes, with b = dr_out + rstd_pre dx w_pre, v = w_post
// gate[c] (per channel) and s_t = alpha gate[t] rstd_post (per row):
//   M = sum rstd_pre dx w_pre r',  E1 = sum o v b,  E2 = sum o v r'
// one reduction of three values per row, since G = b - k r' with k =
// rstd_pre^2 M / d is linear in M: sum o v G = E1 - k E2.  Then
//   do = s_t v G - o s_t rstd_post^2 (E1 - k E2) / d,
// and the gradients per channel come from one more column sum besides
// dw_pre's: Q = sum_t s_t G o;  dw_post = gate[c] Q, dgate[c] = w_post Q.
//
// Bound by HBM (four rows in, two out), and next by instruction issue.  A CTA
// walks groups of `rows` consecutive token rows, blockIdx.x, + gridDim.x, ...;
// a group's inputs are contiguous and come by bulk copies into a ring in shared
// memory, several groups ahead, so that the row's latency chain (load, reduce,
// store) does not hold back the reads.  A group's barrier says that the stage of
// the group before it has been read; one lane then fills that stage again, of
// another warp each time, as the copies' issue would make one warp late at every
// barrier.  A row has `lanes` threads (whole warps), one vector of 8 channels
// each (VPT = 2: two).  Each thread keeps its channels' column sums in
// registers; its CTA leaves them, the rows of a group added, in
// part[CTA][2][d], which a second kernel adds in order (deterministic).
// T = 16384, d = 2048, bf16: 67.5 us with the columns, 6.0 TB/s (0.88 of the copy
// rate); with an fp32 stream, half as many instructions per byte, 0.95.
constexpr int kBwdThreads = 512;
struct BwdPlan {
  int rows;    // token rows of a group
  int lanes;   // threads of a row
  int stages;  // groups in flight
  int per_sm;  // CTAs of an SM
};

template <bool RF32>
struct BwdStage {  // one group's inputs: dx | o | dr_out | r_out
  static constexpr int RB = RF32 ? 4 : 2;
  __host__ __device__ static int bytes(int rows, int d) { return rows * d * (4 + 2 * RB); }
};

// The CTA's barrier, and whether any of its threads failed.
__device__ __forceinline__ bool cta_failed(bool failed) { return __syncthreads_or(failed) != 0; }

// FULL: dx, dr_out, o and dr are all given (the step between two blocks).
template <int VPT, bool RF32, bool FULL>
__global__ void __launch_bounds__(kBwdThreads, 1) residual_norm_bwd_kernel(const NormBwdArgs A, const BwdPlan L) {
  constexpr int RB = BwdStage<RF32>::RB;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[8];
  __shared__ float slots[2][4][kBwdThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int row_warps = L.lanes >> 5, warps = blockDim.x >> 5;
  const int nv = A.d >> 3, d = A.d;
  const int stage_bytes = BwdStage<RF32>::bytes(L.rows, d), unit = L.rows * d;
  const int groups = (A.T + L.rows - 1) / L.rows;
  const bool has_dx = FULL || A.dx, has_o = FULL || A.o, has_up = FULL || A.dr_out;
  if (tid == 0) {
    for (int s = 0; s < L.stages; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbarrier_init();
  }
  dependency_wait();
  __syncthreads();

  // the bulk copies of group g into stage s
  auto fetch = [&](int g, int s) {
    if (g >= groups) return;
    const long long at = (long long)g * unit;  // first element
    const unsigned n = (unsigned)min((long long)unit, (long long)A.T * d - at);
    uint8_t* dst = ring + s * stage_bytes;
    uint64_t* bar = &full[s];
    ptx::mbar_arrive_expect_tx(bar, (has_dx ? n * (2 + RB) : 0u) + (has_o ? n * 2 : 0u) + (has_up ? n * RB : 0u));
    if (has_dx) {
      ptx::bulk_load(dst, static_cast<const uint8_t*>(A.dx) + at * 2, n * 2, bar);
      ptx::bulk_load(dst + unit * (4 + RB), static_cast<const uint8_t*>(A.r_out) + at * RB, n * RB, bar);
    }
    if (has_o) ptx::bulk_load(dst + unit * 2, static_cast<const uint8_t*>(A.o) + at * 2, n * 2, bar);
    if (has_up) ptx::bulk_load(dst + unit * 4, static_cast<const uint8_t*>(A.dr_out) + at * RB, n * RB, bar);
  };
  if (tid == 0)
    for (int q = 0; q < L.stages - 1; ++q) fetch(blockIdx.x + q * gridDim.x, q);

  F2 s_pre[VPT][4], s_q[VPT][4];
  const int sub = tid / L.lanes, lt = tid - sub * L.lanes;  // row of the group, thread of the row
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s_pre[j][e] = s_q[j][e] = 0;
  {
    const float inv_d = 1.0f / (float)d;
    F2 wp[VPT][4], wv[VPT][4];  // w_pre, v
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lt + j * L.lanes;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        wp[j][e] = 0;
        wv[j][e] = both(1.0f);
      }
      if (v >= nv) continue;
      if (has_dx) load2<false>(A.w_pre, v, wp[j]);
      if (A.w_post) load2<false>(A.w_post, v, wv[j]);
      if (A.gate_kind == MOE_GATE_CHANNEL) {
        F2 g[4];
        load2<true>(A.gate, v, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) wv[j][e] = mul2(wv[j][e], g[e]);
      }
    }
    // per-row scalars, read one row ahead (1, 1 and 0 where absent)
    const float* p_pre = has_dx ? A.rstd_pre : nullptr;
    const float* p_post = A.w_post ? A.rstd_post : nullptr;
    const float* p_gate = A.gate_kind == MOE_GATE_TOKEN ? A.gate : nullptr;
    const int t_step = gridDim.x * L.rows;
    int t = blockIdx.x * L.rows + sub;
    float rstd_n = 0.0f, ro_n = 1.0f, scale_n = 1.0f;
    if (t < A.T) {
      if (p_pre) rstd_n = __ldg(p_pre + t);
      if (p_post) ro_n = __ldg(p_post + t);
      if (p_gate) scale_n = __ldg(p_gate + t);
    }
    int stage = 0, last = L.stages - 1, par = 0, turn = 0;
    uint32_t phase = 0;
    volatile int never = 0;
    for (int g = blockIdx.x; g < groups; g += gridDim.x) {
      const bool live = t < A.T;
      const float rstd = rstd_n, ro = ro_n, scale = A.alpha * scale_n;
      const int tn = t + t_step;
      if (tn < A.T && g + (int)gridDim.x < groups) {
        if (p_pre) rstd_n = __ldg(p_pre + tn);
        if (p_post) ro_n = __ldg(p_post + tn);
        if (p_gate) scale_n = __ldg(p_gate + tn);
      }
      const bool failed = !ptx::mbar_wait_bounded(&full[stage], phase, &never, kWaitLimitNs);
      const uint8_t* st = ring + stage * stage_bytes;
      F2 b[VPT][4], r[VPT][4], o[VPT][4];
      F2 m2 = 0, e12 = 0, e22 = 0;
      const F2 rstd2 = both(rstd);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = lt + j * L.lanes;
        if (v >= nv || !live) {
#pragma unroll
          for (int e = 0; e < 4; ++e) b[j][e] = r[j][e] = o[j][e] = 0;
          continue;
        }
        const int at = sub * nv + v;
        if (!FULL)
#pragma unroll
          for (int e = 0; e < 4; ++e) b[j][e] = r[j][e] = o[j][e] = 0;
        if (has_up) load2<RF32>(st + unit * 4, at, b[j]);
        if (has_o) load2<false>(st + unit * 2, at, o[j]);
        if (has_dx) {
          F2 a[4];
          load2<RF32>(st + unit * (4 + RB), at, r[j]);
          load2<false>(st, at, a);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = mul2(a[e], rstd2);
            s_pre[j][e] = fma2(a[e], r[j][e], s_pre[j][e]);
            b[j][e] = fma2(a[e], wp[j][e], b[j][e]);
            m2 = fma2(mul2(a[e], wp[j][e]), r[j][e], m2);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const F2 n = mul2(o[j][e], wv[j][e]);
          e12 = fma2(n, b[j][e], e12);
          e22 = fma2(n, r[j][e], e22);
        }
      }
      // the three sums over the warp: halves of the lanes take over one value
      // of a pair at a time, so that six shuffles do the work of fifteen
      const float m0 = sum2(m2), e10 = sum2(e12), e20 = sum2(e22);
      const bool hi = lane & 16, hi2 = lane & 8;
      const float u = (hi ? e10 : m0) + __shfl_xor_sync(0xffffffffu, hi ? m0 : e10, 16);
      const float w = e20 + __shfl_xor_sync(0xffffffffu, e20, 16);
      float x = (hi2 ? w : u) + __shfl_xor_sync(0xffffffffu, hi2 ? u : w, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      // lanes 0..7: M, 16..23: E1, 8..15 and 24..31: E2
      if ((lane & 7) == 0) slots[par][lane >> 3][tid >> 5] = x;
      if (cta_failed(failed)) {
        if (tid == 0) {
          record_status(A.status, MOE_ERR_TIMEOUT);
          // the copies in flight land before the CTA's shared memory goes away
          for (int q = 0; q < L.stages; ++q) ptx::mbar_wait_bounded(&full[q], q < stage ? phase ^ 1u : phase, &never, 100000000ull);
        }
        break;
      }
      if (turn == (tid >> 5) && lane == 0) {
        ptx::fence_proxy_async_smem();
        fetch(g + (L.stages - 1) * (int)gridDim.x, last);
      }
      if (++turn == warps) turn = 0;
      last = stage;
      if (++stage == L.stages) {
        stage = 0;
        phase ^= 1u;
      }
      if (row_warps > 1) {
        const int k = lane & 7;  // each eighth of the lanes adds one value over the row's warps
        const float* sl = slots[par][lane >> 3] + sub * row_warps;
        x = k < row_warps ? sl[k] : 0.0f;
        if (k + 8 < row_warps) x += sl[k + 8];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        x += __shfl_xor_sync(0xffffffffu, x, 1);
      }
      par ^= 1;
      const float M = __shfl_sync(0xffffffffu, x, 0), E1 = __shfl_sync(0xffffffffu, x, 16),
                  E2 = __shfl_sync(0xffffffffu, x, 8);
      if (live) {
        const float k = rstd * rstd * M * inv_d;  // M = sum rstd dx w_pre r'
        const float og = E1 - k * E2;             // sum o v G
        if (p_gate && A.dgate && lt == 0) A.dgate[t] = A.alpha * ro * og;
        const F2 st2 = both(scale * ro), k2 = both(-k);
        const F2 c2 = both(p_post ? -scale * ro * ro * ro * og * inv_d : 0.0f);
        const long long row = (long long)t * nv;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int v = lt + j * L.lanes;
          if (v >= nv) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) b[j][e] = fma2(k2, r[j][e], b[j][e]);  // G
          if (FULL || A.dr) store2<RF32>(A.dr, row + v, b[j]);
          if (!has_o) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const F2 y = mul2(st2, b[j][e]);
            s_q[j][e] = fma2(y, o[j][e], s_q[j][e]);
            b[j][e] = fma2(y, wv[j][e], mul2(c2, o[j][e]));
          }
          store2<false>(A.d_o, row + v, b[j]);
        }
      }
      t = tn;
    }
  }
  // the rows' sums meet in shared memory: every copy has landed and been read
  float* part = A.part + (long long)blockIdx.x * 2 * d;
  if (L.rows > 1) {
    __syncthreads();
    float* meet = reinterpret_cast<float*>(ring);  // [rows][2][d]
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = lt + j * L.lanes;
      if (v >= nv) continue;
      store2<true>(meet + (2 * sub) * d, v, s_pre[j]);
      store2<true>(meet + (2 * sub + 1) * d, v, s_q[j]);
    }
    __syncthreads();
    for (int c = tid; c < 2 * d; c += blockDim.x) {
      float v = meet[c];
      for (int k = 1; k < L.rows; ++k) v += meet[2 * k * d + c];
      part[c] = v;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = lt + j * L.lanes;
    if (v >= nv) continue;
    store2<true>(part, v, s_pre[j]);
    store2<true>(part + d, v, s_q[j]);
  }
}

constexpr int kColumnWarps = 32;

// The column sums: 32 columns per CTA, each of its warps adds every
// kColumnWarps-th partial, then the warps' sums are added in order (8 warps: 2 us
// more for 304 partials).  blockIdx.y = 0: dw_pre; 1: Q, of which dw_post =
// gate Q and dgate = w_post Q (a gate per channel).  304 partials of 2 d values
// (5 MB at d = 2048), bound by latency: 4 us.
__global__ void __launch_bounds__(32 * kColumnWarps)
    norm_bwd_columns_kernel(const float* part, int parts, int d, const float* gate, const __nv_bfloat16* w_post,
                            float* dw_pre, float* dw_post, float* dgate) {
  __shared__ float sums[kColumnWarps][32];
  dependency_wait();
  const bool q = blockIdx.y == 1;
  if (q ? !dw_post && !dgate : !dw_pre) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // d is a multiple of 64
  const float g = q && w == 0 && gate ? gate[c] : 1.0f;  // on their way meanwhile
  const float wp = q && w == 0 && w_post ? __bfloat162float(w_post[c]) : 1.0f;
  float v = 0.0f;
#pragma unroll 4
  for (int i = w; i < parts; i += kColumnWarps) v += __ldg(part + ((long long)i * 2 + blockIdx.y) * d + c);
  sums[w][lane] = v;
  __syncthreads();
  if (w) return;
#pragma unroll
  for (int i = 1; i < kColumnWarps; ++i) v += sums[i][lane];
  if (!q) {
    dw_pre[c] = v;
    return;
  }
  if (dw_post) dw_post[c] = g * v;
  if (dgate) dgate[c] = wp * v;
}

int round_warp(int n) { return (n + 31) / 32 * 32; }

template <bool RF32>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  const int nv = a.d / 8;
  if (nv <= 64) {  // a warp per row, eight rows per CTA
    const dim3 grid((a.T + 7) / 8);
    return nv <= 32 ? launch_pdl(residual_norm_kernel<1, RF32, true>, grid, dim3(256), 0, s, a)
                    : launch_pdl(residual_norm_kernel<2, RF32, true>, grid, dim3(256), 0, s, a);
  }
  const dim3 grid(a.T);
  return launch_pdl(residual_norm_kernel<1, RF32, false>, grid, dim3(round_warp(nv)), 0, s, a);
}

// Backward: a row's threads are whole warps, one vector per thread up to 4096
// channels, two above.  A CTA takes as many rows as fit 256 threads (at least
// one), an SM as many CTAs as fit kBwdThreads, which share its shared memory for
// their rings: while one waits at its barrier another computes.  T = 16384, d =
// 2048: two CTAs of 256 threads 67 us, one of 512 70, three 76, four 90
// (registers); T = 16384, d = 1280: three of 160 47, one of 480 49, two 55.  Two
// vectors per thread spill 84 to 132 bytes (128 registers): T = 8192, d = 8192:
// 173 us, 0.69 of the copy rate (fp32 stream 243, 0.73), d = 4096: 70, 0.85.
BwdPlan plan_of(int d, bool r_f32) {
  BwdPlan L;
  const int nv = d / 8;
  L.lanes = d <= 4096 ? round_warp(nv) : round_warp((nv + 1) / 2);
  L.rows = L.lanes < kBwdThreads / 2 ? kBwdThreads / 2 / L.lanes : 1;
  L.per_sm = kBwdThreads / (L.rows * L.lanes);
  const int stage = r_f32 ? BwdStage<true>::bytes(L.rows, d) : BwdStage<false>::bytes(L.rows, d);
  const int room = 220 * 1024 / L.per_sm / stage;
  L.stages = room < 8 ? room : 8;
  return L;
}
int bwd_ctas(int T, int d) {
  const BwdPlan L = plan_of(d, false);
  const int groups = (T + L.rows - 1) / L.rows, most = L.per_sm * kNormSms;
  return groups < most ? groups : most;
}

template <int VPT, bool RF32, bool FULL>
cudaError_t bwd_as(const NormBwdArgs& a, const BwdPlan& L, int ctas, cudaStream_t s) {
  const size_t smem = (size_t)L.stages * BwdStage<RF32>::bytes(L.rows, a.d);
  auto kern = residual_norm_bwd_kernel<VPT, RF32, FULL>;
  static std::atomic<unsigned long long> devices{0};
  const cudaError_t e = allow_smem(kern, devices, 220 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(L.rows * L.lanes), smem, s, a, L);
}
template <int VPT>
cudaError_t bwd(const NormBwdArgs& a, bool r_f32, const BwdPlan& L, int ctas, cudaStream_t s) {
  const bool full = a.dx && a.dr_out && a.o && a.dr;
  if (r_f32)
    return full ? bwd_as<VPT, true, true>(a, L, ctas, s)
                : bwd_as<VPT, true, false>(a, L, ctas, s);
  return full ? bwd_as<VPT, false, true>(a, L, ctas, s)
              : bwd_as<VPT, false, false>(a, L, ctas, s);
}

}  // namespace

size_t residual_norm_ws_bytes(int T, int d) {
  return up256((size_t)bwd_ctas(T, d) * 2 * d * 4);
}

cudaError_t launch_residual_norm(const NormArgs& a, bool r_f32, cudaStream_t s) {
  timing_mark(s, "residual_norm");
  return r_f32 ? fwd<true>(a, s) : fwd<false>(a, s);
}

cudaError_t launch_residual_norm_bwd(const NormBwdArgs& a, bool r_f32, cudaStream_t s) {
  const BwdPlan L = plan_of(a.d, r_f32);
  const int ctas = bwd_ctas(a.T, a.d);
  timing_mark(s, "residual_norm_bwd");
  cudaError_t e = a.d <= 4096 ? bwd<1>(a, r_f32, L, ctas, s) : bwd<2>(a, r_f32, L, ctas, s);
  if (e != cudaSuccess) return e;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  float* dg = channel ? a.dgate : nullptr;
  if (!a.dw_pre && !a.dw_post && !dg) return cudaSuccess;
  timing_mark(s, "residual_norm_bwd_columns");
  return launch_pdl(norm_bwd_columns_kernel, dim3(a.d / 32, 2), dim3(32 * kColumnWarps), 0, s, (const float*)a.part, ctas,
                    a.d, channel ? a.gate : nullptr, static_cast<const __nv_bfloat16*>(a.w_post), a.dw_pre, a.dw_post,
                    dg);
}

}  // namespace moe
