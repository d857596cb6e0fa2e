// Global norm of a list of gradients and their clipping:
//   norm = sqrt(sum over all tensors of sum g^2)
//   coef = min(1, max_norm / (norm + 1e-6));  out = coef g
// One kernel sums squares (a fixed grid walks fixed chunks, one partial per
// CTA), a second adds the partials in order and scales.  Elements are squared
// and added in fp32 within a chunk and joined in fp64; a chunk whose fp32 sum
// left the range is summed again with its elements scaled, so the norm holds
// for gradients of any magnitude.
#include "common.cuh"
#include "step.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;                              // 16-byte vectors in flight per thread
constexpr int kChunkBytes = kThreads * kVecs * 16;    // 32 KB
constexpr int kCtas = 608;                            // four per SM of the 152-SM part
constexpr int kMaxList = 512;                         // tensors of one launch

// Work list of one launch, in the kernel's parameters.  A tensor's bytes are
// cut at 16-byte aligned addresses: chunk 0 starts at its first element, the
// k-th ends 32 KB after the aligned address at or below that element.
template <int CAP>
struct List {
  const void* in[CAP];
  void* out[CAP];
  long long bytes_type[CAP];  // bytes << 2 | type
  int first_chunk[CAP + 1];
  int n;
};

struct Piece {
  const char* p;     // first byte, element-aligned
  char* out;
  int bytes;
  int type;
};

// The c-th chunk of the list (binary search over first_chunk).
template <int CAP>
__device__ __forceinline__ Piece piece_of(const List<CAP>& L, int c) {
  int lo = 0, hi = L.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.first_chunk[mid] <= c) lo = mid; else hi = mid - 1;
  }
  const long long bt = L.bytes_type[lo];
  const char* base = static_cast<const char*>(L.in[lo]);
  const long long head = (long long)(reinterpret_cast<uintptr_t>(base) & 15u);
  const long long total = bt >> 2;
  long long b0 = (long long)(c - L.first_chunk[lo]) * kChunkBytes - head, b1 = b0 + kChunkBytes;
  if (b0 < 0) b0 = 0;
  if (b1 > total) b1 = total;
  Piece q;
  q.p = base + b0;
  q.out = L.out[lo] ? static_cast<char*>(L.out[lo]) + b0 : nullptr;
  q.bytes = (int)(b1 - b0);
  q.type = (int)(bt & 3);
  return q;
}

template <int TYPE>
struct Elem {  // bf16
  static constexpr int N = 8, SIZE = 2;
  __device__ static float get(const char* p) { return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p)); }
  __device__ static void put(char* p, float v) { *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v); }
  __device__ static void unpack(const uint4& v, float (&f)[8]) { unpack8(v, f); }
  __device__ static uint4 pack(const float (&f)[8]) { return pack8(f); }
};
template <>
struct Elem<MOE_GRAD_F16> {
  static constexpr int N = 8, SIZE = 2;
  __device__ static float get(const char* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }
  __device__ static void put(char* p, float v) { *reinterpret_cast<__half*>(p) = __float2half_rn(v); }
  __device__ static void unpack(const uint4& v, float (&f)[8]) { unpack_f16x8(v, f); }
  __device__ static uint4 pack(const float (&f)[8]) {
    const uint2 a = f16x4(make_float4(f[0], f[1], f[2], f[3])), b = f16x4(make_float4(f[4], f[5], f[6], f[7]));
    return make_uint4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Elem<MOE_GRAD_F32> {
  static constexpr int N = 4, SIZE = 4;
  __device__ static float get(const char* p) { return *reinterpret_cast<const float*>(p); }
  __device__ static void put(char* p, float v) { *reinterpret_cast<float*>(p) = v; }
  __device__ static void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// A chunk as this thread sees it: single elements before the first 16-byte
// boundary and after the last one, whole vectors between.
struct Split {
  int head, vecs, tail;  // elements, vectors, elements
};
template <int TYPE>
__device__ __forceinline__ Split split_of(const Piece& q) {
  using E = Elem<TYPE>;
  const int to16 = (int)((16u - (unsigned)(reinterpret_cast<uintptr_t>(q.p) & 15u)) & 15u);
  const int head = min(to16, q.bytes), rest = q.bytes - head;
  return Split{head / E::SIZE, rest / 16, (rest % 16) / E::SIZE};
}

// The squares of one vector, scaled, added to four fp32 sums.
template <int TYPE>
__device__ __forceinline__ void add_squares(const uint4& v, float scale, float (&s)[4]) {
  using E = Elem<TYPE>;
  float f[E::N];
  E::unpack(v, f);
#pragma unroll
  for (int e = 0; e < E::N; ++e) {
    const float g = f[e] * scale;
    s[e & 3] = fmaf(g, g, s[e & 3]);
  }
}

// The single elements of the chunk that fall to this thread: one before its
// first vector, one after its last.
template <int TYPE>
__device__ __forceinline__ void edge_elements(const Piece& q, const Split& sp, float (&f)[2]) {
  using E = Elem<TYPE>;
  const int t = threadIdx.x;
  f[0] = t < sp.head ? E::get(q.p + t * E::SIZE) : 0.0f;
  f[1] = t < sp.tail ? E::get(q.p + sp.head * E::SIZE + sp.vecs * 16 + t * E::SIZE) : 0.0f;
}

// This thread's part of the chunk's sum of (scale g)^2, in fp32, read again:
// for the chunks whose plain squares left the range (out of line: rare).
template <int TYPE>
__device__ __noinline__ float scaled_squares(const Piece q, float scale) {
  using E = Elem<TYPE>;
  const Split sp = split_of<TYPE>(q);
  const uint4* vec = reinterpret_cast<const uint4*>(q.p + sp.head * E::SIZE);
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, f[2];
  for (int i = threadIdx.x; i < sp.vecs; i += kThreads) add_squares<TYPE>(vec[i], scale, s);
  edge_elements<TYPE>(q, sp, f);
  s[0] = fmaf(f[0] * scale, f[0] * scale, s[0]);
  s[1] = fmaf(f[1] * scale, f[1] * scale, s[1]);
  return (s[0] + s[1]) + (s[2] + s[3]);
}

constexpr float kSmall = 8.0779356694631609e-28f;  // 2^-90
constexpr float kUp = 1.2379400392853803e27f;      // 2^90
constexpr float kDown = 8.0779356694631609e-28f;   // 2^-90

// The chunk's part of the sum for this thread in fp64: fp32 squares unless
// they overflowed or may have lost small values (elements below 2^-63 have no
// normal square; next to a sum of 2^-90 the at most 66 of them weigh 2^-30),
// then the same with scaled elements: 2^90 x an element of at most 2^-45, or
// 2^-90 x one of up to 2^128, whose squares are in range.
template <int TYPE>
__device__ __forceinline__ double chunk_sum(const Piece& q) {
  using E = Elem<TYPE>;
  const Split sp = split_of<TYPE>(q);
  const uint4* vec = reinterpret_cast<const uint4*>(q.p + sp.head * E::SIZE);
  uint4 raw[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int i = threadIdx.x + j * kThreads;
    raw[j] = i < sp.vecs ? vec[i] : make_uint4(0, 0, 0, 0);
  }
  float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f}, f[2];
  edge_elements<TYPE>(q, sp, f);
  s4[0] = f[0] * f[0];
  s4[1] = f[1] * f[1];
  unsigned bits = __float_as_uint(f[0]) | __float_as_uint(f[1]);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    bits |= raw[j].x | raw[j].y | raw[j].z | raw[j].w;
    add_squares<TYPE>(raw[j], 1.0f, s4);
  }
  const float s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
  if (s >= kSmall && s <= 3.0e38f) return (double)s;
  if (bits == 0u) return 0.0;
  if (s < kSmall) return (double)scaled_squares<TYPE>(q, kUp) * ((double)kDown * (double)kDown);
  return (double)scaled_squares<TYPE>(q, kDown) * ((double)kUp * (double)kUp);  // inf and NaN stay what they are
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}
// Sum over the CTA, for warp 0 (the fp64 units take 16 cycles per warp and
// instruction, so the other warps stay out of the second half).
__device__ __forceinline__ double cta_sum_d(double v) {
  __shared__ double w[kThreads / 32];
  v = warp_sum_d(v);
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  return warp_sum_d(threadIdx.x < kThreads / 32 ? w[threadIdx.x] : 0.0);
}
// sqrt(v) in fp32 for v >= 0 of fp64's range: the square root of the mantissa
// (1 to 4, fp32) times half the exponent.  inf and NaN stay; beyond fp32: inf.
__device__ __forceinline__ float sqrt_f(double v) {
  const int hi = __double2hiint(v);
  const int e = (hi >> 20) & 0x7FF;
  if (e == 0 || e == 0x7FF) return (float)v;  // 0 (squares are no fp64 subnormals), inf, NaN
  const int half = (e - 1023) >> 1;
  const float m = (float)__hiloint2double(hi - (half << 21), __double2loint(v));
  return ldexpf(sqrtf(m), half);
}

// Bound by HBM: four CTAs per SM, each with 32 KB of one chunk in flight.  The
// gradients of a 64-expert layer (818 MB): 116 us, 7.0 TB/s.
template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) grad_squares_kernel(const __grid_constant__ List<CAP> L, double* part) {
  dependency_wait();
  double sum = 0.0;
  const int chunks = L.first_chunk[L.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Piece q = piece_of(L, c);
    sum += q.type == MOE_GRAD_BF16 ? chunk_sum<MOE_GRAD_BF16>(q)
           : q.type == MOE_GRAD_F32 ? chunk_sum<MOE_GRAD_F32>(q)
                                    : chunk_sum<MOE_GRAD_F16>(q);
  }
  sum = cta_sum_d(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// Element by element (out of line): bytes [b0, b1) of the piece.
template <int TYPE>
__device__ __noinline__ void scale_elements(const char* in, char* out, int b0, int b1, float coef) {
  using E = Elem<TYPE>;
  for (int b = b0 + threadIdx.x * E::SIZE; b < b1; b += kThreads * E::SIZE) E::put(out + b, E::get(in + b) * coef);
}
// The same unscaled: the bits, as a product by 1 rewrites a NaN's.
template <typename U>
__device__ __noinline__ void copy_elements(const char* in, char* out, int b0, int b1) {
  for (int b = b0 + threadIdx.x * (int)sizeof(U); b < b1; b += kThreads * (int)sizeof(U))
    *reinterpret_cast<U*>(out + b) = *reinterpret_cast<const U*>(in + b);
}
__device__ __forceinline__ void scale_range(const Piece& q, int b0, int b1, float coef) {
  if (b0 >= b1) return;
  if (coef == 1.0f) {
    if (q.type == MOE_GRAD_F32) copy_elements<uint32_t>(q.p, q.out, b0, b1);
    else copy_elements<uint16_t>(q.p, q.out, b0, b1);
    return;
  }
  if (q.type == MOE_GRAD_BF16) scale_elements<MOE_GRAD_BF16>(q.p, q.out, b0, b1, coef);
  else if (q.type == MOE_GRAD_F32) scale_elements<MOE_GRAD_F32>(q.p, q.out, b0, b1, coef);
  else scale_elements<MOE_GRAD_F16>(q.p, q.out, b0, b1, coef);
}
template <int TYPE>
__device__ __forceinline__ void scale_vec(uint4& v, float coef) {
  using E = Elem<TYPE>;
  float f[E::N];
  E::unpack(v, f);
#pragma unroll
  for (int e = 0; e < E::N; ++e) f[e] *= coef;
  v = E::pack(f);
}

// The whole vectors of a chunk, as this thread holds them.
struct Vecs {
  uint4 raw[kVecs];
  int head, n;  // bytes before the first vector; vectors of the chunk
  bool aligned;  // the output lies at the same offset from a 16-byte boundary
};
__device__ __forceinline__ void load_chunk(const Piece& q, Vecs& v) {
  v.head = min((int)((16u - (unsigned)(reinterpret_cast<uintptr_t>(q.p) & 15u)) & 15u), q.bytes);
  v.n = (q.bytes - v.head) / 16;
  v.aligned = ((reinterpret_cast<uintptr_t>(q.p) ^ reinterpret_cast<uintptr_t>(q.out)) & 15u) == 0;
  const uint4* vec = reinterpret_cast<const uint4*>(q.p + v.head);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int i = threadIdx.x + j * kThreads;
    v.raw[j] = i < v.n ? vec[i] : make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void scale_chunk(const Piece& q, Vecs& v, float coef) {
  if (!q.out || (coef == 1.0f && q.out == q.p)) return;
  if (!v.aligned) {
    scale_range(q, 0, q.bytes, coef);
    return;
  }
  uint4* out = reinterpret_cast<uint4*>(q.out + v.head);
  if (coef != 1.0f) {  // 1: bit copies
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (q.type == MOE_GRAD_BF16) scale_vec<MOE_GRAD_BF16>(v.raw[j], coef);
      else if (q.type == MOE_GRAD_F32) scale_vec<MOE_GRAD_F32>(v.raw[j], coef);
      else scale_vec<MOE_GRAD_F16>(v.raw[j], coef);
    }
  }
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < v.n) out[i] = v.raw[j];
  }
  scale_range(q, 0, v.head, coef);
  scale_range(q, v.head + 16 * v.n, q.bytes, coef);
}

// Every CTA adds the partials in the same order, so all scale by the same
// bits.  A norm that is not finite leaves the gradients as they are (coef 1)
// and is recorded.  In place and coef 1: nothing is written.  818 MB in and
// out: 254 us, 6.4 TB/s; small lists cost the latency of the two kernels (8 us
// together, 11 with the root and the quotient in fp64 by every thread).  Without
// outputs one CTA walks the list alone: 805 MB 16 ms.
template <int CAP>
__global__ void __launch_bounds__(kThreads, 4)
    grad_scale_kernel(const __grid_constant__ List<CAP> L, const double* part, int n_part, float max_norm, float* norm,
                      float* coef_out, int write, int* status) {
  dependency_wait();
  // from the end: the chunks the sum read last are still in L2; the first one
  // is on its way while the partials are added
  int c = L.first_chunk[L.n] - 1 - (int)blockIdx.x;
  Piece q;
  Vecs v;
  if (c >= 0) {
    q = piece_of(L, c);
    load_chunk(q, v);
  }
  double sum = 0.0;
  for (int i = threadIdx.x; i < n_part; i += kThreads) sum += part[i];
  sum = cta_sum_d(sum);
  __shared__ float coef_s;
  if (threadIdx.x == 0) {
    const float nrm = sqrt_f(sum);
    const bool finite = isfinite(nrm);
    const float c1 = finite ? fminf(1.0f, max_norm / (nrm + 1e-6f)) : 1.0f;
    coef_s = c1;
    if (blockIdx.x == 0 && write) {
      *norm = nrm;
      if (coef_out) *coef_out = c1;
      if (!finite) record_status(status, MOE_ERR_RANGE);
    }
  }
  __syncthreads();
  const float coef = coef_s;
  while (c >= 0) {
    scale_chunk(q, v, coef);
    c -= gridDim.x;
    if (c < 0) break;
    q = piece_of(L, c);
    load_chunk(q, v);
  }
}

template <int CAP>
int fill(List<CAP>& L, const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types,
         int n) {
  long long chunks = 0;
  for (int i = 0; i < n; ++i) {
    const long long bytes = sizes[i] * (types[i] == MOE_GRAD_F32 ? 4 : 2);
    const long long head = (long long)(reinterpret_cast<uintptr_t>(grads[i]) & 15u);
    L.in[i] = grads[i];
    L.out[i] = outs ? outs[i] : nullptr;
    L.bytes_type[i] = bytes << 2 | types[i];
    L.first_chunk[i] = (int)chunks;
    if (bytes > 0) chunks += (bytes + head + kChunkBytes - 1) / kChunkBytes;
  }
  L.n = n;
  L.first_chunk[n] = (int)chunks;
  return (int)chunks;
}

int grid_of(int chunks) { return chunks < 1 ? 1 : chunks < kCtas ? chunks : kCtas; }
int lists_of(long long n) { return n < 1 ? 1 : (int)((n + kMaxList - 1) / kMaxList); }

template <int CAP>
cudaError_t run(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int n,
                float max_norm, float* norm, float* coef, double* part, int* status, cudaStream_t s) {
  const int lists = n <= CAP ? 1 : lists_of(n);
  List<CAP> L;
  int parts = 0, chunks = 0;
  for (int l = 0; l < lists; ++l) {
    const int i0 = l * CAP, m = n - i0 < CAP ? n - i0 : CAP;
    chunks = fill(L, grads + i0, outs ? outs + i0 : nullptr, sizes + i0, types + i0, m);
    const int grid = grid_of(chunks);
    timing_mark(s, "grad_squares");
    cudaError_t e = launch_pdl(grad_squares_kernel<CAP>, dim3(grid), dim3(kThreads), 0, s, L, part + parts);
    if (e != cudaSuccess) return e;
    parts += grid;
  }
  for (int l = outs ? lists - 1 : 0; l >= 0; --l) {
    const int i0 = l * CAP, m = n - i0 < CAP ? n - i0 : CAP;
    if (lists > 1) chunks = fill(L, grads + i0, outs ? outs + i0 : nullptr, sizes + i0, types + i0, m);
    timing_mark(s, "grad_scale");
    cudaError_t e = launch_pdl(grad_scale_kernel<CAP>, dim3(outs ? grid_of(chunks) : 1), dim3(kThreads), 0, s, L,
                               (const double*)part, parts, max_norm, norm, coef, l == 0 ? 1 : 0, status);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_clip_ws_bytes(long long n_tensors) { return up256((size_t)lists_of(n_tensors) * kCtas * 8); }

cudaError_t launch_grad_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types,
                             int n, float max_norm, float* norm, float* coef, void* ws, int* status, cudaStream_t s) {
  double* part = static_cast<double*>(ws);
  // The list travels in the kernels' parameters, in the smallest block that
  // holds it: their size is host time in each of the two launches (7 to 14 KB
  // less: 0.6 us of 8 for lists of 17 to 224 small tensors).
  if (n <= 16) return run<16>(grads, outs, sizes, types, n, max_norm, norm, coef, part, status, s);
  if (n <= 64) return run<64>(grads, outs, sizes, types, n, max_norm, norm, coef, part, status, s);
  if (n <= 256) return run<256>(grads, outs, sizes, types, n, max_norm, norm, coef, part, status, s);
  return run<kMaxList>(grads, outs, sizes, types, n, max_norm, norm, coef, part, status, s);
}

}  // namespace moe
