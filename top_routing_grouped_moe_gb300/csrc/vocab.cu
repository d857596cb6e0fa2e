// Softmax cross entropy of the vocabulary head, z = x W^T, without the [T, V]
// logits in memory, and its gradient.
//
//   forward   lse[t] = log sum_v exp(z[t,v]),
//             loss[t] = lse[t] - z[t,target] + z_weight lse[t]^2
//   backward  dz[t,v] = dloss[t] (p[t,v] (1 + 2 z_weight lse[t]) - [v = target]),
//             p = exp(z - lse);   dx = dz W,  dW = dz^T x
//
// The forward is one GEMM whose epilogue keeps, per row and 256-column tile,
// the maximum and the sum of exponentials; a small kernel joins the tiles.
// The backward takes the vocabulary in pieces: the piece's logits are computed
// again, their epilogue writes dz in bf16 (the operand of two more GEMMs), and
// the piece's rows of dW and its share of dx follow.
//
// All four products (the logits, the logits again, dx, dW) run on one kernel,
// bound by the tensor cores and, in a loop, by the board's power: T = 8192, V =
// 50257, d = 4096: 8.1 ms forward and backward, 1.67 PFLOP/s over the 8 T V d
// issued (a plain bf16 product of cuBLAS in a loop: 1.71); T = 2047, V = 32003,
// d = 1024: 0.373 ms, 1.44 PFLOP/s.  CTA pairs on 256 x 256 tiles (tcgen05.mma
// cta_group::2, fp32 accumulators in tensor memory, two of them so that a tile's
// epilogue runs beside the next tile's products), operands by TMA into a
// six-stage ring (a seventh stage, and clusters of two pairs that share B by
// multicast, changed nothing; the issuing thread's instructions did, see
// mma_stage).
//
// The tensor cores truncate when they add into an accumulator, which biases a
// long sum toward zero: over K = 2048 a logit is low by about 3e-6 of itself,
// several times fp32's own error.  The logits are therefore contracted 512
// columns at a time into alternating accumulators and the epilogue adds these
// parts in registers (round to nearest).  The backward forms its logits the same
// way, so that they are the forward's bit for bit and their own error cancels in
// z - lse: dz at the target is p - 1, in which an error of z is absolute (with
// one accumulator through d = 4096 and a logit of 105, a token with 1 - p = 2e-5
// got 1e-3).  dx and dW are sums of dz, already rounded to bf16, whose terms do
// not cancel like that: they run through.
#include <type_traits>

#include "gemm_host.cuh"
#include "step.h"

namespace moe {
namespace {

using gemm::A_BYTES;
using gemm::BK;
using gemm::BM;
using gemm::BN;
using gemm::MN_BLOCK_BYTES;
using gemm::UMMA_K;

constexpr int TILE = 256;          // rows and columns of a pair's tile
constexpr int EPI_WARPS = 8;       // two per 32 rows: columns [0, 128) and [128, 256)
constexpr int THREADS = 64 + 32 * EPI_WARPS;  // TMA warp, MMA warp, epilogue
constexpr int SEG = 8;             // logits: K steps per accumulator
constexpr float kLog2e = 1.44269504088896340736f;
// 1 / kLog2e, the float, in two parts: what takes a base-2 maximum back exactly
constexpr float kLn2 = 0.69314718246459961f, kLn2Lo = 7.3486932e-09f;

enum Mode : int {
  LSE = 0,  // A = x (K = d), B = W: per-row partials of the log-sum-exp
  DZ = 1,   // the same product: dz in bf16
  GRAD = 2,  // both products of dz, in one launch:
             //   dx: A = dz (K = the piece's columns), B = W by columns of d
             //   dW: A = dz by its columns (K = tokens), B = x by columns of d
};

constexpr int STAGES = 6;
constexpr int STAGE_BYTES = 2 * A_BYTES;  // this CTA's 128 rows of A and 128 of B, 64 K

// One product: its operand maps (and that of its bf16 stores), its output and
// its tiles.
struct Product {
  CUtensorMap a, b, out;
  int rows, cols;           // valid rows and columns of the output
  int m_tiles, n_tiles, group_m, per_group;
  unsigned group_magic, per_group_magic;  // for n / group_m, n / per_group (0: divide)
  int k_steps, splits;      // K steps of 64 in all, cut into `splits` ranges
};

struct VParams {
  Product p;                // LSE, DZ: the logits; GRAD: dx (splits = 0: none)
  Product w;                // GRAD: dW (m_tiles = 0: none)
  int late_rounds;          // GRAD: see tile_of
  // LSE, DZ
  const int32_t* targets;
  int v0, V;                // first column's vocabulary index; vocabulary size
  float2* part;             // [2 n_tiles][rows]: maximum (base 2), sum of a half tile
  float* target_logit;      // [rows]
  const float* lse;
  const float* dloss;
  float z_weight;
  // dz is kept divided by the largest |dloss| (DZ writes it here), the outputs
  // of GRAD are multiplied by it
  float* scale;
  // GRAD
  float* slab;              // dx: [splits][rows][cols] fp32 (NULL: store bf16 through `out`)
  int add;                  // add to the slab
  int* status;
};

struct Tail {
  float4 stage[EPI_WARPS][256];  // per epilogue warp: 4 KB staging
  uint64_t full[STAGES], empty[STAGES];
  uint64_t acc_full[2], acc_empty[2];
  float peak[EPI_WARPS];  // DZ: the warps' largest |dloss|
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kSmem = 1024 + STAGES * STAGE_BYTES + sizeof(Tail);
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");

struct TileAt {
  int m0, n0, n, split, k0, k1;
  bool dw;  // GRAD: a tile of dW
};
// Tile t of a product.  Tiles go in groups of group_m row tiles: within a group
// the row index runs fastest, so that the 76 tiles running at one time are about
// 16 x 5, and share their rows of A and of B in L2 as they move along K.  (T =
// 8192, V = 50257, d = 4096, the backward: 6.06 ms with 4 row tiles per group,
// 5.96 with 8 to 16, 6.15 with 32: power spent on DRAM reads is clock lost.)
constexpr int GROUP_M = 16;
__device__ __forceinline__ TileAt tile_at(const Product& P, int t) {
  TileAt at;
  at.split = 0;
  at.k0 = 0;
  at.k1 = P.k_steps;
  int w = t;
  if (P.splits > 1) {
    const int per_split = P.m_tiles * P.n_tiles;
    at.split = t / per_split;
    w -= at.split * per_split;
    at.k0 = (int)((long long)P.k_steps * at.split / P.splits);
    at.k1 = (int)((long long)P.k_steps * (at.split + 1) / P.splits);
  }
  // quotients by multiplication: the thread that loads works this out between
  // two tiles, while nothing new is on its way
  const int g = P.per_group_magic ? __umulhi(w, P.per_group_magic) : w / P.per_group;
  w -= g * P.per_group;
  const int first = g * P.group_m, left = P.m_tiles - first;
  int m;
  if (left >= P.group_m) {
    at.n = P.group_magic ? __umulhi(w, P.group_magic) : w / P.group_m;
    m = w - at.n * P.group_m;
  } else {
    at.n = w / left;
    m = w - at.n * left;
  }
  at.n0 = at.n * TILE;
  at.m0 = (first + m) * TILE;
  at.dw = false;
  return at;
}

// The i-th tile of CTA pair `pair`; false when it has no more.  Tiles are dealt
// round by round.  GRAD deals dx's tiles first (the longer ones); in their last
// round only `late` pairs get one, and the others go on to dW: they have
// late_rounds rounds of it to themselves, about as long as one tile of dx, and
// from then on every pair takes part.
template <int MODE>
__device__ __forceinline__ bool tile_of(const VParams& P, int pair, int i, TileAt& at) {
  const int pairs = gridDim.x / 2;
  const int n = P.p.m_tiles * P.p.n_tiles * P.p.splits, t = pair + i * pairs;
  if (t < n) {
    at = tile_at(P.p, t);
    return true;
  }
  if (MODE != GRAD) return false;
  const int mine = pair < n ? (n - pair + pairs - 1) / pairs : 0, late = n % pairs;
  int r = i - mine;  // the pair's round of dW, counted from its first
  int u;
  if (late == 0) u = r * pairs + pair;
  else if (pair >= late && r < P.late_rounds) u = r * (pairs - late) + (pair - late);
  else u = P.late_rounds * (pairs - late) + (pair < late ? r : r - P.late_rounds) * pairs + pair;
  if (u >= P.w.m_tiles * P.w.n_tiles) return false;
  at = tile_at(P.w, u);
  at.dw = true;
  return true;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 consecutive fp32 columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_get16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The products of one stage: four pair MMAs of 16 K each, then the commit that
// frees the stage in both CTAs, in one asm statement.  One thread issues them
// all and its instructions per stage, not the tensor cores, are what a stage
// costs if they are many (85% of the rate with descriptors built for every MMA):
// here a descriptor is its low word (shared-memory address / 16 and leading
// offset; a_lo, b_lo for the stage) plus a constant, over a constant high word
// (1024 bytes between groups of eight rows, 128-byte swizzle).
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t desc_lead(bool mn) { return (mn ? (uint32_t)MN_BLOCK_BYTES >> 4 : 1u) << 16; }
template <int A_MN, int B_MN>
__device__ __forceinline__ void mma_stage(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t more,
                                          uint32_t empty_bar) {
  constexpr uint32_t SA = A_MN ? 2048 >> 4 : 32 >> 4, SB = B_MN ? 2048 >> 4 : 32 >> 4;
  constexpr uint32_t idesc = ptx::idesc_bf16(TILE, TILE, A_MN, B_MN);
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 da, db;\n\t.reg .b32 a, b;\n\t.reg .b16 both;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "setp.eq.b32 t, %3, %3;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t"
      "add.u32 a, %1, %6;\n\tadd.u32 b, %2, %7;\n\tmov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, t;\n\t"
      "add.u32 a, a, %6;\n\tadd.u32 b, b, %7;\n\tmov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, t;\n\t"
      "add.u32 a, a, %6;\n\tadd.u32 b, b, %7;\n\tmov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, t;\n\t"
      "mov.b16 both, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%8], both;\n\t"
      "}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(more), "r"(DESC_HI), "r"(idesc), "n"(SA), "n"(SB), "r"(empty_bar)
      : "memory");
}
// TMA loads of a CTA pair: 64 K columns of 128 rows, or 64 K rows of two blocks
// of 64 columns (a block view); bytes counted on the leader's barrier.
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* m, uint32_t bar, int k, int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(k), "r"(row)
      : "memory");
}
__device__ __forceinline__ void load_blocks(uint32_t dst, const CUtensorMap* m, uint32_t bar, int k, int block) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(k), "r"(block)
      : "memory");
}
__device__ __forceinline__ bool bar_ready(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

template <int MODE>
__global__ void __launch_bounds__(THREADS, 1) vocab_gemm_kernel(const __grid_constant__ VParams P) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Tail* tail = reinterpret_cast<Tail*>(smem + STAGES * STAGE_BYTES);
  volatile int* abort_flag = &tail->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int pair = blockIdx.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&tail->full[s], 1);
      ptx::mbar_init(&tail->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tail->acc_full[a], 1);
      ptx::mbar_init(&tail->acc_empty[a], EPI_WARPS * 2);  // every epilogue warp of each CTA
    }
    tail->abort_flag = 0;
    ptx::fence_mbarrier_init();
    ptx::prefetch_tmap(&P.p.a);
    ptx::prefetch_tmap(&P.p.b);
    if (MODE == GRAD) {
      ptx::prefetch_tmap(&P.w.a);
      ptx::prefetch_tmap(&P.w.b);
    }
  }
  if (warp == 1) {
    ptx::tmem_alloc<2>(&tail->tmem_base, 2 * BN);
    ptx::tmem_relinquish<2>();
    ptx::tc_fence_before();
  }
  dependency_wait();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      TileAt at{};
      const uint32_t smem0 = ptx::smem_u32(smem), empty0 = ptx::smem_u32(tail->empty);
      const uint32_t full0 = ptx::mapa(ptx::smem_u32(tail->full), 0);  // the leader's
      // the stages of one tile; its kind is a constant of the loop (a branch
      // on it per stage cost 4% of the launch)
      auto load_tile = [&](auto kind) {
        constexpr bool dw = decltype(kind)::value;
        const CUtensorMap* ma = dw ? &P.w.a : &P.p.a;
        const CUtensorMap* mb = dw ? &P.w.b : &P.p.b;
        const int am = at.m0 + rank * BM, bn = at.n0 + rank * BM;
        for (int kb = at.k0; kb < at.k1; ++kb) {
          if (!bar_ready(empty0 + 8 * stage, phase ^ 1u) &&
              !ptx::mbar_wait_bounded(&tail->empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          if (rank == 0) ptx::mbar_arrive_expect_tx(&tail->full[stage], 2 * STAGE_BYTES);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          const uint32_t a_dst = smem0 + stage * STAGE_BYTES, bar = full0 + 8 * stage;
          const int k = kb * BK;
          // by columns: two blocks of 64 columns x 64 K rows in one box
          if (dw) load_blocks(a_dst, ma, bar, k, am >> 6);
          else load_rows(a_dst, ma, bar, k, am);
          if (MODE == GRAD) load_blocks(a_dst + A_BYTES, mb, bar, k, bn >> 6);
          else load_rows(a_dst + A_BYTES, mb, bar, k, bn);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      };
      for (int i = 0; ok && tile_of<MODE>(P, pair, i, at); ++i) {
        if (MODE == GRAD && at.dw) load_tile(std::true_type{});
        else load_tile(std::false_type{});
      }
      if (!ok) {
        *abort_flag = 1;
        record_status(P.status, MOE_ERR_TIMEOUT);
        // copies in flight land before the CTA's shared memory goes away (the
        // leader's barriers count both CTAs' bytes)
        for (int s = 0; s < STAGES; ++s)
          if (rank == 0 && (issued & (1u << s))) {
            volatile int never = 0;
            ptx::mbar_wait_bounded(&tail->full[s], (issued_phase >> s) & 1u, &never, 100000000ull);
          }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    if (lane == 0 && rank == 0) {
      constexpr int b_mn = MODE == GRAD;
      const uint32_t smem0 = ptx::smem_u32(smem) >> 4;
      const uint32_t full0 = ptx::smem_u32(tail->full), empty0 = ptx::smem_u32(tail->empty);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int it = 0;  // accumulators filled
      TileAt at{};
      auto multiply_tile = [&](auto kind) {
        constexpr int a_mn = decltype(kind)::value;
        const uint32_t a_lo0 = smem0 | desc_lead(a_mn), b_lo0 = (smem0 + (A_BYTES >> 4)) | desc_lead(b_mn);
        for (int ks = at.k0; ok && ks < at.k1; ++it) {
          const int ke = MODE == GRAD ? at.k1 : min(ks + SEG, at.k1);
          const int acc = it & 1;
          if (!ptx::mbar_wait_cluster_bounded(&tail->acc_empty[acc], ((it >> 1) & 1) ^ 1u, abort_flag,
                                              kWaitLimitNs)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * BN;
          for (int kb = ks; kb < ke; ++kb) {
            if (!bar_ready(full0 + 8 * stage, phase) &&
                !ptx::mbar_wait_bounded(&tail->full[stage], phase, abort_flag, kWaitLimitNs)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            mma_stage<a_mn, b_mn>(d_tmem, a_lo0 + stage * (STAGE_BYTES >> 4), b_lo0 + stage * (STAGE_BYTES >> 4),
                                  kb > ks ? 1u : 0u, empty0 + 8 * stage);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) ptx::mma_commit_pair(&tail->acc_full[acc], 0x3);
          ks = ke;
        }
      };
      for (int i = 0; ok && tile_of<MODE>(P, pair, i, at); ++i) {
        if (MODE == GRAD && at.dw) multiply_tile(std::true_type{});
        else multiply_tile(std::false_type{});
      }
      if (!ok) {
        *abort_flag = 1;
        record_status(P.status, MOE_ERR_TIMEOUT);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    // Tensor memory gives a warp the lanes of its index mod 4: rows
    // [32 q, 32 q + 32) of the CTA's; `half` picks its 128 columns.  A thread
    // holds one row.
    const int q = warp & 3, half = (warp - 2) >> 2;
    float4* stg = tail->stage[warp - 2];
    uint32_t stores = 0;
    int it = 0;  // accumulators taken
    bool ok = true;
    auto take = [&](int acc) {
      if (!ptx::mbar_wait_cluster_bounded(&tail->acc_full[acc], (it >> 1) & 1, abort_flag, kWaitLimitNs)) {
        *abort_flag = 1;
        record_status(P.status, MOE_ERR_TIMEOUT);
        return false;
      }
      ptx::tc_fence_after();
      return true;
    };
    auto give = [&](int acc) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) ptx::mbar_arrive(&tail->acc_empty[acc]);
        else ptx::mbar_arrive_remote(ptx::mapa(ptx::smem_u32(&tail->acc_empty[acc]), 0));
      }
    };
    float scale = 1.0f;
    if (MODE == DZ) {
      // The largest |dloss| of the rows with a target.  Divided by it, equal
      // weights (a mean) leave dz = p - 1 at the target, which bf16 holds far
      // better than that times an arbitrary 1 / N.
      const int et = threadIdx.x - 64;
      float top = 0.0f;
      for (int i = et; i < P.p.rows; i += 32 * EPI_WARPS) {
        const int tg = __ldg(P.targets + i);
        if (tg >= 0 && tg < P.V) top = fmaxf(top, fabsf(__ldg(P.dloss + i)));
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      if (lane == 0) tail->peak[warp - 2] = top;
      asm volatile("bar.sync 1, %0;" ::"n"(32 * EPI_WARPS) : "memory");
#pragma unroll
      for (int w = 0; w < EPI_WARPS; ++w) top = fmaxf(top, tail->peak[w]);
      if (top > 0.0f && top < INFINITY) scale = top;
      if (blockIdx.x == 0 && et == 0) *P.scale = scale;
    } else if (MODE == GRAD) {
      scale = *P.scale;
    }
    TileAt at{};
    for (int i = 0; ok && tile_of<MODE>(P, pair, i, at); ++i) {
      const Product& pr = MODE == GRAD && at.dw ? P.w : P.p;
      const bool to_slab = !at.dw && P.slab;
      const int out_rows = pr.rows, out_cols = pr.cols;
      const int row0 = at.m0 + rank * BM + q * 32, row = row0 + lane;
      const int col0 = at.n0 + half * 128;  // this warp's first column
      const int ncol = min(128, out_cols - col0);  // valid ones (may be <= 0)
      const bool in = row < out_rows;
      const uint32_t lane_addr = (static_cast<uint32_t>(q * 32) << 16) + half * 128;
      // this row's constants, read while the products run
      int target = -1;
      float l = 0.0f, mult = 0.0f, up = 0.0f;
      if (MODE == LSE || MODE == DZ) {
        if (in) target = __ldg(P.targets + row);
        if (target >= P.V) target = -1;
        if (MODE == DZ && target >= 0) {
          l = __ldg(P.lse + row);
          up = __ldg(P.dloss + row) / scale;
          mult = up * fmaf(2.0f * P.z_weight, l, 1.0f);
        }
        target = target < 0 ? -1 : target - (P.v0 + col0);  // column of this warp's, or outside
      }
      // a chunk of 32 columns as bf16 into a 32 x 32 box (64-byte swizzle, two
      // boxes in turn), out by TMA
      auto store_box = [&](int c, auto value) {
        uint8_t* box = reinterpret_cast<uint8_t*>(stg) + (stores & 1) * 2048;
        if (stores >= 2) {
          if (lane == 0) ptx::bulk_wait_read<1>();
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 v = make_uint4(pack_bf16(value(8 * j), value(8 * j + 1)), pack_bf16(value(8 * j + 2), value(8 * j + 3)),
                                     pack_bf16(value(8 * j + 4), value(8 * j + 5)), pack_bf16(value(8 * j + 6), value(8 * j + 7)));
          *reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = v;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::tma_store_3d(&pr.out, box, col0 + 32 * c, row0, 0);
          ptx::bulk_commit();
        }
        ++stores;
      };
      if constexpr (MODE != GRAD) {
        const bool work = row0 < out_rows && ncol > 0;
        float z[128];
#pragma unroll
        for (int e = 0; e < 128; ++e) z[e] = 0.0f;
        for (int ks = at.k0; ks < at.k1; ks += SEG, ++it) {
          const int acc = it & 1;
          if (!take(acc)) {
            ok = false;
            break;
          }
          if (work) {
            const uint32_t taddr = tmem_base + acc * BN + lane_addr;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (16 * c >= ncol) break;
              uint32_t r[16];
              tmem_get16(taddr + 16 * c, r);
#pragma unroll
              for (int e = 0; e < 16; ++e) z[16 * c + e] += __uint_as_float(r[e]);
            }
          }
          give(acc);
        }
        if (!ok) break;
        if (row0 >= out_rows) continue;
        if constexpr (MODE == DZ) {
          // dz: z - lse first (exact where they are close), then the exponential.
          // Rows without a target and columns past the vocabulary are zero
          // whatever their logits are.
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int e = 32 * c; e < 32 * c + 32; ++e) z[e] = mult * exp2_fast((z[e] - l) * kLog2e);
            if (__any_sync(0xffffffffu, (unsigned)(target - 32 * c) < 32u)) {
#pragma unroll
              for (int e = 32 * c; e < 32 * c + 32; ++e)
                if (target == e) z[e] -= up;
            }
            if (ncol < 32 * c + 32 || up == 0.0f) {
#pragma unroll
              for (int e = 32 * c; e < 32 * c + 32; ++e)
                if (e >= ncol || up == 0.0f) z[e] = 0.0f;
            }
            store_box(c, [&](int e) { return z[32 * c + e]; });
          }
          continue;
        }
        if (__any_sync(0xffffffffu, target >= 0 && target < ncol)) {
          float zt = 0.0f;
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (target == e) zt = z[e];
          if (target >= 0 && target < ncol) P.target_logit[row] = zt;
        }
        float mx[4], sum[4];
        if (ncol < 128) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e >= ncol) z[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = z[e], sum[e] = 0.0f;
#pragma unroll
        for (int e = 4; e < 128; ++e) mx[e & 3] = fmaxf(mx[e & 3], z[e]);
        // the reference exponent, in base 2; a row of -inf takes 0
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kLog2e;
        const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int e = 0; e < 128; ++e) sum[e & 3] += exp2_fast(fmaf(z[e], kLog2e, -ref));
        if (in) P.part[(long long)(2 * at.n + half) * out_rows + row] = make_float2(top, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        continue;
      }
      const int acc = it & 1;
      if (!take(acc)) {
        ok = false;
        break;
      }
      ++it;
      const uint32_t taddr = tmem_base + acc * BN + lane_addr;
      if (row0 < out_rows && ncol > 0) {
        const int nch = (ncol + 31) / 32;
        uint32_t r[2][32];
        ptx::tmem_ld32(taddr, r[0]);
        ptx::tmem_ld_wait(r[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c >= nch) break;
          uint32_t(&cur)[32] = r[c & 1];
          uint32_t(&nxt)[32] = r[(c + 1) & 1];
          if (c + 1 < nch) ptx::tmem_ld32(taddr + 32 * (c + 1), nxt);
#pragma unroll
          for (int e = 0; e < 32; ++e) cur[e] = __float_as_uint(__uint_as_float(cur[e]) * scale);
          if (to_slab) {
            // fp32 share of dx: eight lanes per row through the staging buffer
            // (16-byte pieces XOR-swizzled by the row: no bank conflicts)
            __syncwarp();
#pragma unroll
            for (int m = 0; m < 8; ++m)
              stg[lane * 8 + (m ^ (lane & 7))] =
                  make_float4(__uint_as_float(cur[4 * m]), __uint_as_float(cur[4 * m + 1]),
                              __uint_as_float(cur[4 * m + 2]), __uint_as_float(cur[4 * m + 3]));
            __syncwarp();
            const int rs = lane >> 3, cg = lane & 7;
            float* out = P.slab + ((long long)at.split * out_rows + row0) * out_cols + col0 + 32 * c + 4 * cg;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int rr = 4 * j + rs;
              if (row0 + rr >= out_rows) continue;
              float4 v = stg[rr * 8 + (cg ^ (rr & 7))];
              float4* p = reinterpret_cast<float4*>(out + (long long)rr * out_cols);
              if (P.add) {
                const float4 o = *p;
                v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
              }
              *p = v;
            }
          } else {
            store_box(c, [&](int e) { return __uint_as_float(cur[e]); });
          }
          if (c + 1 < nch) ptx::tmem_ld_wait(nxt);
        }
      }
      give(acc);
    }
    if (MODE != LSE && lane == 0) ptx::bulk_wait_all();
  }

  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc<2>(tmem_base, 2 * BN);
  }
}

// ------------------------------------------------------------ few tokens
// The forward of at most 128 tokens reads W once and is bound by that read.
// Here the vocabulary is the row index of the tile (128 lanes of tensor memory)
// and the tokens its columns, so that a stage is a slice of W and little else:
// with 16 tokens eleven stages of 18 KB are in flight per SM (as columns of a
// 128-token tile: four of 48 KB).  5 tokens, d = 2048, V = 50257: 34 us for the
// 206 MB of W (0.9 of the copy rate) and 2 for the join; as columns 48.
// The width of a tile (rows of W) gives every SM nearly the same number of rows.
constexpr int kFewTokens = 128;
constexpr int FEW_STAGES = 12;
constexpr int FEW_RING = 200 * 1024;
constexpr int FEW_THREADS = 64 + 128;

struct FewParams {
  CUtensorMap w, x;        // boxes: tile_rows x 64 of W, n x 64 of x
  int T, V, n;             // n: tokens rounded up to 16
  int tile_rows, tiles;
  int k_steps, stages, stage_bytes;
  const int32_t* targets;
  float2* part;            // [4 CTAs][T]
  float* target_logit;     // [T]
  int* status;
};

struct FewTail {
  float stage[4][32 * 32];  // per epilogue warp: a 32 x 32 block
  uint64_t full[FEW_STAGES], empty[FEW_STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kFewSmem = 1024 + FEW_RING + sizeof(FewTail);
static_assert(kFewSmem <= 227 * 1024, "shared memory of one CTA");

__global__ void __launch_bounds__(FEW_THREADS, 1) vocab_few_kernel(const __grid_constant__ FewParams P) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewTail* tail = reinterpret_cast<FewTail*>(smem + FEW_RING);
  volatile int* abort_flag = &tail->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      ptx::mbar_init(&tail->full[s], 1);
      ptx::mbar_init(&tail->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tail->acc_full[a], 1);
      ptx::mbar_init(&tail->acc_empty[a], 4);
    }
    tail->abort_flag = 0;
    ptx::fence_mbarrier_init();
    ptx::prefetch_tmap(&P.w);
    ptx::prefetch_tmap(&P.x);
  }
  if (warp == 1) {
    ptx::tmem_alloc<1>(&tail->tmem_base, 256);
    ptx::tmem_relinquish<1>();
    ptx::tc_fence_before();
  }
  dependency_wait();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      const uint32_t tx = (P.tile_rows + P.n) * BK * 2;
      for (int t = blockIdx.x; ok && t < P.tiles; t += gridDim.x) {
        for (int kb = 0; kb < P.k_steps; ++kb) {
          if (!ptx::mbar_wait_bounded(&tail->empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          uint64_t* fb = &tail->full[stage];
          ptx::mbar_arrive_expect_tx(fb, tx);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          uint8_t* dst = smem + stage * P.stage_bytes;
          ptx::tma_load_2d(dst, &P.w, fb, kb * BK, t * P.tile_rows);
          ptx::tma_load_2d(dst + A_BYTES, &P.x, fb, kb * BK, 0);
          if (++stage == P.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        record_status(P.status, MOE_ERR_TIMEOUT);
        for (int s = 0; s < P.stages; ++s)  // copies in flight land first
          if (issued & (1u << s)) {
            volatile int never = 0;
            ptx::mbar_wait_bounded(&tail->full[s], (issued_phase >> s) & 1u, &never, 100000000ull);
          }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // rows of the tile past tile_rows hold what the stage held before: their
      // accumulator rows are not read
      const uint32_t idesc = ptx::idesc_bf16(BM, P.n, 0, 0);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < P.tiles; t += gridDim.x) {
        for (int ks = 0; ok && ks < P.k_steps; ++it) {
          const int ke = min(ks + SEG, P.k_steps), acc = it & 1;
          if (!ptx::mbar_wait_bounded(&tail->acc_empty[acc], ((it >> 1) & 1) ^ 1u, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * 128;
          for (int kb = ks; kb < ke; ++kb) {
            if (!ptx::mbar_wait_bounded(&tail->full[stage], phase, abort_flag, kWaitLimitNs)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint32_t a_addr = ptx::smem_u32(smem + stage * P.stage_bytes), b_addr = a_addr + A_BYTES;
#pragma unroll
            for (int s = 0; s < BK / UMMA_K; ++s)
              ptx::mma_bf16(d_tmem, ptx::smem_desc(a_addr + s * 32, 16, 1024), ptx::smem_desc(b_addr + s * 32, 16, 1024),
                            idesc, (kb > ks || s > 0) ? 1u : 0u);
            ptx::mma_commit(&tail->empty[stage]);
            if (++stage == P.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) ptx::mma_commit(&tail->acc_full[acc]);
          ks = ke;
        }
      }
      if (!ok) {
        *abort_flag = 1;
        record_status(P.status, MOE_ERR_TIMEOUT);
      }
    }
  } else {
    // A thread holds one row of W against all tokens; blocks of 32 x 32 go
    // through shared memory so that a lane then holds one token against the
    // warp's 32 rows.  m2, sum: the token's running maximum (base 2) and sum
    // over all tiles of this CTA, tokens lane, lane + 32, ...
    const int q = warp & 3;
    float* stg = tail->stage[q];
    float m2[4], sum[4];
    int target[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      m2[c] = -INFINITY, sum[c] = 0.0f;
      const int tok = 32 * c + lane;
      target[c] = tok < P.T ? __ldg(P.targets + tok) : -1;
      if (target[c] >= P.V) target[c] = -1;
    }
    int it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < P.tiles; t += gridDim.x) {
      const int v0 = t * P.tile_rows + 32 * q;  // this warp's first row of W
      const int rows = min(P.tile_rows - 32 * q, P.V - v0);  // its rows of this tile (may be <= 0)
      float z[128];
#pragma unroll
      for (int e = 0; e < 128; ++e) z[e] = 0.0f;
      for (int ks = 0; ks < P.k_steps; ks += SEG, ++it) {
        const int acc = it & 1;
        if (!ptx::mbar_wait_bounded(&tail->acc_full[acc], (it >> 1) & 1, abort_flag, kWaitLimitNs)) {
          *abort_flag = 1;
          record_status(P.status, MOE_ERR_TIMEOUT);
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if (rows > 0) {
          const uint32_t taddr = tmem_base + acc * 128 + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (16 * c >= P.n) break;
            uint32_t r[16];
            tmem_get16(taddr + 16 * c, r);
#pragma unroll
            for (int e = 0; e < 16; ++e) z[16 * c + e] += __uint_as_float(r[e]);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&tail->acc_empty[acc]);
      }
      if (!ok || rows <= 0) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (32 * c >= P.T) break;
        // row `lane`, token e at column e ^ lane: no bank conflicts either way
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 32; ++e) stg[lane * 32 + (e ^ lane)] = lane < rows ? z[32 * c + e] : -INFINITY;
        __syncwarp();
        float v[32], mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          v[e] = stg[e * 32 + (lane ^ e)];
          mx = fmaxf(mx, v[e]);
        }
        const float top = fmaxf(m2[c], mx * kLog2e), ref = top == -INFINITY ? 0.0f : top;
        float s4[4] = {sum[c] * exp2_fast(m2[c] - ref), 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 32; ++e) s4[e & 3] += exp2_fast(fmaf(v[e], kLog2e, -ref));
        sum[c] = (s4[0] + s4[1]) + (s4[2] + s4[3]);
        m2[c] = top;
        const int at = target[c] - v0;
        if (target[c] >= 0 && at >= 0 && at < min(rows, 32)) P.target_logit[32 * c + lane] = stg[at * 32 + (lane ^ at)];
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int tok = 32 * c + lane;
      if (tok < P.T) P.part[(long long)(4 * blockIdx.x + q) * P.T + tok] = make_float2(m2[c], sum[c]);
    }
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc<1>(tmem_base, 256);
  }
}

// Joins the partials of a row: ROWS rows per CTA, each lane of a row's
// 256 / ROWS on every (256 / ROWS)-th partial; the lanes of a warp that share a
// row join by shuffles, the warps in order.  Bound by latency; with the exponentials
// one after another and the target read at the end the loss of 5 tokens (V =
// 50257, d = 2048) took 38.7 us instead of 37.3.
template <int ROWS>
__global__ void __launch_bounds__(256)
    vocab_join_kernel(const float2* part, const float* target_logit, const int32_t* targets, int T, int V, int parts,
                      float z_weight, float* loss, float* lse, int* status) {
  constexpr int GROUPS = 256 / ROWS, AHEAD = 4;
  __shared__ float2 sh[8][ROWS];
  dependency_wait();
  const int r = threadIdx.x % ROWS, g = threadIdx.x / ROWS;
  const int row = blockIdx.x * ROWS + r;
  // what the last step needs is on its way meanwhile (no target: not used)
  const bool writes = threadIdx.x < ROWS && row < T;
  const int t = writes ? __ldg(targets + row) : -1;
  const float target = writes ? __ldg(target_logit + row) : 0.0f;
  // (m, s) of several pairs: the largest m first, then every s against it, so
  // that the exponentials do not wait for each other
  float m = -INFINITY, s = 0.0f;
  auto join = [&](const float2* p, int n) {
    float top = m;
#pragma unroll
    for (int j = 0; j < n; ++j) top = fmaxf(top, p[j].x);
    const float ref = top == -INFINITY ? 0.0f : top;
    s *= exp2_fast(m - ref);
#pragma unroll
    for (int j = 0; j < n; ++j) s = fmaf(p[j].y, exp2_fast(p[j].x - ref), s);
    m = top;
  };
  if (row < T) {
    for (int i0 = g; i0 < parts; i0 += AHEAD * GROUPS) {
      float2 p[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int i = i0 + j * GROUPS;
        p[j] = i < parts ? __ldg(part + (long long)i * T + row) : make_float2(-INFINITY, 0.0f);
      }
      join(p, AHEAD);
    }
  }
  float top = m;
#pragma unroll
  for (int k = ROWS; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  s *= exp2_fast(m - (top == -INFINITY ? 0.0f : top));
  m = top;
#pragma unroll
  for (int k = ROWS; k < 32; k <<= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  if ((threadIdx.x & 31) < ROWS) sh[threadIdx.x >> 5][r] = make_float2(m, s);
  __syncthreads();
  if (!writes) return;
  float2 q[7];
#pragma unroll
  for (int w = 1; w < 8; ++w) q[w - 1] = sh[w][r];
  join(q, 7);
  const float l = fmaf(m, kLn2, fmaf(m, kLn2Lo, log2f(s) * kLn2));  // one rounding at the size of l
  if (t >= V) record_status(status, MOE_ERR_DEVICE_BOUNDS);
  lse[row] = l;
  loss[row] = t >= 0 && t < V ? fmaf(z_weight * l, l, l - target) : 0.0f;
}

// dx = the slabs' sum in their order, four columns per thread (T = 2047, d =
// 1024, three slabs: 5 us)
__global__ void __launch_bounds__(256) vocab_slab_sum_kernel(const float4* slab, int splits, long long n4, uint2* dx) {
  dependency_wait();
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n4; i += (long long)gridDim.x * 256) {
    float4 v = __ldg(slab + i);
    for (int k = 1; k < splits; ++k) {
      const float4 u = __ldg(slab + k * n4 + i);
      v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
    }
    dx[i] = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  }
}

int cdiv_i(long long a, long long b) { return (int)((a + b - 1) / b); }

// m with n / d = (n m) >> 32 for n <= most (0 if there is none of 32 bits):
// m = floor(2^32 / d) + 1 overshoots by at most d / 2^32 per unit of n
unsigned magic_of(unsigned d, unsigned long long most) {
  return d > 1 && most * d < (1ull << 32) ? (unsigned)((1ull << 32) / d + 1) : 0u;
}
void set_tiles(Product& p, int rows, int cols, int k_steps, int splits) {
  p.rows = rows;
  p.cols = cols;
  p.k_steps = k_steps;
  p.splits = splits;
  p.m_tiles = cdiv_i(rows, TILE);
  p.n_tiles = cdiv_i(cols, TILE);
  p.group_m = p.m_tiles < GROUP_M ? p.m_tiles : GROUP_M;
  p.per_group = p.group_m * p.n_tiles;
  p.group_magic = magic_of(p.group_m, p.per_group);
  p.per_group_magic = magic_of(p.per_group, (unsigned long long)p.m_tiles * p.n_tiles);
}

template <int MODE>
cudaError_t launch_gemm(VParams& P, cudaStream_t s, const char* name) {
  auto kern = vocab_gemm_kernel<MODE>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.attrs = attr;
  static std::mutex mu;
  static int resident[64] = {0};
  int clusters;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!resident[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
      if (e != cudaSuccess) return e;
      cfg.gridDim = dim3(device_sm_count() / 2 * 2, 1, 1);
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
      resident[dev] = n > 0 ? n : 1;
    }
    clusters = resident[dev];
  }
  const long long tiles =
      (long long)P.p.m_tiles * P.p.n_tiles * P.p.splits + (long long)P.w.m_tiles * P.w.n_tiles;
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
  if (tiles < clusters) clusters = (int)tiles;
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.stream = s;
  cfg.numAttrs = 2;
  timing_mark(s, name);
  return cudaLaunchKernelEx(&cfg, kern, P);
}

// The time of GRAD's tiles on kPairs pairs, in K steps (0.3 us), with dx's
// contraction in s pieces: the rounds of tile_of; a tile's own epilogue and
// start-up are worth about four steps, the kernel that adds the s slabs twelve
// and its traffic.
constexpr int kPairs = 76;  // of the 152-SM part
constexpr int kTileSteps = 4;
constexpr int kMaxSplits = 16;
int late_rounds(int dx_steps, int dw_steps) { return cdiv_i(dx_steps + kTileSteps, dw_steps + kTileSteps); }
double grad_steps(int T, int d, int piece, int s, bool dw) {
  const long long nx = (long long)cdiv_i(T, TILE) * cdiv_i(d, TILE) * s;
  const long long nw = dw ? (long long)cdiv_i(piece, TILE) * cdiv_i(d, TILE) : 0;
  const int cx = cdiv_i(cdiv_i(piece, BK), s), cw = cdiv_i(T, BK), late = (int)(nx % kPairs);
  const long long alone = late ? (long long)late_rounds(cx, cw) * (kPairs - late) : 0;
  const long long rest = nw > alone ? nw - alone : 0;
  const double rounds_x = (double)cdiv_i(nx, kPairs), rounds_w = (double)cdiv_i(rest, kPairs);
  return rounds_x * (cx + kTileSteps) + rounds_w * (cw + kTileSteps) +
         (s > 1 ? 12.0 + (double)s * T * d / 5.0e5 : 0.0);
}
int dx_splits(int T, int d, int piece, bool dw) {
  int best = 1;
  for (int s = 2; s <= kMaxSplits && s * 8 <= cdiv_i(piece, BK); ++s)
    if (grad_steps(T, d, piece, s, dw) < grad_steps(T, d, piece, best, dw)) best = s;
  return best;
}

struct BwdWs {
  size_t scale, dz, slab, total;
  int piece, pieces, splits;
};
// no batch of up to T tokens keeps more of dz
size_t bwd_dz_limit(int T, int V, int piece_in) {
  const long long all = (long long)cdiv_i(V, TILE) * TILE;
  const long long cols = piece_in > 0 ? vocab_piece(T, V, piece_in) : all;
  size_t n = (size_t)T * cols * 2;
  const size_t limit = (size_t)1 << 30, narrow = (size_t)T * TILE * 2;
  if (piece_in <= 0 && n > limit) n = narrow > limit ? narrow : limit;
  return 256 + up256(n);
}
BwdWs bwd_ws(int T, int d, int V, int piece_in) {
  // (the same splits whether dW is wanted or not: the workspace's size and dx's
  // bits do not depend on it)
  BwdWs w;
  w.piece = vocab_piece(T, V, piece_in);
  w.pieces = cdiv_i(V, w.piece);
  w.splits = dx_splits(T, d, w.piece, true);
  w.scale = 0;
  w.dz = 256;
  w.slab = w.dz + up256((size_t)T * w.piece * 2);
  w.total = w.slab + (w.pieces > 1 || w.splits > 1 ? up256((size_t)w.splits * T * d * 4) : 0);
  return w;
}

}  // namespace

int vocab_piece(int T, int V, int piece) {
  const long long all = (long long)cdiv_i(V, TILE) * TILE;
  long long p = piece;
  if (p <= 0) p = (1LL << 29) / T;  // dz of one piece: 1 GiB
  p = p / TILE * TILE;
  if (p < TILE) p = TILE;
  return (int)(p < all ? p : all);
}

namespace {
// Few tokens: rows of W per tile (a multiple of 8, at most 128) and tiles
void few_tiles(int V, int* rows, int* tiles) {
  const int rounds = cdiv_i(V, 2LL * kPairs * BM);
  *rows = cdiv_i(cdiv_i(V, 2LL * kPairs * rounds), 8) * 8;
  *tiles = cdiv_i(V, *rows);
}
int fwd_parts(int T, int V) {
  if (T > kFewTokens) return 2 * cdiv_i(V, TILE);
  int rows, tiles;
  few_tiles(V, &rows, &tiles);
  return 4 * (tiles < 2 * kPairs ? tiles : 2 * kPairs);
}

cudaError_t launch_few(const VocabArgs& a, float2* part, float* target_logit, int* status, cudaStream_t s) {
  FewParams P;
  std::memset(&P, 0, sizeof(P));
  P.T = a.T;
  P.V = a.V;
  P.n = cdiv_i(a.T, 16) * 16;
  few_tiles(a.V, &P.tile_rows, &P.tiles);
  if (!gemm::encode_2d(&P.w, a.W, a.d, a.V, (uint64_t)a.d * 2, 64, P.tile_rows)) return cudaErrorInvalidValue;
  if (!gemm::encode_2d(&P.x, a.x, a.d, a.T, (uint64_t)a.d * 2, 64, P.n)) return cudaErrorInvalidValue;
  P.k_steps = a.d / BK;
  P.stage_bytes = A_BYTES + P.n * BK * 2;
  P.stages = FEW_RING / P.stage_bytes < FEW_STAGES ? FEW_RING / P.stage_bytes : FEW_STAGES;
  P.targets = a.targets;
  P.part = part;
  P.target_logit = target_logit;
  P.status = status;
  static std::atomic<unsigned long long> devices{0};
  cudaError_t e = allow_smem(vocab_few_kernel, devices, (int)kFewSmem);
  if (e != cudaSuccess) return e;
  timing_mark(s, "vocab_few");
  return launch_pdl(vocab_few_kernel, dim3(fwd_parts(a.T, a.V) / 4), dim3(FEW_THREADS), kFewSmem, s, P);
}
}  // namespace

size_t vocab_fwd_ws_bytes(int T, int d, int V) {
  (void)d;
  return up256((size_t)T * fwd_parts(T, V) * 8) + up256((size_t)T * 4);
}
size_t vocab_bwd_ws_bytes(int T, int d, int V, int piece) { return bwd_ws(T, d, V, piece).total; }

// Few tokens keep four partials per CTA, more of them than the half tiles of
// the other form: the most is at one of the two ends.
size_t vocab_fwd_ws_bytes_up_to(int T, int d, int V) {
  const size_t own = vocab_fwd_ws_bytes(T, d, V);
  const size_t few = T > kFewTokens ? vocab_fwd_ws_bytes(kFewTokens, d, V) : 0;
  return own > few ? own : few;
}

// dz grows with the tokens (up to a piece's limit), but dx's slabs come and go
// with the splits.  Walks down the ranges of tokens in which the tiles and K
// steps and the piece are constant.  Within one the slabs' cost in grad_steps
// grows with the tokens, so the shortest batch has the most splits: its splits
// with the longest batch's rows bound them all.  Ends when even the most splits
// would not need more (8192 tokens: 30 us of host time, 65536: 400).
size_t vocab_bwd_ws_bytes_up_to(int T, int d, int V, int piece_in) {
  size_t most = 0;
  for (int hi = T; hi >= 1;) {
    const int piece = vocab_piece(hi, V, piece_in);
    int lo = (hi - 1) / BK * BK + 1;  // BK divides TILE: one number of row tiles too
    while (vocab_piece(lo, V, piece_in) != piece) ++lo;
    const auto need = [&](int splits) {
      const bool slabs = splits > 1 || piece < V;
      return 256 + up256((size_t)hi * piece * 2) + (slabs ? up256((size_t)splits * hi * d * 4) : 0);
    };
    const size_t n = need(dx_splits(lo, d, piece, true));
    if (n > most) most = n;
    hi = lo - 1;
    // below: no more dz than this (a piece is at most V rounded up, and its dz
    // 1 GiB unless it is 256 columns or the caller's), no more slabs than kMaxSplits
    if (hi >= 1 && bwd_dz_limit(hi, V, piece_in) + up256((size_t)kMaxSplits * hi * d * 4) <= most) break;
  }
  return most;
}

namespace {
bool fill_logits(VParams& P, const VocabArgs& a, int v0, int nv) {
  std::memset(&P, 0, sizeof(P));
  const char* W = static_cast<const char*>(a.W) + (size_t)v0 * a.d * 2;
  if (!gemm::encode_2d(&P.p.a, a.x, a.d, a.T, (uint64_t)a.d * 2, 64, BM)) return false;
  if (!gemm::encode_2d(&P.p.b, W, a.d, nv, (uint64_t)a.d * 2, 64, BM)) return false;
  set_tiles(P.p, a.T, nv, a.d / BK, 1);
  P.targets = a.targets;
  P.v0 = v0;
  P.V = a.V;
  P.z_weight = a.z_weight;
  return true;
}
}  // namespace

cudaError_t launch_cross_entropy(const VocabArgs& a, float* loss, float* lse, void* ws, int* status, cudaStream_t s) {
  const int parts = fwd_parts(a.T, a.V);
  float2* part = static_cast<float2*>(ws);
  float* target_logit = reinterpret_cast<float*>(static_cast<char*>(ws) + up256((size_t)a.T * parts * 8));
  cudaError_t e;
  if (a.T <= kFewTokens) {
    e = launch_few(a, part, target_logit, status, s);
  } else {
    VParams P;
    if (!fill_logits(P, a, 0, a.V)) return cudaErrorInvalidValue;
    P.part = part;
    P.target_logit = target_logit;
    P.status = status;
    e = launch_gemm<LSE>(P, s, "vocab_lse");
  }
  if (e != cudaSuccess) return e;
  timing_mark(s, "vocab_join");
  // the fewer rows, the more threads of each
  const int rows = a.T <= kFewTokens ? 1 : a.T < 32 * 152 ? 4 : 32;
  return launch_pdl(rows == 1 ? vocab_join_kernel<1> : rows == 4 ? vocab_join_kernel<4> : vocab_join_kernel<32>,
                    dim3(cdiv_i(a.T, rows)), dim3(256), 0, s, (const float2*)part, (const float*)target_logit,
                    a.targets, a.T, a.V, parts, a.z_weight, loss, lse, status);
}

cudaError_t launch_cross_entropy_bwd(const VocabArgs& a, const float* lse, const float* dloss, int piece_in, void* dx,
                                     void* dW, void* ws, int* status, cudaStream_t s) {
  const BwdWs w = bwd_ws(a.T, a.d, a.V, piece_in);
  char* base = static_cast<char*>(ws);
  void* dz = base + w.dz;
  const bool slabs = w.pieces > 1 || w.splits > 1;
  float* slab = reinterpret_cast<float*>(base + w.slab);
  float* scale = reinterpret_cast<float*>(base + w.scale);
  cudaError_t e = cudaSuccess;
  for (int p = 0; p < w.pieces; ++p) {
    const int v0 = p * w.piece, nv = a.V - v0 < w.piece ? a.V - v0 : w.piece;
    const char* W = static_cast<const char*>(a.W) + (size_t)v0 * a.d * 2;
    VParams P;
    if (!fill_logits(P, a, v0, nv)) return cudaErrorInvalidValue;
    if (!gemm::encode_store_3d(&P.p.out, dz, w.piece, a.T, 1)) return cudaErrorInvalidValue;
    P.lse = lse;
    P.dloss = dloss;
    P.scale = scale;
    P.status = status;
    e = launch_gemm<DZ>(P, s, "vocab_dz");
    if (e != cudaSuccess) return e;
    VParams Q;
    std::memset(&Q, 0, sizeof(Q));
    const uint64_t dz_row = (uint64_t)w.piece * 2;
    if (dx) {
      if (!gemm::encode_2d(&Q.p.a, dz, w.piece, a.T, dz_row, 64, BM)) return cudaErrorInvalidValue;
      if (!gemm::encode_blocks(&Q.p.b, W, a.d, nv, BK, 2)) return cudaErrorInvalidValue;
      if (!gemm::encode_store_3d(&Q.p.out, dx, a.d, a.T, 1)) return cudaErrorInvalidValue;
      const int steps = cdiv_i(nv, BK);
      set_tiles(Q.p, a.T, a.d, steps, w.splits < steps ? w.splits : steps);
    }
    if (dW) {
      char* out = static_cast<char*>(dW) + (size_t)v0 * a.d * 2;
      if (!gemm::encode_blocks(&Q.w.a, dz, w.piece, a.T, BK, 2)) return cudaErrorInvalidValue;
      if (!gemm::encode_blocks(&Q.w.b, a.x, a.d, a.T, BK, 2)) return cudaErrorInvalidValue;
      if (!gemm::encode_store_3d(&Q.w.out, out, a.d, nv, 1)) return cudaErrorInvalidValue;
      set_tiles(Q.w, nv, a.d, cdiv_i(a.T, BK), 1);
    }
    Q.late_rounds = dx && dW ? late_rounds(cdiv_i(Q.p.k_steps, Q.p.splits), Q.w.k_steps) : 0;
    Q.slab = slabs ? slab : nullptr;
    Q.add = p > 0;
    Q.scale = scale;
    Q.status = status;
    e = launch_gemm<GRAD>(Q, s, "vocab_grad");
    if (e != cudaSuccess) return e;
  }
  if (dx && slabs) {
    const long long n4 = (long long)a.T * a.d / 4;
    long long ctas = (n4 + 255) / 256;
    if (ctas > 8LL * device_sm_count()) ctas = 8LL * device_sm_count();
    timing_mark(s, "vocab_dx_sum");
    return launch_pdl(vocab_slab_sum_kernel, dim3((unsigned)ctas), dim3(256), 0, s, (const float4*)slab, w.splits, n4,
                      static_cast<uint2*>(dx));
  }
  return e;
}

}  // namespace moe
