// Softmax cross entropy of a frozen head over a large vocabulary, with its gradient, without
// keeping the logits.
//
// Mathematics.  z[t][v] = x[t] . W[v]; for a token t with target y and any reference value R,
//   others = sum over v != y of exp(z[t][v] - R),   own = exp(z[t][y] - R),
//   loss = log((others + own) / own) = log1p(others / own),       lse = z[t][y] + loss,
//   dx[t] = g / (others + own) * ( sum over v != y of exp(z[t][v] - R) W[v]  -  others W[y] ).
// The sums do not depend on R, so one pass over pieces of the vocabulary computes both: the
// exponentials of a piece are written as 16-bit values P [tokens][piece], and P . W[piece]
// joins an fp32 sum of dx.  4 M V D operations in all; recomputing the logits for the gradient
// would take 6 M V D.  The target's own term stays out of P: near a sure token
// 1 - own / (others + own) cancels, others / (others + own) does not.
//
// R starts as the target's logit (for half, whose largest value is 65504, the largest of it and
// of 8 other entries' logits).  Only range matters: a bf16 P holds exp(z - R) up to z - R = 88,
// a half one up to 11.  A logit further above R than that is found when it is met: the row's
// largest is recorded, and once the piece's logits are done, the token tiles with such a row take
// them once more with the raised R; the sums taken so far are scaled by exp(R_old - R_new).  R
// never exceeds the largest logit, so the largest term never vanishes.  Exponentials are powers
// of two of z log2(e) - R2 with R2 the reference in those units: the rounding of R2 is common to
// every term and cancels.
//
// Kernels.
//   lm_prep       z[t][y], the tokens that count, R's start
//   lm_gemm       one persistent launch over all pieces: clusters of two CTAs, 2-SM tcgen05.mma
//                 on tiles of 256 x 256, fed by TMA, two accumulators in TMEM.
//       scores    256 tokens x 256 entries: x as A (each token's logits in one TMEM lane, so a
//                 thread owns a row), W as B, both K-major.  The epilogue takes exponentials, row
//                 sums and P (16 bits, through a swizzled box and a TMA store), or, without a
//                 gradient, each half tile's row maximum and sum.
//       gradient  256 features x 256 tokens: A = W[piece] read MN-major, B = P; the contraction
//                 (the piece) is split in `slices` parts with an fp32 sum each when there are too
//                 few tiles for the SMs.
//     A piece's gradient starts when every cluster has finished its scores: a counter in global
//     memory that the clusters wait for, which needs them all resident, so the launch is
//     cooperative.  The next piece's scores need no such wait (P has two buffers), so a cluster
//     that has fewer gradient tiles goes on to more of the scores.
//   lm_finish     each token's totals, loss and lse, and dx = a (sum of the slices) - b W[y],
//                 rounded once to 16 bits
//
// Roundings to 16 bits: P (a relative 2^-9 of each term of the sum, the target's excepted)
// and dx itself; logits, exponentials, sums and statistics are fp32.
//
// Every mbarrier wait is bounded in time; one that gives up sets NF4_ERR_TIMEOUT in the status
// word and the CTA winds down, freeing its TMEM.
#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "lm_loss.cuh"
#include "tc_ptx.cuh"

namespace qnf4 {
namespace {

using namespace tc;

constexpr int kSub = 64;                    // 64 deep: one 128-byte swizzled row of 16-bit values
constexpr int kSubs = 2;                    // sub-blocks per step
constexpr int kStepK = kSub * kSubs;
constexpr int kTile = 256;                  // MMA M (128 rows in each CTA) and N
constexpr int kHalf = 128;
constexpr int kCluster = 2;
constexpr int kSubBytes = kHalf * kSub * 2; // 16 KB: 128 rows of A, or the CTA's half of B
constexpr int kHalfSub = kSubBytes / 2;     // one 64-feature half of an MN-major sub-block
constexpr int kStageBytes = 2 * kSubs * kSubBytes;
constexpr int kStages = 3;
// TMA warp, MMA warp, 8 epilogue warps: two for each 32 TMEM lanes, half of the columns each
// (with 4 warps the epilogue of a 576-deep tile took longer than its products)
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kEpiCols = kTile / 2;
constexpr int kTmemCols = 512;
constexpr int kBoxCols = 32;                // a warp's store box: 32 tokens x 32 values
constexpr int kBoxBytes = 32 * kBoxCols * 2;
constexpr int kBoxes = 2;                   // per epilogue warp
constexpr int kBarFull = 0, kBarEmpty = kStages, kBarAccFull = 2 * kStages, kBarAccEmpty = kBarAccFull + 2,
              kBarDone = kBarAccEmpty + 2, kBarPhase = kBarDone + 1, kBarAck = kBarPhase + 1, kNumBars = kBarAck + 1;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kEpiWarps * kBoxes * kBoxBytes + kNumBars * 8 + 16;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// how far above R a logit may lie, as powers of two: 2^86 leaves the fp32 sums of any vocabulary
// finite; 2^15.9 is below half's 65504
constexpr float kRangeBf16 = 86.0f, kRangeF16 = 15.9f;
constexpr int kSamples = 8;                 // entries whose logits half's R starts from, beside the target

struct LmParams {
  int64_t M, D, V;
  int Mp;               // rows of a buffer of P: M rounded up to whole tiles
  int cols;             // vocabulary entries of a piece (the last may have fewer)
  int c0, c1;           // the pieces of this launch
  int w_row0;           // the first entry that the W maps hold
  int make_scores;      // 0: P is there already, only the gradient is taken (one piece a launch)
  int tiles_t, tiles_d; // token tiles; feature tiles
  int d_steps;          // 128-deep steps of the hidden size
  int slices;           // parts of the gradient's contraction
  int band;             // token tiles of the gradient in bands of `band` (0: token tiles fastest)
  int piece_parts;      // part_sum rows of a piece
  int f16;
  float range;
  const int64_t* targets;   // clean: the target, or -1 for a token that does not count
  float* refs;              // [pieces + 1][M] R, times log2(e); row 0 is the start
  int* piece_ref;           // [pieces] the row of refs that holds R after a piece
  float* spike;             // [pieces][M] largest logit beyond the range in a piece, or -inf
  int* flags;               // [pieces][tiles_t] a row of the tile went beyond the range
  int* any;                 // [pieces] one of them is set
  unsigned* arrived;        // [pieces] the counter of a launch that starts with this piece
  float* part_sum;          // [half vocabulary tile][M]
  float* part_max;          // without a gradient: [half vocabulary tile][M], times log2(e)
  float* acc;               // [slices][M][D]
  int* status;
  uint64_t wait_ns;
  int skip_stage0;
};

struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void advance() {
    if (++s == kStages) s = 0, ph ^= 1u;
  }
};

// One tile's work.
struct Unit {
  int t, f;             // token tile; vocabulary tile of the piece, or feature tile
  int k0;               // first contraction element (of the hidden size, or of the piece)
  int nsub;             // 64-deep sub-blocks
  int slice;
};

// The units of one piece that a cluster takes, in order.  Scores after another piece's gradient:
// the first `extra` clusters have one gradient unit more than the others, which is worth `skew`
// units of scores, so the others go on for that many rounds alone.
struct Piece {
  int v0, cols, tiles_v;
  int n_scores, n_grad, g_steps;
  int full;             // rounds of scores that every cluster takes part in
  int extra;
  __device__ Piece(const LmParams& p, int c, int clusters, int first) {
    v0 = c * p.cols;
    cols = static_cast<int>(min(static_cast<int64_t>(p.cols), p.V - v0));
    tiles_v = (cols + kTile - 1) / kTile;
    n_scores = p.make_scores ? p.tiles_t * tiles_v : 0;
    n_grad = p.tiles_t * p.tiles_d * p.slices;
    g_steps = (cols + kStepK - 1) / kStepK;
    extra = c > first && p.slices > 0 ? n_grad % clusters : 0;
    const int skew = extra > 0 ? (p.cols / kStepK / p.slices + p.d_steps / 2) / p.d_steps : 0;
    const int others = clusters - extra;
    full = skew > 0 ? max(0, (n_scores - others * skew + clusters - 1) / clusters) : (n_scores + clusters - 1) / clusters;
  }
  // The cluster's score unit of round r, or -1.
  __device__ __forceinline__ int score(int r, int cluster, int clusters) const {
    int u;
    if (r < full) u = r * clusters + cluster;
    else if (cluster < extra) return -1;
    else u = full * clusters + (r - full) * (clusters - extra) + cluster - extra;
    return u < n_scores ? u : -1;
  }
};

__device__ __forceinline__ Unit score_unit(const LmParams& p, int u) {
  Unit x;
  x.t = u % p.tiles_t;
  x.f = u / p.tiles_t;
  x.k0 = 0;
  x.nsub = static_cast<int>((p.D + kSub - 1) / kSub);
  x.slice = 0;
  return x;
}

__device__ __forceinline__ Unit grad_unit(const LmParams& p, const Piece& pc, int u) {
  Unit x;
  const int tiles = p.tiles_t * p.tiles_d;
  x.slice = u / tiles;
  u -= x.slice * tiles;
  if (p.band > 0) {
    const int per = p.band * p.tiles_d;
    const int bi = u / per, t0 = bi * p.band;
    const int bt = min(p.band, p.tiles_t - t0);
    const int idx = u - bi * per;
    x.t = t0 + idx % bt;
    x.f = idx / bt;
  } else {
    x.t = u % p.tiles_t;
    x.f = u / p.tiles_t;
  }
  // slices differ by a step at most; none is empty (slices <= g_steps)
  const int s0 = static_cast<int>(static_cast<int64_t>(pc.g_steps) * x.slice / p.slices);
  const int s1 = static_cast<int>(static_cast<int64_t>(pc.g_steps) * (x.slice + 1) / p.slices);
  x.k0 = s0 * kStepK;
  x.nsub = (min(pc.cols, s1 * kStepK) - x.k0 + kSub - 1) / kSub;
  return x;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int f16) {
  uint32_t r;
  if (f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The larger of *a and v (finite or +-inf, never NaN): the order of floats as integers.
__device__ __forceinline__ void atomic_max_float(float* a, float v) {
  if (v >= 0.0f) atomicMax(reinterpret_cast<int*>(a), __float_as_int(v));
  else atomicMin(reinterpret_cast<unsigned*>(a), __float_as_uint(v));
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Maps: x and W for the scores (K-major boxes of 128 rows), W for the gradient (64 features x 64
// entries, MN-major), P as it is stored (boxes of 32 x 32) and read (128 rows).
template <bool kGradient>
__global__ void __launch_bounds__(kThreads, 1)
lm_gemm(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
        const __grid_constant__ CUtensorMap tm_wg, const __grid_constant__ CUtensorMap tm_p,
        const __grid_constant__ CUtensorMap tm_pg, const LmParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const uint32_t boxes = base + kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base_ptr + kStages * kStageBytes + kEpiWarps * kBoxes * kBoxBytes);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kNumBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars) + 1;
  volatile int* raise = reinterpret_cast<volatile int*>(bars + kNumBars) + 2;   // the piece has flags
  auto bar = [&](int i) { return smem_u32(bars + i); };
  auto stage_a = [&](int s) { return base + s * kStageBytes; };
  auto stage_b = [&](int s) { return base + s * kStageBytes + kSubs * kSubBytes; };
  const uint32_t rank = cluster_ctarank();
  auto lead_bar = [&](int i) { return mapa_shared(bar(i), 0); };
  const int cluster = blockIdx.x / kCluster;
  const int clusters = gridDim.x / kCluster;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(kBarAccFull + b), 1);
      mbar_init(bar(kBarAccEmpty + b), kEpiWarps * kCluster);
    }
    mbar_init(bar(kBarDone), 1);
    mbar_init(bar(kBarPhase), 1);
    mbar_init(bar(kBarAck), 1);
    *abort_flag = 0;
    *raise = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_allow_next();
  // TMEM is taken only after the preceding grid has completed (see linear_tc.cu)
  pdl_wait();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity, abort_flag, p.status, p.wait_ns); };

  // Every role walks the same units: each piece's scores, the phase that ends them, the flagged
  // tiles' scores again and their phase, the gradient.  `scores`, `phase` and `grad` return false
  // when a wait gave up.
  unsigned phases = 0;
  bool raised = false;      // the piece has flags (each role's copy, taken at its phase)
  auto walk = [&](auto&& scores, auto&& phase, auto&& grad) {
    for (int c = p.c0; c < p.c1; ++c) {
      const Piece pc(p, c, clusters, p.c0);
      for (int r = 0;; ++r) {
        const int u = pc.score(r, cluster, clusters);
        if (u < 0) break;
        if (!scores(pc, c, score_unit(p, u), false)) return;
      }
      if (!kGradient) continue;
      if (p.make_scores) {
        if (!phase(c, false)) return;
        if (raised) {
          for (int u = cluster; u < pc.n_scores; u += clusters) {
            const Unit un = score_unit(p, u);
            if (__ldcg(p.flags + c * p.tiles_t + un.t) != 0 && !scores(pc, c, un, true)) return;
          }
          if (!phase(c, true)) return;
        }
      }
      for (int u = cluster; u < pc.n_grad; u += clusters)
        if (!grad(pc, c, grad_unit(p, pc, u))) return;
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer, and the CTA's look-out for phases ----------------
      Ring r;
      int64_t issued = 0;
      int64_t lt = 0;
      bool ok = true;
      auto load = [&](const Unit& un, auto&& copy) {
        const int nsteps = (un.nsub + kSubs - 1) / kSubs;
        for (int st = 0; st < nsteps; ++st, r.advance()) {
          if (!wait(kBarEmpty + r.s, r.ph ^ 1u)) return ok = false;
          if (p.skip_stage0 && blockIdx.x == 0 && issued == 0) {   // the stage's waits will run out
            ++issued;
            continue;
          }
          // odd units walk the contraction backwards, so a round starts on what the last one
          // left in L2
          const int kst = (lt & 1) ? nsteps - 1 - st : st;
          const int subs = min(kSubs, un.nsub - kst * kSubs);
          if (rank == 0) mbar_expect_tx(bar(kBarFull + r.s), kCluster * 2 * subs * kSubBytes);
          for (int q = 0; q < subs; ++q)
            copy(stage_a(r.s) + q * kSubBytes, stage_b(r.s) + q * kSubBytes, lead_bar(kBarFull + r.s),
                 un.k0 + (kst * kSubs + q) * kSub);
          ++issued;
        }
        ++lt;
        return true;
      };
      const int half = static_cast<int>(rank) * kHalf;
      walk(
          [&](const Piece& pc, int, const Unit& un, bool) {
            const int t = un.t * kTile + half, v = pc.v0 - p.w_row0 + un.f * kTile + half;
            return load(un, [&](uint32_t a, uint32_t b, uint32_t full, int k) {
              tma_load_2d_pair(a, &tm_x, full, k, t);
              tma_load_2d_pair(b, &tm_w, full, k, v);
            });
          },
          [&](int c, bool again) {
            // every epilogue warp of the launch has arrived: P is written, and who went beyond the
            // range is known
            ++phases;
            const unsigned target = phases * kEpiWarps * gridDim.x;
            const uint64_t t0 = global_ns();
            for (uint32_t i = 1; ld_acquire(p.arrived + p.c0) < target; ++i) {
              __nanosleep(64);
              if ((i & 15u) == 0 && (*abort_flag || global_ns() - t0 > p.wait_ns)) {
                *abort_flag = 1;
                atomicCAS(p.status, 0, static_cast<int>(NF4_ERR_TIMEOUT));
                return ok = false;
              }
            }
            asm volatile("fence.proxy.async;" ::: "memory");   // P's stores before this CTA's TMA loads
            // the issuer has taken the phase before (the epilogue's arrival says so itself)
            if (rank == 0 && phases > 1 && !wait(kBarAck, (phases - 2) & 1u)) return ok = false;
            raised = !again && __ldcg(p.any + c) != 0;
            *raise = raised;
            mbar_arrive(bar(kBarPhase));
            return true;
          },
          [&](const Piece& pc, int c, const Unit& un) {
            const int t = (c & 1) * p.Mp + un.t * kTile + half, f = un.f * kTile + half, v = pc.v0 - p.w_row0;
            return load(un, [&](uint32_t a, uint32_t b, uint32_t full, int k) {
              tma_load_2d_pair(a, &tm_wg, full, f, v + k);
              tma_load_2d_pair(a + kHalfSub, &tm_wg, full, f + 64, v + k);
              tma_load_2d_pair(b, &tm_pg, full, k, t);
            });
          });
      if (ok) {
        for (int k = 0; k < kStages; ++k) {
          if (!wait(kBarEmpty + r.s, r.ph ^ 1u)) break;
          r.advance();
        }
      } else if (rank == 0) {   // let copies in flight land before the CTA exits
        for (int64_t k = 0; k < kStages && k < issued; ++k) {
          if (r.s == 0) r.s = kStages - 1, r.ph ^= 1u;
          else --r.s;
          mbar_drain(bar(kBarFull + r.s), r.ph);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer (even CTA) ----------------
      Ring r;
      int64_t lt = 0;
      auto issue = [&](const Unit& un, bool mn_major) {
        const uint32_t idesc = idesc_16(kTile, kTile, mn_major ? 1u : 0u, p.f16 ? 1u : 0u);
        const int nsteps = (un.nsub + kSubs - 1) / kSubs;
        const uint32_t b = static_cast<uint32_t>(lt) & 1u;
        if (!wait(kBarAccEmpty + b, (static_cast<uint32_t>(lt >> 1) & 1u) ^ 1u)) return false;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + b * kTile;
        for (int st = 0; st < nsteps; ++st, r.advance()) {
          if (!wait(kBarFull + r.s, r.ph)) return false;
          tc_fence_after();
          const int kst = (lt & 1) ? nsteps - 1 - st : st;
          const int subs = min(kSubs, un.nsub - kst * kSubs);
          for (int q = 0; q < subs; ++q)
#pragma unroll
            for (int kk = 0; kk < kSub / 16; ++kk) {
              const uint32_t sa = stage_a(r.s) + q * kSubBytes;
              const uint64_t adesc =
                  mn_major ? smem_desc(sa + kk * 2048, kHalfSub, 1024) : smem_desc(sa + kk * 32, 16, 1024);
              const uint64_t bdesc = smem_desc(stage_b(r.s) + q * kSubBytes + kk * 32, 16, 1024);
              umma_bf16_pair(d_tmem, adesc, bdesc, idesc, (st > 0 || q > 0 || kk > 0) ? 1u : 0u);
            }
          umma_commit_pair_mc(bar(kBarEmpty + r.s), 0x3);
          if (st == nsteps - 1) umma_commit_pair_mc(bar(kBarAccFull + b), 0x3);
        }
        ++lt;
        return true;
      };
      walk([&](const Piece&, int, const Unit& un, bool) { return issue(un, false); },
           [&](int, bool) {
             if (!wait(kBarPhase, (phases++) & 1u)) return false;
             raised = *raise != 0;
             mbar_arrive(bar(kBarAck));
             return true;
           },
           [&](const Piece&, int, const Unit& un) { return issue(un, true); });
      umma_commit_pair_mc(bar(kBarDone), 0x1);
      mbar_drain(bar(kBarDone), 0);
    }
  } else {
    // ---------------- epilogue: each warp on 32 TMEM lanes and half of the columns ----------------
    const int quarter = warp & 3;
    const int lrow = quarter * 32 + lane;
    const int half = (warp - 2) >> 2, cb = half * kEpiCols, ce = cb + kEpiCols;
    const uint32_t my_box = boxes + static_cast<uint32_t>((warp - 2) * kBoxes * kBoxBytes);
    uint32_t nst = 0;
    int64_t lt = 0;
    int ref_row = p.c0 == 0 || !kGradient ? 0 : __ldcg(p.piece_ref + p.c0 - 1);   // R of the piece at hand
    int old_row = ref_row;                                                       // R of the sums so far
    // the accumulator of the next unit, ready
    auto ready = [&](uint32_t* taddr) {
      const uint32_t b = static_cast<uint32_t>(lt) & 1u;
      if (!__all_sync(0xffffffffu, wait(kBarAccFull + b, static_cast<uint32_t>(lt >> 1) & 1u))) return false;
      tc_fence_after();
      *taddr = tmem_base + b * kTile + (static_cast<uint32_t>(quarter * 32) << 16);
      return true;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(lead_bar(kBarAccEmpty + (static_cast<uint32_t>(lt) & 1u)));
      ++lt;
    };
    walk(
        [&](const Piece& pc, int c, const Unit& un, bool again) {
          // lane: one token; columns: vocabulary entries
          uint32_t taddr;
          if (!ready(&taddr)) return false;
          const int t0w = un.t * kTile + static_cast<int>(rank) * kHalf + quarter * 32, t = t0w + lane;
          const int64_t y = t < p.M ? p.targets[t] : -1;
          const bool live = y >= 0;
          const int64_t yc64 = y - pc.v0 - un.f * kTile;
          const int yc = (live && yc64 >= cb && yc64 < ce) ? static_cast<int>(yc64) : -1;
          const int valid = min(kTile, pc.cols - un.f * kTile);
          const bool masked = __any_sync(0xffffffffu, yc >= 0) || valid < ce;
          const int64_t part = (static_cast<int64_t>(c) * p.piece_parts + un.f * 2 + half) * p.M + t;
          const float* ref = p.refs + static_cast<int64_t>(ref_row) * p.M;
          float* spike = p.spike + static_cast<int64_t>(c) * p.M;
          float r2 = 0.0f;
          if (kGradient && t < p.M) {
            r2 = __ldcg(ref + t);
            if (again) r2 = fmaxf(r2, __ldcg(spike + t));
          }
          const uint32_t keep = live ? 0xffffffffu : 0u;
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          // columns at a time in registers: all of them where their maximum comes first; the last
          // load frees the accumulator for the unit after next
          constexpr int kAt = kGradient ? 2 : kEpiCols / 32;
#pragma unroll
          for (int h0 = 0; h0 < kEpiCols / 32; h0 += kAt) {
            uint32_t v[kAt][32];
            const int cp = cb + 32 * h0;
#pragma unroll
            for (int h = 0; h < kAt; ++h) tmem_ld32(taddr + cp + 32 * h, v[h]);
            tmem_ld_wait();
            if (h0 + kAt == kEpiCols / 32) release();
            if (masked) {
#pragma unroll
              for (int h = 0; h < kAt; ++h)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (cp + 32 * h + j == yc || cp + 32 * h + j >= valid) v[h][j] = 0xff800000u;   // -inf
            }
#pragma unroll
            for (int h = 0; h < kAt; ++h)
#pragma unroll
              for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(v[h][j]));
            if (!kGradient) {
              const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
              const float m2 = mx == -INFINITY ? 0.0f : mx * kLog2e;
#pragma unroll
              for (int h = 0; h < kAt; ++h)
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j & 3] += ex2(fmaf(__uint_as_float(v[h][j]), kLog2e, -m2));
              if (t < p.M) {
                p.part_max[part] = mx == -INFINITY ? mx : m2;
                p.part_sum[part] = (s[0] + s[1]) + (s[2] + s[3]);
              }
              return true;
            }
#pragma unroll
            for (int h = 0; h < kAt; ++h, ++nst) {
              const uint32_t box = my_box + (nst & 1u) * kBoxBytes;
              uint32_t o[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float e0 = ex2(fmaf(__uint_as_float(v[h][2 * k]), kLog2e, -r2));
                const float e1 = ex2(fmaf(__uint_as_float(v[h][2 * k + 1]), kLog2e, -r2));
                s[k & 3] += e0;
                s[k & 3] += e1;
                o[k] = pack2(e0, e1, p.f16) & keep;
              }
              if (lane == 0) bulk_wait_read<1>();      // the store that last used this box has read it
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // row `lane` of the box, 16-byte column k, 64-byte swizzle
                const uint32_t col = static_cast<uint32_t>(k) ^ ((static_cast<uint32_t>(lane) >> 1) & 3u);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * (kBoxCols * 2) + col * 16),
                             "r"(o[4 * k]), "r"(o[4 * k + 1]), "r"(o[4 * k + 2]), "r"(o[4 * k + 3])
                             : "memory");
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) {   // (rows past M fill the buffer's last tile with zeros)
                tma_store_2d(&tm_p, box, un.f * kTile + cp + h * kBoxCols, (c & 1) * p.Mp + t0w);
                bulk_commit();
              }
            }
          }
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          if (t < p.M) {
            p.part_sum[part] = live ? (s[0] + s[1]) + (s[2] + s[3]) : 0.0f;
            const float m2 = mx * kLog2e;
            if (live && !again && m2 > r2 + p.range) {
              atomic_max_float(spike + t, m2);
              p.flags[c * p.tiles_t + un.t] = 1;
              p.any[c] = 1;
            }
          }
          return true;
        },
        [&](int c, bool again) {
          if (!again) old_row = ref_row;
          if (again) {   // the raised R, for the pieces after this one
            if (blockIdx.x == 0)
              for (int64_t t = threadIdx.x - 64; t < p.M; t += 32 * kEpiWarps)
                p.refs[(c + 1) * p.M + t] = fmaxf(__ldcg(p.refs + ref_row * p.M + t), __ldcg(p.spike + c * p.M + t));
            ref_row = c + 1;
          }
          if (lane == 0) bulk_wait_all();     // this warp's stores of P are complete
          __syncwarp();
          __threadfence();
          if (lane == 0) atomicAdd(p.arrived + p.c0, 1u);
          const bool got = wait(kBarPhase, (phases++) & 1u);
          if (!__all_sync(0xffffffffu, got)) return false;
          raised = *raise != 0;
          if (blockIdx.x == 0 && threadIdx.x == 64) p.piece_ref[c] = ref_row;
          return true;
        },
        [&](const Piece&, int c, const Unit& un) {
          // lane: one feature; columns: tokens.  The sums so far are in units of 2^-refs[old_row],
          // this piece's in 2^-refs[row]
          uint32_t taddr;
          if (!ready(&taddr)) return false;
          const int row = p.make_scores ? ref_row : c + 1;
          const int before = p.make_scores ? old_row : c;
          const float* r0 = p.refs + static_cast<int64_t>(before) * p.M;
          const float* r1 = p.refs + static_cast<int64_t>(row) * p.M;
          const int64_t f = static_cast<int64_t>(un.f) * kTile + static_cast<int64_t>(rank) * kHalf + lrow;
          float* dst = p.acc + static_cast<int64_t>(un.slice) * p.M * p.D + f;
          const int64_t t0 = static_cast<int64_t>(un.t) * kTile;
#pragma unroll 1
          for (int c0 = cb; c0 < ce && t0 + c0 < p.M; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(taddr + c0, v);
            float old[16];
            if (c > 0) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int64_t t = t0 + c0 + j;
                old[j] = (t < p.M && f < p.D) ? dst[t * p.D] : 0.0f;
                if (row != before && t < p.M) {
                  const float a = __ldcg(r0 + t), b = __ldcg(r1 + t);
                  if (a != b) old[j] *= exp2f(a - b);
                }
              }
            }
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int64_t t = t0 + c0 + j;
              float s = __uint_as_float(v[j]);
              if (c > 0) s += old[j];
              if (t < p.M && f < p.D) dst[t * p.D] = s;
            }
          }
          release();
          return true;
        });
    if (kGradient && lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                 : "memory");
  }
}

__device__ __forceinline__ float lo16(uint32_t w, int f16) {
  return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(w & 0xffffu))) : __uint_as_float(w << 16);
}
__device__ __forceinline__ float hi16(uint32_t w, int f16) {
  return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16))) : __uint_as_float(w & 0xffff0000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The target of a token, or -1 where it does not count.
__device__ __forceinline__ int64_t clean_target(int64_t y, int64_t V, int64_t ignore) {
  return y >= 0 && y < V && y != ignore ? y : -1;
}
// Entry i of the kSamples of a vocabulary.
__device__ __forceinline__ int64_t sample_of(int i, int64_t V) { return V * i / kSamples; }

// Rows of a stored head: out[t][d..d+7] = T16(nf4[code] * a'), the bits nf4_dequantize writes, of
// the targets' rows (0 for a token that does not count) and then of the samples'.
__global__ void lm_stored_rows(const Nf4View W, const DecodeTables tabs, const int64_t* targets, int64_t M, int64_t V,
                               int64_t ignore, int64_t D8, int f16, uint4* out) {
  __shared__ float dyn8[256];
  __shared__ float nf4[16];
  for (int i = threadIdx.x; i < 256; i += blockDim.x) dyn8[i] = tabs.dyn8[i];
  if (threadIdx.x < 16) nf4[threadIdx.x] = tabs.nf4[threadIdx.x];
  __syncthreads();
  pdl_allow_next();
  pdl_wait();
  const float offset = W.dq ? *W.offset : 0.0f;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < (M + kSamples) * D8;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t t = i / D8;
    const int64_t row = t < M ? max(clean_target(targets[t], V, ignore), int64_t(0)) : sample_of(static_cast<int>(t - M), V);
    const int64_t e = row * D8 * 8 + i % D8 * 8;   // 8 elements of one 64-element block
    const float s = block_scale(W, e / kBlock, dyn8, offset);
    const uint32_t q = *reinterpret_cast<const uint32_t*>(W.packed + e / 2);
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t b = q >> (8 * k);
      o[k] = pack2(nf4[(b >> 4) & 15u] * s, nf4[b & 15u] * s, f16);
    }
    out[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__device__ __forceinline__ float dot8(uint4 u, uint4 v, int f16, float s) {
  const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    s = fmaf(lo16(uu[k], f16), lo16(vv[k], f16), s);
    s = fmaf(hi16(uu[k], f16), hi16(vv[k], f16), s);
  }
  return s;
}

constexpr int kPrepThreads = 128;

// One CTA per token: clean[t]; zt[t] = x[t] . W[y] in fp32; R's start (ref, times log2(e), where a
// gradient is asked for: kSample takes the samples' logits too); the pieces' spikes and flags.
// A target outside [0, V) that is not ignore_index sets NF4_ERR_ARG.
// rows: W, or with by_token the decoded rows of the targets and then of the samples.
template <bool kSample>
__global__ void __launch_bounds__(kPrepThreads)
lm_prep(const uint4* x, const uint4* rows, int by_token, const int64_t* targets, int64_t M, int64_t V, int64_t ignore,
        int64_t D8, int f16, int64_t* clean, float* zt, float* ref, float* spike, int* flags, int* any,
        unsigned* arrived, int* piece_ref, int pieces, int tiles_t, int* status) {
  constexpr int kDots = kSample ? 1 + kSamples : 1;
  __shared__ float red[kPrepThreads / 32][kDots];
  pdl_allow_next();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int64_t given = targets[t], y = clean_target(given, V, ignore);
  float s[kDots];
#pragma unroll
  for (int k = 0; k < kDots; ++k) s[k] = 0.0f;
  if (y >= 0) {
    const uint4* a = x + t * D8;
    const uint4* w = rows + (by_token ? t : y) * D8;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < D8; i += kPrepThreads) {
      const uint4 u = a[i];
      s[0] = dot8(u, w[i], f16, s[0]);
      if (kSample) {
#pragma unroll
        for (int k = 0; k < kDots - 1; ++k)
          s[1 + k] = dot8(u, rows[(by_token ? M + k : sample_of(k, V)) * D8 + i], f16, s[1 + k]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kDots; ++k) {
    s[k] = warp_sum(s[k]);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][k] = s[k];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float z = 0.0f, top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kDots; ++k) {
      float v = 0.0f;
      for (int q = 0; q < kPrepThreads / 32; ++q) v += red[q][k];
      if (k == 0) z = v;
      top = fmaxf(top, v);
    }
    clean[t] = y;
    zt[t] = z;
    if (ref != nullptr) ref[t] = (kSample ? top : z) * kLog2e;
    if (y < 0 && given != ignore) atomicCAS(status, 0, static_cast<int>(NF4_ERR_ARG));
  }
  for (int c = threadIdx.x; c < pieces; c += kPrepThreads) {
    spike[static_cast<int64_t>(c) * M + t] = -INFINITY;
    if (t < tiles_t) flags[c * tiles_t + t] = 0;
    if (t == 0) any[c] = 0, arrived[c] = 0, piece_ref[c] = c + 1;
  }
}

struct FinishArgs {
  int64_t M, D8;
  const float* part_sum;    // [parts][M]
  const float* part_max;    // given: each part's sum is relative to it; else to its piece's R
  const float* refs;        // [pieces + 1][M]: R after a piece is row piece_ref[piece], the last what dx's sums are relative to
  const int* piece_ref;
  int parts, piece_parts, pieces;
  const float* zt;
  const int64_t* clean;
  const float* gscale;
  int gscale_per_row;
  float* loss;
  float* lse;
  const float4* acc;        // nullptr: no gradient
  int slices;
  const uint4* rows;
  int by_token, f16;
  uint4* dx;
};
constexpr int kFinThreads = 256, kFinTokens = 4;

// kFinTokens tokens a CTA: each one's totals (64 threads down the parts, 16 bytes of neighbouring
// tokens at a time), loss and lse, then dx of the CTA's share of the features (blockIdx.y):
// dx[t][d] = a (sum of the slices) - b W[y][d], a = g / (others + own), b = others a.
__global__ void __launch_bounds__(kFinThreads) lm_finish(const FinishArgs f) {
  __shared__ float red[kFinThreads / 32][kFinTokens];
  __shared__ float2 coef[kFinTokens];
  __shared__ int64_t target[kFinTokens];
  pdl_allow_next();
  pdl_wait();
  const int k = threadIdx.x % kFinTokens, i0 = threadIdx.x / kFinTokens, warp = threadIdx.x >> 5;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kFinTokens, t = t0 + k;
  const bool in = t < f.M;
  const float z = in ? f.zt[t] : 0.0f;
  float ref = in && f.part_max == nullptr ? f.refs[static_cast<int64_t>(f.piece_ref[f.pieces - 1]) * f.M + t] : z * kLog2e;
  if (f.part_max != nullptr) {
    if (in)
      for (int i = i0; i < f.parts; i += kFinThreads / kFinTokens)
        ref = fmaxf(ref, f.part_max[static_cast<int64_t>(i) * f.M + t]);
#pragma unroll
    for (int o = 16; o >= kFinTokens; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    if ((threadIdx.x & 31) < kFinTokens) red[warp][k] = ref;
    __syncthreads();
    for (int q = 0; q < kFinThreads / 32; ++q) ref = fmaxf(ref, red[q][k]);
    __syncthreads();
  }
  // dx's items of this CTA (8 features of one token each); a thread's first one is gathered while
  // the totals' loads are under way
  const int64_t n = f.M * f.D8;
  const int64_t d0 = f.D8 * blockIdx.y / gridDim.y;
  const int dn = f.acc == nullptr ? 0 : static_cast<int>(f.D8 * (blockIdx.y + 1) / gridDim.y - d0);
  const int items = static_cast<int>(min(static_cast<int64_t>(kFinTokens), f.M - t0)) * dn;
  float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v = u;
  uint4 w = make_uint4(0, 0, 0, 0);
  auto gather = [&](int j) {
    const int tk = j / dn;
    const int64_t d = d0 + j - tk * dn, at = (t0 + tk) * f.D8 + d, y = f.clean[t0 + tk];
    w = f.rows[(f.by_token ? t0 + tk : max(y, int64_t(0))) * f.D8 + d];
    u = f.acc[2 * at], v = f.acc[2 * at + 1];
#pragma unroll 4
    for (int q = 1; q < f.slices; ++q) {
      const float4 a = f.acc[2 * (q * n + at)], b = f.acc[2 * (q * n + at) + 1];
      u.x += a.x, u.y += a.y, u.z += a.z, u.w += a.w;
      v.x += b.x, v.y += b.y, v.z += b.z, v.w += b.w;
    }
  };
  if (threadIdx.x < items) gather(threadIdx.x);
  float s = 0.0f;
  if (in) {
#pragma unroll 4
    for (int i = i0; i < f.parts; i += kFinThreads / kFinTokens) {
      const float q = f.part_sum[static_cast<int64_t>(i) * f.M + t];
      const float r = f.part_max != nullptr ? f.part_max[static_cast<int64_t>(i) * f.M + t]
                                            : f.refs[static_cast<int64_t>(f.piece_ref[i / f.piece_parts]) * f.M + t];
      s += r == ref ? q : q == 0.0f ? 0.0f : q * exp2f(r - ref);
    }
  }
#pragma unroll
  for (int o = 16; o >= kFinTokens; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) < kFinTokens) red[warp][k] = s;
  __syncthreads();
  if (threadIdx.x < kFinTokens) {
    const bool live = in && f.clean[t] >= 0;
    float others = 0.0f;
    for (int q = 0; q < kFinThreads / 32; ++q) others += red[q][k];
    const float d = fmaf(z, kLog2e, -ref);      // log2 of own
    const float own = exp2f(d);
    const float total = others + own;
    // the quotient keeps the digits of a sure token's loss; far below the largest logit own vanishes
    const float l = d > -28.0f ? log1pf(others / own) : fmaf(-kLn2, d, logf(total));
    const float g = !live ? 0.0f : f.gscale == nullptr ? 1.0f : f.gscale[f.gscale_per_row ? t : 0];
    coef[k] = make_float2(g / total, g * (others / total));
    target[k] = live ? f.clean[t] : -1;
    if (in && blockIdx.y == 0) {
      f.loss[t] = live ? l : 0.0f;
      if (f.lse != nullptr) f.lse[t] = live ? z + l : 0.0f;
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < items; j += kFinThreads) {
    if (j != threadIdx.x) gather(j);
    const int tk = j / dn;
    uint4 o = make_uint4(0, 0, 0, 0);
    if (target[tk] >= 0) {
      const float2 c = coef[tk];
      o.x = pack2(c.x * u.x - c.y * lo16(w.x, f.f16), c.x * u.y - c.y * hi16(w.x, f.f16), f.f16);
      o.y = pack2(c.x * u.z - c.y * lo16(w.y, f.f16), c.x * u.w - c.y * hi16(w.y, f.f16), f.f16);
      o.z = pack2(c.x * v.x - c.y * lo16(w.z, f.f16), c.x * v.y - c.y * hi16(w.z, f.f16), f.f16);
      o.w = pack2(c.x * v.z - c.y * lo16(w.w, f.f16), c.x * v.w - c.y * hi16(w.w, f.f16), f.f16);
    }
    f.dx[(t0 + tk) * f.D8 + d0 + j - tk * dn] = o;
  }
}

// ---- host side --------------------------------------------------------------------------

size_t a1024(size_t b) { return (b + 1023) & ~static_cast<size_t>(1023); }

constexpr int64_t kBlockTokens = 8192;              // tokens of one pass over the vocabulary
constexpr int64_t kPieceBytes = 128ll << 20;        // P of one piece at most (two are held)

// Clusters that are resident at once (one CTA an SM); looked up once per device.
int max_clusters() {
  constexpr int kMaxDev = 64;
  static std::atomic<int> cache[kMaxDev];
  int dev = 0;
  cudaGetDevice(&dev);
  const bool slot = dev >= 0 && dev < kMaxDev;
  if (slot && cache[dev].load(std::memory_order_relaxed) > 0) return cache[dev].load(std::memory_order_relaxed);
  int n = 0;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(device_sm_count() / kCluster * kCluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(lm_gemm<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, lm_gemm<true>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return std::max(1, device_sm_count() / kCluster);    // sizes can be asked without a device
  }
  if (slot) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a block of M tokens runs: vocabulary tiles of a piece and parts of the gradient's
// contraction.  Costs are in 128-deep steps of a cluster: for each piece the rounds of gradient
// tiles (and 6 steps for each one's ends), then the scores, which even out what the gradient of
// the piece before left uneven; a phase ends with the last score, so half a tile is lost there.
struct LmPlan {
  int piece_tiles, slices;
};
LmPlan lm_plan(int64_t M, int64_t V, int64_t D, bool stored, bool grad) {
  const int64_t tiles = ceil_div(V, kTile), tt = ceil_div(M, kTile), td = ceil_div(D, kTile);
  const int64_t d_steps = ceil_div(D, kStepK), n = max_clusters();
  int64_t fit = std::max<int64_t>(1, kPieceBytes / (2 * tt * kTile) / kTile);
  if (stored) fit = std::max<int64_t>(1, std::min(fit, 2 * kPieceBytes / (2 * D) / kTile));   // and its decoded copy
  if (!grad) return LmPlan{static_cast<int>(std::min(fit, tiles)), 0};
  LmPlan best{1, 1};
  double best_cost = 1e300;
  const int64_t fewest = ceil_div(tiles, fit);
  for (int64_t pieces = fewest; pieces <= 2 * fewest && pieces <= tiles; ++pieces) {
    const int64_t pt = ceil_div(tiles, pieces), last = tiles - (ceil_div(tiles, pt) - 1) * pt, count = ceil_div(tiles, pt);
    for (int s = 1; s <= 16 && (s == 1 || last * 2 / s >= 8); ++s) {
      const double g = static_cast<double>(ceil_div(pt * 2, s)) + 6.0;        // steps of a gradient tile
      const int64_t grads = tt * td * s;
      const double scores = static_cast<double>(tt * pt) / n * d_steps;
      const double first = static_cast<double>(ceil_div(tt * pt, n)) * d_steps;
      const double middle = std::max(static_cast<double>(grads) / n * g + scores + 0.5 * d_steps,
                                     static_cast<double>(ceil_div(grads, n)) * g);
      const double end = static_cast<double>(ceil_div(grads, n)) * (static_cast<double>(ceil_div(last * 2, s)) + 6.0);
      // each further slice is fp32 sums read and written once more a piece: about 2 steps a round
      const double cost = first + (count - 1) * (middle + 6.0) + end + count * (s - 1) * 2.0 * grads / n / s;
      if (cost < best_cost * 0.995) best = LmPlan{static_cast<int>(pt), s}, best_cost = cost;
    }
  }
  return best;
}

struct LmLayout {
  int64_t Mb, cols, Mp;
  int pieces, tiles, slices;
  bool stream;              // the logits come from lm_stream.cu
  int parts, piece_parts;   // sums a token has, in all and from one piece
  size_t clean, zt, refs, piece_ref, spike, flags, any, arrived, part_sum, part_max, wy, wb, P, acc, total;
  LmLayout(int64_t M, int64_t V, int64_t D, bool stored, bool grad) {
    Mb = std::min(M, kBlockTokens);
    Mp = ceil_div(Mb, kTile) * kTile;
    tiles = static_cast<int>(ceil_div(V, kTile));
    // without a gradient a piece only bounds the decoded copy of a stored head
    const LmPlan plan = grad || stored ? lm_plan(Mb, V, D, stored, grad) : LmPlan{tiles, 0};
    cols = static_cast<int64_t>(plan.piece_tiles) * kTile;
    slices = plan.slices;
    pieces = static_cast<int>(ceil_div(tiles, plan.piece_tiles));
    stream = Mb <= kLmStreamMaxM && D <= kLmStreamMaxD;
    piece_parts = stream ? lm_stream_ctas() : 2 * plan.piece_tiles;
    parts = stream ? pieces * piece_parts : 2 * tiles;
    size_t off = 0;
    auto take = [&](size_t b) {
      const size_t at = off;
      off += a1024(b);
      return at;
    };
    const size_t m = static_cast<size_t>(Mb), np = static_cast<size_t>(pieces);
    clean = take(8 * m);
    zt = take(4 * m);
    refs = take(grad ? 4 * m * (np + 1) : 0);
    piece_ref = take(4 * np);
    spike = take(grad ? 4 * m * np : 0);
    flags = take(grad ? 4 * static_cast<size_t>(Mp / kTile) * np : 0);
    any = take(4 * np);
    arrived = take(4 * np);
    part_sum = take(4 * m * parts);
    part_max = take(grad ? 0 : 4 * m * parts);
    wy = take(stored ? 2 * (m + kSamples) * D : 0);
    wb = take(stored ? 2 * static_cast<size_t>(std::min(cols, V)) * D : 0);
    P = take(grad ? 2 * 2 * static_cast<size_t>(Mp) * cols : 0);
    acc = take(grad ? sizeof(float) * m * D * slices : 0);
    total = off;
  }
};

struct LmMaps {
  CUtensorMap x, w, wg, p, pg;
};

// kGradient: a cooperative launch (its clusters wait for one another), unless it only takes the
// gradient of a P that is there.
template <bool kGradient>
cudaError_t launch_lm_gemm(const LmParams& p, const LmMaps& m, cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [&] {
    attr_err = cudaFuncSetAttribute(lm_gemm<kGradient>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (attr_err != cudaSuccess) return attr_err;
  const int64_t scores = static_cast<int64_t>(p.tiles_t) * (p.cols / kTile);
  const int64_t grads = kGradient ? static_cast<int64_t>(p.tiles_t) * p.tiles_d * p.slices : 0;
  const int64_t clusters = std::min<int64_t>(std::max(p.make_scores ? scores : 0, grads), max_clusters());
  LmParams q = p;
  const WaitSettings ws = take_wait_settings();
  q.wait_ns = ws.wait_ns;
  q.skip_stage0 = ws.skip_stage0;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  if (kGradient && p.make_scores) {
    at[1].id = cudaLaunchAttributeCooperative;
    at[1].val.cooperative = 1;
  } else {
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kCluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  note_launch();
  return cudaLaunchKernelEx(&cfg, lm_gemm<kGradient>, m.x, m.w, m.wg, m.p, m.pg, q);
}

}  // namespace

size_t lm_loss_ws_bytes(int64_t M, int64_t V, int64_t D, bool stored, bool grad) {
  return LmLayout(M, V, D, stored, grad).total;
}

cudaError_t lm_loss(const LmLossArgs& a, void* ws, int* status, cudaStream_t st) {
  const bool grad = a.dx != nullptr, stored = a.w16 == nullptr;
  const LmLayout L(a.M, a.V, a.D, stored, grad);
  char* w = static_cast<char*>(ws);
  auto* clean = reinterpret_cast<int64_t*>(w + L.clean);
  auto* zt = reinterpret_cast<float*>(w + L.zt);
  auto* refs = reinterpret_cast<float*>(w + L.refs);
  auto* spike = reinterpret_cast<float*>(w + L.spike);
  auto* part_sum = reinterpret_cast<float*>(w + L.part_sum);
  auto* part_max = reinterpret_cast<float*>(w + L.part_max);
  auto* acc = reinterpret_cast<float*>(w + L.acc);
  const CUtensorMapDataType dt = a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const int64_t D8 = a.D / 8;
  cudaError_t e = cudaSuccess;
  for (int64_t m0 = 0; m0 < a.M; m0 += L.Mb) {
    const int64_t M = std::min(L.Mb, a.M - m0);
    const char* x = static_cast<const char*>(a.x) + 2 * m0 * a.D;
    const void* rows = a.w16;
    const int f16 = a.f16 ? 1 : 0;
    if (stored) {
      rows = w + L.wy;
      const int64_t ctas = std::min<int64_t>(((M + kSamples) * D8 + 255) / 256, static_cast<int64_t>(device_sm_count()) * 8);
      note_launch();
      if ((e = launch_pdl(lm_stored_rows, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, st, 1, a.W, decode_tables(),
                          a.targets + m0, M, a.V, a.ignore_index, D8, f16, reinterpret_cast<uint4*>(w + L.wy))) !=
          cudaSuccess)
        return e;
    }
    LmParams p{};
    p.M = M;
    p.D = a.D;
    p.V = a.V;
    p.Mp = static_cast<int>(L.Mp);
    p.cols = static_cast<int>(L.cols);
    p.tiles_t = static_cast<int>(ceil_div(M, kTile));
    p.tiles_d = static_cast<int>(ceil_div(a.D, kTile));
    p.d_steps = static_cast<int>(ceil_div(a.D, kStepK));
    p.slices = L.slices;
    p.band = p.tiles_t > 8 && p.tiles_d > 8 ? 8 : 0;
    p.piece_parts = L.piece_parts;
    p.f16 = f16;
    p.range = a.f16 ? kRangeF16 : kRangeBf16;
    p.targets = clean;
    p.refs = refs;
    p.piece_ref = reinterpret_cast<int*>(w + L.piece_ref);
    p.spike = spike;
    p.flags = reinterpret_cast<int*>(w + L.flags);
    p.any = reinterpret_cast<int*>(w + L.any);
    p.arrived = reinterpret_cast<unsigned*>(w + L.arrived);
    p.part_sum = part_sum;
    p.part_max = part_max;
    p.acc = acc;
    p.status = status;
    note_launch();
    if ((e = launch_pdl(grad && a.f16 ? lm_prep<true> : lm_prep<false>, dim3(static_cast<unsigned>(M)), dim3(kPrepThreads),
                        0, st, 1, reinterpret_cast<const uint4*>(x), static_cast<const uint4*>(rows), stored ? 1 : 0,
                        a.targets + m0, M, a.V, a.ignore_index, D8, f16, clean, zt, grad ? refs : nullptr, spike, p.flags,
                        p.any, p.arrived, p.piece_ref, grad ? L.pieces : 0, p.tiles_t, status)) != cudaSuccess)
      return e;
    // The pieces of a stored head are decoded one at a time, and a streamed piece's logits are a
    // launch of their own; otherwise one launch takes them all.
    const int step = stored || L.stream ? 1 : L.pieces;
    for (int c = 0; c < L.pieces; c += step) {
      const int64_t v0 = c * L.cols, cols = std::min(L.cols * step, a.V - v0);
      const void* wc = static_cast<const char*>(a.w16) + 2 * v0 * a.D;
      if (stored) {
        Nf4View part = a.W;
        const int64_t at = v0 * a.D;   // a multiple of 16384: whole nested blocks
        part.packed += at / 2;
        part.absmax = static_cast<const char*>(part.absmax) + at / kBlock * (part.dq ? 1 : 4);
        if (part.dq) part.nested += at / kGroupElems;
        part.numel = cols * a.D;
        wc = w + L.wb;
        if ((e = launch_dequantize(part, w + L.wb, a.f16 ? NF4_F16 : NF4_BF16, st)) != cudaSuccess) return e;
      }
      LmMaps m;
      bool ok = make_map(&m.x, dt, x, a.D, M, 2 * a.D, kSub, kHalf, sw);
      ok = ok && make_map(&m.w, dt, wc, a.D, cols, 2 * a.D, kSub, kHalf, sw);
      m.wg = m.p = m.pg = m.w;
      if (grad) {
        ok = ok && make_map(&m.wg, dt, wc, a.D, cols, 2 * a.D, kSub, kSub, sw);
        ok = ok && make_map(&m.p, dt, w + L.P, L.cols, 2 * L.Mp, 2 * L.cols, kBoxCols, 32, CU_TENSOR_MAP_SWIZZLE_64B);
        ok = ok && make_map(&m.pg, dt, w + L.P, L.cols, 2 * L.Mp, 2 * L.cols, kSub, kHalf, sw);
      }
      if (!ok) return cudaErrorInvalidValue;
      p.c0 = c;
      p.c1 = c + step;
      p.w_row0 = static_cast<int>(v0);
      p.make_scores = L.stream ? 0 : 1;
      if (L.stream) {
        LmStreamArgs q{};
        q.M = static_cast<int>(M);
        q.D = a.D;
        q.cols = cols;
        q.v0 = v0;
        q.x = x;
        q.W = wc;
        q.targets = clean;
        q.range = p.range;
        q.ref = refs + static_cast<int64_t>(c) * M;
        q.ref_next = refs + static_cast<int64_t>(c + 1) * M;
        q.spike = spike + static_cast<int64_t>(c) * M;
        q.flags = p.flags + static_cast<int64_t>(c) * p.tiles_t;
        q.P = w + L.P + 2 * (c & 1) * L.Mp * L.cols;
        q.ldp = L.cols;
        q.part_sum = part_sum + static_cast<int64_t>(c) * L.piece_parts * M;
        q.part_max = part_max + static_cast<int64_t>(c) * L.piece_parts * M;
        if ((e = launch_lm_stream(q, grad, a.f16, st)) != cudaSuccess) return e;
        if (!grad) continue;
        q.redo = 1;
        if ((e = launch_lm_stream(q, true, a.f16, st)) != cudaSuccess) return e;
      }
      if ((e = grad ? launch_lm_gemm<true>(p, m, st) : launch_lm_gemm<false>(p, m, st)) != cudaSuccess) return e;
    }
    FinishArgs f{};
    f.M = M;
    f.D8 = D8;
    f.part_sum = part_sum;
    f.part_max = grad ? nullptr : part_max;
    f.refs = refs;
    f.piece_ref = p.piece_ref;
    f.parts = L.parts;
    f.piece_parts = L.piece_parts;
    f.pieces = L.pieces;
    f.zt = zt;
    f.clean = clean;
    f.gscale = a.grad_scale == nullptr ? nullptr : a.grad_scale + (a.grad_scale_per_row ? m0 : 0);
    f.gscale_per_row = a.grad_scale_per_row;
    f.loss = a.loss + m0;
    f.lse = a.lse == nullptr ? nullptr : a.lse + m0;
    f.acc = grad ? reinterpret_cast<const float4*>(acc) : nullptr;
    f.slices = L.slices;
    f.rows = static_cast<const uint4*>(rows);
    f.by_token = stored ? 1 : 0;
    f.f16 = f16;
    f.dx = reinterpret_cast<uint4*>(static_cast<char*>(a.dx) + 2 * m0 * a.D);
    // few tokens: their features are shared among CTAs, each taking the totals again
    const int64_t gx = (M + kFinTokens - 1) / kFinTokens;
    const int64_t gy = grad ? std::max<int64_t>(1, std::min<int64_t>(4 * device_sm_count() / gx, D8 / 16)) : 1;
    note_launch();
    if ((e = launch_pdl(lm_finish, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(kFinThreads), 0, st, 1,
                        f)) != cudaSuccess)
      return e;
  }
  return cudaGetLastError();
}

}  // namespace qnf4
