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
// R starts as the target's logit (for half, whose largest value is 65504, the larger of it and
// of the logits of the vocabulary's first 256 tokens).  Only range matters: a bf16 P holds
// exp(z - R) up to z - R = 88, a half one up to 11.  A logit further above R than that is found
// by the pass that meets it, which records the row's largest; the token tiles with such a row
// run that piece once more with the raised R, and the sums taken so far are scaled by
// exp(R_old - R_new).  R never exceeds the largest logit, so the largest term never vanishes.
//
// Kernels.
//   lm_target     z[t][y], the tokens that count, R's start
//   lm_gemm<kScores / kMax>  clusters of two CTAs, persistent over tiles of 256 tokens x 256
//                 vocabulary entries: 2-SM tcgen05.mma with x as A (each token's logits in one
//                 TMEM lane, so a thread owns a row), W as B, both K-major through TMA.  The
//                 epilogue takes exponentials, row sums and P (bf16 / half through a swizzled
//                 shared-memory box and a TMA store), or, without a gradient, each tile's row
//                 maximum and sum.
//   lm_gemm<kGrad>   tiles of 256 features x 256 tokens: A = W[piece] read MN-major, B = P;
//                 the contraction (the piece) is split in `slices` parts with an fp32 sum each
//                 when there are too few tiles for the SMs.
//   lm_rows       each token's totals, loss, lse and the two factors of dx
//   lm_dx         dx = a (sum of the slices) - b W[y], rounded once to 16 bits
//
// Roundings to 16 bits: P (a relative 2^-9 of each term of the sum, the target's excepted)
// and dx itself; logits, exponentials, sums and statistics are fp32.
//
// Every mbarrier wait is bounded in time; one that gives up sets NF4_ERR_TIMEOUT in the status
// word and the CTA winds down, freeing its TMEM.
#include <algorithm>

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
constexpr int kThreads = 192;               // TMA warp, MMA warp, 4 epilogue warps
constexpr int kTmemCols = 512;
constexpr int kBoxBytes = 32 * 128;         // a warp's store box: 32 tokens x 64 values
constexpr int kBoxes = 2;                   // per epilogue warp
constexpr int kBarFull = 0, kBarEmpty = kStages, kBarAccFull = 2 * kStages, kBarAccEmpty = kBarAccFull + 2,
              kBarDone = kBarAccEmpty + 2, kNumBars = kBarDone + 1;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 4 * kBoxes * kBoxBytes + kNumBars * 8 + 16;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

constexpr float kLog2e = 1.4426950408889634f;
// how far above R a logit may lie: exp(60) leaves the fp32 sums of any vocabulary finite;
// exp(11) is the largest integer power below half's 65504
constexpr float kRangeBf16 = 60.0f, kRangeF16 = 11.0f;

enum { kScores = 0, kMax = 1, kGrad = 2 };

struct LmParams {
  int64_t M;            // tokens of this block
  int64_t D;            // hidden size
  int64_t cols;         // vocabulary entries of this piece
  int64_t v0;           // the piece's first vocabulary entry
  int red_steps;        // 128-deep steps of the whole contraction
  int64_t red_len;      // contraction length (D, or cols)
  int tiles_t, tiles_f; // token tiles; vocabulary tiles or feature tiles (256)
  int slices;           // kGrad: parts of the contraction
  int band;             // kGrad: token tiles in bands of `band` (0: token tiles fastest)
  int f16;
  int redo;             // kScores: only the token tiles whose flag is set, with the raised R
  int add;              // kGrad: add to the sums of the pieces before
  float range;
  const int64_t* targets;   // clean: the target, or -1 for a token that does not count
  const float* ref;         // [M] R for this piece
  float* ref_next;          // [M] redo: R after this piece
  float* spike;             // [M] largest logit beyond the range in this piece, or -inf
  int* flags;               // [tiles_t] a row of the tile went beyond the range
  float* part_sum;          // [vocabulary tile][M]
  float* part_max;          // kMax: [vocabulary tile][M]
  float* acc;               // kGrad: [slices][M][D]
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

struct Unit {
  int64_t t, f;         // token tile; vocabulary or feature tile
  int64_t k0;           // first contraction element
  int nsub;             // 64-deep sub-blocks
  int slice;
};

template <int MODE>
__device__ __forceinline__ Unit unit_of(const LmParams& p, int64_t u) {
  Unit x;
  x.slice = 0;
  if (MODE == kGrad) {
    const int64_t tiles = static_cast<int64_t>(p.tiles_t) * p.tiles_f;
    x.slice = static_cast<int>(u / tiles);
    u -= x.slice * tiles;
  }
  if (MODE == kGrad && p.band > 0) {
    const int64_t per = static_cast<int64_t>(p.band) * p.tiles_f;
    const int64_t bi = u / per, t0 = bi * p.band;
    const int64_t bt = min(static_cast<int64_t>(p.band), static_cast<int64_t>(p.tiles_t) - t0);
    const int64_t idx = u - bi * per;
    x.t = t0 + idx % bt;
    x.f = idx / bt;
  } else {
    x.t = u % p.tiles_t;
    x.f = u / p.tiles_t;
  }
  int s0 = 0, s1 = p.red_steps;
  if (MODE == kGrad) {   // slices differ by a step at most; none is empty (slices <= red_steps)
    s0 = static_cast<int>(static_cast<int64_t>(p.red_steps) * x.slice / p.slices);
    s1 = static_cast<int>(static_cast<int64_t>(p.red_steps) * (x.slice + 1) / p.slices);
  }
  x.k0 = static_cast<int64_t>(s0) * kStepK;
  const int64_t len = min(p.red_len, static_cast<int64_t>(s1) * kStepK) - x.k0;
  x.nsub = static_cast<int>((len + kSub - 1) / kSub);
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

// tm_a / tm_b: kScores, kMax: x and W[piece] (K-major); kGrad: W[piece] (MN-major) and P.
// tm_p: P as the kScores epilogue stores it.
template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
lm_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
        const __grid_constant__ CUtensorMap tm_p, const LmParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const uint32_t boxes = base + kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base_ptr + kStages * kStageBytes + 4 * kBoxes * kBoxBytes);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kNumBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars) + 1;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  auto stage_a = [&](int s) { return base + s * kStageBytes; };
  auto stage_b = [&](int s) { return base + s * kStageBytes + kSubs * kSubBytes; };
  const uint32_t rank = cluster_ctarank();
  auto lead_bar = [&](int i) { return mapa_shared(bar(i), 0); };
  const int64_t cluster_id = blockIdx.x / kCluster;
  const int64_t n_clusters = gridDim.x / kCluster;
  const int64_t total = static_cast<int64_t>(p.tiles_t) * p.tiles_f * (MODE == kGrad ? p.slices : 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(kBarAccFull + b), 1);
      mbar_init(bar(kBarAccEmpty + b), 4 * kCluster);
    }
    mbar_init(bar(kBarDone), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_allow_next();
  // TMEM is taken only after the preceding grid has completed (see linear_tc.cu)
  pdl_wait();
  if (MODE == kScores && p.redo) {
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; t < p.M;
         t += static_cast<int64_t>(gridDim.x) * kThreads)
      p.ref_next[t] = fmaxf(p.ref[t], p.spike[t]);
  }
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

  // every role walks the same units; a repeated pass leaves out the token tiles without a flag
  auto runs = [&](const Unit& un) { return !(MODE == kScores && p.redo) || p.flags[un.t] != 0; };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      bool ok = true;
      Ring c;
      int64_t issued = 0;
      int64_t lt = 0;
      for (int64_t u = cluster_id; ok && u < total; u += n_clusters) {
        const Unit un = unit_of<MODE>(p, u);
        if (!runs(un)) continue;
        // A rows / B rows of this CTA, as tensor coordinates
        const int t_row = static_cast<int>(un.t * kTile) + static_cast<int>(rank) * kHalf;
        const int f_row = static_cast<int>(un.f * kTile) + static_cast<int>(rank) * kHalf;
        const int nsteps = (un.nsub + kSubs - 1) / kSubs;
        for (int st = 0; st < nsteps; ++st, c.advance()) {
          const int s = c.s;
          if (!mbar_wait(bar(kBarEmpty + s), c.ph ^ 1u, abort_flag, p.status, p.wait_ns)) { ok = false; break; }
          const uint32_t full = lead_bar(kBarFull + s);
          if (p.skip_stage0 && blockIdx.x == 0 && issued == 0) {
            ++issued;
            continue;
          }
          // odd units walk the contraction backwards, so a round starts on what the last one
          // left in L2
          const int kst = (lt & 1) ? nsteps - 1 - st : st;
          const int k0 = static_cast<int>(un.k0) + kst * kStepK;
          const int subs = min(kSubs, un.nsub - kst * kSubs);
          if (rank == 0) mbar_expect_tx(bar(kBarFull + s), kCluster * 2 * subs * kSubBytes);
          for (int q = 0; q < subs; ++q) {
            const uint32_t a = stage_a(s) + q * kSubBytes;
            const uint32_t b = stage_b(s) + q * kSubBytes;
            if (MODE == kGrad) {
              tma_load_2d_pair(a, &tm_a, full, f_row, k0 + q * kSub);
              tma_load_2d_pair(a + kHalfSub, &tm_a, full, f_row + 64, k0 + q * kSub);
              tma_load_2d_pair(b, &tm_b, full, k0 + q * kSub, t_row);
            } else {
              tma_load_2d_pair(a, &tm_a, full, k0 + q * kSub, t_row);
              tma_load_2d_pair(b, &tm_b, full, k0 + q * kSub, f_row);
            }
          }
          ++issued;
        }
        ++lt;
      }
      if (ok) {
        for (int k = 0; k < kStages; ++k) {
          if (!mbar_wait(bar(kBarEmpty + c.s), c.ph ^ 1u, abort_flag, p.status, p.wait_ns)) break;
          c.advance();
        }
      } else if (rank == 0) {
        int ds = c.s;
        uint32_t dph = c.ph;
        for (int64_t k = 0; k < kStages && k < issued; ++k) {
          if (ds == 0) ds = kStages - 1, dph ^= 1u;
          else --ds;
          mbar_drain(bar(kBarFull + ds), dph);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer (even CTA) ----------------
      const uint32_t idesc = idesc_16(kTile, kTile, MODE == kGrad ? 1u : 0u, p.f16 ? 1u : 0u);
      bool ok = true;
      Ring c;
      int64_t lt = 0;
      for (int64_t u = cluster_id; ok && u < total; u += n_clusters) {
        const Unit un = unit_of<MODE>(p, u);
        if (!runs(un)) continue;
        const int nsteps = (un.nsub + kSubs - 1) / kSubs;
        const uint32_t b = static_cast<uint32_t>(lt) & 1u;
        if (!mbar_wait(bar(kBarAccEmpty + b), (static_cast<uint32_t>(lt >> 1) & 1u) ^ 1u, abort_flag, p.status,
                       p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + b * kTile;
        for (int st = 0; st < nsteps; ++st, c.advance()) {
          if (!mbar_wait(bar(kBarFull + c.s), c.ph, abort_flag, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int kst = (lt & 1) ? nsteps - 1 - st : st;
          const int subs = min(kSubs, un.nsub - kst * kSubs);
          for (int q = 0; q < subs; ++q)
#pragma unroll
            for (int kk = 0; kk < kSub / 16; ++kk) {
              const uint32_t sa = stage_a(c.s) + q * kSubBytes;
              const uint64_t adesc = MODE == kGrad ? smem_desc(sa + kk * 2048, kHalfSub, 1024)
                                                   : smem_desc(sa + kk * 32, 16, 1024);
              const uint64_t bdesc = smem_desc(stage_b(c.s) + q * kSubBytes + kk * 32, 16, 1024);
              umma_bf16_pair(d_tmem, adesc, bdesc, idesc, (st > 0 || q > 0 || kk > 0) ? 1u : 0u);
            }
          umma_commit_pair_mc(bar(kBarEmpty + c.s), 0x3);
          if (st == nsteps - 1) umma_commit_pair_mc(bar(kBarAccFull + b), 0x3);
        }
        ++lt;
      }
      umma_commit_pair_mc(bar(kBarDone), 0x1);
      mbar_drain(bar(kBarDone), 0);
    }
  } else {
    // ---------------- epilogue: each warp on its own 32 TMEM lanes ----------------
    const int quarter = warp & 3;
    const int lrow = quarter * 32 + lane;
    const uint32_t my_box = boxes + static_cast<uint32_t>(quarter * kBoxes * kBoxBytes);
    uint32_t nst = 0;
    int64_t lt = 0;
    for (int64_t u = cluster_id; u < total; u += n_clusters) {
      const Unit un = unit_of<MODE>(p, u);
      if (!runs(un)) continue;
      const uint32_t b = static_cast<uint32_t>(lt) & 1u;
      const uint32_t aph = static_cast<uint32_t>(lt >> 1) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarAccFull + b), aph, abort_flag, p.status, p.wait_ns))) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + b * kTile + (static_cast<uint32_t>(quarter * 32) << 16);
      if (MODE == kGrad) {
        // lane: one feature; columns: tokens.  Sums of the pieces before are in units of
        // exp(-ref); this piece's in exp(-ref_next)
        const int64_t f = un.f * kTile + static_cast<int64_t>(rank) * kHalf + lrow;
        float* dst = p.acc + static_cast<int64_t>(un.slice) * p.M * p.D + f;
        const int64_t t0 = un.t * kTile;
#pragma unroll 1
        for (int c0 = 0; c0 < kTile && t0 + c0 < p.M; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(taddr + c0, v);
          float old[16];
          if (p.add) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int64_t t = t0 + c0 + j;
              old[j] = (t < p.M && f < p.D) ? dst[t * p.D] : 0.0f;
              const float r0 = t < p.M ? p.ref[t] : 0.0f, r1 = t < p.M ? p.ref_next[t] : 0.0f;
              if (r0 != r1) old[j] *= __expf(r0 - r1);
            }
          }
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int64_t t = t0 + c0 + j;
            float s = __uint_as_float(v[j]);
            if (p.add) s += old[j];
            if (t < p.M && f < p.D) dst[t * p.D] = s;
          }
        }
      } else {
        // lane: one token; columns: vocabulary entries
        const int64_t t0w = un.t * kTile + static_cast<int64_t>(rank) * kHalf + quarter * 32;
        const int64_t t = t0w + lane;
        const int64_t c_tile = un.f * kTile;                         // first column within the piece
        const int64_t y = t < p.M ? p.targets[t] : -1;
        const bool live = y >= 0;
        const int64_t yc64 = y - p.v0 - c_tile;
        const int yc = (live && yc64 >= 0 && yc64 < kTile) ? static_cast<int>(yc64) : -1;
        const int valid = static_cast<int>(min(static_cast<int64_t>(kTile), p.cols - c_tile));
        const bool masked = __any_sync(0xffffffffu, yc >= 0) || valid < kTile;
        auto mask = [&](uint32_t (&v)[32], int c0) {
          if (masked) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c0 + j == yc || c0 + j >= valid) v[j] = 0xff800000u;   // -inf
          }
        };
        if (MODE == kMax) {
          float mx = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < kTile; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + c0, v);
            tmem_ld_wait();
            mask(v, c0);
#pragma unroll
            for (int j = 0; j < 32; ++j) mx = fmaxf(mx, __uint_as_float(v[j]));
          }
          const float m2 = mx == -INFINITY ? 0.0f : mx * kLog2e;
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
          for (int c0 = 0; c0 < kTile; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + c0, v);
            tmem_ld_wait();
            mask(v, c0);
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j & 3] += ex2(fmaf(__uint_as_float(v[j]), kLog2e, -m2));
          }
          if (t < p.M) {
            p.part_max[un.f * p.M + t] = mx;
            p.part_sum[un.f * p.M + t] = (s[0] + s[1]) + (s[2] + s[3]);
          }
        } else {
          float ref = t < p.M ? p.ref[t] : 0.0f;
          if (p.redo && t < p.M) ref = fmaxf(ref, p.spike[t]);
          const float r2 = ref * kLog2e;
          const uint32_t keep = live ? 0xffffffffu : 0u;
          float mx = -INFINITY;
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
          for (int c0 = 0; c0 < kTile; c0 += 64, ++nst) {
            const uint32_t box = my_box + (nst & 1u) * kBoxBytes;
            if (lane == 0) bulk_wait_read<1>();      // the store that last used this box has read it
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[32];
              tmem_ld32(taddr + c0 + h * 32, v);
              tmem_ld_wait();
              mask(v, c0 + h * 32);
#pragma unroll
              for (int j = 0; j < 32; j += 8) {
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float z0 = __uint_as_float(v[j + 2 * k]), z1 = __uint_as_float(v[j + 2 * k + 1]);
                  mx = fmaxf(mx, fmaxf(z0, z1));
                  const float e0 = ex2(fmaf(z0, kLog2e, -r2)), e1 = ex2(fmaf(z1, kLog2e, -r2));
                  s[k] += e0;
                  s[k] += e1;
                  o[k] = pack2(e0, e1, p.f16) & keep;
                }
                // row `lane` of the box, 16-byte column h * 4 + j / 8, 128-byte swizzle
                const uint32_t col = static_cast<uint32_t>(h * 4 + j / 8) ^ (static_cast<uint32_t>(lane) & 7u);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 128 + col * 16), "r"(o[0]),
                             "r"(o[1]), "r"(o[2]), "r"(o[3])
                             : "memory");
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              // columns past the piece hold zeros up to the next 64
              if (t0w < p.M && c0 < valid) tma_store_2d(&tm_p, box, static_cast<int>(c_tile) + c0, static_cast<int>(t0w));
              bulk_commit();
            }
          }
          if (t < p.M) {
            p.part_sum[un.f * p.M + t] = live ? (s[0] + s[1]) + (s[2] + s[3]) : 0.0f;
            if (live && !p.redo && mx > ref + p.range) {
              atomic_max_float(p.spike + t, mx);
              p.flags[un.t] = 1;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(lead_bar(kBarAccEmpty + b));
      ++lt;
    }
    if (MODE == kScores && lane == 0) bulk_wait_all();
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

// A clean copy of the targets (-1: the token does not count), and the rows of a stored head to
// decode (0 for those).  A target outside [0, V) that is not ignore_index sets NF4_ERR_ARG.
__global__ void lm_clean(const int64_t* targets, int64_t M, int64_t V, int64_t ignore, int64_t* clean, int64_t* ids,
                         int* status) {
  pdl_allow_next();
  pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= M) return;
  const int64_t y = targets[t];
  const bool in = y >= 0 && y < V && y != ignore;
  if (!in && y != ignore) atomicCAS(status, 0, static_cast<int>(NF4_ERR_ARG));
  clean[t] = in ? y : -1;
  ids[t] = in ? y : 0;
}

// The targets' rows of a stored head: out[t][d..d+7] = T16(nf4[code] * a') of row ids[t], the
// bits nf4_dequantize writes.
__global__ void lm_stored_rows(const Nf4View W, const DecodeTables tabs, const int64_t* ids, int64_t M, int64_t D8,
                               int f16, uint4* out) {
  __shared__ float dyn8[256];
  __shared__ float nf4[16];
  for (int i = threadIdx.x; i < 256; i += blockDim.x) dyn8[i] = tabs.dyn8[i];
  if (threadIdx.x < 16) nf4[threadIdx.x] = tabs.nf4[threadIdx.x];
  __syncthreads();
  pdl_allow_next();
  pdl_wait();
  const float offset = W.dq ? *W.offset : 0.0f;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < M * D8;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t e = ids[i / D8] * D8 * 8 + i % D8 * 8;   // 8 elements of one 64-element block
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

// One warp per token: zt[t] = x[t] . W[y] in fp32; R's start (ref[0]); the pieces' spikes.
// rows: W (row y), or with by_token the targets' decoded rows (row t).
__global__ void lm_target(const uint4* x, const uint4* rows, int by_token, const int64_t* clean, int64_t M, int64_t D8,
                          int f16, float* zt, float* ref, float* spike, int pieces) {
  pdl_allow_next();
  pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= M) return;
  const int64_t y = clean[t];
  float s = 0.0f;
  if (y >= 0) {
    const uint4* a = x + t * D8;
    const uint4* w = rows + (by_token ? t : y) * D8;
    float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t i = lane; i < D8; i += 32) {
      const uint4 u = a[i], v = w[i];
      const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q[k] = fmaf(lo16(uu[k], f16), lo16(vv[k], f16), q[k]);
        q[k] = fmaf(hi16(uu[k], f16), hi16(vv[k], f16), q[k]);
      }
    }
    s = (q[0] + q[1]) + (q[2] + q[3]);
  }
  s = warp_sum(s);
  if (lane == 0) {
    zt[t] = s;
    if (ref != nullptr) ref[t] = s;
  }
  for (int c = lane; c < pieces; c += 32) spike[static_cast<int64_t>(c) * M + t] = -INFINITY;
}

// ref[t] = the larger of it and the first vocabulary tile's largest logit.
__global__ void lm_raise_ref(float* ref, const float* part_max, int64_t M) {
  pdl_allow_next();
  pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t < M) ref[t] = fmaxf(ref[t], part_max[t]);
}

// One warp per token: its totals, loss, lse and dx's factors
// coef[t] = {g / (others + own), g others / (others + own)}.
// part_max given: each tile's sum is relative to that maximum; else to the R of its piece
// (refs[piece + 1]), piece_tiles tiles a piece, and the result to the last R.
__global__ void lm_rows(const float* part_sum, const float* part_max, const float* refs, int64_t M, int tiles,
                        int piece_tiles, int pieces, const float* zt, const int64_t* clean, const float* gscale,
                        int gscale_per_row, float* loss, float* lse, float2* coef) {
  pdl_allow_next();
  pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= M) return;
  const bool live = clean[t] >= 0;
  const float z = zt[t];
  float ref;
  float s = 0.0f;
  if (part_max != nullptr) {
    ref = z;
    for (int i = lane; i < tiles; i += 32) ref = fmaxf(ref, part_max[static_cast<int64_t>(i) * M + t]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    for (int i = lane; i < tiles; i += 32) {
      const float q = part_sum[static_cast<int64_t>(i) * M + t];
      if (q != 0.0f) s += q * expf(part_max[static_cast<int64_t>(i) * M + t] - ref);
    }
  } else {
    ref = refs[static_cast<int64_t>(pieces) * M + t];
    for (int i = lane; i < tiles; i += 32) {
      const float r = refs[static_cast<int64_t>(i / piece_tiles + 1) * M + t];
      const float q = part_sum[static_cast<int64_t>(i) * M + t];
      s += r == ref ? q : q * expf(r - ref);
    }
  }
  const float others = warp_sum(s);
  if (lane != 0) return;
  const float own = expf(z - ref);
  const float total = others + own;
  // the quotient keeps the digits of a sure token's loss; far below the largest logit own vanishes
  const float l = z - ref > -20.0f ? log1pf(others / own) : logf(total) + (ref - z);
  loss[t] = live ? l : 0.0f;
  if (lse != nullptr) lse[t] = live ? z + l : 0.0f;
  if (coef != nullptr) {
    const float g = gscale == nullptr ? 1.0f : gscale[gscale_per_row ? t : 0];
    coef[t] = live ? make_float2(g / total, g * (others / total)) : make_float2(0.0f, 0.0f);
  }
}

// dx[t][d..d+7] = a (sum of the slices) - b W[y][d..d+7]; zero for a token that does not count.
__global__ void lm_dx(const float4* acc, int slices, const uint4* rows, int by_token, const int64_t* clean,
                      const float2* coef, int64_t M, int64_t D8, int f16, uint4* dx) {
  pdl_allow_next();
  pdl_wait();
  const int64_t n = M * D8;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t t = i / D8, d = i - t * D8;
    const int64_t y = clean[t];
    uint4 o = make_uint4(0, 0, 0, 0);
    if (y >= 0) {
      const uint4 w = rows[(by_token ? t : y) * D8 + d];
      float4 u = acc[2 * i], v = acc[2 * i + 1];
      for (int q = 1; q < slices; ++q) {
        const float4 a = acc[2 * (q * n + i)], b = acc[2 * (q * n + i) + 1];
        u.x += a.x, u.y += a.y, u.z += a.z, u.w += a.w;
        v.x += b.x, v.y += b.y, v.z += b.z, v.w += b.w;
      }
      const float2 c = coef[t];
      o.x = pack2(c.x * u.x - c.y * lo16(w.x, f16), c.x * u.y - c.y * hi16(w.x, f16), f16);
      o.y = pack2(c.x * u.z - c.y * lo16(w.y, f16), c.x * u.w - c.y * hi16(w.y, f16), f16);
      o.z = pack2(c.x * v.x - c.y * lo16(w.z, f16), c.x * v.y - c.y * hi16(w.z, f16), f16);
      o.w = pack2(c.x * v.z - c.y * lo16(w.w, f16), c.x * v.w - c.y * hi16(w.w, f16), f16);
    }
    dx[i] = o;
  }
}

// ---- host side --------------------------------------------------------------------------

size_t a1024(size_t b) { return (b + 1023) & ~static_cast<size_t>(1023); }

constexpr int64_t kBlockTokens = 8192;              // tokens of one pass over the vocabulary
constexpr int64_t kPieceBytes = 256ll << 20;        // P of one piece

// Vocabulary entries of a piece: P stays within kPieceBytes, the pieces are about equal, and
// each starts at a multiple of 256 (a whole tile; 256 stored rows of a multiple of 64 elements
// are whole nested blocks of the NF4 format).
int64_t piece_cols(int64_t M, int64_t V) {
  const int64_t fit = std::max<int64_t>(kTile, kPieceBytes / (2 * M) / kTile * kTile);
  const int64_t pieces = (V + fit - 1) / fit;
  return ((V + pieces - 1) / pieces + kTile - 1) / kTile * kTile;
}

int max_clusters() { return device_sm_count() / kCluster; }

// Parts of the gradient's contraction: enough that the tiles fill the SMs, each part at least
// eight steps long; among those up to 16 the count whose last round of clusters is fullest.
int grad_slices(int64_t tiles, int64_t cols) {
  const int64_t steps = (cols + kStepK - 1) / kStepK;
  const int64_t n = max_clusters();
  int best = 1;
  double best_cost = 1e30;
  for (int s = 1; s <= 64 && (s == 1 || steps / s >= 8); ++s) {
    const int64_t rounds = (tiles * s + n - 1) / n;
    const double cost = static_cast<double>(rounds) * (static_cast<double>((steps + s - 1) / s) + 6.0);
    if (cost < best_cost * 0.97) best = s, best_cost = cost;
  }
  return best;
}

struct LmLayout {
  int64_t Mb, cols;
  int pieces, tiles, slices, piece_tiles;
  size_t clean, ids, zt, refs, spike, flags, part_sum, part_max, coef, wy, wb, P, acc, total;
  LmLayout(int64_t M, int64_t V, int64_t D, bool stored, bool grad) {
    Mb = std::min(M, kBlockTokens);
    // without a gradient a piece only bounds the decoded copy of a stored head
    cols = grad || stored ? piece_cols(Mb, V) : (V + kTile - 1) / kTile * kTile;
    pieces = static_cast<int>((V + cols - 1) / cols);
    piece_tiles = static_cast<int>(cols / kTile);
    tiles = static_cast<int>((V + kTile - 1) / kTile);
    const int64_t tt = (Mb + kTile - 1) / kTile, ft = (D + kTile - 1) / kTile;
    slices = grad ? grad_slices(tt * ft, V - (pieces - 1) * cols) : 0;   // the last piece is the smallest
    size_t off = 0;
    auto take = [&](size_t b) {
      const size_t at = off;
      off += a1024(b);
      return at;
    };
    const size_t m = static_cast<size_t>(Mb);
    clean = take(8 * m);
    ids = take(8 * m);
    zt = take(4 * m);
    refs = take(4 * m * (pieces + 1));
    spike = take(4 * m * pieces);
    flags = take(sizeof(int) * static_cast<size_t>(tt) * pieces);
    part_sum = take(4 * m * tiles);
    part_max = take(4 * m * (grad ? 1 : tiles));
    coef = take(grad ? 8 * m : 0);
    wy = take(stored ? 2 * m * D : 0);
    wb = take(stored ? 2 * static_cast<size_t>(std::min(cols, V)) * D : 0);
    P = take(grad ? 2 * m * cols : 0);
    acc = take(grad ? sizeof(float) * m * D * slices : 0);
    total = off;
  }
};

template <int MODE>
cudaError_t launch_lm_gemm(const LmParams& p, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& pm,
                           cudaStream_t st) {
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [&] {
    attr_err = cudaFuncSetAttribute(lm_gemm<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (attr_err != cudaSuccess) return attr_err;
  const int64_t units = static_cast<int64_t>(p.tiles_t) * p.tiles_f * (MODE == kGrad ? p.slices : 1);
  const int64_t clusters = std::min<int64_t>(units, max_clusters());
  LmParams q = p;
  const WaitSettings ws = take_wait_settings();
  q.wait_ns = ws.wait_ns;
  q.skip_stage0 = ws.skip_stage0;
  note_launch();
  return launch_pdl(lm_gemm<MODE>, dim3(static_cast<unsigned>(clusters * kCluster)), dim3(kThreads), kSmemBytes, st,
                    kCluster, a, b, pm, q);
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
  auto* ids = reinterpret_cast<int64_t*>(w + L.ids);
  auto* zt = reinterpret_cast<float*>(w + L.zt);
  auto* refs = reinterpret_cast<float*>(w + L.refs);
  auto* spike = reinterpret_cast<float*>(w + L.spike);
  auto* flags = reinterpret_cast<int*>(w + L.flags);
  auto* part_sum = reinterpret_cast<float*>(w + L.part_sum);
  auto* part_max = reinterpret_cast<float*>(w + L.part_max);
  auto* coef = grad ? reinterpret_cast<float2*>(w + L.coef) : nullptr;
  auto* acc = reinterpret_cast<float*>(w + L.acc);
  const CUtensorMapDataType dt = a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const int64_t D8 = a.D / 8;
  cudaError_t e = cudaSuccess;
  for (int64_t m0 = 0; m0 < a.M; m0 += L.Mb) {
    const int64_t M = std::min(L.Mb, a.M - m0);
    const char* x = static_cast<const char*>(a.x) + 2 * m0 * a.D;
    const int tt = static_cast<int>((M + kTile - 1) / kTile);
    note_launch();
    if ((e = launch_pdl(lm_clean, dim3(static_cast<unsigned>((M + 255) / 256)), dim3(256), 0, st, 1, a.targets + m0, M,
                        a.V, a.ignore_index, clean, ids, status)) != cudaSuccess)
      return e;
    const void* rows = a.w16;
    if (stored) {   // the targets' rows of a stored head
      rows = w + L.wy;
      const int64_t ctas = std::min<int64_t>((M * D8 + 255) / 256, static_cast<int64_t>(device_sm_count()) * 8);
      note_launch();
      if ((e = launch_pdl(lm_stored_rows, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, st, 1, a.W, decode_tables(),
                          static_cast<const int64_t*>(ids), M, D8, a.f16 ? 1 : 0,
                          reinterpret_cast<uint4*>(w + L.wy))) != cudaSuccess)
        return e;
    }
    note_launch();
    if ((e = launch_pdl(lm_target, dim3(static_cast<unsigned>((M + 7) / 8)), dim3(256), 0, st, 1,
                        reinterpret_cast<const uint4*>(x), static_cast<const uint4*>(rows), stored ? 1 : 0,
                        static_cast<const int64_t*>(clean), M, D8, a.f16 ? 1 : 0, zt, grad ? refs : nullptr, spike,
                        grad ? L.pieces : 0)) != cudaSuccess)
      return e;
    if (grad && (e = cudaMemsetAsync(flags, 0, sizeof(int) * static_cast<size_t>(tt) * L.pieces, st)) != cudaSuccess)
      return e;
    CUtensorMap xm;
    if (!make_map(&xm, dt, x, a.D, M, 2 * a.D, kSub, kHalf, sw)) return cudaErrorInvalidValue;
    for (int c = 0; c < L.pieces; ++c) {
      const int64_t v0 = c * L.cols, cols = std::min(L.cols, a.V - v0);
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
      CUtensorMap wm, wg, pm, pg;
      bool ok = make_map(&wm, dt, wc, a.D, cols, 2 * a.D, kSub, kHalf, sw);
      if (grad) {
        ok = ok && make_map(&wg, dt, wc, a.D, cols, 2 * a.D, kSub, kSub, sw);
        ok = ok && make_map(&pm, dt, w + L.P, L.cols, M, 2 * L.cols, kSub, 32, sw);
        ok = ok && make_map(&pg, dt, w + L.P, L.cols, M, 2 * L.cols, kSub, kHalf, sw);
      } else {
        wg = pm = pg = wm;
      }
      if (!ok) return cudaErrorInvalidValue;
      LmParams p{};
      p.M = M;
      p.D = a.D;
      p.cols = cols;
      p.v0 = v0;
      p.red_len = a.D;
      p.red_steps = static_cast<int>((a.D + kStepK - 1) / kStepK);
      p.tiles_t = tt;
      p.tiles_f = static_cast<int>((cols + kTile - 1) / kTile);
      p.slices = 1;
      p.f16 = a.f16 ? 1 : 0;
      p.range = a.f16 ? kRangeF16 : kRangeBf16;
      p.targets = clean;
      p.status = status;
      p.part_sum = part_sum + static_cast<int64_t>(c) * L.piece_tiles * M;
      if (!grad) {
        p.part_max = part_max + static_cast<int64_t>(c) * L.piece_tiles * M;
        if ((e = launch_lm_gemm<kMax>(p, xm, wm, pm, st)) != cudaSuccess) return e;
        continue;
      }
      if (c == 0 && a.f16) {   // R's start from the first vocabulary tile too
        LmParams q = p;
        q.tiles_f = 1;
        q.part_max = part_max;
        if ((e = launch_lm_gemm<kMax>(q, xm, wm, pm, st)) != cudaSuccess) return e;
        note_launch();
        if ((e = launch_pdl(lm_raise_ref, dim3(static_cast<unsigned>((M + 255) / 256)), dim3(256), 0, st, 1, refs,
                            static_cast<const float*>(part_max), M)) != cudaSuccess)
          return e;
      }
      p.ref = refs + static_cast<int64_t>(c) * M;
      p.ref_next = refs + static_cast<int64_t>(c + 1) * M;
      p.spike = spike + static_cast<int64_t>(c) * M;
      p.flags = flags + static_cast<int64_t>(c) * tt;
      if ((e = launch_lm_gemm<kScores>(p, xm, wm, pm, st)) != cudaSuccess) return e;
      p.redo = 1;
      if ((e = launch_lm_gemm<kScores>(p, xm, wm, pm, st)) != cudaSuccess) return e;
      LmParams g = p;
      g.red_len = cols;
      g.red_steps = static_cast<int>((cols + kStepK - 1) / kStepK);
      g.tiles_f = static_cast<int>((a.D + kTile - 1) / kTile);
      g.slices = L.slices;
      g.band = g.tiles_t > 8 && g.tiles_f > 8 ? 8 : 0;
      g.add = c > 0 ? 1 : 0;
      g.acc = acc;
      if ((e = launch_lm_gemm<kGrad>(g, wg, pg, pm, st)) != cudaSuccess) return e;
    }
    note_launch();
    if ((e = launch_pdl(lm_rows, dim3(static_cast<unsigned>((M + 7) / 8)), dim3(256), 0, st, 1,
                        static_cast<const float*>(part_sum), grad ? nullptr : static_cast<const float*>(part_max),
                        static_cast<const float*>(refs), M, L.tiles, L.piece_tiles, L.pieces,
                        static_cast<const float*>(zt), static_cast<const int64_t*>(clean),
                        a.grad_scale == nullptr ? nullptr : a.grad_scale + (a.grad_scale_per_row ? m0 : 0),
                        a.grad_scale_per_row, a.loss + m0, a.lse == nullptr ? nullptr : a.lse + m0, coef)) != cudaSuccess)
      return e;
    if (grad) {
      const int64_t n = M * D8;
      const int64_t ctas = std::min<int64_t>((n + 255) / 256, static_cast<int64_t>(device_sm_count()) * 8);
      note_launch();
      if ((e = launch_pdl(lm_dx, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, st, 1,
                          reinterpret_cast<const float4*>(acc), L.slices, static_cast<const uint4*>(rows),
                          stored ? 1 : 0, static_cast<const int64_t*>(clean), static_cast<const float2*>(coef), M, D8,
                          a.f16 ? 1 : 0, reinterpret_cast<uint4*>(static_cast<char*>(a.dx) + 2 * m0 * a.D))) !=
          cudaSuccess)
        return e;
    }
  }
  return cudaGetLastError();
}

}  // namespace qnf4
