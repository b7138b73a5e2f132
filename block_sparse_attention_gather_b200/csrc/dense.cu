// Dense attention of query rows over the video keys and the context keys (tcgen05 + TMEM + TMA),
// and the key ranges it reads.
//
// Spark-H3 blog, section "Spark-Reblock": context/sink tokens stay exact.  Their own queries
// attend every video and context key; the same blog's runs keep the first layer and the warm-up
// steps dense.  Per head h and query row i, over the keys j of the row's two ranges,
//   s_j = sigma q_i . k_j,   out_i = sum_j exp(s_j - lse_i) v_j,   lse_i = log sum_j exp(s_j).
//
// One pass over the keys with a running reference per row (an online softmax):
//   p_j = 2^(s_j log2e - ref),  l = sum p,  O = sum p v,  out = O / l,  lse = (ref + log2 l) ln2.
// ref is the row's maximum over the first two tiles (the first with a live key).  It is raised to
// a later tile's maximum, and O and l rescaled, only when that tile's sum of p reaches 2^8 (or is
// no number): up to there p, rounded to bf16 for the tensor cores, and the fp32 sums keep their
// relative accuracy, so a reference below the true maximum costs none, and the usual tile needs
// no maximum at all.  The scores stay in TMEM until the sum is known, so the tile can be redone.
// A reference at the maximum bounds a tile's sum by 2^7, so large values overflow O at most one
// power of two earlier than they would there (a limit of 2^24 did so from 2^104 on).  A raised
// reference goes 2^16 beyond the maximum, as scores that rose once tend to rise again: 8 heads x
// 8192 x 8192 with scores that rise by 25 nats over the keys take 280 us, 418 if it went to the
// maximum (by 100 nats: 286 and 461; 264 and 277 with the limit of 2^24).  What that costs is the
// lower end: in such rows values under 2^-110 have products below fp32's normal numbers.
//
// One CTA works on one head, one 128-row query tile and one slice of the key tiles.  12 warps:
// 0-3 / 4-7 the softmax groups, which take the even and the odd key tiles (warp w owns TMEM lanes
// 32*(w%4)..), 8 the TMA producer, 9 the MMA issuer, 10 the watch of the loaded tiles.  TMEM
// columns: three S buffers (P is written over S as bf16) and one O for both groups.  S(t + 3) is
// issued behind the PV that reads P(t) in the same buffer, so a group finds the next S of its
// own waiting when it has handed a tile over, and the commit that announces S(t + 3) also tells
// that PV(t) is complete.  The groups hand their tiles over in turn (tile t after tile t - 1):
// only then does a group look at the rows' common reference, which the other may have raised,
// and raise it itself.
//
// Keys beyond a row's ranges are masked to -inf by value, so what they hold (NaN included) does
// not matter; rows of V that no row of the query tile sees are zeroed in shared memory before the
// product, as 0 * NaN would not be 0: those past the hull of the ranges, and, where the ranges of
// neighbouring rows do not touch (padding between segments), those in the gaps.
//
// p is rounded to bf16 because the tensor cores take P and V in one type and V is bf16; a P of two
// bf16 parts would double the second product.  The sums l stay fp32 and take p unrounded.  Against
// 64 bits the relative error of a bf16 output is 2.3e-3, where the rounding of the output alone
// is 1.7e-3.
//
// What bounds it.  Few rows: reading K and V once (24 heads x 60480 keys, one row: 116 us =
// 6.4 TB/s, and 5 us for the join of the slices that the keys are split into).  Many rows, d = 128:
// no unit, but two chains of about the same length.  A key tile takes 1514 cycles (the slope of a
// CTA's cycles over the keys; 1606 with its start and end).  The MMA warp needs nearly all of them,
// 1480 by clock stamps: 1150 to issue the tile's 16 MMAs (which execute in 1024; their operands and
// the loads of K, V take 1280 of shared memory's cycles), 150 for a barrier test that has long come
// true and 180 around them.  A softmax warp has one tile in two such periods and is busy for 2670
// of the 2960 cycles: 1800 to load the scores and exponentiate, 330 for its turn, 230 for the
// reference, 140 to store P, 170 to see S.  The special-function unit works 700 of a period's
// cycles (88 of the 128 exponentials of a row's tile; the others by polynomial), and a scheduler
// issues in half of them (840 instructions a tile).  d = 64: the products halve, the softmax does
// not, and a tile takes 1570 cycles by the stamps.
// 24 heads x 30240 x 30240 take 8.6 to 9.05 ms alone (1305 to 1241 TFLOP/s) and 9.7 to 10.0 ms in
// a loop at the 1000 W power cap (1126 to 1163 TFLOP/s, 1470 MHz); with d = 64 7.7 ms and 8.1 ms.
//
// The steps, on that case unless named: running maximum, pair of query tiles per CTA 10.9 ms;
// no maximum per tile 10.3; registers moved to the softmax warps, polynomial 9.7; tile waits in a
// warp of their own 9.3 (a barrier test takes a few hundred cycles while the MMAs read shared
// memory); one query tile per CTA, three S buffers, common reference 9.5 against 10.6 on one box,
// and packed prompts 58 -> 40 us; late query tiles first 327 -> 310 us (8191 causal rows, in a
// loop); masks over the scores instead of in the exponentials 10.0 -> 9.7.
// Measured and not kept: S in 64-key units (an M = 128 MMA takes 64 cycles for N = 64 too), P
// handed over in halves, CTA pairs with M = 256 (no faster, though they halve the reads of K, V).
//
// Every wait is bounded (see spark_ptx.cuh); on expiry the kernel flags kErrTimeout, drains its
// copies and MMAs, frees TMEM and returns.
#include <atomic>
#include <climits>

#include "spark_kernels.cuh"

namespace spark {

namespace {

constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpTiles = 10;
constexpr int kThreads = 384;                // three warpgroups; warp 11 only gives registers
// Registers a thread: 168 at launch (all the SM has for 384 threads), then moved from the third
// warpgroup to the softmax ones; 2 * kRegsSoftmax + kRegsOther == 3 * kRegsLaunch.  The softmax is
// a few short at its peak: 20 bytes are spilled (24 for d = 64).
constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther == 3 * kRegsLaunch, "register split");
constexpr uint32_t kColO = 384;              // S/P buffers at TMEM columns 0, 128, 256
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxSum = 0x1p8f;            // a tile's sum of p from which the reference is raised
constexpr float kRoom = 16.f;                // powers of two from the maximum to a raised reference
constexpr int kMaxSplits = 64;
constexpr int kPolyEvery = 3;                // every third pair of exponentials by polynomial

template <int D>
struct Cfg {
  static constexpr int kTile = 128 * D * 2;                  // bytes of one Q, K or V tile
  static constexpr int kStages = D == 128 ? 6 : 12;          // what 227 KB hold next to Q
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(1 + kStages) * kTile;
};

template <int kStages>
struct __align__(8) Bars {
  uint64_t qfull, full[kStages], empty[kStages], sfull[3], pready[3], done;
  uint32_t tmem;
  int abort_flag;
};

// The key tiles of a CTA: the hull of its rows' video range, then of their context range, each
// cut into tiles of 128 rows from its own start.
struct Tiles {
  int vb, ve, cb, ce;      // hulls
  int tv;                  // video tiles
  int first, count;        // this CTA's slice of them all

  __device__ __forceinline__ bool video(int t) const { return first + t < tv; }
  __device__ __forceinline__ int row(int t) const {
    const int a = first + t;
    return a < tv ? vb + a * 128 : cb + (a - tv) * 128;
  }
};

// Warp-wide bounded wait (all lanes): true once the phase of `bar` with parity `parity` is
// complete, false after an abort, as mbar_wait.  The lanes test together, so the warp stays
// converged, and only a few tests apart from the abort checks, which read global memory.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t* err, uint64_t limit_ns) {
  constexpr uint32_t kAll = 0xffffffffu;
  if (limit_ns != 0 && __all_sync(kAll, mbar_test(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    bool ok = true;
    if (limit_ns == 0 || globaltimer_ns() - t0 >= limit_ns) {
      flag_error(err, kErrTimeout);
      *abort_flag = 1;
      ok = false;
    } else if (*abort_flag) {
      ok = false;
    } else if (launch_timed_out(err)) {
      *abort_flag = 1;
      ok = false;
    }
    if (!__all_sync(kAll, ok)) return false;
    for (int i = 0; i < 8; ++i)
      if (__all_sync(kAll, mbar_test_sleep(bar, parity, 20000u))) return true;
  }
}

__device__ __forceinline__ bool drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}

// NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 2^a of two values without the special-function unit: 2^a = 2^n 2^f, n the nearest integer
// (taken by adding 1.5 * 2^23, which leaves n in the low bits), 2^f on [-1/2, 1/2] by a degree-4
// polynomial that is 1 at 0, fitted for the least largest relative error (2.9e-6 in fp32; the
// result is rounded to bf16, 2^-8).  Arguments from -127 down give 0 exactly (n = -127 takes the
// exponent of 1.0 away), so that a masked key adds none of its value, however large.  Those from
// 128 on and NaN give anything: `top`, the largest argument so far, tells the caller.
__device__ __forceinline__ void ex2_poly2(uint64_t a2, float& top, float& p0, float& p1) {
  float a0, a1;
  f2_unpack(a2, a0, a1);
  top = max3_nan(top, a0, a1);
  a2 = f2_pack(fmaxf(a0, -127.f), fmaxf(a1, -127.f));
  const uint64_t r2 = f2_add(a2, f2_splat(12582912.f));
  const uint64_t f2 = f2_fma(f2_add(r2, f2_splat(-12582912.f)), f2_splat(-1.f), a2);
  uint64_t y = f2_fma(f2_splat(0.009585382416844368f), f2, f2_splat(0.05590662732720375f));
  y = f2_fma(y, f2, f2_splat(0.24024038016796112f));
  y = f2_fma(y, f2, f2_splat(0.6931241750717163f));
  y = f2_fma(y, f2, f2_splat(1.f));
  float y0, y1, r0, r1;
  f2_unpack(y, y0, y1);
  f2_unpack(r2, r0, r1);
  p0 = __int_as_float(__float_as_int(y0) + (__float_as_int(r0) << 23));
  p1 = __int_as_float(__float_as_int(y1) + (__float_as_int(r1) << 23));
}

// Order of the tiles in the shared-memory ring, that of their first use by the MMA warp:
// K0 K1 K2 V0 K3 V1 K4 ... K(T-1) V(T-4) V(T-3) V(T-2) V(T-1).
__device__ __forceinline__ int slot_k(int t) { return t < 3 ? t : 2 * t - 2; }
__device__ __forceinline__ int slot_v(int t, int T) { return min(2 * t + 3, T + t); }

// 32 columns of this thread's TMEM row without waiting; tmem_wait32 completes it (the registers
// pass through the wait, so that no use moves before it).
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SPARK_R8(0), SPARK_R8(8), SPARK_R8(16), SPARK_R8(24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SPARK_R8(0), SPARK_R8(8)
      : "r"(taddr)
      : "memory");
}
#define SPARK_RW8(b) "+r"(r[b + 0]), "+r"(r[b + 1]), "+r"(r[b + 2]), "+r"(r[b + 3]), \
                     "+r"(r[b + 4]), "+r"(r[b + 5]), "+r"(r[b + 6]), "+r"(r[b + 7])
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : SPARK_RW8(0), SPARK_RW8(8), SPARK_RW8(16), SPARK_RW8(24)
               :
               : "memory");
}

// Bits lo .. hi-1 of 32 (either bound may lie outside).
__device__ __forceinline__ uint32_t bits32(int lo, int hi) {
  auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
  return below(hi) & ~below(lo);
}

// p of 32 scores (raw) as packed bf16 pairs; returns their sum (two partial ones).  One pair in
// kPolyEvery takes the polynomial (its largest argument goes to `top`), the others the
// special-function unit.  A masked score (-inf) gives 0; a row without a live key is known by its
// reference.
__device__ __forceinline__ uint64_t exp32(const uint32_t (&r)[32], uint64_t c2, uint64_t nm2,
                                          float& top, uint32_t (&pk)[16]) {
  uint64_t sum2[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint64_t a2 = f2_fma(f2_pack(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])),
                               c2, nm2);
    float p0, p1;
    if (j % kPolyEvery == kPolyEvery - 1) {
      ex2_poly2(a2, top, p0, p1);
    } else {
      float a0, a1;
      f2_unpack(a2, a0, a1);
      p0 = ex2_approx(a0), p1 = ex2_approx(a1);
    }
    sum2[j & 1] = f2_add(sum2[j & 1], f2_pack(p0, p1));
    pk[j] = pack_bf16(p0, p1);
  }
  return f2_add(sum2[0], sum2[1]);
}

// The tile's 128 scores at `sbuf` -> packed pairs, returning the sum of p, which is no number
// under 2^8 when a score is NaN or its p reaches that.  The load of the second half's columns is
// in flight while the first half's are exponentiated.
__device__ __forceinline__ float exp_tile(uint32_t sbuf, float c, float m, uint32_t (&pk)[4][16]) {
  float top = -INFINITY;
  const uint64_t c2 = f2_splat(c), nm2 = f2_splat(-m);
  uint32_t r[4][32];
  tmem_ld32_issue(sbuf, r[0]);
  tmem_ld32_issue(sbuf + 32, r[1]);
  tmem_wait32(r[0]);
  tmem_wait32(r[1]);
  tmem_ld32_issue(sbuf + 64, r[2]);
  tmem_ld32_issue(sbuf + 96, r[3]);
  uint64_t s = exp32(r[0], c2, nm2, top, pk[0]);
  s = f2_add(s, exp32(r[1], c2, nm2, top, pk[1]));
  tmem_wait32(r[2]);
  tmem_wait32(r[3]);
  s = f2_add(s, exp32(r[2], c2, nm2, top, pk[2]));
  s = f2_add(s, exp32(r[3], c2, nm2, top, pk[3]));
  float s0, s1;
  f2_unpack(s, s0, s1);
  return top < 120.f ? s0 + s1 : INFINITY;
}

// Sets the tile's scores outside columns [lo, hi) to -inf where they stand (a pass of its own, so
// that the exponentials have one form: with a second, masking one the loop outgrew the
// instruction caches).
__device__ __forceinline__ void mask_tile(uint32_t sbuf, int lo, int hi) {
#pragma unroll 1
  for (int cc = 0; cc < 128; cc += 32) {
    uint32_t r[32], q[16];
    tmem_ld32(sbuf + cc, r);
    const uint32_t live = bits32(lo - cc, hi - cc);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        q[j] = live & (1u << (16 * half + j)) ? r[16 * half + j] : 0xff800000u;
      tmem_st16_issue(sbuf + cc + 16 * half, q);
    }
  }
  tmem_wait_st();
}

// Maximum of the tile's scores (raw), NaN if one is.
__device__ __forceinline__ float max_tile(uint32_t sbuf) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int cc = 0; cc < 128; cc += 32) {
    uint32_t r[32];
    tmem_ld32(sbuf + cc, r);
#pragma unroll
    for (int j = 0; j < 32; ++j) mx = max_nan(mx, __uint_as_float(r[j]));
  }
  return mx;
}

// Whether two ranges leave keys between them (they neither overlap nor touch).
__device__ __forceinline__ bool apart(int a0, int a1, int b0, int b1) {
  return a0 < a1 && b0 < b1 && (b0 > a1 || a0 > b1);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attend_dense_kernel(
    const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_kc,
    const __grid_constant__ CUtensorMap map_vc, int nq, int nk, int nc,
    const int4* __restrict__ ranges, int nsplit, void* __restrict__ out, int out_dtype,
    float* __restrict__ lse, float* __restrict__ part, float2* __restrict__ part_ml,
    uint32_t* err, uint64_t wait_ns) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  constexpr int kAtoms = D / 64;
  constexpr uint32_t kAll = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* qst = smem;
  uint8_t* ring = qst + C::kTile;
  __shared__ Bars<kStages> bars;
  __shared__ int s_skip;
  __shared__ int hull[8][4], hull_gaps[8];
  __shared__ float row_ref[128];             // the rows' reference as of the last tile handed over
  __shared__ float first_max[2][128];        // the rows' maxima of each group's first tile
  // sums of the groups' rows, over the query tile once every MMA has read it
  float(*ex_l)[128] = reinterpret_cast<float(*)[128]>(qst);
  volatile int* abort_flag = &bars.abort_flag;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int h = blockIdx.z, split = blockIdx.y;
  // late query tiles first: under causal ranges they have the most keys, and a launch should not
  // end with its longest CTAs (8191 causal rows, 16 heads, in a loop: 327 -> 310 us)
  const int q0 = static_cast<int>(gridDim.x - 1 - blockIdx.x) * 128;

  // This thread's row and its key ranges; rows past nq count as unmasked and are never stored.
  const int grp = (warp >> 2) & 1, q4 = warp & 3;
  const int row = q4 * 32 + lane;
  const int qi = q0 + row;
  const bool live = warp < 8 && qi < nq;
  int4 rg = make_int4(0, INT_MAX, 0, INT_MAX);
  // launched while the kernel before it ends: nothing of global memory is touched up to here
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp < 8) {
    int4 r = make_int4(INT_MAX, 0, INT_MAX, 0);
    if (live) {
      if (ranges != nullptr) rg = ranges[qi];
      rg.x = max(rg.x, 0), rg.y = max(min(rg.y, nk), 0);
      rg.z = max(rg.z, 0), rg.w = max(min(rg.w, nc), 0);
      if (rg.x < rg.y) r.x = rg.x, r.y = rg.y;
      if (rg.z < rg.w) r.z = rg.z, r.w = rg.w;
    }
    const int a = __reduce_min_sync(kAll, r.x), b = __reduce_max_sync(kAll, r.y);
    const int c = __reduce_min_sync(kAll, r.z), e = __reduce_max_sync(kAll, r.w);
    // Whether this row's ranges and those of the last row before it that has any leave keys
    // between them: where none do, the rows see every key between the hull's ends.
    auto gap = [&](int b, int e) {
      const uint32_t before = __ballot_sync(kAll, b < e) & ((1u << lane) - 1);
      const int src = before != 0 ? 31 - __clz(before) : lane;
      return apart(__shfl_sync(kAll, b, src), __shfl_sync(kAll, e, src), b, e);
    };
    const bool gap_v = gap(r.x, r.y), gap_c = gap(r.z, r.w);
    const int gaps = __any_sync(kAll, gap_v || gap_c);
    if (lane == 0) hull[warp][0] = a, hull[warp][1] = b, hull[warp][2] = c, hull[warp][3] = e;
    if (lane == 0) hull_gaps[warp] = gaps;
    if (grp == 0) row_ref[row] = -INFINITY;
  }
  if (tid == 0) {
    s_skip = launch_timed_out(err) ? 1 : 0;               // an earlier CTA gave up
    bars.abort_flag = 0;
    mbar_init(&bars.qfull, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int b = 0; b < 3; ++b) {
      mbar_init(&bars.sfull[b], 1);
      mbar_init(&bars.pready[b], 4 + 1);                  // the group's warps and the tile watch
    }
    mbar_init(&bars.done, 1);
    mbar_fence_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&bars.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = bars.tmem;
  if (s_skip) {                                            // uniform: give back TMEM and leave
    if (warp == kWarpMma) tmem_dealloc(tbase, 512);
    return;
  }
  Tiles tl{INT_MAX, 0, INT_MAX, 0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    tl.vb = min(tl.vb, hull[w][0]), tl.ve = max(tl.ve, hull[w][1]);
    tl.cb = min(tl.cb, hull[w][2]), tl.ce = max(tl.ce, hull[w][3]);
  }
  {
    tl.tv = tl.ve > tl.vb ? (tl.ve - tl.vb + 127) / 128 : 0;
    const long long n = tl.tv + (tl.ce > tl.cb ? (tl.ce - tl.cb + 127) / 128 : 0);
    tl.first = static_cast<int>(n * split / nsplit);
    tl.count = static_cast<int>(n * (split + 1) / nsplit) - tl.first;
  }
  const int T = tl.count;
  // waits of a whole warp for a tile's slot, its S, its P
  auto wait_slot = [&](int i) {
    return wait_warp(&bars.full[i % kStages], (i / kStages) & 1, abort_flag, err, wait_ns);
  };
  auto wait_s = [&](int t) {
    return wait_warp(&bars.sfull[t % 3], (t / 3) & 1, abort_flag, err, wait_ns);
  };
  auto wait_p = [&](int t) {
    return wait_warp(&bars.pready[t % 3], (t / 3) & 1, abort_flag, err, wait_ns);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------------ TMA producer
      int issued = 0;
      if (T > 0) {
        if (elect_one()) {
          tma_prefetch_desc(&map_k);
          tma_prefetch_desc(&map_v);
          mbar_arrive_expect_tx(&bars.qfull, C::kTile);
          for (int a = 0; a < kAtoms; ++a)
            tma_load_3d(qst + a * 16384, &map_q, &bars.qfull, a * 64, q0, h);
        }
        __syncwarp();
        int nk_done = 0, nv_done = 0;                      // K and V tiles issued
        for (int i = 0; i < 2 * T; ++i) {
          const bool is_k = nk_done < T && slot_k(nk_done) == i;
          const int t = is_k ? nk_done++ : nv_done++;
          const int s = i % kStages;
          if (i >= kStages &&
              !wait_warp(&bars.empty[s], ((i / kStages) - 1) & 1, abort_flag, err, wait_ns))
            break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&bars.full[s], C::kTile);
            const CUtensorMap* m = tl.video(t) ? (is_k ? &map_k : &map_v)
                                               : (is_k ? &map_kc : &map_vc);
            for (int a = 0; a < kAtoms; ++a)
              tma_load_3d(ring + s * C::kTile + a * 16384, m, &bars.full[s], a * 64, tl.row(t), h);
          }
          __syncwarp();
          issued = i + 1;
        }
        // every load has landed before the CTA ends (after an abort some were never consumed)
        for (int i = max(0, issued - kStages); i < issued; ++i)
          drain(&bars.full[i % kStages], (i / kStages) & 1);
        drain(&bars.qfull, 0);
      }
    } else if (warp == kWarpMma) {
      // -------------------------------------------------------------------- MMA issuer
      // S(0), S(1), S(2), then per tile O += P V(t) and S(t + 3) over that P (MMAs of one thread
      // execute in order).  One wait a tile, for P and what the tile watch has seen land.
      constexpr uint32_t idS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idO = idesc_bf16(128, D, false, true);
      const uint64_t qd = sdesc_sw128(smem_u32(qst), 16, 1024);
      const uint64_t kd0 = sdesc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t vd0 = sdesc_sw128(smem_u32(ring), 16384, 1024);
      auto mma_s = [&](int t) {                            // one lane
        const int i = slot_k(t);
        const uint64_t kd = kd0 + static_cast<uint64_t>((i % kStages) * (C::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * 16384 + (kk % 4) * 32) / 16;
          mma_ss(tbase + (t % 3) * 128, qd + off, kd + off, idS, kk > 0 ? 1u : 0u);
        }
        tc_commit(&bars.empty[i % kStages]);
      };
      bool ok = T > 0 && wait_warp(&bars.qfull, 0, abort_flag, err, wait_ns);
      for (int t = 0; ok && t < min(T, 3); ++t) {
        if (!(ok = wait_slot(slot_k(t)))) break;
        if (elect_one()) {
          mma_s(t);
          tc_commit(&bars.sfull[t]);
        }
        __syncwarp();
      }
      for (int t = 0; ok && t < T; ++t) {
        if (!(ok = wait_p(t))) break;
        tc_fence_after_sync();
        if (elect_one()) {
          const int i = slot_v(t, T);
          const uint64_t vd = vd0 + static_cast<uint64_t>((i % kStages) * (C::kTile >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tbase + kColO, tbase + (t % 3) * 128 + kk * 8, vd + (kk * 2048) / 16, idO,
                   (kk > 0 || t > 0) ? 1u : 0u);
          tc_commit(&bars.empty[i % kStages]);
          if (t + 3 < T) mma_s(t + 3);
          tc_commit(&bars.sfull[t % 3]);                   // S(t + 3) is there, PV(t) complete
        }
        __syncwarp();
      }
      // every MMA complete: the epilogue reads O, and TMEM is freed after
      if (elect_one()) tc_commit(&bars.done);
      __syncwarp();
      drain(&bars.done, 0);
    } else if (warp == kWarpTiles) {
      // -------------------------------------------------------------------- tile watch
      // Waits for V(t) and K(t + 3) in the MMA warp's stead and arrives at pready for them: a
      // barrier test takes a few hundred cycles while the MMAs read shared memory, and the MMA
      // warp's are all in the way.  Zeros the rows of V that no query row sees: those past the
      // hull that are not past the tensor (those TMA fills with zeros), or all of them where the
      // ranges have gaps.
      bool gaps = false;
      for (int w = 0, v = 0, c = 0; w < 4; ++w) {          // v, c: the last warp with such keys
        gaps |= hull_gaps[w] || apart(hull[v][0], hull[v][1], hull[w][0], hull[w][1]) ||
                apart(hull[c][2], hull[c][3], hull[w][2], hull[w][3]);
        if (hull[w][0] < hull[w][1]) v = w;
        if (hull[w][2] < hull[w][3]) c = w;
      }
      for (int t = 0; t < T; ++t) {
        if (!wait_slot(slot_v(t, T))) break;
        const int y = tl.row(t);
        const bool video = tl.video(t);
        const int end = (video ? tl.ve : tl.ce) - y, rows = (video ? nk : nc) - y;
        if (gaps || (end < 128 && end < rows)) {
          uint8_t* v = ring + (slot_v(t, T) % kStages) * C::kTile;
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {                    // keys y + 32 w .. of the tile
            uint32_t seen = 0;
            for (int i = q0 + lane; i < min(q0 + 128, nq); i += 32) {
              const int4 o = ranges[i];
              const int key = y + 32 * w;
              seen |= bits32(max(video ? o.x : o.z, 0) - key, max(video ? o.y : o.w, 0) - key);
            }
            seen = __reduce_or_sync(kAll, seen);
            if (!(seen >> lane & 1))
              for (int k = 0; k < kAtoms * 8; ++k)
                *reinterpret_cast<uint4*>(v + (k / 8) * 16384 + (32 * w + lane) * 128 +
                                          (k % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (t + 3 < T && !wait_slot(slot_k(t + 3))) break;
        // the phase before has to be over, or this would count for it: S(t) is behind PV(t - 3)
        if (!wait_s(t)) break;
        if (elect_one()) mbar_arrive(&bars.pready[t % 3]);
        __syncwarp();
      }
    }
  } else {
    // -------------------------------------------------------------------- softmax rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t obuf = tbase + lane_off + kColO;
    const float c = kLog2e * rsqrtf(static_cast<float>(D));
    const bool warp_live = __any_sync(kAll, live);         // else nothing of this warp is stored
    float ref = -INFINITY, l = 0.f;                        // log2 units; the group's sum of p
    bool ok = true;
    // The reference to start with: the maximum over both groups' first tiles.
    if (T > 0) {
      float mx = -INFINITY;
      if (grp < T && (ok = wait_s(grp)) && warp_live) {
        tc_fence_after_sync();
        const uint32_t sbuf = tbase + lane_off + grp * 128;
        const int y = tl.row(grp);
        const bool video = tl.video(grp);
        mask_tile(sbuf, (video ? rg.x : rg.z) - y, (video ? rg.y : rg.w) - y);
        mx = c * max_tile(sbuf);
      }
      first_max[grp][row] = mx;
      named_bar_sync(1 + q4, 64);                          // the two groups of this quarter
      ref = max_nan(first_max[0][row], first_max[1][row]);
      if (!(ref < INFINITY)) ref = NAN;                    // a score that nothing compares with
      if (grp == 0) row_ref[row] = ref;
    }
    for (int t = grp; ok && t < T; t += 2) {
      if (!(ok = wait_s(t))) break;
      tc_fence_after_sync();
      const uint32_t sbuf = tbase + lane_off + (t % 3) * 128;
      const int y = tl.row(t);
      const bool video = tl.video(t);
      const int lo = (video ? rg.x : rg.z) - y, hi = (video ? rg.y : rg.w) - y;
      const bool some = max(lo, 0) < min(hi, 128);
      uint32_t pk[4][16];
      if (!__any_sync(kAll, some && warp_live)) {
        // no row of this warp has a key here: zeros, whatever the reference
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[i][j] = 0u;
      } else {
        if (__any_sync(kAll, lo > 0 || hi < 128)) mask_tile(sbuf, lo, hi);
        float sum;
        for (int pass = 0;; ++pass) {
          // no live key yet: every p is (next to) 0
          sum = exp_tile(sbuf, c, ref == -INFINITY ? 0.f : ref, pk);
          if (pass == 0) {
            // The other group hands its tile over first; it may have raised the reference, which
            // what is here then has to follow.
            if (t > 0 && !(ok = wait_p(t - 1))) break;
            const float cur = row_ref[row];
            const bool moved = __float_as_uint(cur) != __float_as_uint(ref);
            if (__any_sync(kAll, moved)) {
              if (moved) l *= ref == -INFINITY ? 1.f : ex2_approx(ref - cur);
              ref = cur;
              continue;
            }
          }
          // the reference is too low, or a row sees its first keys without one
          if (pass == 2 || !__any_sync(kAll, !(sum < kMaxSum) || (ref == -INFINITY && some)))
            break;
          const float mx = max_tile(sbuf) * c;
          const bool grow = !(mx <= ref);                  // a NaN among the scores too
          // a score of +inf leaves no number to compare the others with, and a row that met one, or
          // a NaN, keeps none: its masked tiles (maximum -inf) must not make it a row without keys
          const float room = ref == -INFINITY ? 0.f : kRoom;
          const float next = grow ? (ref == ref && mx < INFINITY ? mx + room : NAN) : ref;
          const float f = grow ? ex2_approx(ref - next) : 1.f;
          ref = next;
          l *= f;
          if (t > 0) {
            // PV(t - 1) is complete when the S behind it, or its place, is announced
            if (!(ok = wait_s(t + 2))) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int cc = 0; cc < D; cc += 16) {
              uint32_t o[16];
              tmem_ld16(obuf + cc, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16_issue(obuf + cc, o);
            }
          }
          row_ref[row] = ref;
          pass = 1;                                        // once more, then it stands
        }
        if (!ok) break;
        l += sum;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_st16_issue(sbuf + 16 * i, pk[i]);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.pready[t % 3]);
    }
    // ---- epilogue: each group's warps store half of the columns
    if (ok && T > 0)
      ok = wait_warp(&bars.done, 0, abort_flag, err, wait_ns);
    {
      const float last = row_ref[row];                     // the tiles are all handed over
      if (__float_as_uint(last) != __float_as_uint(ref))
        l *= ref == -INFINITY ? 1.f : ex2_approx(ref - last);
      ref = last;
    }
    ex_l[grp][row] = l;
    named_bar_sync(1 + q4, 64);                            // the two groups of this quarter
    l = ex_l[0][row] + ex_l[1][row];
    if (ok && warp_live) {
      tc_fence_after_sync();
      const size_t at = static_cast<size_t>(h) * nq + qi;
      const size_t prow = (static_cast<size_t>(h) * nsplit + split) * nq + qi;
      // one slice: the output; several: unnormalised partial sums for the join
      const float inv = nsplit > 1 ? 1.f : 1.f / l;
      const bool none = ref == -INFINITY;                  // no live key: zeros
#pragma unroll
      for (int cc = 0; cc < D / 2; cc += 32) {
        const int col = grp * (D / 2) + cc;
        float o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0.f;
        if (T > 0) {
          uint32_t a[32];
          tmem_ld32(obuf + col, a);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = none ? 0.f : __uint_as_float(a[j]) * inv;
        }
        if (live) {
          if (nsplit > 1 || out_dtype == 1) {
            float4* dst = reinterpret_cast<float4*>(
                nsplit > 1 ? part + prow * D + col : static_cast<float*>(out) + at * D + col);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          } else {
            uint4* dst =
                reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at * D + col);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              dst[j] = make_uint4(pack_bf16(o[8 * j], o[8 * j + 1]),
                                  pack_bf16(o[8 * j + 2], o[8 * j + 3]),
                                  pack_bf16(o[8 * j + 4], o[8 * j + 5]),
                                  pack_bf16(o[8 * j + 6], o[8 * j + 7]));
          }
        }
      }
      if (live && grp == 0) {
        if (nsplit > 1)
          part_ml[prow] = make_float2(ref, l);
        else if (lse != nullptr)
          lse[at] = none ? -INFINITY : (ref + log2f(l)) * kLn2;
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, 512);
  }
}

// Joins the slices of a row: out = sum_s 2^(ref_s - ref) O_s / sum_s 2^(ref_s - ref) l_s with
// ref the largest, in the order of the slices.  One warp per row, D/32 columns per lane; the
// slices' references come a lane each (up to 64), and eight slices' columns are loaded at once
// (one at a time: packed prompts 40 us, one query 137 us; so 37 and 135).
template <int D>
__global__ void __launch_bounds__(256) attend_dense_join_kernel(
    const float* __restrict__ part, const float2* __restrict__ part_ml, int nq, int nsplit,
    long long rows, void* __restrict__ out, int out_dtype, float* __restrict__ lse) {
  constexpr int kPer = D / 32;
  constexpr uint32_t kAll = 0xffffffffu;
  static_assert(kMaxSplits == 64, "two slices a lane");
  // a kernel behind this one may be set up from here on; the attention kernel's partial sums are
  // there after the wait
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const long long r = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (r >= rows) return;
  const size_t base = static_cast<size_t>(r / nq) * nsplit * nq + static_cast<size_t>(r % nq);
  float2 ml[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = lane + 32 * i;
    ml[i] = s < nsplit ? part_ml[base + static_cast<size_t>(s) * nq] : make_float2(-INFINITY, 0.f);
  }
  float m = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  float w[2], l = 0.f, acc[kPer] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // a slice without a live key has no reference, and zeros
    w[i] = ml[i].x == -INFINITY ? 0.f : ex2_approx(ml[i].x - m);
    ml[i].y *= w[i];
  }
  for (int s0 = 0; s0 < nsplit; s0 += 8) {
    float v[8][kPer];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = min(s0 + j, nsplit - 1);
      const float* src = part + (base + static_cast<size_t>(s) * nq) * D + lane * kPer;
      if constexpr (kPer == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[j][0] = f.x, v[j][1] = f.y, v[j][2] = f.z, v[j][3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        v[j][0] = f.x, v[j][1] = f.y;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = s0 + j;
      const float ws = __shfl_sync(kAll, s < 32 ? w[0] : w[1], s & 31);
      const float ls = __shfl_sync(kAll, s < 32 ? ml[0].y : ml[1].y, s & 31);
      if (s >= nsplit) break;                              // uniform
      l += ls;
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(ws, v[j][k], acc[k]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t at = static_cast<size_t>(r) * D + lane * kPer;
#pragma unroll
  for (int j = 0; j < kPer; j += 2) {
    if (out_dtype == 1)
      *reinterpret_cast<float2*>(static_cast<float*>(out) + at + j) =
          make_float2(acc[j] * inv, acc[j + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(out) + at + j) =
          pack_bf16(acc[j] * inv, acc[j + 1] * inv);
  }
  if (lane == 0 && lse != nullptr) lse[r] = (m + log2f(l)) * kLn2;
}

// Slices of the key tiles per query tile: the count with the least estimated time on 148 SMs, one
// CTA each.  A tile (0.9 us) is taken as 1 unit, a CTA's start and end as 4, the join kernel as 5
// plus the partial sums' traffic.
int attend_dense_splits(int H, int nq, int nk, int nc, int d) {
  constexpr int kSms = 148;
  const long long qt = (static_cast<long long>(nq) + 127) / 128;
  const long long units = static_cast<long long>(H) * qt;
  const long long T = (static_cast<long long>(nk) + 127) / 128 + (nc + 127) / 128;
  int best = 1;
  double least = 0;
  for (int s = 1; s <= kMaxSplits && (s == 1 || 2 * s <= T); ++s) {
    const long long waves = (units * s + kSms - 1) / kSms;
    const double bytes = static_cast<double>(H) * nq * d * 8.0 * s;
    if (s > 1 && bytes > 512e6) break;
    const double cost = static_cast<double>(waves) *
                            (static_cast<double>((T + s - 1) / s) + 4) +
                        (s > 1 ? 5 + bytes / 4e6 : 0);
    if (s == 1 || cost < least) least = cost, best = s;
  }
  return best;
}

size_t attend_dense_workspace(int H, int nq, int nk, int nc, int d) {
  const int s = attend_dense_splits(H, nq, nk, nc, d);
  if (s == 1) return 256;
  const size_t rows = static_cast<size_t>(H) * nq * s;
  return (rows * d * 4 + 255) / 256 * 256 + (rows * 8 + 255) / 256 * 256;
}

template <int D>
static cudaError_t launch_dense_t(const DenseMaps& m, int H, int nq, int nk, int nc,
                                  const int32_t* ranges, int nsplit, void* out, int out_dtype,
                                  float* lse, float* part, float2* ml, uint32_t* err,
                                  cudaStream_t s) {
  auto kern = attend_dense_kernel<D>;
  constexpr size_t smem = Cfg<D>::kSmem;
  // The kernel's attributes are set once per device (bit per device; every thread that finds the
  // bit clear sets the same values).
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit == 0 || !(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    // The register split would wait for ever for registers that a launch with fewer does not have:
    // a compiler that gives the kernel fewer than it may use gets an error here.
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((nq + 127) / 128, nsplit, H);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, m.q, m.k, m.v, m.kc, m.vc, nq, nk, nc,
                            reinterpret_cast<const int4*>(ranges), nsplit, out, out_dtype, lse,
                            part, ml, err, wait_limit_ns());
}

// The join's launch overlaps the attention kernel's end, which it waits for (asking for it any
// earlier, from the attention kernel's start, measured 8% slower on packed prompts); a kernel
// behind the join, such as the next attention, is set up while it runs (77 rows x 1101 keys, back
// to back: 14.5 -> 12.0 us).
template <int D>
static cudaError_t launch_join_t(const float* part, const float2* ml, int nq, int nsplit,
                                 long long rows, void* out, int out_dtype, float* lse,
                                 cudaStream_t s) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_dense_join_kernel<D>, part, ml, nq, nsplit, rows, out,
                            out_dtype, lse);
}

cudaError_t launch_attend_dense(const DenseMaps& maps, int H, int nq, int nk, int nc, int d,
                                const int32_t* ranges, void* out, int out_dtype, float* lse,
                                void* workspace, uint32_t* err, cudaStream_t s) {
  const int nsplit = attend_dense_splits(H, nq, nk, nc, d);
  const long long rows = static_cast<long long>(H) * nq;
  float* part = static_cast<float*>(workspace);
  const size_t part_bytes = (static_cast<size_t>(rows) * nsplit * d * 4 + 255) / 256 * 256;
  float2* ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + part_bytes);
  cudaError_t e;
  e = d == 128 ? launch_dense_t<128>(maps, H, nq, nk, nc, ranges, nsplit, out, out_dtype, lse, part,
                                     ml, err, s)
               : launch_dense_t<64>(maps, H, nq, nk, nc, ranges, nsplit, out, out_dtype, lse, part,
                                    ml, err, s);
  if (e != cudaSuccess || nsplit == 1) return e;
  return d == 128 ? launch_join_t<128>(part, ml, nq, nsplit, rows, out, out_dtype, lse, s)
                  : launch_join_t<64>(part, ml, nq, nsplit, rows, out, out_dtype, lse, s);
}

// ------------------------------------------------------------------------------ key ranges

// One thread per row, a binary search over the segments' offsets (which stay in L1) and one
// 16-byte store: bound by latency.
// Row i of segment b (the one whose queries q_offsets[b] .. q_offsets[b+1]-1 hold i): the whole
// of the segment's video keys and of its context keys, the latter ended at
// max(prefix_b, i - first + 1 + context - queries) when causal.  Rows of no segment are empty.
__global__ void __launch_bounds__(256) attend_ranges_kernel(
    int nq, int nseg, const int32_t* __restrict__ q_offsets,
    const int32_t* __restrict__ k_offsets, const int32_t* __restrict__ c_offsets,
    const int32_t* __restrict__ prefix, int causal, int4* __restrict__ ranges, uint32_t* err) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= nq) return;
  // the last b with q_offsets[b] <= i
  int lo = 0, hi = nseg + 1;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;        // lo + hi passes 2^31 at 2^30 segments
    if (q_offsets[mid] <= i) lo = mid + 1; else hi = mid;
  }
  const int b = lo - 1;
  int4 r = make_int4(0, 0, 0, 0);
  if (b >= 0 && b < nseg) {
    const int q0 = q_offsets[b], q1 = q_offsets[b + 1];
    bool bad = false;
    if (k_offsets != nullptr) {
      r.x = k_offsets[b], r.y = k_offsets[b + 1];
      bad |= r.x < 0 || r.y < r.x;
    }
    if (c_offsets != nullptr) {
      const int c0 = c_offsets[b], c1 = c_offsets[b + 1];
      bad |= c0 < 0 || c1 < c0;
      r.z = c0, r.w = c1;
      if (causal) {
        long long end = static_cast<long long>(i) - q0 + 1 + (static_cast<long long>(c1) - c0) -
                        (static_cast<long long>(q1) - q0);
        if (prefix != nullptr) end = max(end, static_cast<long long>(prefix[b]));
        end = min(max(end, 0ll), static_cast<long long>(c1) - c0);
        r.w = static_cast<int>(c0 + end);
      }
    }
    if (bad) {
      r = make_int4(0, 0, 0, 0);
      flag_error(err, kErrOffsets);
    }
  }
  ranges[i] = r;
}

cudaError_t launch_attend_ranges(int nq, int nseg, const int32_t* q_offsets,
                                 const int32_t* k_offsets, const int32_t* c_offsets,
                                 const int32_t* prefix, int causal, int32_t* ranges,
                                 uint32_t* err, cudaStream_t s) {
  attend_ranges_kernel<<<(nq + 255) / 256, 256, 0, s>>>(nq, nseg, q_offsets, k_offsets, c_offsets,
                                                        prefix, causal,
                                                        reinterpret_cast<int4*>(ranges), err);
  return cudaGetLastError();
}

}  // namespace spark
