// Per-head norm and position rotation of queries and keys, with the layout change to [H,N,d]
// that every other kernel here reads (values are laid out along).
//
// Row (h, n), x its d values, w the weights, pair i of the rotated part at angle
// t_i = pos[n, axis(i)] * inv_freq[i]:
//   y = x * rsqrt(mean x^2 + eps) * w
//   (a, b) -> scale * (a cos t - b sin t, a sin t + b cos t)
// over pairs (y_i, y_{i+pairs}) (half layout) or (y_{2i}, y_{2i+1}) (interleaved); the values
// behind the 2*pairs rotated ones pass.  Everything is fp32 with one rounding at the end; the
// angle is taken modulo a turn in fp64, as a far position's fp32 angle has lost its low bits.
//
// Bound by HBM: each value is read and written once.  A thread owns the same columns of a token
// in every head (8 pairs at the widest access), so cosines, sines and weights stay in registers
// while it walks the heads of one of Q, K and V; neighbouring lane groups take neighbouring
// tokens, which makes a head's writes contiguous over a CTA's tokens.  The next rows come by
// asynchronous copies into shared memory: 4 under way per thread.  On 60480 tokens, 20 heads,
// d = 128, bf16, Q, K and V from a fused projection, the steps to that measured 479 us (all
// three tensors in a thread, loads into registers), 401 us (one tensor per CTA), 380 us
// (accesses that cover whole sectors), 333 us (asynchronous copies) and 299 us (streaming stores,
// 6 CTAs of 128 threads an SM).  It now takes 308 to 311 us in a loop = 6.0 TB/s, 91% of the
// measured copy bandwidth.
#include <type_traits>

#include "spark_kernels.cuh"

namespace spark {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 6;                       // per SM
constexpr int kRopeDepth = 4;                      // rows a thread has under way

template <typename T, int V>
struct __align__(sizeof(T) * V) Vec {
  T v[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

template <typename Vt, typename T>
__device__ __forceinline__ void put(T* dst, const Vt& v) {
  if constexpr (sizeof(Vt) == 16)                  // streamed: nothing here reads it again
    __stcs(reinterpret_cast<uint4*>(dst), *reinterpret_cast<const uint4*>(&v));
  else
    *reinterpret_cast<Vt*>(dst) = v;
}

// Asynchronous copy of one vector from global to this thread's own place in shared memory; the
// thread alone reads it again, after cp_wait, so no barrier is needed.
template <int kBytes>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "n"(kBytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

}  // namespace

// V: values per access (the two halves of V pairs are V values each); C: such accesses per
// thread and half; kPart: some vector of an interleaved row is rotated in part, which takes a test
// per pair (with the test in every row 60480 tokens took 6% longer; without vectors rotated in
// part, by narrower accesses, 16384 tokens with 33 pairs took 75 us in place of 40).
template <typename T, int D, int V, int C, bool kPart>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    qk_norm_rope_kernel(const RopeArgs a, int heads_per_cta) {
  constexpr int kLanes = D / 2 / (V * C);          // threads per row
  constexpr int kTokens = kRopeThreads / kLanes;   // tokens per CTA
  using Vt = Vec<T, V>;
  const int t = blockIdx.z == 0 ? 0 : (a.in[1] != nullptr ? blockIdx.z : 2);   // Q, K or V
  const int lane = threadIdx.x % kLanes;
  const long long n = static_cast<long long>(blockIdx.x) * kTokens + threadIdx.x / kLanes;
  const bool live = n < a.N;
  const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, a.H);
  const float* weight = t < 2 ? a.weight[t] : nullptr;
  // set up while the kernel before it ends, and so may the one behind it be: no global memory is
  // touched before the wait (back to back: 16384 tokens 41.5 -> 39.6 us, one token 12.2 -> 11.7)
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");

  // Columns of the thread's two vectors.  Half layout: the two sides of V pairs.  Interleaved (and
  // unrotated) rows: one vector in each half of the row with V/2 whole pairs each, so that a
  // warp's access covers whole sectors; a single value per access (V = 1) takes the two values
  // of one pair.
  constexpr int kInner = V > 1 ? V / 2 : 1;        // whole pairs in a vector
  int col[C][2];
  // whether each vector is rotated (half layout and V = 1: rot[.][0] counts for both), or with
  // kPart how many of its pairs are
  std::conditional_t<kPart, int, bool> rot[C][2];
  float cs[C][V], sn[C][V], w[C][2][V];
  const bool half = !a.interleaved && a.pairs > 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int p = (c * kLanes + lane) * V;
    if (half && p < a.pairs) {
      col[c][0] = p, col[c][1] = p + a.pairs;
      rot[c][0] = rot[c][1] = t < 2;
    } else if (half || V == 1) {
      col[c][0] = 2 * p, col[c][1] = 2 * p + V;
      rot[c][0] = rot[c][1] = t < 2 && !half && p < a.pairs;
    } else {
      col[c][0] = p, col[c][1] = p + D / 2;
      rot[c][0] = t < 2 && col[c][0] < 2 * a.pairs;
      rot[c][1] = t < 2 && col[c][1] < 2 * a.pairs;
      if constexpr (kPart) {
        rot[c][0] *= min(kInner, a.pairs - col[c][0] / 2);
        rot[c][1] *= min(kInner, a.pairs - col[c][1] / 2);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      cs[c][j] = sn[c][j] = 0.f;
      const int e = half || V == 1 ? 0 : j / kInner;
      bool here = rot[c][e] && live;
      if constexpr (kPart) here = here && j % kInner < rot[c][e];
      if (here) {
        const int i = half || V == 1 ? p + j : col[c][e] / 2 + j % kInner;
        int axis = 0;
        for (int k = 1; k < a.naxes; ++k) axis += i >= a.first[k];
        const size_t at = static_cast<size_t>(n) * a.naxes + axis;
        const double pos = a.positions_f32
                               ? static_cast<double>(static_cast<const float*>(a.positions)[at])
                               : static_cast<double>(static_cast<const int32_t*>(a.positions)[at]);
        double turns = pos * static_cast<double>(a.inv_freq[i]) * 0.15915494309189535;
        turns -= rint(turns);
        float s, k;
        sincospif(2.f * static_cast<float>(turns), &s, &k);
        cs[c][j] = k * a.scale, sn[c][j] = s * a.scale;
      }
      w[c][0][j] = weight != nullptr ? weight[col[c][0] + j] : 1.f;
      w[c][1][j] = weight != nullptr ? weight[col[c][1] + j] : 1.f;
    }
  }
  const T* src = static_cast<const T*>(a.in[t]) + n * a.token_stride[t];
  T* dst = static_cast<T*>(a.out[t]) + n * D;
  const long long hs = a.head_stride[t], hd = static_cast<long long>(a.N) * D;
  // kDepth - 1 rows ahead of the one at work are on their way (accesses under the 4 bytes that an
  // asynchronous copy takes are loaded as they are needed)
  constexpr bool kAsync = sizeof(Vt) >= 4;
  constexpr int kDepth = kAsync ? kRopeDepth : 1;
  __shared__ Vt ring[kDepth][C][2][kRopeThreads];
  auto fetch = [&](int h) {
    if (kAsync && h < h1 && live) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          cp_async<kAsync ? sizeof(Vt) : 4>(&ring[(h - h0) % kDepth][c][e][threadIdx.x],
                                            src + h * hs + col[c][e]);
    }
    if (kAsync) cp_commit();
  };
  for (int i = 0; i < kDepth - 1; ++i) fetch(h0 + i);
  for (int h = h0; h < h1; ++h) {
    fetch(h + kDepth - 1);
    if (kAsync) cp_wait<kDepth - 1>();
    Vt x[C][2];
    if (live) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[c][e] = kAsync ? ring[(h - h0) % kDepth][c][e][threadIdx.x]
                           : *reinterpret_cast<const Vt*>(src + h * hs + col[c][e]);
    }
    if (t < 2) {
      float r = 1.f;
      if (weight != nullptr) {
        float ss = 0.f;
        if (live) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < V; ++j) {
                const float v = to_f(x[c][e].v[j]);
                ss = fmaf(v, v, ss);
              }
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = rsqrtf(ss * (1.f / D) + a.eps);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float y[2 * V];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < V; ++j) y[e * V + j] = to_f(x[c][e].v[j]) * r * w[c][e][j];
        if (half || V == 1) {
          if (rot[c][0]) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const float p = y[j], q = y[V + j];
              y[j] = p * cs[c][j] - q * sn[c][j];
              y[V + j] = p * sn[c][j] + q * cs[c][j];
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!rot[c][e]) continue;
#pragma unroll
            for (int i = 0; i < kInner; ++i) {
              if constexpr (kPart) {
                if (i >= rot[c][e]) break;
              }
              const int j = e * kInner + i;
              const float p = y[e * V + 2 * i], q = y[e * V + 2 * i + 1];
              y[e * V + 2 * i] = p * cs[c][j] - q * sn[c][j];
              y[e * V + 2 * i + 1] = p * sn[c][j] + q * cs[c][j];
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < V; ++j) from_f(x[c][e].v[j], y[e * V + j]);
      }
    }
    if (live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        put(dst + h * hd + col[c][0], x[c][0]);
        put(dst + h * hd + col[c][1], x[c][1]);
      }
    }
  }
}

template <typename T, int D, int V, int C>
static cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t s) {
  constexpr int kTokens = kRopeThreads / (D / 2 / (V * C));
  const int blocks = (a.N + kTokens - 1) / kTokens;
  const int tensors = 1 + (a.in[1] != nullptr) + (a.in[2] != nullptr);
  // Few tokens: the heads go to more CTAs, until each SM has its share.  Every CTA computes its
  // tokens' cosines again, so no more than that (16384 tokens, 8 heads: 43 us at one to two
  // splits, 53 us at four).
  const long long ctas = static_cast<long long>(blocks) * tensors;
  int splits = static_cast<int>((kRopeCtas * 148 + ctas - 1) / ctas);
  if (splits > a.H) splits = a.H;
  const int per = (a.H + splits - 1) / splits;
  const auto kern = V > 1 && a.interleaved && a.pairs % (V > 1 ? V / 2 : 1) != 0
                        ? qk_norm_rope_kernel<T, D, V, C, (V > 1)>
                        : qk_norm_rope_kernel<T, D, V, C, false>;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, (a.H + per - 1) / per, tensors);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, per);
}

// The widest access that every row start, stride and half allows.
static int rope_vec(const RopeArgs& a, int esize, int d) {
  int v = esize == 2 ? 8 : 4;
  auto fits = [&](int n) {
    // the two sides of a half layout's pairs have to start at whole vectors
    if ((!a.interleaved && a.pairs % n != 0) || (d / 2) % n != 0) return false;
    for (int t = 0; t < 3; ++t) {
      if (a.in[t] == nullptr) continue;
      const uintptr_t bytes = static_cast<uintptr_t>(n) * esize;
      const uintptr_t in = reinterpret_cast<uintptr_t>(a.in[t]);
      if (in % bytes || reinterpret_cast<uintptr_t>(a.out[t]) % bytes) return false;
      if (a.head_stride[t] % n || a.token_stride[t] % n) return false;
    }
    return true;
  };
  while (v > 1 && !fits(v)) v /= 2;
  return v;
}

template <typename T, int D>
static cudaError_t launch_rope_d(const RopeArgs& a, cudaStream_t s) {
  const int v = rope_vec(a, sizeof(T), D);
  if constexpr (sizeof(T) == 2) {
    if (v == 8) return launch_rope_t<T, D, 8, 1>(a, s);
  }
  if (v >= 4) return launch_rope_t<T, D, 4, 1>(a, s);
  if (v == 2) return launch_rope_t<T, D, 2, 2>(a, s);
  return launch_rope_t<T, D, 1, 4>(a, s);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, int dtype, int d, cudaStream_t s) {
  if (dtype == 0)
    return d == 128 ? launch_rope_d<__nv_bfloat16, 128>(a, s)
                    : launch_rope_d<__nv_bfloat16, 64>(a, s);
  return d == 128 ? launch_rope_d<float, 128>(a, s) : launch_rope_d<float, 64>(a, s);
}

}  // namespace spark
