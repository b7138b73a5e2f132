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
// Bound by HBM: each value is read and written once.  A thread owns kPairs pairs of a token and
// walks the heads with them, so the cosines, sines and weights stay in registers; the rows of
// one (token, head) are read by d/2/kPairs neighbouring lanes, and neighbouring lane groups take
// neighbouring tokens, which makes the writes of a head contiguous over a CTA's tokens.
#include "spark_kernels.cuh"

namespace spark {

namespace {

constexpr int kRopeThreads = 256;

template <typename T, int V>
struct __align__(sizeof(T) * V) Vec {
  T v[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

}  // namespace

// V: values per access (the two halves of V pairs are V values each); C: such accesses per
// thread and half; U: heads whose rows a thread holds at once.
template <typename T, int D, int V, int C, int U>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a,
                                                                    int heads_per_cta) {
  constexpr int kLanes = D / 2 / (V * C);          // threads per row
  constexpr int kTokens = kRopeThreads / kLanes;   // tokens per CTA
  using Vt = Vec<T, V>;
  const int t = blockIdx.z == 0 ? 0 : (a.in[1] != nullptr ? blockIdx.z : 2);   // Q, K or V
  const int lane = threadIdx.x % kLanes;
  const long long n = static_cast<long long>(blockIdx.x) * kTokens + threadIdx.x / kLanes;
  const bool live = n < a.N;
  const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, a.H);
  const float* weight = t < 2 ? a.weight[t] : nullptr;

  // columns of the thread's two vectors, cos and sin of their pairs, norm weights
  int ca[C], cb[C];
  bool rot[C];
  float cs[C][V], sn[C][V], w[C][2][V];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int p = (c * kLanes + lane) * V;         // first pair
    rot[c] = t < 2 && p < a.pairs;
    const bool half = rot[c] && !a.interleaved;
    ca[c] = half ? p : 2 * p;
    cb[c] = half ? p + a.pairs : 2 * p + V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      cs[c][j] = 1.f, sn[c][j] = 0.f;
      if (rot[c] && live) {
        int axis = 0;
        for (int k = 1; k < a.naxes; ++k) axis += p + j >= a.first[k];
        const size_t at = static_cast<size_t>(n) * a.naxes + axis;
        const double pos = a.positions_f32
                               ? static_cast<double>(static_cast<const float*>(a.positions)[at])
                               : static_cast<double>(static_cast<const int32_t*>(a.positions)[at]);
        double turns = pos * static_cast<double>(a.inv_freq[p + j]) * 0.15915494309189535;
        turns -= rint(turns);
        float s, k;
        sincospif(2.f * static_cast<float>(turns), &s, &k);
        cs[c][j] = k * a.scale, sn[c][j] = s * a.scale;
      }
      w[c][0][j] = weight != nullptr ? weight[ca[c] + j] : 1.f;
      w[c][1][j] = weight != nullptr ? weight[cb[c] + j] : 1.f;
    }
  }
  const T* src = static_cast<const T*>(a.in[t]) + n * a.token_stride[t];
  T* dst = static_cast<T*>(a.out[t]) + n * D;
  const long long hs = a.head_stride[t], hd = static_cast<long long>(a.N) * D;
  for (int h = h0; h < h1; h += U) {
    Vt x[U][C][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= h1 || !live) continue;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        x[u][c][0] = *reinterpret_cast<const Vt*>(src + (h + u) * hs + ca[c]);
        x[u][c][1] = *reinterpret_cast<const Vt*>(src + (h + u) * hs + cb[c]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= h1) break;                      // uniform
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
                  const float v = to_f(x[u][c][e].v[j]);
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
            for (int j = 0; j < V; ++j) y[e * V + j] = to_f(x[u][c][e].v[j]) * r * w[c][e][j];
          if (rot[c]) {
            if (a.interleaved) {
#pragma unroll
              for (int j = 0; j < V; ++j) {
                const float p = y[2 * j], q = y[2 * j + 1];
                y[2 * j] = p * cs[c][j] - q * sn[c][j];
                y[2 * j + 1] = p * sn[c][j] + q * cs[c][j];
              }
            } else {
#pragma unroll
              for (int j = 0; j < V; ++j) {
                const float p = y[j], q = y[V + j];
                y[j] = p * cs[c][j] - q * sn[c][j];
                y[V + j] = p * sn[c][j] + q * cs[c][j];
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < V; ++j) from_f(x[u][c][e].v[j], y[e * V + j]);
        }
      }
      if (live) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          *reinterpret_cast<Vt*>(dst + (h + u) * hd + ca[c]) = x[u][c][0];
          *reinterpret_cast<Vt*>(dst + (h + u) * hd + cb[c]) = x[u][c][1];
        }
      }
    }
  }
}

#ifndef RU
#define RU 4
#endif
#ifndef RW
#define RW 8
#endif
template <typename T, int D, int V, int C>
static cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t s) {
  constexpr int kTokens = kRopeThreads / (D / 2 / (V * C));
  const int blocks = (a.N + kTokens - 1) / kTokens;
  const int tensors = 1 + (a.in[1] != nullptr) + (a.in[2] != nullptr);
  // few tokens: the heads go to more CTAs, until there are RW per SM
  int splits = (RW * 148 + blocks * tensors - 1) / (blocks * tensors);
  if (splits > a.H) splits = a.H;
  const int per = (a.H + splits - 1) / splits;
  qk_norm_rope_kernel<T, D, V, C, RU>
      <<<dim3(blocks, (a.H + per - 1) / per, tensors), kRopeThreads, 0, s>>>(a, per);
  return cudaGetLastError();
}

// The widest access that every row start, stride and half allows.
static int rope_vec(const RopeArgs& a, int esize, int d) {
  int v = esize == 2 ? 8 : 4;
  auto fits = [&](int n) {
    if (a.pairs % n != 0 || (d / 2) % n != 0) return false;
    for (int t = 0; t < 3; ++t) {
      if (a.in[t] == nullptr) continue;
      const uintptr_t bytes = static_cast<uintptr_t>(n) * esize;
      if (reinterpret_cast<uintptr_t>(a.in[t]) % bytes || reinterpret_cast<uintptr_t>(a.out[t]) % bytes)
        return false;
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
